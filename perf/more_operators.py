"""The operators of a serving step around the paged latent cache, as a benchmark: plain forms and the framework's calls.

  tables   block table, slot map, positions and row offsets of a step from the requests' lengths, with the
           pages taken from and given back to a free stack
  attend   absorbed latent attention of new tokens where groups of requests share a long prefix
  sample   temperature, top-k, top-p and min-p, then a token drawn with a given random number (or the filtered
           distribution, as the verification of drafted tokens takes it)
"""
import math
import random

import torch

own = False

PAGE = 64
LATENT, VALUE = 576, 512
SCALE = 192 ** -0.5          # 128 nope + 64 rope dims of the expanded query


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request, one new token: the latency of the smallest step
        {"name": "tables_b1", "op": "tables", "batch": 1, "new_lo": 1, "new_hi": 1, "ctx_hi": 5000, "ended": 0,
         "pad": 0, "prefix": 0, "lens_seed": 1},
        # a decode step of 500 requests with drafts behind a common system prompt, some of them ended, the rows
        # padded to a captured graph's size
        {"name": "tables_b500_drafts", "op": "tables", "batch": 500, "new_lo": 1, "new_hi": 4, "ctx_hi": 65536,
         "ended": 40, "pad": 131, "prefix": 1024, "lens_seed": 2},
        # prompts of 1 to 16K tokens that start together
        {"name": "tables_prompts_b48", "op": "tables", "batch": 48, "new_lo": 1, "new_hi": 16384, "ctx_hi": 4096,
         "ended": 2, "pad": 0, "prefix": 0, "lens_seed": 3},
        # four requests just started behind a short common prompt, on one rank of a head-parallel group
        {"name": "attend_b4_1k_h16", "op": "attend", "groups": 1, "batch": 4, "prefix_lo": 1024, "prefix_hi": 1024,
         "own_lo": 1, "own_hi": 100, "q_len": 1, "heads": 16, "idle": 0, "lens_seed": 4},
        # 64 conversations behind one long document, 16 heads a rank
        {"name": "attend_b64_32k_h16", "op": "attend", "groups": 1, "batch": 64, "prefix_lo": 32768,
         "prefix_hi": 32768, "own_lo": 64, "own_hi": 4096, "q_len": 1, "heads": 16, "idle": 0, "lens_seed": 5},
        # several documents with a few requests each, drafted tokens, 32 heads a rank, the batch padded with two idle
        # requests as a captured graph pads it
        {"name": "attend_g5_mtp_h32", "op": "attend", "groups": 5, "batch": 60, "prefix_lo": 2048,
         "prefix_hi": 32768, "own_lo": 1, "own_hi": 8192, "q_len": 2, "heads": 32, "idle": 2, "lens_seed": 6},
        # all heads on one GPU
        {"name": "attend_b32_16k_h128", "op": "attend", "groups": 1, "batch": 32, "prefix_lo": 16384,
         "prefix_hi": 16384, "own_lo": 100, "own_hi": 1000, "q_len": 1, "heads": 128, "idle": 0, "lens_seed": 7},
        # many samples of one very long prompt
        {"name": "attend_b200_128k_h16", "op": "attend", "groups": 1, "batch": 200, "prefix_lo": 131008,
         "prefix_hi": 131008, "own_lo": 1, "own_hi": 2000, "q_len": 1, "heads": 16, "idle": 0, "lens_seed": 8},
        # one request, the usual filters
        {"name": "sample_b1_32k", "op": "sample", "rows": 1, "vocab": 32000, "bf16": True, "mode": "usual",
         "probs": False, "pad": 0, "masked": 0.0, "rows_seed": 9},
        # 64 requests with settings of their own, some under a grammar's mask
        {"name": "sample_b64_131k", "op": "sample", "rows": 64, "vocab": 131072, "bf16": False, "mode": "mixed",
         "probs": False, "pad": 0, "masked": 0.5, "rows_seed": 10},
        # a large batch of an odd vocabulary, top-p only: most of the mass counts
        {"name": "sample_b300_100003", "op": "sample", "rows": 300, "vocab": 100003, "bf16": True, "mode": "top_p",
         "probs": False, "pad": 5, "masked": 0.0, "rows_seed": 11},
        # the target distributions of 64 requests with three drafts each, for their verification
        {"name": "sample_probs_b256_131k", "op": "sample", "rows": 256, "vocab": 131072, "bf16": False,
         "mode": "usual", "probs": True, "pad": 0, "masked": 0.0, "rows_seed": 12},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "attend", "sample"])
    seed = rng.randrange(1 << 30)
    if op == "tables":
        while True:
            case = {"op": op, "batch": _log_uniform(rng, 1, 2000), "new_lo": 1, "new_hi": _log_uniform(rng, 1, 16384),
                    "ctx_hi": _log_uniform(rng, 64, 65536), "ended": rng.choice([0, 0, 1, 7]),
                    "pad": rng.choice([0, 1, 200]), "prefix": rng.choice([0, 0, 64, 1024]), "lens_seed": seed}
            if sum(n for _, n, _ in _table_lens(case)) <= 150000:
                return case
    if op == "attend":
        while True:
            case = {"op": op, "groups": rng.choice([1, 1, 2, 5]), "batch": _log_uniform(rng, 1, 256),
                    "prefix_lo": _log_uniform(rng, 1, 60000), "prefix_hi": 0, "own_lo": 1,
                    "own_hi": _log_uniform(rng, 1, 8192), "q_len": rng.choice([1, 1, 2, 3, 4]),
                    "heads": rng.choice([16, 16, 32, 64, 128]), "idle": rng.choice([0, 0, 1]), "lens_seed": seed}
            case["prefix_hi"] = _log_uniform(rng, case["prefix_lo"], 131072)
            w = work(case)
            if w["flops"] <= 9e11 and w["bytes"] <= 6e8:
                return case
    while True:
        case = {"op": op, "rows": _log_uniform(rng, 1, 512), "vocab": _log_uniform(rng, 1000, 160000),
                "bf16": rng.random() < 0.5, "mode": rng.choice(["usual", "mixed", "top_p", "all"]),
                "probs": rng.random() < 0.3, "pad": rng.choice([0, 0, 3, 64]), "masked": rng.choice([0.0, 0.0, 0.5, 0.99]),
                "rows_seed": seed}
        if case["rows"] * case["vocab"] <= 256 * 131072:
            return case


def _table_lens(case):
    """(cached tokens, new tokens, mapped pages) of every request; new = -1: the request ends."""
    rng = random.Random(case["lens_seed"])
    out = []
    for b in range(case["batch"]):
        ctx = case["prefix"] + _log_uniform(rng, 1, case["ctx_hi"]) - 1
        new = min(case["new_hi"], max(case["new_lo"], _log_uniform(rng, case["new_lo"], case["new_hi"])))
        if b % 7 == 3 and b // 7 < case["ended"]:
            new = -1
        # rejected drafts leave a page mapped ahead of the cached tokens now and then
        out.append((ctx, new, (ctx + PAGE - 1) // PAGE + (1 if rng.random() < 0.1 else 0)))
    return out


def _attend_lens(case):
    """(requests, prefix) of every group, (cached tokens, new tokens) of every request; the last `idle` ones, a
    group of their own, pad the batch."""
    rng = random.Random(case["lens_seed"])
    cuts = sorted(rng.randrange(case["batch"] + 1) for _ in range(case["groups"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["batch"]])]
    groups, reqs = [], []
    for n in sizes:
        prefix = _log_uniform(rng, case["prefix_lo"], case["prefix_hi"]) // PAGE * PAGE
        groups.append((n, prefix))
        for _ in range(n):
            reqs.append((prefix + _log_uniform(rng, case["own_lo"], case["own_hi"]) + case["q_len"] - 1, case["q_len"]))
    if case["idle"]:
        groups.append((case["idle"], 0))
        reqs += [(0, case["q_len"])] * case["idle"]
    return groups, reqs


def work(case):
    if case["op"] == "tables":
        lens = _table_lens(case)
        tokens = sum(max(0, n) for _, n, _ in lens)
        pages = sum(max(0, (c + n + PAGE - 1) // PAGE - m) if n >= 0 else m - case["prefix"] // PAGE for c, n, m in lens)
        return {"bytes": (tokens + case["pad"]) * 16 + pages * 8 + case["batch"] * 28 + 12, "flops": 0}
    if case["op"] == "attend":
        groups, reqs = _attend_lens(case)
        h, keys, pairs, rows, b = case["heads"], 0, 0, 0, 0
        for n, prefix in groups:
            keys += prefix if n else 0
            for length, q in reqs[b:b + n]:
                keys += max(0, length - prefix)
                pairs += sum(max(0, length - q + j + 1) for j in range(q))
                rows += q
            b += n
        return {"bytes": keys * LATENT * 2 + rows * h * (LATENT * 2 + VALUE * 2 + 4),
                "flops": pairs * h * 2 * (LATENT + VALUE)}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (2 if case["bf16"] else 4) + (n * 4 if case["probs"] else 0) + case["rows"] * 24,
            "flops": n * 4}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _cum(ns):
    c = [0]
    for n in ns:
        c.append(c[-1] + n)
    return c


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"tables": _prepare_tables, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](case, seed)


def _prepare_tables(case, seed):
    lens, g = _table_lens(case), _gen(seed, 1)
    shared = case["prefix"] // PAGE
    need = [max(m, (c + max(0, n) + PAGE - 1) // PAGE) for c, n, m in lens]
    mapped = shared + sum(m - shared for _, _, m in lens)
    num_pages = shared + sum(n - shared for n in need) + 10
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = shared
    for b, (_, _, m) in enumerate(lens):
        table[b, :shared] = perm[:shared]
        table[b, shared:m] = perm[at:at + m - shared]
        at += m - shared
    free = torch.full((num_pages,), -1, dtype=torch.int32, device="cuda")
    free[:num_pages - mapped] = perm[mapped:]
    rows = sum(max(0, n) for _, n, _ in lens) + case["pad"]
    return {"op": "tables", "cached": _i32([c for c, _, _ in lens]), "q_lens": _i32([n for _, n, _ in lens]),
            "counts": _i32([m for _, _, m in lens]), "keep": _i32([shared] * len(lens)), "table": table,
            "num_pages": num_pages, "free": free, "free_count": _i32([num_pages - mapped]),
            "seq_lens": _i32([0] * len(lens)), "counts_out": _i32([0] * len(lens)), "free_count_out": _i32([0]),
            "cu_q": _i32([0] * (len(lens) + 1)), "positions": torch.zeros(rows, dtype=torch.int64, device="cuda"),
            "slots": torch.zeros(rows, dtype=torch.int64, device="cuda")}


def _prepare_attend(case, seed):
    groups, reqs = _attend_lens(case)
    h, g = case["heads"], _gen(seed, 2)
    need = [(n + PAGE - 1) // PAGE for n, _ in reqs]
    total = sum(prefix // PAGE for n, prefix in groups if n)
    b = 0
    for n, prefix in groups:
        total += sum(max(0, need[i] - prefix // PAGE) for i in range(b, b + n))
        b += n
    num_pages = total + 3
    # normed latents and rotated rope keys: unit variance
    pool = torch.empty(num_pages, PAGE, LATENT, dtype=torch.bfloat16, device="cuda")
    for p0 in range(0, num_pages, 4096):
        n = min(4096, num_pages - p0)
        pool[p0:p0 + n] = torch.randn((n, PAGE, LATENT), generator=g, device="cuda").to(torch.bfloat16)
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(reqs), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = b = 0
    for n, prefix in groups:
        if n:
            table[b:b + n, :prefix // PAGE] = perm[at:at + prefix // PAGE]
            at += prefix // PAGE
        for i in range(b, b + n):
            k = max(0, need[i] - prefix // PAGE)
            table[i, prefix // PAGE:prefix // PAGE + k] = perm[at:at + k]
            at += k
        b += n
    rows = sum(q for _, q in reqs)
    st = {"op": "attend", "groups": groups, "reqs": reqs, "pool": pool, "table": table,
          "seq_lens": _i32([n for n, _ in reqs]), "cu_q": _i32(_cum([q for _, q in reqs])),
          "cu_group": _i32(_cum([n for n, _ in groups])), "shared": _i32([p for _, p in groups]),
          "q": torch.randn((rows, h, LATENT), generator=g, device="cuda").to(torch.bfloat16),
          "out": torch.empty(rows, h, VALUE, dtype=torch.bfloat16, device="cuda"),
          "lse": torch.empty(rows, h, dtype=torch.float32, device="cuda")}
    if own:
        from deepseek_sparse_attention_paged_gb300 import capi
        st["ws"] = torch.empty(max(16, capi.dsa_dense_mla_decode_shared_workspace_size(rows, h)), dtype=torch.uint8,
                               device="cuda")
    return st


def _settings(case):
    """(temperature, top_k, top_p, min_p) of every row."""
    rng = random.Random(case["rows_seed"])
    out = []
    for _ in range(case["rows"]):
        t = round(rng.uniform(0.6, 1.3), 3)
        if case["mode"] == "usual":
            out.append((t, 50, 0.95, 0.0))
        elif case["mode"] == "top_p":
            out.append((t, 0, rng.choice([0.9, 0.95, 0.99]), 0.0))
        elif case["mode"] == "all":
            out.append((t, 0, 1.0, 0.0))
        else:
            out.append((rng.choice([0.0, t, t, t]), rng.choice([0, 1, 20, 50, 1000]), rng.choice([0.5, 0.9, 0.99, 1.0]),
                        rng.choice([0.0, 0.0, 0.02, 0.1])))
    return out


def _prepare_sample(case, seed):
    r, v, g = case["rows"], case["vocab"], _gen(seed, 3)
    # logits of a language model: a broad bulk, and a few tokens far above it
    buf = torch.randn((r, v + case["pad"]), generator=g, device="cuda") * 2.0
    top = torch.randint(0, v, (r, 24), generator=g, device="cuda")
    buf.scatter_(1, top, 7.0 + 3.0 * torch.randn((r, 24), generator=g, device="cuda"))
    if case["masked"]:
        # a grammar that forbids tokens in every other row (one token at least stays)
        off = torch.rand((r, v + case["pad"]), generator=g, device="cuda") < case["masked"]
        off[1::2] = False
        off.scatter_(1, top[:, :1], False)
        buf.masked_fill_(off, -math.inf)
    rows = _settings(case)
    f32 = lambda i: torch.tensor([x[i] for x in rows], dtype=torch.float32, device="cuda")
    filters = case["mode"] != "all"
    return {"op": "sample", "logits": (buf.to(torch.bfloat16) if case["bf16"] else buf)[:, :v], "temperature": f32(0),
            "top_k": _i32([x[1] for x in rows]) if filters and case["mode"] != "top_p" else None,
            "top_p": f32(2) if filters else None, "min_p": f32(3) if case["mode"] == "mixed" else None,
            "u": torch.rand(r, generator=g, device="cuda"), "tokens": torch.empty(r, dtype=torch.int32, device="cuda"),
            "probs": torch.empty(r, v, dtype=torch.float32, device="cuda") if case["probs"] else None}


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return {"tables": _own_tables, "attend": _own_attend, "sample": _own_sample}[state["op"]](state)
    return {"tables": _plain_tables, "attend": _plain_attend, "sample": _plain_sample}[state["op"]](state)


_TABLE_OUTPUTS = ("seq_lens", "counts_out", "free_count_out", "cu_q", "positions", "slots", "table", "free")


def _own_tables(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_step_tables(st["cached"], st["q_lens"], st["counts"], st["table"], st["num_pages"], st["free"],
                         st["free_count"], st["seq_lens"], st["counts_out"], st["free_count_out"], st["cu_q"],
                         st["positions"], st["slots"], keep_pages=st["keep"])
    return {k: st[k] for k in _TABLE_OUTPUTS}


def _own_attend(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_dense_mla_decode_shared(st["q"], st["pool"], st["table"], st["seq_lens"], st["cu_q"], st["cu_group"],
                                     st["shared"], SCALE, st["out"], st["ws"], lse=st["lse"])
    return st["out"], st["lse"]


def _own_sample(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_sample_tokens(st["logits"], st["u"], st["tokens"], temperature=st["temperature"], top_k=st["top_k"],
                           top_p=st["top_p"], min_p=st["min_p"], probs=st["probs"])
    return st["tokens"] if st["probs"] is None else (st["tokens"], st["probs"])


def _plain_tables(st):
    cached, q, counts, keep = (st[k].long() for k in ("cached", "q_lens", "counts", "keep"))
    table, free, have, rows = st["table"], st["free"], st["free_count"].long(), st["slots"].numel()
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    ended = q < 0
    cu = torch.cat([zero, torch.cumsum(q.clamp_min(0), 0)]).clamp_max(rows)
    total = torch.where(ended, 0, cached + cu[1:] - cu[:-1])
    page = torch.arange(table.shape[1], device="cuda")[None]
    # pages given back: pushed on the stack in order
    back = ended[:, None] & (page >= keep[:, None]) & (page < counts[:, None])
    place = torch.cumsum(back.reshape(-1), 0).view(back.shape)
    at = torch.where(back, have + place - 1, free.numel())
    stack = torch.cat([free, free[:1]]).scatter(0, at.reshape(-1), table.reshape(-1))[:-1]
    have = have + place[-1, -1]
    # pages taken: from the top of the stack
    need = (total + PAGE - 1) // PAGE
    take = (page >= counts[:, None]) & (page < need[:, None])
    rank = torch.cumsum(take.reshape(-1), 0).view(take.shape)
    table.copy_(torch.where(take, stack[(have - rank).clamp_min(0)], table))
    free.copy_(stack)
    row = torch.arange(rows, device="cuda")
    req = torch.searchsorted(cu, row, right=True).clamp_max(cached.numel()) - 1
    used = row < cu[-1]
    pos = torch.where(used, cached[req] + row - cu[req], 0)
    slots = torch.where(used, table[req, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    new = {"seq_lens": total, "counts_out": torch.where(ended, 0, torch.maximum(counts, need)),
           "free_count_out": have - rank[-1, -1:], "cu_q": cu, "positions": pos, "slots": slots}
    for k, v in new.items():
        st[k].copy_(v)
    return {k: st[k] for k in _TABLE_OUTPUTS}


def _plain_attend(st):
    out, lse = torch.zeros_like(st["out"]), torch.full_like(st["lse"], -math.inf)
    h, b, r = st["q"].shape[1], 0, 0
    for n, prefix in st["groups"]:
        if n == 0:
            continue
        common = st["pool"][st["table"][b, :prefix // PAGE].long()].reshape(-1, LATENT).float()
        for i in range(b, b + n):
            length, ql = st["reqs"][i]
            if length == 0:
                r += ql
                continue
            rest = st["table"][i, prefix // PAGE:(length + PAGE - 1) // PAGE].long()
            rest = st["pool"][rest].reshape(-1, LATENT)[:length - prefix].float()
            q = st["q"][r:r + ql].reshape(-1, LATENT).float()
            vis = length - ql + 1 + torch.arange(ql, device="cuda").repeat_interleave(h)
            s = torch.cat([q @ common.t(), q @ rest.t()], 1) * SCALE
            s = torch.where(torch.arange(length, device="cuda")[None] < vis[:, None], s, -math.inf)
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - m)
            tot = e.sum(1, keepdim=True)
            o = (e[:, :prefix] @ common[:, :VALUE] + e[:, prefix:] @ rest[:, :VALUE]) / tot
            out[r:r + ql] = o.view(ql, h, VALUE).to(torch.bfloat16)
            lse[r:r + ql] = (m + torch.log(tot)).view(ql, h)
            r += ql
        b += n
    return out, lse


def _plain_sample(st):
    rows, v = st["logits"].shape
    tokens, probs = torch.empty_like(st["tokens"]), None
    if st["probs"] is not None:
        probs = torch.empty_like(st["probs"])
    rank = torch.arange(v, device="cuda")[None]
    for r in range(0, rows, 64):
        part = slice(r, min(rows, r + 64))
        z = st["logits"][part].double()
        t = st["temperature"][part].double()[:, None]
        zs, order = torch.sort(z, dim=1, descending=True, stable=True)
        ws = torch.exp((zs - zs[:, :1]) / torch.where(t > 0, t, 1.0))
        keep = (t > 0) | (rank == 0)
        if st["top_k"] is not None:
            k = st["top_k"][part, None]
            keep = keep & ((k <= 0) | (rank < k))
        ws = torch.where(keep, ws, 0.0)
        if st["top_p"] is not None:
            p = st["top_p"][part].double()[:, None]
            c = torch.cumsum(ws, 1)
            before = torch.cat([torch.zeros_like(c[:, :1]), c[:, :-1]], 1)
            ws = torch.where((p >= 1.0) | (rank == 0) | (before < p * c[:, -1:]), ws, 0.0)
        if st["min_p"] is not None:
            ws = torch.where(ws >= st["min_p"][part].double()[:, None], ws, 0.0)
        w = torch.zeros_like(ws).scatter_(1, order, ws)
        c = torch.cumsum(w, 1)
        tokens[part] = (c <= st["u"][part].double()[:, None] * c[:, -1:]).sum(1).clamp_max(v - 1).to(torch.int32)
        if probs is not None:
            probs[part] = (w / c[:, -1:]).float()
    return tokens if probs is None else (tokens, probs)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    return {"tables": _exact_tables, "attend": _exact_attend, "sample": _exact_sample}[case["op"]](
        prepare(case, seed), case)


def _exact_tables(st, case):
    cached, q, counts, keep = (st[k].tolist() for k in ("cached", "q_lens", "counts", "keep"))
    table, stack = st["table"].cpu().numpy().copy(), st["free"].tolist()
    have, rows, cu, seq, mapped, pos, slots = st["free_count"].item(), st["slots"].numel(), [0], [], [], [], []
    for b, n in enumerate(q):
        if n < 0:
            for i in range(keep[b], counts[b]):
                stack[have] = int(table[b, i])
                have += 1
    for b, n in enumerate(q):
        n = max(-1, min(n, rows - cu[-1]))
        cu.append(cu[-1] + max(0, n))
        if n < 0:
            seq.append(0)
            mapped.append(0)
            continue
        m = counts[b]
        while m * PAGE < cached[b] + n:
            have -= 1
            table[b, m] = stack[have]
            m += 1
        seq.append(cached[b] + n)
        mapped.append(m)
        for p in range(cached[b], cached[b] + n):
            pos.append(p)
            slots.append(int(table[b, p // PAGE]) * PAGE + p % PAGE)
    left = rows - len(pos)
    i64 = lambda x: torch.tensor(x, dtype=torch.int64, device="cuda")
    return {"seq_lens": _i32(seq), "counts_out": _i32(mapped), "free_count_out": _i32([have]), "cu_q": _i32(cu),
            "positions": i64(pos + [0] * left), "slots": i64(slots + [-1] * left),
            "table": torch.from_numpy(table).cuda(), "free": _i32(stack)}


def _exact_attend(st, case):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    flat, cu, at = st["pool"].view(-1, LATENT), st["cu_q"].tolist(), 0
    owner = [g for g, (n, _) in enumerate(st["groups"]) for _ in range(n)]
    cache, last = None, None
    for b, (length, ql) in enumerate(st["reqs"]):
        prefix = st["groups"][owner[b]][1]
        if owner[b] != last:
            pos = torch.arange(prefix, device="cuda")
            cache, last = flat[st["table"][b].long()[pos // PAGE] * PAGE + pos % PAGE].double(), owner[b]
        pos = torch.arange(prefix, max(prefix, length), device="cuda")
        keys = torch.cat([cache, flat[st["table"][b].long()[pos // PAGE] * PAGE + pos % PAGE].double()])
        for j in range(ql):
            v = length - ql + j + 1
            if v <= 0:
                continue
            row = cu[b] + j
            s = torch.einsum("hd,nd->hn", st["q"][row].double(), keys[:v]) / math.sqrt(192.0)
            lse[row] = torch.logsumexp(s, 1)
            out[row] = torch.einsum("hn,ne->he", torch.exp(s - lse[row][:, None]), keys[:v, :VALUE])
    return out, lse


def _exact_sample(st, case):
    rows, v = st["logits"].shape
    tokens, probs = [], None
    if st["probs"] is not None:
        probs = torch.zeros(rows, v, dtype=torch.float64, device="cuda")
    for r, (t, k, p, least) in enumerate(_settings(case)):
        z = st["logits"][r].double()
        t, u = float(st["temperature"][r]), float(st["u"][r])
        if t <= 0:
            best = int((z == z.max()).nonzero()[0])
            tokens.append(best)
            if probs is not None:
                probs[r, best] = 1.0
            continue
        z = z / t
        order = torch.argsort(-z, stable=True)[:k if 0 < k < v else v]
        w = torch.exp(z[order] - z[order[0]])
        if st["top_p"] is not None and p < 1:
            c = torch.cumsum(w, 0)
            n = 1 + int(torch.searchsorted(c[:-1].contiguous(), float(st["top_p"][r]) * c[-1:]))
            order, w = order[:n], w[:n]
        if st["min_p"] is not None:
            n = int((w >= float(st["min_p"][r])).sum())
            order, w = order[:n], w[:n]
        order, at = torch.sort(order)
        c = torch.cumsum(w[at], 0)
        i = min(int(torch.searchsorted(c, u * c[-1:], right=True)), order.numel() - 1)
        tokens.append(int(order[i]))
        if probs is not None:
            probs[r, order] = w[at] / c[-1]
    return _i32(tokens) if probs is None else (_i32(tokens), probs)
