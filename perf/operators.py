"""The dense latent-attention operators as a benchmark: their plain forms and the framework's calls.

Four operators that run one after the other around the paged latent cache of an MLA layer:
  store    norm + rotary embedding of the latent rows, written into the paged cache
  prefill  attention of a prompt in expanded form (per-head keys and values, one shared rope key)
  decode   attention of one or a few new tokens in absorbed form over the whole paged cache
  verify   acceptance of drafted tokens and the draw of the token after them
"""
import math
import random

import torch

own = False

PAGE = 64
LATENT, VALUE, ROPE, NOPE = 576, 512, 64, 128
SCALE = 192 ** -0.5          # 128 nope + 64 rope dims of the expanded query
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one request with a short context: the latency of the smallest decode step
        {"name": "decode_b1_4k", "op": "decode", "batch": 1, "lo": 4096, "hi": 4096, "q_len": 1, "heads": 128,
         "idle": 0, "lens_seed": 1},
        # 32 requests of 8K tokens, one new token each
        {"name": "decode_b32_8k", "op": "decode", "batch": 32, "lo": 8192, "hi": 8192, "q_len": 1, "heads": 128,
         "idle": 0, "lens_seed": 1},
        # 64 requests with contexts spread over 4K to 64K: the main serving batch
        {"name": "decode_b64_logu64k", "op": "decode", "batch": 64, "lo": 4096, "hi": 65536, "q_len": 1,
         "heads": 128, "idle": 0, "lens_seed": 2},
        # drafted tokens over long contexts on one rank of a head-parallel group, the batch padded with
        # two idle requests (length 0) as a captured graph pads it
        {"name": "decode_mtp_b8_128k_h16", "op": "decode", "batch": 8, "lo": 100000, "hi": 131072, "q_len": 2,
         "heads": 16, "idle": 2, "lens_seed": 3},
        # a few very short prompts on one rank of a head-parallel group
        {"name": "prefill_short_h16", "op": "prefill", "batch": 4, "lo": 1, "hi": 200, "prefix": 0, "heads": 16,
         "causal": True, "lens_seed": 4},
        # an ordinary batch of ragged prompts
        {"name": "prefill_ragged_b8", "op": "prefill", "batch": 8, "lo": 128, "hi": 2048, "prefix": 0, "heads": 128,
         "causal": True, "lens_seed": 5},
        # one long prompt
        {"name": "prefill_8k", "op": "prefill", "batch": 1, "lo": 8192, "hi": 8192, "prefix": 0, "heads": 128,
         "causal": True, "lens_seed": 6},
        # a chunk of a prompt whose earlier part is in the cache already
        {"name": "prefill_chunk_1k_after_15k", "op": "prefill", "batch": 1, "lo": 1000, "hi": 1000, "prefix": 15001,
         "heads": 128, "causal": True, "lens_seed": 7},
        # the new tokens of one decode step
        {"name": "store_64", "op": "store", "tokens": 64, "pad": 0, "interleaved": True, "skip": 4},
        # the tokens of a long prefill, read out of a wider projection output
        {"name": "store_32k", "op": "store", "tokens": 32768, "pad": 64, "interleaved": False, "skip": 0},
        # one request, one draft that was taken greedily (no draft distribution)
        {"name": "verify_b1_greedy", "op": "verify", "batch": 1, "drafts": 1, "vocab": 32000, "draft_probs": False,
         "uneven": False},
        # 64 requests with three sampled drafts each
        {"name": "verify_b64_k3", "op": "verify", "batch": 64, "drafts": 3, "vocab": 131072, "draft_probs": True,
         "uneven": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "prefill", "store", "verify"])
    seed = rng.randrange(1 << 30)
    if op == "decode":
        while True:
            case = {"op": op, "batch": _log_uniform(rng, 1, 128), "lo": _log_uniform(rng, 1, 60000), "hi": 0,
                    "q_len": rng.choice([1, 1, 2, 3, 4]), "heads": rng.choice([16, 32, 64, 128]),
                    "idle": rng.choice([0, 0, 1]), "lens_seed": seed}
            case["hi"] = _log_uniform(rng, case["lo"], 131072)
            if _cost(case) <= 0.9:
                return case
    if op == "prefill":
        while True:
            case = {"op": op, "batch": _log_uniform(rng, 1, 16), "lo": _log_uniform(rng, 1, 4000), "hi": 0,
                    "prefix": rng.choice([0, 0, _log_uniform(rng, 1, 12000)]),
                    "heads": rng.choice([1, 8, 16, 20, 64, 128]), "causal": rng.random() < 0.8, "lens_seed": seed}
            case["hi"] = _log_uniform(rng, case["lo"], 8192)
            if _cost(case) <= 0.9:
                return case
    if op == "store":
        return {"op": op, "tokens": _log_uniform(rng, 1, 32768), "pad": rng.choice([0, 8, 64, 1536]),
                "interleaved": rng.random() < 0.5, "skip": rng.choice([0, 1, 3])}
    while True:
        case = {"op": op, "batch": _log_uniform(rng, 1, 128), "drafts": rng.choice([0, 1, 2, 3, 5]),
                "vocab": _log_uniform(rng, 1000, 160000), "draft_probs": rng.random() < 0.7,
                "uneven": rng.random() < 0.5}
        if case["batch"] * (case["drafts"] + 1) * case["vocab"] <= 64 * 4 * 131072:
            return case


def _cost(case):
    """A drawn case's work over that of the largest listed one of its operator."""
    w = work(case)
    if case["op"] == "decode":
        return max(w["bytes"] / 1.6e9, w["flops"] / 3.5e11)
    return max(w["flops"] / 2.7e12, w["bytes"] / 2.2e9)


def _lens(case):
    rng = random.Random(case["lens_seed"])
    return [min(case["hi"], max(case["lo"], _log_uniform(rng, case["lo"], case["hi"]))) for _ in range(case["batch"])]


def _decode_lens(case):
    """(cached tokens, new tokens) of every request; the last `idle` ones pad the batch."""
    return _lens(case) + [0] * case["idle"], [case["q_len"]] * (case["batch"] + case["idle"])


def _draft_counts(case):
    """Drafts of every request."""
    k = case["drafts"]
    return [k - (b % (k + 1)) if case["uneven"] and b % 3 == 2 else k for b in range(case["batch"])]


def work(case):
    if case["op"] == "decode":
        lens, q_lens = _decode_lens(case)
        rows, h = sum(q_lens), case["heads"]
        pairs = sum(max(0, n - q + j + 1) for n, q in zip(lens, q_lens) for j in range(q))
        return {"bytes": sum(lens) * LATENT * 2 + rows * h * (LATENT * 2 + VALUE * 2 + 4),
                "flops": pairs * h * 2 * (LATENT + VALUE)}
    if case["op"] == "prefill":
        lens, h, pre = _lens(case), case["heads"], case["prefix"]
        rows, keys = sum(lens), sum(n + pre for n in lens)
        pairs = sum(n * pre + (n * (n + 1) // 2 if case["causal"] else n * n) for n in lens)
        return {"bytes": rows * h * (192 * 2 + 128 * 2 + 4) + keys * (h * 256 + ROPE) * 2,
                "flops": pairs * h * 2 * (192 + 128)}
    if case["op"] == "store":
        n = case["tokens"]
        return {"bytes": n * (3 * LATENT * 2 + ROPE * 4 + 16) + VALUE * 4, "flops": n * (VALUE * 4 + ROPE * 3)}
    counts = _draft_counts(case)
    read = case["vocab"] * 4 * (2 if case["draft_probs"] else 1)
    return {"bytes": case["batch"] * read + sum(k + 1 for k in counts) * 20,
            "flops": case["batch"] * case["vocab"] * 3}


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _randn(shape, g, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _cum(ns):
    c = [0]
    for n in ns:
        c.append(c[-1] + n)
    return c


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"decode": _prepare_decode, "prefill": _prepare_prefill, "store": _prepare_store,
            "verify": _prepare_verify}[case["op"]](case, seed)


def _prepare_decode(case, seed):
    lens, q_lens = _decode_lens(case)
    h, g = case["heads"], _gen(seed, 1)
    pages = [(n + PAGE - 1) // PAGE for n in lens]
    num_pages = sum(pages) + 3
    # normed latents and rotated rope keys: unit variance
    pool = torch.empty(num_pages, PAGE, LATENT, dtype=torch.bfloat16, device="cuda")
    for p0 in range(0, num_pages, 4096):
        n = min(4096, num_pages - p0)
        pool[p0:p0 + n] = _randn((n, PAGE, LATENT), g)
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(1, max(pages))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    rows = sum(q_lens)
    st = {"op": "decode", "lens": lens, "q_lens": q_lens, "pool": pool, "table": table, "seq_lens": _i32(lens),
          "cu_q": _i32(_cum(q_lens)), "q": _randn((rows, h, LATENT), g),
          "out": torch.empty(rows, h, VALUE, dtype=torch.bfloat16, device="cuda"),
          "lse": torch.empty(rows, h, dtype=torch.float32, device="cuda")}
    if own:
        from deepseek_sparse_attention_paged_gb300 import capi
        st["ws"] = torch.empty(max(16, capi.dsa_dense_mla_decode_workspace_size(rows, h)), dtype=torch.uint8,
                               device="cuda")
    return st


def _prepare_prefill(case, seed):
    lens, h, pre, g = _lens(case), case["heads"], case["prefix"], _gen(seed, 2)
    rows, keys = sum(lens), sum(n + pre for n in lens)
    latent = _randn((keys, LATENT), g)                    # normed latents, the rotated rope keys behind them
    kv = torch.empty(keys, h, 256, dtype=torch.bfloat16, device="cuda")     # up-projected: keys, then values
    step = max(1, (1 << 27) // (h * 256))
    for s in range(0, keys, step):
        n = min(step, keys - s)
        kv[s:s + n] = _randn((n, h, 256), g)
    return {"op": "prefill", "lens": lens, "prefix": pre, "causal": case["causal"], "q": _randn((rows, h, 192), g),
            "k_nope": kv[..., :NOPE], "v": kv[..., NOPE:], "k_pe": latent[:, VALUE:], "cu_q": _i32(_cum(lens)),
            "cu_k": _i32(_cum([n + pre for n in lens])),
            "out": torch.empty(rows, h, NOPE, dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty(rows, h, dtype=torch.float32, device="cuda")}


def _prepare_store(case, seed):
    n, g = case["tokens"], _gen(seed, 3)
    # projection outputs before the norm: a different size for every token
    raw = torch.randn((n, LATENT + case["pad"]), generator=g, device="cuda")
    raw = (raw * torch.exp(torch.randn((n, 1), generator=g, device="cuda") * 0.5)).to(torch.bfloat16)
    weight = 1.0 + 0.1 * torch.randn(VALUE, generator=g, device="cuda")
    max_pos = 40000
    freq = 10000.0 ** (-torch.arange(ROPE // 2, dtype=torch.float64, device="cuda") * 2 / ROPE)
    ang = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
    num_pages = (n + PAGE - 1) // PAGE + 2
    slots = torch.randperm(num_pages * PAGE, generator=g, device="cuda")[:n].contiguous()
    if case["skip"]:
        slots[:: max(2, n // case["skip"])] = -1          # padding tokens of the batch
    pos = torch.randint(0, max_pos, (n,), generator=g, device="cuda")
    return {"op": "store", "raw": raw[:, :LATENT], "weight": weight, "cs": cs, "pos": pos, "slots": slots,
            "interleaved": case["interleaved"],
            "pool": torch.zeros(num_pages, PAGE, LATENT, dtype=torch.bfloat16, device="cuda"),
            "latent": torch.zeros(n, LATENT, dtype=torch.bfloat16, device="cuda")}


def _prepare_verify(case, seed):
    counts, v, g = _draft_counts(case), case["vocab"], _gen(seed, 4)
    rows = sum(k + 1 for k in counts)
    # target: a softmax of spread logits with its tail cut off; draft: a softmax of logits near the target's
    logits = torch.randn((rows, v), generator=g, device="cuda") * 3.0
    target = torch.softmax(logits, 1)
    target = torch.where(target < 1e-7, torch.zeros_like(target), target)
    target = target / target.sum(1, keepdim=True)
    logits += torch.randn((rows, v), generator=g, device="cuda") * 0.7
    draft = torch.softmax(logits, 1)
    if case["draft_probs"]:
        tokens = torch.multinomial(draft, 1, generator=g)[:, 0].to(torch.int32)
    else:
        tokens = draft.argmax(1).to(torch.int32)
    return {"op": "verify", "target": target, "draft": draft if case["draft_probs"] else None, "tokens": tokens,
            "cu_q": _i32(_cum([k + 1 for k in counts])),
            "u": torch.rand(rows, generator=g, device="cuda"),
            "u_sample": torch.rand(len(counts), generator=g, device="cuda"),
            "out": torch.empty(rows, dtype=torch.int32, device="cuda"),
            "accepted": torch.empty(len(counts), dtype=torch.int32, device="cuda")}


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return {"decode": _own_decode, "prefill": _own_prefill, "store": _own_store, "verify": _own_verify}[
            state["op"]](state)
    return {"decode": _plain_decode, "prefill": _plain_prefill, "store": _plain_store, "verify": _plain_verify}[
        state["op"]](state)


def _own_decode(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_dense_mla_decode(st["q"], st["pool"], st["table"], st["seq_lens"], st["cu_q"], SCALE, st["out"],
                              st["ws"], lse=st["lse"])
    return st["out"], st["lse"]


def _own_prefill(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_dense_mla_prefill(st["q"], st["k_nope"], st["k_pe"], st["v"], st["cu_q"], st["cu_k"], SCALE, st["out"],
                               lse=st["lse"], causal=st["causal"])
    return st["out"], st["lse"]


def _own_store(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_store_latent_prologue(st["raw"], st["weight"], EPS, st["cs"], st["pos"], st["slots"], st["pool"],
                                   latent_out=st["latent"],
                                   flags=capi.DSA_ROPE_INTERLEAVED if st["interleaved"] else 0)
    return st["pool"], st["latent"]


def _own_verify(st):
    from deepseek_sparse_attention_paged_gb300 import capi
    capi.dsa_verify_drafts(st["target"], st["tokens"], st["cu_q"], st["u"], st["u_sample"], st["out"],
                           st["accepted"], draft_probs=st["draft"])
    return st["out"], st["accepted"]


def _softmax_av(s, v):
    """(softmax of the last axis times v, log-sum-exp); rows of -inf give 0 and -inf."""
    m = s.amax(-1, keepdim=True) if s.shape[-1] else s.new_full(s.shape[:-1] + (1,), -math.inf)
    m0 = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(s - m0)
    tot = e.sum(-1, keepdim=True)
    return (e @ v) / torch.where(tot == 0, torch.ones_like(tot), tot), (m0 + torch.log(tot)).squeeze(-1)


def _plain_decode(st):
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    r = 0
    for b, (n, ql) in enumerate(zip(st["lens"], st["q_lens"])):
        pages = st["table"][b, :(n + PAGE - 1) // PAGE].long()
        c = st["pool"][pages].reshape(-1, LATENT)[:n].float()
        s = st["q"][r:r + ql].float() @ c.t() * SCALE                       # [ql, H, n]
        pos = torch.arange(n, device="cuda")
        last = n - ql + torch.arange(ql, device="cuda")
        s = torch.where((pos[None] <= last[:, None])[:, None], s, -math.inf)
        o, l = _softmax_av(s, c[:, :VALUE])
        out[r:r + ql], lse[r:r + ql] = o.to(torch.bfloat16), l
        r += ql
    return out, lse


def _plain_prefill(st):
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    h, r, k0 = st["q"].shape[1], 0, 0
    for n in st["lens"]:
        nk = n + st["prefix"]
        pe = st["k_pe"][k0:k0 + nk].float()
        seen = torch.arange(nk, device="cuda")[None] <= nk - n + torch.arange(n, device="cuda")[:, None]
        step = max(1, (1 << 29) // (n * nk))
        for h0 in range(0, h, step):
            hs = slice(h0, min(h, h0 + step))
            q = st["q"][r:r + n, hs].float().transpose(0, 1)
            k = st["k_nope"][k0:k0 + nk, hs].float().transpose(0, 1)
            v = st["v"][k0:k0 + nk, hs].float().transpose(0, 1)
            s = (q[..., :NOPE] @ k.transpose(1, 2) + q[..., NOPE:] @ pe.t()) * SCALE
            if st["causal"]:
                s = torch.where(seen, s, -math.inf)
            o, l = _softmax_av(s, v)
            out[r:r + n, hs] = o.transpose(0, 1).to(torch.bfloat16)
            lse[r:r + n, hs] = l.t()
        r, k0 = r + n, k0 + nk
    return out, lse


def _plain_store(st):
    x = st["raw"].float()
    lat = x[:, :VALUE]
    lat = lat * (1.0 / torch.sqrt((lat * lat).mean(1, keepdim=True) + EPS)) * st["weight"]
    c, s = st["cs"][st["pos"]].chunk(2, 1)
    rope = x[:, VALUE:]
    if st["interleaved"]:
        a, b = rope[:, 0::2], rope[:, 1::2]
        rope = torch.stack([a * c - b * s, b * c + a * s], 2).reshape(-1, ROPE)
    else:
        a, b = rope.chunk(2, 1)
        rope = torch.cat([a * c - b * s, b * c + a * s], 1)
    latent = torch.cat([lat, rope], 1).to(torch.bfloat16)
    st["latent"].copy_(latent)
    keep = st["slots"] >= 0
    st["pool"].view(-1, LATENT)[st["slots"][keep]] = latent[keep]
    return st["pool"], st["latent"]


def _plain_verify(st):
    target, draft, x = st["target"], st["draft"], st["tokens"].long()
    cu = st["cu_q"].long()
    rows, v = target.shape
    row = torch.arange(rows, device="cuda")
    req = torch.searchsorted(cu, row, right=True) - 1
    has = (row != cu[req + 1] - 1) & (x >= 0) & (x < v)                     # the row has a draft after it
    xs = torch.where(has, x, torch.zeros_like(x))
    px = target[row, xs].double()
    qx = draft[row, xs].double() if draft is not None else torch.ones_like(px)
    taken = has & (st["u"].double() * qx < px)
    first = torch.full_like(cu[:-1], rows).scatter_reduce(0, req, torch.where(taken, rows, row), "amin")
    p = target[first].double()
    if draft is not None:
        left = (p - draft[first].double()).clamp_min(0.0)
    else:
        left = p.scatter(1, xs[first][:, None], 0.0)
    use = has[first][:, None] & (left.sum(1, keepdim=True) > 0)
    w = torch.where(use, left, p)
    c = torch.cumsum(w, 1)
    t = st["u_sample"].double() * c[:, -1]
    tok = (c <= t[:, None]).sum(1).clamp_max(v - 1)
    out = torch.where(row < first[req], x, torch.where(row == first[req], tok[req], torch.full_like(x, -1)))
    return out.to(torch.int32), (first - cu[:-1]).to(torch.int32)


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 4e12:
        return None
    return {"decode": _exact_decode, "prefill": _exact_prefill, "store": _exact_store, "verify": _exact_verify}[
        case["op"]](prepare(case, seed), case)


def _attend(q, k, v, vis):
    """One head group: q [n, d], k [m, d], v [m, e] in 64 bits; row i sees the first vis[i] keys."""
    s = torch.einsum("nd,md->nm", q, k) * (1.0 / math.sqrt(192.0))
    s.masked_fill_(torch.arange(k.shape[0], device="cuda")[None, :] >= vis[:, None], -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.exp(s - torch.where(vis > 0, lse, torch.zeros_like(lse))[:, None])
    return torch.einsum("nm,me->ne", p, v), torch.where(vis > 0, lse, torch.full_like(lse, -math.inf))


def _exact_decode(st, case):
    h = case["heads"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    flat = st["pool"].view(-1, LATENT)
    row = 0
    for b, (n, ql) in enumerate(zip(st["lens"], st["q_lens"])):
        pos = torch.arange(n, device="cuda")
        c = flat[st["table"][b].long()[pos // PAGE] * PAGE + pos % PAGE].double()
        for j in range(ql):
            v = n - ql + j + 1
            if v > 0:
                vis = torch.full((h,), v, device="cuda")
                out[row], lse[row] = _attend(st["q"][row].double(), c[:v], c[:v, :VALUE], vis)
            row += 1
    return out, lse


def _exact_prefill(st, case):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
    for b in range(len(cu_q) - 1):
        ks = slice(cu_k[b], cu_k[b + 1])
        nk, nq = cu_k[b + 1] - cu_k[b], cu_q[b + 1] - cu_q[b]
        for h in range(case["heads"]):
            k = torch.cat([st["k_nope"][ks, h], st["k_pe"][ks]], 1).double()
            v = st["v"][ks, h].double()
            for i in range(0, nq, 2048):
                j = min(nq, i + 2048)
                end = nk - nq + j if case["causal"] else nk
                vis = nk - nq + 1 + torch.arange(i, j, device="cuda")
                if not case["causal"]:
                    vis = torch.full_like(vis, nk)
                rows = slice(cu_q[b] + i, cu_q[b] + j)
                out[rows, h], lse[rows, h] = _attend(st["q"][rows, h].double(), k[:end], v[:end], vis)
    return out, lse


def _exact_store(st, case):
    x = st["raw"].double()
    inv = torch.rsqrt(x[:, :VALUE].square().sum(1) / VALUE + EPS)
    y = torch.empty_like(x)
    y[:, :VALUE] = x[:, :VALUE] * inv[:, None] * st["weight"].double()
    turn = torch.complex(st["cs"][:, :32].double(), st["cs"][:, 32:].double())[st["pos"]]
    lo, hi = (slice(VALUE, None, 2), slice(VALUE + 1, None, 2)) if case["interleaved"] else (
        slice(VALUE, VALUE + 32), slice(VALUE + 32, None))
    z = torch.complex(x[:, lo].contiguous(), x[:, hi].contiguous()) * turn
    y[:, lo], y[:, hi] = z.real, z.imag
    pool = torch.zeros(st["pool"].shape, dtype=torch.float64, device="cuda")
    for t, slot in enumerate(st["slots"].tolist()):
        if slot >= 0:
            pool[slot // PAGE, slot % PAGE] = y[t]
    return pool, y


def _exact_verify(st, case):
    cu = st["cu_q"].tolist()
    toks, u, us = st["tokens"].tolist(), st["u"].tolist(), st["u_sample"].tolist()
    out, acc = [-1] * cu[-1], []
    for b in range(len(cu) - 1):
        j, end = cu[b], cu[b + 1] - 1
        while j < end:
            p = float(st["target"][j, toks[j]])
            q = float(st["draft"][j, toks[j]]) if st["draft"] is not None else 1.0
            if not u[j] * q < p:
                break
            out[j] = toks[j]
            j += 1
        w = st["target"][j].double()
        if j < end:
            if st["draft"] is not None:
                rest = torch.relu(w - st["draft"][j].double())
            else:
                rest = w.clone()
                rest[toks[j]] = 0.0
            if bool(rest.any()):
                w = rest
        c = torch.cumsum(w, 0)
        out[j] = min(int(torch.searchsorted(c, us[b] * c[-1:], right=True)), case["vocab"] - 1)
        acc.append(j - cu[b])
    return _i32(out), _i32(acc)
