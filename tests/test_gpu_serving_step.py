"""GPU tests of the calls around a serving step against plain definitions: the step's tables, the attention behind
shared prefixes, the sampling, and a run of them together.  Bounds: dense_mla_ref (attention), serving_step_ref (sampling)."""
import math
import random

import numpy as np
import pytest
import torch

import dense_mla_ref
import serving_step_ref as ref
from deepseek_sparse_attention_paged_gb300 import capi

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _f32(v):
    return torch.tensor(v, dtype=torch.float32, device="cuda")


def _cum(ns):
    c = [0]
    for n in ns:
        c.append(c[-1] + n)
    return c


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- step tables

def _run_tables(cached, q, counts, keep, table, num_pages, stack, have, T, stream=None):
    """The call's outputs as lists, like the definition's; table and stack are updated."""
    B = len(cached)
    tb, st = _i32(table), _i32(stack)
    seq, co, ho, cu = _i32([7] * B), _i32([7] * B), _i32([7]), _i32([7] * (B + 1))
    pos = torch.full((T,), 7, dtype=torch.int64, device="cuda")
    slots = torch.full((T,), 7, dtype=torch.int64, device="cuda")
    err = _err()
    capi.dsa_step_tables(_i32(cached), _i32(q), _i32(counts), tb, num_pages, st, _i32([have]), seq, co, ho, cu, pos, slots,
                         keep_pages=None if keep is None else _i32(keep), dev_err=err)
    table[:], stack[:] = tb.tolist(), st.tolist()
    return seq.tolist(), co.tolist(), ho.item(), cu.tolist(), pos.tolist(), slots.tolist(), err.item()


def _check_tables(cached, q, counts, keep, table, num_pages, stack, have, T):
    want_table, want_stack = [list(r) for r in table], list(stack)
    want = ref.tables(cached, q, counts, keep or [0] * len(q), want_table, num_pages, want_stack, have, T)
    got = _run_tables(cached, q, counts, keep, table, num_pages, stack, have, T)
    assert got == want
    assert table == want_table and stack == want_stack


def _random_tables(B, new, ctx, seed, ended, keep, slack=10, max_pages=None):
    rng = random.Random(seed)
    cached = [rng.randrange(ctx + 1) for _ in range(B)]
    q = [-1 if rng.random() < ended else rng.randrange(new + 1) for _ in range(B)]
    counts = [(c + 63) // 64 + rng.choice([0, 0, 0, 1]) for c in cached]
    kept = [rng.randrange(c + 1) for c in counts] if keep else None
    need = [max(m, (c + max(0, n) + 63) // 64) for c, n, m in zip(cached, q, counts)]
    width = max_pages or max(1, max(need))
    num_pages = sum(need) + slack
    perm = list(range(num_pages))
    rng.shuffle(perm)
    table, at = [], 0
    for m in counts:
        table.append((perm[at:at + m] + [-1] * width)[:width])
        at += m
    free = perm[at:]
    return cached, q, counts, kept, table, num_pages, free + [-1] * (num_pages - len(free)), len(free)


@pytest.mark.parametrize("B,new,ctx,ended,keep,pad", [
    (1, 1, 0, 0.0, False, 0), (1, 1, 63, 0.0, False, 0), (1, 1, 64, 0.0, True, 3), (1, 0, 100, 1.0, False, 2),
    (2, 200, 300, 0.5, True, 1), (31, 5, 1000, 0.2, True, 0), (511, 3, 700, 0.1, False, 100), (512, 1, 200, 0.0, True, 0),
    (513, 2, 64, 0.9, True, 7), (1025, 130, 130, 0.3, True, 0), (3000, 4, 256, 0.1, True, 513), (40, 9000, 4096, 0.1, True, 5)])
def test_tables(B, new, ctx, ended, keep, pad):
    for seed in range(3):
        case = _random_tables(B, new, ctx, seed, ended, keep)
        _check_tables(*case, sum(max(0, n) for n in case[1]) + pad)


def test_tables_largest_batch():
    case = _random_tables(16384, 2, 70, 5, 0.3, True)
    _check_tables(*case, sum(max(0, n) for n in case[1]))


def test_tables_without_rows():
    """T = 0: no request gets tokens, pages still move."""
    case = list(_random_tables(20, 0, 500, 6, 0.5, True))
    _check_tables(*case, 0)


def test_tables_take_what_is_given_back():
    """An empty stack: everything that is taken was given back in the same call; the whole stack turned over."""
    cached, q = [640, 64 * 9, 0, 0, 0], [-1, -1, 300, 640, 64]
    table = [list(range(0, 10)), list(range(10, 20)), [-1] * 10, [-1] * 10, [-1] * 10]
    _check_tables(cached, q, [10, 9, 0, 0, 0], [0, 1, 0, 0, 0], table, 20, [-1] * 20, 0, 1010)


def test_tables_run_out():
    """Fewer pages than needed: later pages in order get none."""
    for have in (0, 1, 3, 8):
        table = [[-1] * 6 for _ in range(4)]
        _check_tables([0, 0, 10, 0], [130, 64, 60, 300], [0, 0, 0, 0], None, table, 9, list(range(9)), have, 560)


def test_tables_out_of_range():
    """Rows cut at T, tokens past the table, counts and lengths out of range, a stack that overflows, bad page ids."""
    t = lambda: [[0, 1], [2, 3], [-1, -1]]
    _check_tables([0, 100, 5], [100, 28, 7], [2, 2, 0], None, t(), 8, [4, 5, 6, 7, -1, -1, -1, -1], 4, 110)
    _check_tables([100, 60, 0], [60, 70, 200], [2, 2, 0], None, t(), 8, [4, 5, 6, 7, -1, -1, -1, -1], 4, 330)
    _check_tables([-5, 3, -2 ** 31], [1, 1, 1], [9, -3, 2 ** 31 - 1], [7, -7, 1], t(), 8, [4, 5, 6, 7, -1, -1, -1, -1], 4, 3)
    _check_tables([100, 100, 0], [-1, -2 ** 31, 1], [2, 2, 0], None, t(), 5, [4, 4, 4, 4, 4], 3, 1)
    _check_tables([0, 0, 0], [64, 64, 64], [0, 0, 0], None, t(), 8, [9, -4, 5, -1, -1, -1, -1, -1], 3, 192)
    _check_tables([64, 70, 0], [1, 1, 1], [2, 2, 0], None, [[0, 99], [2, -1], [-1, -1]], 8, [4, 5, 6, 7, -1, -1, -1, -1], 4, 3)
    _check_tables([1, 1, 1], [1, 1, 1], [1, 1, 1], None, t(), 8, [4] * 8, 1000, 3)
    _check_tables([1, 1, 1], [1, 1, 1], [1, 1, 1], None, t(), 8, [4] * 8, -1000, 3)
    _check_tables([2 ** 31 - 1, 0, 0], [2 ** 31 - 1, 0, 0], [2, 0, 0], None, t(), 8, [4] * 8, 4, 0)


def test_tables_lengths_pass_32_bits():
    """2^31 - 1 cached tokens and one more: the length stays at the largest number, the slot is -1."""
    got = _run_tables([2 ** 31 - 1], [1], [2], None, [[0, 1]], 4, [2, 3, -1, -1], 2, 1)
    assert got == ([2 ** 31 - 1], [2], 2, [0, 1], [2 ** 31 - 1], [-1], ref.INDEX_RANGE)


def test_tables_captured_steps():
    """Two steps with swapped buffers in one graph, replayed: a loop of decode steps on one request batch."""
    B, num_pages, width = 70, 2000, 24
    rng = random.Random(8)
    cached = [rng.randrange(600) for _ in range(B)]
    counts = [(c + 63) // 64 for c in cached]
    perm = list(range(num_pages))
    rng.shuffle(perm)
    table, at = [], 0
    for m in counts:
        table.append(perm[at:at + m] + [-1] * (width - m))
        at += m
    stack, have = perm[at:] + [-1] * at, num_pages - at
    q = [rng.choice([0, 1, 2, 40]) for _ in range(B)]
    T = sum(q) + 5
    lens = [_i32(cached), _i32(cached)]
    cnt = [_i32(counts), _i32(counts)]
    top = [_i32([have]), _i32([have])]
    tb, st, qt, cu, err = _i32(table), _i32(stack), _i32(q), _i32([0] * (B + 1)), _err()
    pos = [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2)]
    slots = [torch.zeros(T, dtype=torch.int64, device="cuda") for _ in range(2)]

    def step(i):
        capi.dsa_step_tables(lens[i], qt, cnt[i], tb, num_pages, st, top[i], lens[1 - i], cnt[1 - i], top[1 - i], cu, pos[i],
                             slots[i], dev_err=err)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
        step(1)
    for _ in range(2):
        graph.replay()
        for i in range(2):
            cached, counts, have, _, p, s, bits = ref.tables(cached, q, counts, [0] * B, table, num_pages, stack, have, T)
            assert bits == 0 and pos[i].tolist() == p and slots[i].tolist() == s
        assert lens[0].tolist() == cached and cnt[0].tolist() == counts and top[0].item() == have
        assert tb.tolist() == table and st.tolist() == stack
    assert err.item() == 0


# ---------------------------------------------------------------- shared prefixes

def _shared_inputs(groups, H, seed, alone=0, stale=None):
    """groups: (prefix, [(own tokens behind the prefix, q_len), ..]); a request's length may end inside the prefix (own
    < 0).  `alone` requests outside all groups follow.  Cache rows past a request's length hold `stale`."""
    g = torch.Generator().manual_seed(seed)
    lens, q_lens, cu_group, shared, tables = [], [], [0], [], []
    page = 0

    def take(n):
        nonlocal page
        page += n
        return list(range(page - n, page))

    fill = []
    for prefix, reqs in groups:
        common = take(prefix // 64)
        fill += [(p, 64) for p in common]
        for own, ql in reqs:
            n = max(0, prefix + own)
            rest = take(max(0, (n + 63) // 64 - len(common)))
            fill += [(p, min(64, n - (len(common) + i) * 64)) for i, p in enumerate(rest)]
            tables.append(common + rest)
            lens.append(n)
            q_lens.append(ql)
        cu_group.append(len(lens))
        shared.append(prefix)
    for _ in range(alone):
        n = 1 + int(torch.randint(0, 300, (1,), generator=g))
        rest = take((n + 63) // 64)
        fill += [(p, min(64, n - i * 64)) for i, p in enumerate(rest)]
        tables.append(rest)
        lens.append(n)
        q_lens.append(1)
    total = page + 2
    perm = torch.randperm(total, generator=g)
    pool = torch.randn(total, 64, 576, generator=g).to(torch.bfloat16)
    if stale is not None:
        for p, n in fill:
            pool[perm[p], n:] = stale
        pool[perm[page:]] = stale
    width = max(1, max(len(t) for t in tables))
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    for b, t in enumerate(tables):
        table[b, :len(t)] = perm[t].to(torch.int32) if t else torch.zeros(0, dtype=torch.int32)
    q = torch.randn(sum(q_lens), H, 576, generator=g).to(torch.bfloat16)
    return q, pool, table, lens, q_lens, cu_group, shared


def _run_shared(inp, T=None, stream=None, ws=None, cu_group=None, shared=None):
    q, pool, table, lens, q_lens, cg, sh = inp
    T = T or q.shape[0]
    H = q.shape[1]
    full = torch.randn(T, H, 576).to(torch.bfloat16)
    full[:q.shape[0]] = q
    out = torch.full((T, H, 512), 9.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 9.0, device="cuda")
    err = _err()
    if ws is None:
        ws = torch.full((max(16, capi.dsa_dense_mla_decode_shared_workspace_size(T, H)),), 255, dtype=torch.uint8, device="cuda")
    capi.dsa_dense_mla_decode_shared(full.cuda(), pool.cuda(), table.cuda(), _i32(lens), _i32(_cum(q_lens)),
                                     _i32(cg if cu_group is None else cu_group), _i32(sh if shared is None else shared), SCALE,
                                     out, ws, lse=lse, dev_err=err)
    return out, lse, err.item()


def _check_shared(inp, **kw):
    out, lse, err = _run_shared(inp, **kw)
    q, pool, table, lens, q_lens, _, _ = inp
    n = q.shape[0]
    want = dense_mla_ref.decode(q.cuda(), pool.cuda(), table.cuda(), lens, q_lens, SCALE)
    dense_mla_ref.check(out[:n], lse[:n], want)
    assert bool((out[n:] == 9.0).all()) and bool((lse[n:] == 9.0).all())
    assert err == 0


@pytest.mark.parametrize("groups,H", [
    ([(64, [(1, 1)])], 16),
    ([(64, [(1, 1), (1, 1)])], 128),
    ([(128, [(5, 1)] * 9)], 16),
    ([(1024, [(1, 1), (64, 1), (65, 1), (200, 1)])], 16),
    ([(320, [(7, 2), (130, 3), (1, 1), (64, 4)]), (64, [(1, 1)] * 3), (0, [(90, 2), (1, 1)])], 32),
    ([(0, [(3, 1), (400, 1)]), (2048, [(10, 1)] * 17), (0, []), (192, [(1000, 2)])], 64),
    ([(4096, [(3 * i, 1 + i % 3) for i in range(1, 40)])], 16),
    ([(20000, [(100 + i, 1) for i in range(12)])], 128),
    ([(64 * 50, [(i, 1) for i in range(1, 101)]), (64 * 7, [(0 + i, 5) for i in range(5, 30)])], 16),
])
def test_shared(groups, H):
    _check_shared(_shared_inputs(groups, H, 11), T=sum(q for _, r in groups for _, q in r) + 3)


def test_shared_requests_outside_groups():
    _check_shared(_shared_inputs([(640, [(9, 1)] * 5), (128, [(3, 2)] * 2)], 32, 12, alone=4))


def test_shared_short_and_idle_requests():
    """Requests that end inside their group's prefix see their own length of it; idle ones (length 0) nothing; requests
    without rows among the others; more query tokens than cached ones."""
    groups = [(640, [(20, 1), (-100, 1), (-640, 1), (30, 0), (-576, 2), (-639, 3), (0, 1), (1, 4)]), (64, [(-64, 2), (-64, 1)]),
              (128, [(5, 0), (7, 0)])]
    _check_shared(_shared_inputs(groups, 16, 13))
    _check_shared(_shared_inputs(groups, 128, 14))


def test_shared_prefix_that_ends_inside_a_page():
    """The part of a prefix past its last whole page is read per request."""
    inp = _shared_inputs([(640, [(9, 1)] * 5)], 16, 15)
    _check_shared(inp, shared=[640 - 1])
    _check_shared(inp, shared=[63])
    _check_shared(inp, shared=[-5])
    _check_shared(inp, cu_group=[0], shared=[])
    _check_shared(inp, cu_group=[2, 4], shared=[640])


def test_shared_stale_rows():
    """Cache rows past the last visible position hold NaN."""
    _check_shared(_shared_inputs([(320, [(1, 1), (63, 1), (64, 1), (65, 2), (100, 3)]), (0, [(10, 1)])], 16, 16, stale=math.nan))


@pytest.mark.parametrize("n_groups", [1, 70])
def test_shared_prefix_that_no_request_sees_whole(n_groups):
    """What lies behind the longest request of a group is not read: pages that are not there, rows that hold NaN."""
    lens = [540, 100, 448, 541, 1]
    q, pool, table, seq, q_lens, cu_group, shared = _shared_inputs([(1024, [(n - 1024, 1) for n in lens])] * n_groups, 16, 19)
    for g in range(n_groups):
        first = table[5 * g]
        pool[first[8], 541 - 512:] = math.nan
        table[5 * g:5 * g + 5, 9:] = -1
    _check_shared((q, pool, table, seq, q_lens, cu_group, shared))


def test_shared_equals_the_plain_call_on_copied_pages():
    """Pages are taken from the first request's row: other rows' entries below the prefix are not read."""
    inp = list(_shared_inputs([(256, [(9, 1)] * 6)], 64, 17))
    want = dense_mla_ref.decode(inp[0].cuda(), inp[1].cuda(), inp[2].cuda(), inp[3], inp[4], SCALE)
    inp[2] = inp[2].clone()
    inp[2][1:, :4] = -7
    out, lse, err = _run_shared(tuple(inp))
    dense_mla_ref.check(out, lse, want)
    assert err == 0


def test_shared_bad_pages_and_ranges():
    inp = list(_shared_inputs([(256, [(9, 1)] * 6)], 16, 18))
    table = inp[2].clone()
    table[:, 1] = 10 ** 6                       # in the prefix
    table[3, 4] = -1                            # behind it
    inp[2] = table
    out, lse, err = _run_shared(tuple(inp))
    want = dense_mla_ref.decode(inp[0].cuda(), inp[1].cuda(), table.cuda(), inp[3], inp[4], SCALE)
    dense_mla_ref.check(out, lse, want)
    assert err == capi.DSA_DEVERR_PAGE_RANGE
    # ranges that leave the batch are cut; a prefix past the table is cut to it
    inp = _shared_inputs([(256, [(9, 1)] * 6)], 16, 19)
    want = dense_mla_ref.decode(inp[0].cuda(), inp[1].cuda(), inp[2].cuda(), inp[3], inp[4], SCALE)
    for cg, sh in (([-2, 9], [256]), ([0, 100], [256])):
        out, lse, err = _run_shared(inp, cu_group=cg, shared=sh)
        dense_mla_ref.check(out, lse, want)
        assert err == capi.DSA_DEVERR_INDEX_RANGE
    _, _, err = _run_shared(inp, cu_group=[0, 6], shared=[10 ** 6])
    assert err & capi.DSA_DEVERR_INDEX_RANGE


def test_shared_streams_graph_and_dirty_workspace():
    """The same workspace for calls of different batches, on a side stream, captured and replayed on other inputs."""
    inp = _shared_inputs([(1280, [(30 + i, 1) for i in range(20)])], 16, 20)
    other = _shared_inputs([(64, [(300, 2)] * 3), (640, [(1, 1)] * 4)], 16, 21)
    T = max(inp[0].shape[0], other[0].shape[0])
    ws = torch.full((capi.dsa_dense_mla_decode_shared_workspace_size(T, 16),), 127, dtype=torch.uint8, device="cuda")
    for x in (inp, other, inp):
        _check_shared(x, ws=ws)
    q, pool, table, lens, q_lens, cg, sh = inp
    dq, dp, dt, dl, dc, dg, ds = (q.cuda(), pool.cuda(), table.cuda(), _i32(lens), _i32(_cum(q_lens)), _i32(cg), _i32(sh))
    out, lse = torch.zeros(q.shape[0], 16, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(q.shape[0], 16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        capi.dsa_dense_mla_decode_shared(dq, dp, dt, dl, dc, dg, ds, SCALE, out, ws, lse=lse)
    for seed in (1, 2):
        fresh = torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        dq.copy_(fresh)
        graph.replay()
        dense_mla_ref.check(out, lse, dense_mla_ref.decode(dq, dp, dt, lens, q_lens, SCALE))


# ---------------------------------------------------------------- sampling

def _logits(R, V, seed, bf16, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, V + pad, generator=g) * 2.0
    top = torch.randint(0, V, (R, 24), generator=g)
    x.scatter_(1, top, 7.0 + 3.0 * torch.randn(R, 24, generator=g))
    return x.to(torch.bfloat16) if bf16 else x


def _run_sample(x, V, u, temperature=None, top_k=None, top_p=None, min_p=None, probs=True, pad_p=0):
    R = x.shape[0]
    tokens = _i32([-5] * R)
    buf = torch.full((R, V + pad_p), 3.0, device="cuda") if probs else None
    err = _err()
    f = lambda v: None if v is None else _f32(v)
    capi.dsa_sample_tokens(x.cuda()[:, :V], _f32(u), tokens, f(temperature), None if top_k is None else _i32(top_k), f(top_p),
                           f(min_p), probs=None if buf is None else buf[:, :V], dev_err=err)
    if buf is not None:
        assert bool((buf[:, V:] == 3.0).all())
    return tokens.tolist(), None if buf is None else buf[:, :V].double().cpu().numpy(), err.item()


def _check_sample(x, V, u, temperature=None, top_k=None, top_p=None, min_p=None, probs=True, pad_p=0):
    got, p, err = _run_sample(x, V, u, temperature, top_k, top_p, min_p, probs, pad_p)
    none = 0
    for r in range(x.shape[0]):
        row = x[r, :V].double().numpy()
        pick = lambda v, d: d if v is None else float(np.float32(v[r]))
        token, want = ref.sample(row, pick(temperature, 1.0), 0 if top_k is None else top_k[r], pick(top_p, 1.0),
                                 pick(min_p, 0.0), float(np.float32(u[r])))
        assert got[r] == token, (r, got[r], token)
        none += token < 0
        if probs:
            e = np.abs(p[r] - want)
            assert np.all(e <= ref.round_probs_bound(want)), (r, float((e / ref.round_probs_bound(want)).max()))
    assert err == (capi.DSA_DEVERR_PROB if none else 0)


SETTINGS = [dict(), dict(temperature=0.0), dict(top_k=1), dict(top_k=50), dict(top_k=50, top_p=0.95), dict(top_k=700),
            dict(top_k=1000, top_p=0.99, min_p=0.001), dict(top_k=3000), dict(top_k=3000, top_p=0.9), dict(top_p=0.9),
            dict(top_p=0.99, temperature=0.7), dict(top_p=0.999, temperature=1.5), dict(top_p=0.0), dict(top_p=1e-6),
            dict(min_p=0.05), dict(min_p=1.0), dict(min_p=1e-9), dict(min_p=0.02, top_p=0.8, temperature=1.3),
            dict(temperature=0.05, top_k=40, top_p=0.9), dict(temperature=30.0, top_p=0.5), dict(temperature=100.0)]


@pytest.mark.parametrize("V,bf16,pad", [(1, False, 0), (2, True, 1), (7, False, 0), (33, True, 0), (1000, False, 3), (1001, True, 0),
                                        (2048, False, 0), (2049, True, 5), (4100, False, 1), (8191, True, 2), (32000, True, 0),
                                        (32001, False, 3)])
def test_sample_every_setting(V, bf16, pad):
    """One row per setting, and each setting with four random numbers."""
    R = 4 * len(SETTINGS)
    x = _logits(R, V, 100 + V, bf16, pad)
    rows = [s for s in SETTINGS for _ in range(4)]
    get = lambda k, d: [s.get(k, d) for s in rows]
    u = torch.rand(R, generator=torch.Generator().manual_seed(V)).tolist()
    _check_sample(x, V, u, get("temperature", 1.0), get("top_k", 0), get("top_p", 1.0), get("min_p", 0.0), pad_p=pad)


@pytest.mark.parametrize("V,bf16,kw", [(100003, True, dict(top_p=0.95)), (131072, False, dict(top_k=50, top_p=0.95)),
                                       (160000, False, dict(top_p=0.99)), (262144, False, dict()), (262144, False, dict(top_p=0.9)),
                                       (262143, True, dict(top_k=1000, min_p=0.01)), (262144, True, dict(top_k=5000, top_p=0.9))])
def test_sample_large_vocabularies(V, bf16, kw):
    R = 6
    x = _logits(R, V, V, bf16, 5)
    u = torch.rand(R, generator=torch.Generator().manual_seed(V + 1)).tolist()
    full = {k: [v] * R for k, v in kw.items()}
    _check_sample(x, V, u, **full)
    _check_sample(x, V, u, probs=False, **full)


def test_sample_defaults():
    """Settings that are not given: temperature 1, nothing filtered; as with neutral values."""
    x = _logits(5, 3001, 3, False)
    u = [0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24]
    _check_sample(x, 3001, u)
    a = _run_sample(x, 3001, u)
    b = _run_sample(x, 3001, u, [1.0] * 5, [0] * 5, [1.0] * 5, [0.0] * 5)
    assert a[0] == b[0] and np.array_equal(a[1], b[1])
    nan = [math.nan] * 5
    c = _run_sample(x, 3001, u, [1.0] * 5, [-3] * 5, nan, nan)
    assert a[0] == c[0] and np.array_equal(a[1], c[1])
    assert _run_sample(x, 3001, u, nan)[0] == x.argmax(1).tolist()


@pytest.mark.parametrize("V", [5, 3000, 40000])
def test_sample_ties(V):
    """Equal logits: the order is the index's, in every filter and at every size (more ties than the list holds)."""
    x = torch.full((8, V), 1.25)
    x[4:] = (torch.arange(V) % 3).float()                 # three values in turn
    x[5, ::2] = -0.0
    x[5, 1::2] = 0.0
    u = [0.0, 0.3, 0.7, 0.999, 0.1, 0.5, 0.9, 0.6]
    k = [0, 3, V // 2, V - 1, 0, V // 2 + 1, 2, V - 1]
    p = [0.5, 0.75, 1.0, 0.25, 1.0, 1.0, 0.9, 1.0]
    _check_sample(x, V, u, top_k=k, top_p=p)
    _check_sample(x, V, u, top_k=[0] * 8, top_p=[0.5, 0.25, 0.125, 1.0, 1.0, 0.5, 1.0, 1.0])
    assert _run_sample(x, V, u, temperature=[0.0] * 8)[0] == [0, 0, 0, 0, 2, 0, 2, 2]


def test_sample_masked_rows():
    """Masks of -infinity and of the type's lowest value; one entry left; none left; NaN; +infinity."""
    V = 5000
    g = torch.Generator().manual_seed(4)
    for bf16 in (False, True):
        low = torch.finfo(torch.bfloat16 if bf16 else torch.float32).min
        x = _logits(9, V, 5, bf16)
        off = torch.rand(9, V, generator=g) < 0.99
        x[0][off[0]] = -math.inf
        x[1][off[1]] = low
        x[2] = -math.inf
        x[2, 4321] = -3.0
        x[3] = -math.inf
        x[4][off[4]] = math.nan
        x[5] = math.nan
        x[6] = low
        x[7, 2:] = low
        x[8] = -math.inf
        x[8, 17:20] = -100.0
        u = [0.1, 0.2, 0.9, 0.5, 0.6, 0.5, 0.7, 0.4, 0.99]
        for kw in ({}, {"top_k": [20] * 9}, {"top_p": [0.9] * 9}, {"top_k": [2000] * 9}, {"min_p": [0.1] * 9},
                   {"temperature": [0.0] * 9}, {"temperature": [1e-30] * 9}, {"temperature": [0.2] * 9, "top_k": [60] * 9}):
            _check_sample(x, V, u, **kw)
    x = torch.zeros(3, V)
    x[0, 100] = x[0, 2000] = math.inf
    x[1, 3] = math.inf
    x[2] = math.inf
    got, p, err = _run_sample(x, V, [0.6, 0.6, 0.5])
    assert got == [2000, 3, 2500] and err == 0 and p[0, 100] == 0.5 and p[1, 3] == 1.0 and np.all(p[2] == np.float32(1 / V))


@pytest.mark.parametrize("kind", ["whole", "halves", "tiny", "low", "high", "mixed", "one", "two"])
def test_sample_bf16_values(kind):
    """bf16 rows with top-p: many equal values (borders within them, in any part of the row), numbers next to 0, far below
    it and past 128, few values."""
    R, V = 8, 20003
    g = torch.Generator().manual_seed(len(kind))
    x = 2.0 * torch.randn(R, V, generator=g)
    if kind == "whole":
        x = x.round()
    elif kind == "halves":
        x = (2 * x).round() / 2 - 6.0
    elif kind == "tiny":
        x = x * 1e-4
        x[:, 5000:5003] = 1.0
    elif kind == "low":
        x = 8 * x - 130.0
    elif kind == "high":
        x = x + 128.0
    elif kind == "mixed":
        x[:, ::2] = x[:, ::2] * 1e-3
        x[:, 1::7] = -500.0
    elif kind == "one":
        x[:] = 3.0
    elif kind == "two":
        x[:] = -1.0
        x[:, 11::3] = 2.0
    x = x.to(torch.bfloat16)
    u = torch.rand(R, generator=g).tolist()
    p = [0.5, 0.9, 0.99, 0.3, 0.75, 0.999, 0.21, 0.95]
    t = [1.0, 0.7, 1.5, 1.0, 3.0, 20.0, 0.1, 1.0]
    _check_sample(x, V, u, top_p=p)
    _check_sample(x, V, u, top_p=p, temperature=t)
    _check_sample(x, V, u, top_p=p, min_p=[0.0, 0.1, 0.5, 0.9, 1.0, 0.3, 0.01, 0.6])
    _check_sample(x[:, 1:], V - 1, u, top_p=p, probs=False)


def test_sample_random_numbers_at_the_ends():
    """u = 0: the first kept entry with weight; u of 1 or more, infinite: the last; negative, NaN: as 0."""
    x = torch.tensor([[-200.0, 1.0, 1.0, 1.0, 3.0, 1.0, -200.0]] * 7)
    u = [0.0, 1.0, 2.0, 1e30, math.inf, -1.0, math.nan]
    for kw in ({}, {"top_k": [6] * 7}, {"top_p": [1.0 - 2.0 ** -24] * 7}):
        assert _run_sample(x, 7, u, **kw)[0] == [1, 5, 5, 5, 5, 1, 1]


def test_sample_extreme_temperatures():
    x = _logits(6, 3000, 6, False)
    t = [1e-45, 1e-38, 3e38, math.inf, -1.0, 1e-4]
    u = [0.3, 0.9, 0.5, 0.5, 0.5, 0.2]
    got, p, err = _run_sample(x, 3000, u, t)
    top = x.argmax(1).tolist()
    assert err == 0 and got[0] == top[0] and got[1] == top[1] and got[4] == top[4] and got[5] == top[5]
    assert got[2] == 1500 and got[3] == 1500 and np.allclose(p[2:4], 1 / 3000, rtol=1e-6)


def test_sample_head_heavy_vocabulary():
    """All large logits at the front (one CTA's share), and more than the list holds within one bin."""
    V = 60000
    x = torch.full((4, V), -5.0)
    g = torch.Generator().manual_seed(9)
    x[:2, :3000] = 4.0 + torch.rand(2, 3000, generator=g)
    x[2:] = 2.0 + 0.01 * torch.rand(2, V, generator=g)
    u = [0.2, 0.8, 0.4, 0.6]
    for kw in ({"top_k": [900] * 4}, {"top_p": [0.6] * 4}, {"top_k": [1024] * 4, "top_p": [0.5] * 4}, {"top_k": [30000] * 4}):
        _check_sample(x, V, u, **kw)


def test_sample_many_rows_strides_and_streams():
    """More rows than fit the GPU at once, odd strides (rows on every alignment), a side stream, replays on other inputs."""
    for bf16 in (False, True):
        R, V = 700, 3003
        x = _logits(R, V, 10, bf16, 6 if bf16 else 2)
        u = torch.rand(R, generator=torch.Generator().manual_seed(2)).tolist()
        _check_sample(x, V, u, top_k=[30] * R, top_p=[0.9] * R, pad_p=1)
        dx, du, tok = x.cuda(), _f32(u), _i32([0] * R)
        tp = _f32([0.9] * R)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            capi.dsa_sample_tokens(dx[:, 1:1 + V], du, tok, top_p=tp)
        for seed in (11, 12):
            y = _logits(R, V, seed, bf16, 6 if bf16 else 2)
            dx.copy_(y)
            graph.replay()
            want = [ref.sample(y[r, 1:1 + V].double().numpy(), 1.0, 0, float(np.float32(0.9)), 0.0, float(np.float32(u[r])))[0]
                    for r in range(R)]
            assert tok.tolist() == want


def test_sample_refuses_probs_over_logits():
    x = torch.zeros(2, 64, device="cuda")
    with pytest.raises(capi.DSAError):
        capi.dsa_sample_tokens(x, _f32([0.5, 0.5]), _i32([0, 0]), probs=x)


# ---------------------------------------------------------------- a run of them together

def test_a_serving_step():
    """Tables, store, attention behind a shared prefix, logits, the filtered distribution, verification of drafts and
    the draw, on one stream without a synchronisation in between; a second step follows from the first's buffers."""
    g = torch.Generator().manual_seed(30)
    B, H, V, prefix, num_pages, width = 6, 16, 5003, 192, 80, 12
    own = [5, 60, 64, 1, 130, 20]
    q = [3, 1, 2, 1, -1, 3]
    shared = prefix // 64
    counts = [shared + (n + 63) // 64 for n in own]
    perm = torch.randperm(num_pages, generator=g).tolist()
    table, at = [], shared
    for m in counts:
        table.append(perm[:shared] + perm[at:at + m - shared] + [-1] * (width - m))
        at += m - shared
    stack, have = perm[at:] + [-1] * at, num_pages - at
    T = sum(max(0, n) for n in q) + 2
    cached = [prefix + n for n in own]
    pool = torch.randn(num_pages, 64, 576, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(T, 576, generator=g).to(torch.bfloat16).cuda()
    qs = torch.randn(T, H, 576, generator=g).to(torch.bfloat16).cuda()
    head = (torch.randn(H * 512, V, generator=g) / 30).cuda()
    norm = torch.ones(512, device="cuda")
    ang = torch.rand(1000, 32, generator=g) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).cuda()
    u = torch.rand(3, T, generator=g).cuda()
    lens, cnt, top = [_i32(cached), _i32([0] * B)], [_i32(counts), _i32([0] * B)], [_i32([have]), _i32([0])]
    tb, st, cu, err, qt = _i32(table), _i32(stack), _i32([0] * (B + 1)), _err(), _i32(q)
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    slots = torch.zeros(T, dtype=torch.int64, device="cuda")
    out = torch.zeros(T, H, 512, dtype=torch.bfloat16, device="cuda")
    probs = torch.zeros(T, V, device="cuda")
    tokens, drafts, res, acc = _i32([0] * T), _i32([0] * T), _i32([0] * T), _i32([0] * B)
    ws = torch.empty(capi.dsa_dense_mla_decode_shared_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    settings = dict(temperature=_f32([0.8] * T), top_k=_i32([40] * T), top_p=_f32([0.9] * T))

    def step(i):
        capi.dsa_step_tables(lens[i], qt, cnt[i], tb, num_pages, st, top[i], lens[1 - i], cnt[1 - i], top[1 - i], cu, pos, slots,
                             keep_pages=_i32([shared] * B), dev_err=err)
        capi.dsa_store_latent_prologue(kv, norm, 1e-6, cs, pos, slots, pool, dev_err=err)
        capi.dsa_dense_mla_decode_shared(qs, pool, tb, lens[1 - i], cu, _i32([0, B]), _i32([prefix]), SCALE, out, ws, dev_err=err)
        logits = out.view(T, -1).float() @ head
        capi.dsa_sample_tokens(logits, u[0], tokens, probs=probs, dev_err=err, **settings)
        drafts.copy_(tokens)
        capi.dsa_verify_drafts(probs, drafts, cu, u[1], u[2, :B].contiguous(), res, acc, dev_err=err)
        return logits

    for i in range(2):
        want = ref.tables(cached, q, counts, [shared] * B, table, num_pages, stack, have, T)
        logits = step(i)
        cached, counts, have = want[0], want[1], want[2]
        assert lens[1 - i].tolist() == cached and cnt[1 - i].tolist() == counts and top[1 - i].item() == have
        assert tb.tolist() == table and st.tolist() == stack and pos.tolist() == want[4] and slots.tolist() == want[5]
        n = want[3][-1]
        dense_mla_ref.check(out[:n], None, dense_mla_ref.decode(qs[:n], pool, tb, cached, [max(0, x) for x in q], SCALE))
        for r in range(n):
            token, p = ref.sample(logits[r].double().cpu().numpy(), float(np.float32(0.8)), 40, float(np.float32(0.9)), 0.0,
                                  float(u[0, r]))
            assert tokens[r].item() == token
            assert np.all(np.abs(probs[r].double().cpu().numpy() - p) <= ref.round_probs_bound(p))
        # a draft drawn from the target itself has probability p(x) > 0: certain drafts are accepted with it
        for b in range(B):
            a, r0, r1 = acc[b].item(), want[3][b], want[3][b + 1]
            assert 0 <= a <= max(0, r1 - r0 - 1)
            if r1 > r0:
                t = res[r0 + a].item()
                assert probs[r0 + a, t].item() > 0 and res[r0:r0 + a].tolist() == drafts[r0:r0 + a].tolist()
        q = [1, 1, 1, 1, 2, 1]                   # the ended request's place is taken by a new one
        qt.copy_(_i32(q))
        # a new request there begins with the prefix
        cached[4], counts[4] = prefix, shared
        lens[1 - i][4] = prefix
        cnt[1 - i][4] = shared
    assert err.item() == 0
