"""GPU tests of the calls around a serving step where requests could reach one another or a setting leaves the usual range.
Bounds as in test_gpu_serving_step."""
import math

import numpy as np
import pytest
import torch

import dense_mla_ref
import serving_step_ref as ref
from deepseek_sparse_attention_paged_gb300 import capi
from test_gpu_serving_step import (SCALE, _check_sample, _cum, _i32, _logits, _run_sample, _run_shared,
                                   _run_tables, _shared_inputs)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- shared prefixes

def _poison(inp, bad, value, dims):
    """`value` in one visible row of the last page that each request of `bad` has for itself."""
    q, pool, table, lens, q_lens, cu_group, shared = inp
    pool = pool.clone()
    for b in bad:
        at = lens[b] - 1 - q_lens[b]                     # seen by every query token of the request
        page = int(table[b, at // 64])
        assert at >= 0 and int((table == page).sum()) == 1
        pool[page, at % 64, dims] = value
    return q, pool, table, lens, q_lens, cu_group, shared


def _check_others(inp, bad, **kw):
    out, lse, err = _run_shared(inp, **kw)
    q, pool, table, lens, q_lens, _, _ = inp
    want = dense_mla_ref.decode(q.cuda(), pool.cuda(), table.cuda(), lens, q_lens, SCALE)
    cu = _cum(q_lens)
    rows = [r for b in range(len(lens)) if b not in bad for r in range(cu[b], cu[b + 1])]
    dense_mla_ref.check(out[rows], lse[rows], tuple(x[rows] for x in want))
    assert err == 0
    for b in bad:
        assert not bool(torch.isfinite(out[cu[b]:cu[b + 1]].float()).all(-1).any()), b


@pytest.mark.parametrize("value,dims", [(math.nan, slice(0, 576)), (math.inf, slice(100, 101)), (-math.inf, slice(500, 512))])
@pytest.mark.parametrize("groups,H", [
    ([(192, [(20 + 37 * i, 1 + i % 2) for i in range(20)])], 16),                    # units of 16 tokens
    ([(64 * 41, [(10 + 3 * i, 1) for i in range(32)]), (64, [(5 + i, 2) for i in range(3)])], 16),   # odd pages: split tiles
    ([(0, [(700 + 64 * i, 1) for i in range(16)])], 16),                             # no prefix: pieces that begin in own pages
    ([(128, [(100, 2), (200, 1), (65, 3), (30, 1)])], 32),
    ([(6400, [(2000 + i, 1) for i in range(8)])], 64),
    ([(1024, [(70, 1), (400, 1), (90, 2), (3, 1)])], 128),
])
def test_shared_values_of_one_request_reach_no_other(groups, H, value, dims):
    """Infinite and NaN values that a request sees in pages of its own: the other requests of its unit, whose weights for
    that page are 0, do not."""
    inp = _shared_inputs(groups, H, 51)
    bad = list(range(1, len(inp[3]), 3))
    inp = _poison(inp, bad, value, dims)
    _check_others(inp, bad, T=inp[0].shape[0] + 2)
    # the same batch with nothing in common, and with the groups' borders elsewhere
    _check_others(inp, bad, cu_group=[0], shared=[])


def test_shared_values_reach_no_request_outside_the_groups():
    inp = _shared_inputs([(320, [(9, 1)] * 5)], 16, 52, alone=13)
    bad = [1, 7, 11]
    _check_others(_poison(inp, bad, math.nan, slice(0, 576)), bad)


@pytest.mark.parametrize("H", [16, 128])
def test_shared_prefix_is_read_through_the_first_row_where_it_is_seen_in_part(H):
    """Requests that end inside their group's prefix, alone in their unit or with longer ones: their own entries below the
    prefix are not read."""
    groups = [(256, [(-1, 1), (-56, 2), (-255, 1), (-64, 1)]),                       # nobody sees the whole of the last page
              (640, [(20 + i, 1) for i in range(16)] + [(-30, 1), (-130, 3), (-577, 1)]),     # the short ones in a unit of their own
              (128, [(-70, 1), (5, 1), (-1, 1)])]
    inp = list(_shared_inputs(groups, H, 53))
    want = dense_mla_ref.decode(inp[0].cuda(), inp[1].cuda(), inp[2].cuda(), inp[3], inp[4], SCALE)
    inp[2], b = inp[2].clone(), 0
    for prefix, reqs in groups:
        inp[2][b + 1:b + len(reqs), :prefix // 64] = -7
        b += len(reqs)
    out, lse, err = _run_shared(tuple(inp))
    dense_mla_ref.check(out, lse, want)
    assert err == 0


# ---------------------------------------------------------------- sampling

@pytest.mark.parametrize("V,R,bf16", [(700, 6, False), (3000, 6, False), (3001, 6, True), (40001, 5, False), (2500, 80, True)])
def test_sample_min_p_at_an_infinite_temperature(V, R, bf16):
    """All weights are 1: every min-p keeps everything that is finite."""
    x = _logits(R, V, 60 + V, bf16)
    u = torch.rand(R, generator=torch.Generator().manual_seed(V)).tolist()
    hot = [math.inf] * R
    for m in (1.0, 5.0, math.inf, 0.5):
        _check_sample(x, V, u, temperature=hot, min_p=[m] * R)
        _check_sample(x, V, u, temperature=hot, min_p=[m] * R, top_k=[7] * R)
    # top-p of equal weights, exact on both sides: the first half in the order of z, rounded up
    got, p, err = _run_sample(x, V, u, hot, None, [0.5] * R, [1.0] * R)
    n = (V + 1) // 2
    for r in range(R):
        kept = np.sort(np.argsort(-x[r, :V].double().numpy(), kind="stable")[:n])
        want = np.zeros(V)
        want[kept] = 1.0 / n
        assert got[r] == kept[math.floor(float(np.float32(u[r])) * n)]
        assert np.all(np.abs(p[r] - want) <= ref.round_probs_bound(want))
    assert err == 0


@pytest.mark.parametrize("V,R,bf16", [(7, 5, True), (701, 6, False), (3001, 6, False), (3002, 6, True), (40001, 5, False), (2501, 80, True),
                                      (9001, 300, False)])
def test_sample_masked_rows_at_an_infinite_temperature(V, R, bf16):
    """Masked entries and the places beside a row, which lies on any alignment, have no weight; all others have the same."""
    g = torch.Generator().manual_seed(V)
    x = _logits(R, V, 70 + V, bf16, 2)
    off = torch.rand(R, V + 2, generator=g) < torch.tensor([0.3, 0.99])[torch.arange(R) % 2][:, None]
    off[:, 3] = False
    x[off] = -math.inf
    x[2, 4:6] = math.nan
    u = torch.rand(R, generator=g).tolist()
    hot = [math.inf] * R
    for kw in ({}, {"top_k": [40] * R}, {"top_p": [0.9] * R}, {"top_k": [V // 2] * R, "top_p": [0.9] * R}, {"min_p": [0.1] * R}):
        for at in (0, 1, 2):
            _check_sample(x[:, at:], V, u, temperature=hot, **kw)


@pytest.mark.parametrize("n", [200, 1000, 1300, 2048, 2300])
def test_sample_border_in_a_bin_of_many_entries(n):
    """A CTA a row, the border among n numbers next to 0, or among n equal ones in a bin of the masses: up to 2048 come
    into the list whole."""
    R, V = 80, 20003
    g = torch.Generator().manual_seed(n)
    small = (torch.arange(n) % 250 + 1).float() * 2.0 ** -18 * (1 - 2 * (torch.arange(n) % 2))
    x = torch.full((R, V), -60.0)
    for r in range(R):
        x[r, torch.randperm(V, generator=g)[:n]] = small
    x[:, 11] = 3.0
    x = x.to(torch.bfloat16)
    u = torch.rand(R, generator=g).tolist()
    _check_sample(x, V, u, top_p=[0.3, 0.7] * (R // 2), probs=False)
    _check_sample(x + 150.0, V, u, top_p=[0.6] * R)              # past the values with bins of their own: masses


@pytest.mark.parametrize("mode", ["usual", "mixed", "top_p", "all"])
@pytest.mark.parametrize("V,R,bf16,masked", [(1000, 300, True, 0.0), (1049, 373, True, 0.99), (1601, 200, False, 0.5), (2808, 150, False, 0.0),
                                             (4005, 120, True, 0.5)])
def test_sample_short_vocabularies(V, R, bf16, masked, mode):
    """Rows with their largest tokens at places of their own and masks in every other row: the definition's tokens, and a
    second call's are the first one's."""
    g = torch.Generator().manual_seed(V)
    x = torch.randn(R, V + 3, generator=g) * 2.0
    top = torch.rand(R, V, generator=g).argsort(1)[:, :24]
    x.scatter_(1, top, 7.0 + 3.0 * torch.randn(R, 24, generator=g))
    off = torch.rand(R, V + 3, generator=g) < masked
    off[1::2] = False
    off.scatter_(1, top[:, :1], False)
    x = x.masked_fill(off, -math.inf)
    x = x.to(torch.bfloat16) if bf16 else x
    u = torch.rand(R, generator=g).tolist()
    pick = lambda v: [v[i] for i in torch.randint(len(v), (R,), generator=g).tolist()]
    kw = {"temperature": (0.6 + 0.7 * torch.rand(R, generator=g)).tolist()}
    if mode == "usual":
        kw.update(top_k=[50] * R, top_p=[0.95] * R)
    elif mode == "top_p":
        kw["top_p"] = pick([0.9, 0.95, 0.99])
    elif mode == "mixed":
        kw.update(top_k=pick([0, 1, 20, 50, 1000]), top_p=pick([0.5, 0.9, 0.99, 1.0]), min_p=pick([0.0, 0.02, 0.1]))
        kw["temperature"][::4] = [0.0] * len(kw["temperature"][::4])
    for probs in (False, True):
        _check_sample(x, V, u, probs=probs, **kw)
    a, b = _run_sample(x, V, u, **kw), _run_sample(x, V, u, **kw)
    assert a[0] == b[0] and np.array_equal(a[1], b[1])


# ---------------------------------------------------------------- step tables

def test_tables_report_bad_pages_that_are_given_back():
    """Ids that are no pages in the rows of requests that end: said in that call, -1 on the stack; those that the request
    does not own, or that are not mapped, are not looked at."""
    table = [[3, 99, 5, 1000], [-1, 7, -5, 2], [0, 1, 4, 6]]
    stack = [8, 9] + [-1] * 8
    got = _run_tables([200, 140, 100], [-1, -1, 10], [3, 3, 2], [0, 1, 0], table, 10, stack, 2, 12)
    assert got == ([0, 0, 110], [0, 0, 2], 7, [0, 0, 0, 10], list(range(100, 110)) + [0, 0],
                   [64 + p % 64 for p in range(100, 110)] + [-1, -1], capi.DSA_DEVERR_PAGE_RANGE)
    assert stack == [8, 9, 3, -1, 5, 7, -1, -1, -1, -1]
    assert table == [[3, 99, 5, 1000], [-1, 7, -5, 2], [0, 1, 4, 6]]
    # outside of what is given back: no error
    stack = [8, 9] + [-1] * 8
    got = _run_tables([200, 140, 100], [-1, -1, 10], [1, 2, 2], [0, 1, 0], table, 10, stack, 2, 10)
    assert got[-1] == 0 and got[2] == 4 and stack[:4] == [8, 9, 3, 7]
    # taken again in the same call: the request that gets the entry has no page there
    table = [[99, 2], [0, -1]]
    got = _run_tables([100, 64], [-1, 1], [2, 1], None, table, 10, [-1] * 10, 0, 1)
    assert got == ([0, 65], [0, 2], 1, [0, 0, 1], [64], [2 * 64], capi.DSA_DEVERR_PAGE_RANGE) and table[1] == [0, 2]


def test_tables_without_requests():
    """An empty batch: nothing is written; rows without requests are refused."""
    stack = [3, 1, -1, -1]
    i64 = lambda n: torch.full((n,), 7, dtype=torch.int64, device="cuda")
    bufs = lambda: (_i32([]), _i32([]), _i32([7]), _i32([7]), i64(0), i64(0))
    st, seq, co, ho, cu, pos, slots = _i32(stack), *bufs()
    none, table, err = _i32([]), torch.zeros(0, 5, dtype=torch.int32, device="cuda"), _i32([0])
    capi.dsa_step_tables(none, none, none, table, 4, st, _i32([2]), seq, co, ho, cu, pos, slots, dev_err=err)
    assert ho.item() == 7 and cu.tolist() == [7] and st.tolist() == stack and err.item() == 0
    with pytest.raises(capi.DSAError):
        capi.dsa_step_tables(none, none, none, table, 4, st, _i32([2]), seq, co, ho, cu, i64(3), i64(3))
