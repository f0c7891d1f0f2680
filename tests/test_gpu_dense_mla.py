"""GPU tests of the dense latent-attention calls against plain float64 definitions (dense_mla_ref): the
latent store, the prompt's attention in expanded form, the absorbed attention over the paged cache, the
verification of drafted tokens, and a run of them together.  Bounds are derived in dense_mla_ref."""
import math

import pytest
import torch

import dense_mla_ref as ref
from deepseek_sparse_attention_paged_gb300 import capi

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _cum(ns):
    c = [0]
    for n in ns:
        c.append(c[-1] + n)
    return c


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- store

def _store_inputs(n, seed, stride=576, pages=None):
    g = _gen(seed)
    raw = (torch.randn(n, stride, generator=g) * torch.exp(torch.randn(n, 1, generator=g))).to(torch.bfloat16)
    w = 1 + 0.2 * torch.randn(512, generator=g)
    ang = torch.rand(300, 32, generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pages = pages or n // 64 + 2
    slots = torch.randperm(pages * 64, generator=g)[:n]
    pos = torch.randint(0, 300, (n,), generator=g)
    return raw, w, cs, pos, slots, pages


@pytest.mark.parametrize("n,stride,interleaved,dense", [(1, 576, True, True), (3, 584, False, False), (64, 576, False, True),
                                                        (777, 640, True, True), (2001, 2112, False, False)])
def test_store_latent(n, stride, interleaved, dense):
    raw, w, cs, pos, slots, pages = _store_inputs(n, 100 + n, stride)
    slots[::7] = -1
    pool = torch.full((pages, 64, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    lat = torch.full((n, 584), 5.0, dtype=torch.bfloat16, device="cuda") if dense else None
    err = _err()
    capi.dsa_store_latent_prologue(raw.cuda()[:, :576], w.cuda(), 1e-6, cs.cuda(), pos.cuda(), slots.cuda(), pool,
                                   latent_out=lat[:, :576] if dense else None,
                                   flags=capi.DSA_ROPE_INTERLEAVED if interleaved else 0, dev_err=err)
    y, bound = ref.store(raw[:, :576], w, 1e-6, cs, pos, interleaved)
    flat = pool.view(-1, 576).cpu().double()
    keep = slots >= 0
    assert bool(((flat[slots[keep]] - y[keep]).abs() <= bound[keep]).all())
    rest = torch.ones(pages * 64, dtype=torch.bool)
    rest[slots[keep]] = False
    assert bool((flat[rest] == 3.0).all())
    if dense:
        assert bool(((lat[:, :576].cpu().double() - y).abs() <= bound).all()) and bool((lat[:, 576:] == 5.0).all())
    assert capi.dsa_read_device_error(err) == (0, 0)


def test_store_latent_in_place_and_extreme_rows():
    """latent_out = kv_a itself; a zero row (0 with eps > 0), tiny and huge rows."""
    raw, w, cs, pos, slots, pages = _store_inputs(6, 31)
    raw[1] = 0
    raw[2] *= 1e-10
    raw[3] = (raw[3].float() * 1e12).to(torch.bfloat16)
    y, bound = ref.store(raw, w, 1e-6, cs, pos, False)
    x = raw.cuda()
    pool = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    capi.dsa_store_latent_prologue(x, w.cuda(), 1e-6, cs.cuda(), pos.cuda(), slots.cuda(), pool, latent_out=x)
    assert bool(((x.cpu().double() - y).abs() <= bound).all())
    assert torch.equal(pool.view(-1, 576)[slots.cuda()], x)


def test_store_latent_bad_positions_and_slots():
    raw, w, cs, pos, slots, pages = _store_inputs(8, 32)
    pos[2], pos[3] = -1, 300
    slots[5], slots[6] = pages * 64, -9
    pool = torch.full((pages, 64, 576), 3.0, dtype=torch.bfloat16, device="cuda")
    lat = torch.full((8, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    err = _err()
    capi.dsa_store_latent_prologue(raw.cuda(), w.cuda(), 1e-6, cs.cuda(), pos.cuda(), slots.cuda(), pool, latent_out=lat,
                                   dev_err=err)
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS,
                                               capi.DSA_DEVERR_POSITION | capi.DSA_DEVERR_SLOT_RANGE)
    assert bool((lat[2:4] == 5.0).all()) and not bool((lat[4:] == 5.0).all(1).any())
    written = (pool.view(-1, 576) != 3.0).any(1).cpu()
    assert sorted(torch.nonzero(written)[:, 0].tolist()) == sorted(slots[[0, 1, 4, 7]].tolist())


# ---------------------------------------------------------------- decode

def _decode_inputs(lens, q_lens, H, seed, extra_pages=3, stale=None):
    """Shuffled pages; cache rows past a request's length hold `stale`."""
    g = _gen(seed)
    pages = [(n + 63) // 64 for n in lens]
    total = sum(pages) + extra_pages
    pool = torch.randn(total, 64, 576, generator=g).to(torch.bfloat16)
    if stale is not None:
        clean = pool.clone()
        pool.fill_(stale)
    perm = torch.randperm(total, generator=g)
    table = torch.full((len(lens), max(pages + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        if stale is not None:
            for i in range(pages[b]):
                m = min(64, n - 64 * i)
                pool[perm[at + i], :m] = clean[perm[at + i], :m]
        at += pages[b]
    q = torch.randn(sum(q_lens), H, 576, generator=g).to(torch.bfloat16)
    return q.cuda(), pool.cuda(), table.cuda()


def _decode(q, pool, table, lens, q_lens, err=None, out=None, lse=None, **kw):
    T, H = q.shape[0], q.shape[1]
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((T, H), 7.0, device="cuda") if lse is None else lse
    capi.dsa_dense_mla_decode(q, pool, table, _i32(lens), _i32(_cum(q_lens)), SCALE, out, lse=lse, dev_err=err, **kw)
    return out, lse


@pytest.mark.parametrize("H", [16, 32, 64, 128])
@pytest.mark.parametrize("lens,q_lens", [
    ([1], [1]), ([64], [1]), ([65], [2]), ([0, 5, 63, 0, 128, 129], [1, 1, 2, 3, 1, 4]),
    ([3, 700, 2], [5, 3, 2]),                       # more queries than tokens: rows that see nothing
    ([1000, 333, 64, 2500], [1, 9, 0, 17]),         # a request without rows, row groups that end inside a tile
])
def test_decode_matches_float64(H, lens, q_lens):
    q, pool, table = _decode_inputs(lens, q_lens, H, 200 + H + sum(lens))
    err = _err()
    out, lse = _decode(q, pool, table, lens, q_lens, err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


@pytest.mark.parametrize("H,lens,q_lens", [(128, [40000], [1]), (16, [30001, 20000], [4, 1]),
                                           (64, [200 + 37 * i for i in range(90)], [1 + i % 3 for i in range(90)]),
                                           (128, [100 + 61 * i for i in range(180)], [1] * 180)])
def test_decode_long_and_many(H, lens, q_lens):
    """One long context split over the whole GPU; more work items than CTAs."""
    q, pool, table = _decode_inputs(lens, q_lens, H, 300 + len(lens))
    out, lse = _decode(q, pool, table, lens, q_lens)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


@pytest.mark.parametrize("stale", [math.nan, math.inf, -math.inf])
def test_decode_ignores_what_is_behind_the_last_token(stale):
    lens, q_lens = [1, 63, 65, 200, 0, 640], [1, 2, 1, 1, 1, 3]
    q, pool, table = _decode_inputs(lens, q_lens, 32, 41, stale=stale)
    out, lse = _decode(q, pool, table, lens, q_lens)
    clean = torch.nan_to_num(pool.float(), 0.0, 0.0, 0.0).to(torch.bfloat16)
    ref.check(out, lse, ref.decode(q, clean, table, lens, q_lens, SCALE))


def test_decode_extreme_scores():
    """One key far above the rest in the last page; keys far below; equal keys."""
    lens, q_lens = [500, 300, 129], [1, 1, 1]
    q, pool, table = _decode_inputs(lens, q_lens, 16, 42)
    pool[table[0, 7].long(), 30] = (q[0, 0].float() * 4).to(torch.bfloat16)
    pool[table[1, :5].long()] = pool[table[1, 0].long(), 0].clone()
    pool[table[2, 0].long()] = (-20 * q[2, 3].float()).to(torch.bfloat16)
    out, lse = _decode(q, pool, table, lens, q_lens)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


def test_decode_bad_pages_and_short_table():
    lens, q_lens = [300, 400, 130], [1, 1, 1]
    q, pool, table = _decode_inputs(lens, q_lens, 16, 43)
    table[0, 1], table[0, 4] = -1, pool.shape[0]
    table[2, :3] = 1 << 30
    err = _err()
    out, lse = _decode(q, pool, table, lens, q_lens, err)
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_PAGE_RANGE)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))
    short = table[:, :2].contiguous()
    err.zero_()
    out, lse = _decode(q, pool, short, lens, q_lens, err)
    assert capi.dsa_read_device_error(err)[1] & capi.DSA_DEVERR_INDEX_RANGE
    ref.check(out, lse, ref.decode(q, pool, short, lens, q_lens, SCALE))


def test_decode_leaves_rows_behind_the_last_request():
    lens, q_lens = [100, 200], [1, 2]
    q, pool, table = _decode_inputs(lens, q_lens + [3], 16, 44)
    out, lse = _decode(q, pool, table, lens, q_lens)
    assert bool((out[3:] == 7.0).all()) and bool((lse[3:] == 7.0).all())
    r = ref.decode(q[:3], pool, table, lens, q_lens, SCALE)
    ref.check(out[:3], lse[:3], r)


def test_decode_equals_sparse_over_all_positions():
    """The framework's sparse call with every position selected, on the same cache."""
    lens, q_lens = [700, 64, 1500], [1, 2, 1]
    q, pool, table = _decode_inputs(lens, q_lens, 128, 45)
    out, lse = _decode(q, pool, table, lens, q_lens)
    idx = torch.full((4, 1536), -1, dtype=torch.int32)
    for r, v in enumerate([700, 63, 64, 1500]):
        idx[r, :v] = torch.arange(v, dtype=torch.int32)
    ws = torch.empty(capi.dsa_sparse_mla_workspace_size(4, 128, 1536) + 16, dtype=torch.uint8, device="cuda")
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    capi.dsa_sparse_mla_decode(q, pool, table, _i32(lens), _i32(_cum(q_lens)), idx.cuda(), SCALE, o2, ws, lse=l2)
    r = ref.decode(q, pool, table, lens, q_lens, SCALE)
    assert bool(((out.double() - o2.double()).abs() <= 2 * r[2]).all())
    assert bool(((lse - l2).abs().double() <= 2 * r[3]).all())


def test_decode_repeats_bit_for_bit_and_in_graphs():
    """Same bits on every run, on another stream, and from two captured graphs with a workspace each,
    replayed on changed lengths."""
    lens, q_lens = [5000, 300, 9000], [1, 1, 2]
    q, pool, table = _decode_inputs(lens, q_lens, 128, 46)
    out, lse = _decode(q, pool, table, lens, q_lens)
    o2, l2 = _decode(q, pool, table, lens, q_lens)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    size = max(16, capi.dsa_dense_mla_decode_workspace_size(4, 128))
    seq, cu = _i32(lens), _i32(_cum(q_lens))
    graphs = []
    for _ in range(2):
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        o, l = torch.zeros_like(out), torch.zeros_like(lse)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            capi.dsa_dense_mla_decode(q, pool, table, seq, cu, SCALE, o, ws, lse=l)
            s.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                capi.dsa_dense_mla_decode(q, pool, table, seq, cu, SCALE, o, ws, lse=l)
        assert torch.equal(o, out) and torch.equal(l, lse)
        graphs.append((gr, o, l, ws))
    seq.copy_(_i32([64, 0, 8999]))
    torch.cuda.synchronize()
    want = ref.decode(q, pool, table, [64, 0, 8999], q_lens, SCALE)
    for gr, o, l, _ in graphs:
        gr.replay()
    torch.cuda.synchronize()
    for gr, o, l, _ in graphs:
        ref.check(o, l, want)
    assert torch.equal(graphs[0][1], graphs[1][1])


def test_decode_far_pages():
    """Row offsets of the cache past 2^31 elements."""
    pages = (1 << 31) // (64 * 576) + 40
    pool = torch.zeros(pages, 64, 576, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    pool[-8:] = torch.randn(8, 64, 576, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.arange(pages - 1, pages - 9, -1, dtype=torch.int32, device="cuda")[None].contiguous()
    q = torch.randn(1, 16, 576, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = _decode(q, pool, table, [500], [1])
    ref.check(out, lse, ref.decode(q, pool, table, [500], [1], SCALE))
    latent = torch.randn(2, 576, generator=g, device="cuda").to(torch.bfloat16)
    cs = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).cuda()
    slots = torch.tensor([pages * 64 - 1, 5], device="cuda")
    capi.dsa_store_latent_prologue(latent, torch.ones(512, device="cuda"), 1e-6, cs, torch.zeros(2, dtype=torch.int64,
                                   device="cuda"), slots, pool)
    y, bound = ref.store(latent.cpu(), torch.ones(512), 1e-6, cs.cpu(), torch.zeros(2, dtype=torch.int64), False)
    assert bool(((pool.view(-1, 576)[slots].cpu().double() - y).abs() <= bound).all())


# ---------------------------------------------------------------- prefill

def _prefill_inputs(q_lens, k_lens, H, seed, extra=0):
    g = _gen(seed)
    T, S = sum(q_lens) + extra, sum(k_lens) + extra
    q = torch.randn(T, H, 192, generator=g).to(torch.bfloat16).cuda()
    kv = torch.randn(S, H, 256, generator=g).to(torch.bfloat16).cuda()
    lat = torch.randn(S, 576, generator=g).to(torch.bfloat16).cuda()
    return q, kv, lat


def _prefill(q, kv, lat, q_lens, k_lens, causal=True, err=None, out=None):
    T, H = q.shape[0], q.shape[1]
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full((T, H), 7.0, device="cuda")
    capi.dsa_dense_mla_prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], _i32(_cum(q_lens)), _i32(_cum(k_lens)), SCALE,
                               out, lse=lse, causal=causal, dev_err=err)
    return out, lse


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,q_lens,k_lens", [
    (1, [1], [1]), (3, [5, 1, 17], [5, 1, 17]), (2, [128, 127, 129], [128, 127, 129]), (16, [300], [300]),
    (2, [1, 7], [400, 257]), (2, [100, 3], [1500, 640]),           # chunks and single tokens after a prefix
    (2, [10, 260, 0, 4], [4, 100, 30, 0]),                          # rows that see nothing, no rows, no keys
    (5, [1000, 513], [1000, 513]), (1, [256, 257], [512, 384]),
])
def test_prefill_matches_float64(H, q_lens, k_lens, causal):
    q, kv, lat = _prefill_inputs(q_lens, k_lens, H, 400 + sum(k_lens))
    err = _err()
    out, lse = _prefill(q, kv, lat, q_lens, k_lens, causal, err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], q_lens, k_lens, SCALE, causal))


def test_prefill_long_and_many_requests():
    q_lens = [3000] + [1 + 11 * i % 300 for i in range(150)]
    q, kv, lat = _prefill_inputs(q_lens, q_lens, 4, 50)
    out, lse = _prefill(q, kv, lat, q_lens, q_lens)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], q_lens, q_lens, SCALE, True))


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_ignores_rows_behind_the_last_request(bad, causal):
    """The buffers are longer than the batch (padded); their tail holds anything and is left as it is."""
    q_lens, k_lens = [70, 200], [90, 200]
    q, kv, lat = _prefill_inputs(q_lens, k_lens, 2, 51, extra=300)
    q[270:], kv[290:], lat[290:] = bad, bad, bad
    out, lse = _prefill(q, kv, lat, q_lens, k_lens, causal)
    assert bool((out[270:] == 7.0).all()) and bool((lse[270:] == 7.0).all())
    want = ref.prefill(q[:270], kv[:290, :, :128], lat[:290, 512:], kv[:290, :, 128:], q_lens, k_lens, SCALE, causal)
    ref.check(out[:270], lse[:270], want)


def test_prefill_bad_values_of_another_request_stay_there():
    q_lens = [70, 130, 200]
    q, kv, lat = _prefill_inputs(q_lens, q_lens, 2, 52)
    clean = [t.clone() for t in (q, kv, lat)]
    for t in (q, kv, lat):
        t[70:200] = math.nan
    out, _ = _prefill(q, kv, lat, q_lens, q_lens)
    want, _ = _prefill(*clean, q_lens, q_lens)
    assert torch.equal(out[:70], want[:70]) and torch.equal(out[200:], want[200:])
    assert bool(out[70:200].isnan().all())


def test_prefill_strides_and_extreme_scores():
    """Head-major queries and outputs, separate key and value arrays with padded rows, one far larger key."""
    g = _gen(53)
    H, n = 3, 400
    q = torch.randn(H, n, 200, generator=g).to(torch.bfloat16).cuda()[..., :192].transpose(0, 1)
    k = torch.randn(n, H, 136, generator=g).to(torch.bfloat16).cuda()[..., :128]
    v = torch.randn(n, H + 2, 128, generator=g).to(torch.bfloat16).cuda()[:, 1:1 + H]
    pe = torch.randn(n, 64, generator=g).to(torch.bfloat16).cuda()
    k[350] = (q[380, :, :128].float() * 6).to(torch.bfloat16)
    k[3] = (q[10, :, :128].float() * -30).to(torch.bfloat16)
    buf = torch.full((H, n, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, H, device="cuda")
    capi.dsa_dense_mla_prefill(q, k, pe, v, _i32([0, n]), _i32([0, n]), SCALE, buf.transpose(0, 1), lse=lse)
    ref.check(buf.transpose(0, 1), lse, ref.prefill(q, k, pe, v, [n], [n], SCALE, True))


def test_prefill_cuts_ranges_outside_the_arrays():
    q, kv, lat = _prefill_inputs([64], [64], 2, 54)
    err = _err()
    out, lse = _prefill(q, kv, lat, [64], [96], False, err)          # cu_k ends past S: keys 0 .. 63
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_INDEX_RANGE)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], [64], [64], SCALE, False))
    err.zero_()
    out, lse = _prefill(q, kv, lat, [80], [64], False, err)          # cu_q ends past T: rows 0 .. 63
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_INDEX_RANGE)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], [64], [64], SCALE, False))


def test_prefill_repeats_bit_for_bit_and_in_a_graph():
    q_lens = [600, 64, 1]
    q, kv, lat = _prefill_inputs(q_lens, q_lens, 8, 55)
    out, lse = _prefill(q, kv, lat, q_lens, q_lens)
    cu = _i32(_cum(q_lens))
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            capi.dsa_dense_mla_prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], cu, cu, SCALE, o, lse=l)
    for _ in range(2):
        gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


# ---------------------------------------------------------------- verify

def _verify_inputs(counts, V, seed, certain=False, pad=0):
    g = _gen(seed)
    T = sum(counts)
    lg = torch.randn(T, V, generator=g) * 2
    p = torch.softmax(lg, 1)
    p = torch.where(p < 0.02 / V, torch.zeros_like(p), p)
    d = torch.softmax(lg + torch.randn(T, V, generator=g) * 0.6, 1)
    tok = d.argmax(1) if certain else torch.multinomial(d, 1, generator=g)[:, 0]

    def wide(x):
        w = torch.full((T, V + pad), math.nan)
        w[:, :V] = x
        return w[:, :V]
    return wide(p), None if certain else wide(d), tok.to(torch.int32), torch.rand(T, generator=g), \
        torch.rand(len(counts), generator=g)


def _padded_cuda(x):
    """A CUDA copy with the CPU tensor's row stride."""
    if x is None:
        return None
    w = torch.full((x.shape[0], x.stride(0)), math.nan, device="cuda")
    w[:, :x.shape[1]] = x.cuda()
    return w[:, :x.shape[1]]


def _verify(p, d, tok, counts, u, us, err=None):
    T = p.shape[0]
    out = torch.full((T,), -7, dtype=torch.int32, device="cuda")
    acc = torch.full((len(counts),), -7, dtype=torch.int32, device="cuda")
    capi.dsa_verify_drafts(_padded_cuda(p), tok.cuda(), _i32(_cum(counts)), u.cuda(), us.cuda(), out, acc,
                           draft_probs=_padded_cuda(d), dev_err=err)
    return out.tolist(), acc.tolist()


@pytest.mark.parametrize("counts,V,pad", [([1], 1, 0), ([2], 7, 0), ([4, 1, 0, 3], 513, 3), ([3] * 20, 1000, 0),
                                          ([4, 2, 1, 6] * 4, 32000, 8), ([40, 1], 4097, 1), ([4] * 6, 131072, 0),
                                          ([2] * 3, 160001, 0)])
@pytest.mark.parametrize("certain", [False, True])
def test_verify_matches_float64(counts, V, pad, certain):
    p, d, tok, u, us = _verify_inputs(counts, V, 500 + V, certain, pad)
    err = _err()
    got = _verify(p, d, tok, counts, u, us, err)
    assert got == ref.verify(p, d, tok.tolist(), _cum(counts), u, us)
    assert capi.dsa_read_device_error(err) == (0, 0)


def test_verify_all_accepted_and_none():
    counts, V = [4, 4], 900
    p, d, tok, u, us = _verify_inputs(counts, V, 61)
    u[:4], u[4:] = 0.0, 1.0 - 2.0 ** -24
    p[0:3, :] = d[0:3, :]
    p[4, tok[4]] = 0.0
    got = _verify(p, d, tok, counts, u, us)
    assert got[1] == [3, 0]
    assert got == ref.verify(p, d, tok.tolist(), _cum(counts), u, us)


def test_verify_draws_at_the_ends():
    """sample_u = 0 draws the first entry with mass, the largest u below 1 the last; leading, trailing
    and inner entries without mass are never drawn."""
    V = 5000
    p = torch.zeros(2, V)
    p[:, 1000:1003] = torch.tensor([0.25, 0.0, 0.25])
    p[:, 4000] = 0.5
    tok = torch.full((2,), -1, dtype=torch.int32)
    us = torch.tensor([0.0, 1.0 - 2.0 ** -24])
    got = _verify(p, None, tok, [1, 1], torch.zeros(2), us)
    assert got == ([1000, 4000], [0, 0])
    got = _verify(p, None, tok, [1, 1], torch.zeros(2), torch.tensor([0.25, 0.5]))   # exactly on the borders
    assert got[0] == [1002, 4000]


def test_verify_no_residual_mass_and_no_mass_at_all():
    V = 600
    p = torch.zeros(4, V)
    p[0, 5], p[0, 9] = 0.5, 0.5
    d = torch.zeros(4, V)
    d[0, 5], d[0, 9] = 1.0, 0.75          # p <= q everywhere, x = 5 rejected by u = 0.9: drawn from p
    p[2, 3] = 1.0
    d[2, 3] = 1.0                          # x = 0 with q(x) = 0 and p(x) = 0: rejected, nothing left, drawn from p
    tok = torch.tensor([5, -1, 0, -1], dtype=torch.int32)
    u, us = torch.tensor([0.9, 0.0, 0.0, 0.0]), torch.tensor([0.6, 0.0])
    err = _err()
    got = _verify(p, d, tok, [2, 2], u, us, err)
    assert got == ([9, -1, 3, -1], [0, 0])
    assert capi.dsa_read_device_error(err) == (0, 0)
    got = _verify(p[1:2], None, tok[1:2], [1], u[:1], us[:1], err)      # a row of zeros
    assert got == ([-1], [0])
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_PROB)


def test_verify_bad_entries_and_tokens():
    """NaN, infinite and negative entries carry no mass; a draft token past the vocabulary is no draft."""
    V = 1024
    p = torch.full((3, V), 1.0 / V)
    p[:, 0], p[:, 1], p[:, 2] = math.nan, math.inf, -4.0
    tok = torch.tensor([V, 0, -5], dtype=torch.int32)
    err = _err()
    u, us = torch.full((3,), 0.5), torch.tensor([0.001, 0.7])
    got = _verify(p, None, tok, [1 + 1, 1], u, us, err)
    assert got == ref.verify(p, None, tok.tolist(), [0, 2, 3], u, us)
    assert got[0][0] >= 3 and got[1] == [0, 0]
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_INDEX_RANGE)
    tok[0] = 0                                                          # p(x) = NaN: rejected
    got = _verify(p, None, tok, [2, 1], u, us)
    assert got == ref.verify(p, None, tok.tolist(), [0, 2, 3], u, us) and got[1] == [0, 0]


def test_verify_leaves_rows_behind_the_last_request():
    p, d, tok, u, us = _verify_inputs([3, 2, 4], 300, 62)
    got = _verify(p, d, tok, [3, 2], u, us[:2])
    assert got[0][5:] == [-7] * 4
    want = ref.verify(p[:5], d[:5], tok.tolist()[:5], [0, 3, 5], u, us)
    assert (got[0][:5], got[1]) == want


# ---------------------------------------------------------------- together

def test_a_layer_of_prompts_then_drafted_tokens():
    """Prompt: store -> expanded attention.  Decode: store of the drafted tokens -> absorbed query ->
    dense attention over the cache -> value up-projection; the decode rows against float64 attention
    over up-projected keys of the stored latents; then the drafts are verified."""
    g = _gen(70)
    H, prompts, q_len = 16, [150, 70], 3
    w_uk = (torch.randn(H, 128, 512, generator=g) / 22).to(torch.bfloat16).cuda()      # [H, nope, latent]
    w_uv = (torch.randn(H, 512, 128, generator=g) / 22).to(torch.bfloat16).cuda()
    w = torch.ones(512).cuda()
    ang = torch.arange(256, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    pool = torch.full((8, 64, 576), math.nan, dtype=torch.bfloat16, device="cuda")      # never written: anything
    table = torch.tensor([[6, 1, 3, -1], [0, 4, -1, -1]], dtype=torch.int32).cuda()

    def slots(b, lo, hi):
        t = torch.arange(lo, hi)
        return table[b].cpu().long()[t // 64] * 64 + t % 64

    # prompts
    n = sum(prompts)
    raw = torch.randn(n, 576, generator=g).to(torch.bfloat16).cuda()
    pos = torch.cat([torch.arange(m) for m in prompts]).cuda()
    lat = torch.empty(n, 576, dtype=torch.bfloat16, device="cuda")
    capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, torch.cat([slots(b, 0, m) for b, m in enumerate(prompts)]).cuda(),
                                   pool, latent_out=lat)
    wk = torch.cat([w_uk.transpose(1, 2), w_uv], 2).float()                              # [H, 512, 256]
    kv = torch.einsum("sl,hlc->shc", lat[:, :512].float(), wk).to(torch.bfloat16)
    q = torch.randn(n, H, 192, generator=g).to(torch.bfloat16).cuda()
    out, lse = _prefill(q, kv, lat, prompts, prompts)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], prompts, prompts, SCALE, True))

    # drafted tokens
    T = 2 * q_len
    raw = torch.randn(T, 576, generator=g).to(torch.bfloat16).cuda()
    lens = [m + q_len for m in prompts]
    pos = torch.cat([torch.arange(m, m + q_len) for m in prompts]).cuda()
    capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, torch.cat([slots(b, m, m + q_len) for b, m in
                                                                     enumerate(prompts)]).cuda(), pool)
    q = torch.randn(T, H, 192, generator=g).to(torch.bfloat16).cuda()
    mq = torch.empty(T, H, 576, dtype=torch.bfloat16, device="cuda")
    mq[..., 512:] = q[..., 128:]
    capi.dsa_mla_absorb_q(q[..., :128], w_uk, mq[..., :512])
    o_lat, lse = _decode(mq, pool, table, lens, [q_len] * 2)
    ref.check(o_lat, lse, ref.decode(mq, pool, table, lens, [q_len] * 2, SCALE))
    o = torch.empty(T, H * 128, dtype=torch.bfloat16, device="cuda")
    capi.dsa_mla_v_up(o_lat, w_uv, o.view(T, H, 128))
    # the expanded definition on the cached latents in float64: differs by the absorbed query's and the
    # latent output's roundings (2^-8 each) and the attention's bound, within 2e-2 on unit-variance data
    for b, m in enumerate(lens):
        c = pool[table[b].long()[torch.arange(m).cuda() // 64], torch.arange(m).cuda() % 64].double()
        k = torch.einsum("sl,hpl->shp", c[:, :512], w_uk.double())
        v = torch.einsum("sl,hlv->shv", c[:, :512], w_uv.double())
        rows = slice(b * q_len, (b + 1) * q_len)
        want, _, _, _ = ref.prefill(q[rows].double(), k, c[:, 512:], v, [q_len], [m], SCALE, True)
        assert float((o.view(T, H, 128)[rows].double() - want).abs().max()) <= 2e-2

    # verification of the drafts against probabilities made from the attention's output
    head = torch.randn(H * 128, 500, generator=g).cuda() / 16
    p = torch.softmax(o.float() @ head, 1)
    d = torch.softmax(o.float() @ head + 0.3 * torch.randn(T, 500, generator=g).cuda(), 1)
    tok = torch.multinomial(d.cpu(), 1, generator=g)[:, 0].to(torch.int32)
    u, us = torch.rand(T, generator=g), torch.rand(2, generator=g)
    got = _verify(p.cpu(), d.cpu(), tok, [q_len] * 2, u, us)
    assert got == ref.verify(p.cpu(), d.cpu(), tok.tolist(), [0, q_len, 2 * q_len], u, us)


# ---------------------------------------------------------------- what else the calls allow

def test_decode_many_requests_without_rows():
    """3000 requests, most of them without query rows or without tokens."""
    lens = [(7 * i) % 200 if i % 3 == 0 else 0 for i in range(3000)]
    q_lens = [1 if i % 7 == 0 else 0 for i in range(3000)]
    q, pool, table = _decode_inputs(lens, q_lens, 16, 80)
    out, lse = _decode(q, pool, table, lens, q_lens)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


@pytest.mark.parametrize("H", [128, 16])
def test_decode_a_chunk_of_many_query_tokens(H):
    """A prompt's chunk through the absorbed call: hundreds of query rows per request."""
    lens, q_lens = [700, 300], [300, 77]
    q, pool, table = _decode_inputs(lens, q_lens, H, 81 + H)
    out, lse = _decode(q, pool, table, lens, q_lens)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


def test_decode_negative_lengths_dirty_workspace_no_lse():
    """A negative length sees nothing; a workspace full of NaN bytes and of an earlier call changes nothing."""
    lens, q_lens = [-5, 3000, 9000, -1], [1, 2, 1, 2]
    q, pool, table = _decode_inputs([max(0, n) for n in lens], q_lens, 64, 82)
    ws = torch.full((capi.dsa_dense_mla_decode_workspace_size(6, 64),), 255, dtype=torch.uint8, device="cuda")
    want = ref.decode(q, pool, table, [max(0, n) for n in lens], q_lens, SCALE)
    for _ in range(2):
        out, lse = _decode(q, pool, table, lens, q_lens, workspace=ws)
        ref.check(out, lse, want)
    o2 = torch.empty_like(out)
    capi.dsa_dense_mla_decode(q, pool, table, _i32(lens), _i32(_cum(q_lens)), SCALE, o2, ws)
    assert torch.equal(out, o2)


def test_decode_on_two_streams_at_once():
    """Two calls in flight, each with its own stream and workspace, give what they give alone."""
    cases = []
    for i, (lens, q_lens, H) in enumerate([([20000, 300], [1, 2], 128), ([5000] * 9, [1] * 9, 32)]):
        q, pool, table = _decode_inputs(lens, q_lens, H, 83 + i)
        out, lse = _decode(q, pool, table, lens, q_lens)
        ws = torch.empty(capi.dsa_dense_mla_decode_workspace_size(q.shape[0], H), dtype=torch.uint8, device="cuda")
        cases.append((q, pool, table, _i32(lens), _i32(_cum(q_lens)), out, lse, torch.zeros_like(out),
                      torch.zeros_like(lse), ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, pool, table, sl, cu, _, _, o, l, ws, s in cases:
            capi.dsa_dense_mla_decode(q, pool, table, sl, cu, SCALE, o, ws, lse=l, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, _, out, lse, o, l, _, _ in cases:
        assert torch.equal(out, o) and torch.equal(lse, l)


def test_prefill_many_short_requests_and_one_head():
    q_lens = [1 + (5 * i) % 9 for i in range(1500)]
    k_lens = [n + (i % 4) * 40 for i, n in enumerate(q_lens)]
    q, kv, lat = _prefill_inputs(q_lens, k_lens, 1, 84)
    out, lse = _prefill(q, kv, lat, q_lens, k_lens)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], q_lens, k_lens, SCALE, True))


def test_prefill_without_keys_and_without_lse():
    q = torch.randn(5, 2, 192, generator=_gen(85)).to(torch.bfloat16).cuda()
    empty = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    pe = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    out = torch.full((5, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    capi.dsa_dense_mla_prefill(q, empty, pe, empty, _i32([0, 5]), _i32([0, 0]), SCALE, out)
    assert bool((out == 0).all())


def test_prefill_twice_in_flight_beside_decode():
    """Two prompts' calls and a decode call on three streams."""
    q_lens = [900, 200]
    q, kv, lat = _prefill_inputs(q_lens, q_lens, 16, 86)
    want, _ = _prefill(q, kv, lat, q_lens, q_lens)
    dq, pool, table = _decode_inputs([9000], [1], 128, 87)
    dwant, _ = _decode(dq, pool, table, [9000], [1])
    outs = [torch.zeros_like(want) for _ in range(2)]
    dout = torch.zeros_like(dwant)
    ws = torch.empty(capi.dsa_dense_mla_decode_workspace_size(1, 128), dtype=torch.uint8, device="cuda")
    cu, sl, dcu = _i32(_cum(q_lens)), _i32([9000]), _i32([0, 1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(4):
        for o, s in zip(outs, streams):
            capi.dsa_dense_mla_prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], cu, cu, SCALE, o, stream=s)
        capi.dsa_dense_mla_decode(dq, pool, table, sl, dcu, SCALE, dout, ws, stream=streams[2])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(dout, dwant)


def test_binding_refuses_what_the_calls_do_not_take():
    f = torch.zeros(4, 16, 576, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(2, 64, 576, dtype=torch.bfloat16, device="cuda")
    table, lens, cu = _i32([[0], [1]]), _i32([3, 4]), _i32([0, 2, 4])
    out = torch.zeros(4, 16, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(capi.dsa_dense_mla_decode_workspace_size(4, 16), dtype=torch.uint8, device="cuda")
    for bad in (dict(q_bf16=f.half()), dict(q_bf16=f[:, :, :512]), dict(kv_pool=pool[:, :, :512]), dict(cu_q=cu[:2]),
                dict(out=out[:3]), dict(lse=torch.zeros(4, 15, device="cuda")), dict(seq_lens=lens.long()),
                dict(block_table=table.t()), dict(workspace=torch.empty(64, dtype=torch.uint8)),
                dict(dev_err=torch.zeros(1, device="cuda"))):
        args = dict(q_bf16=f, kv_pool=pool, block_table=table, seq_lens=lens, cu_q=cu, scale=SCALE, out=out, workspace=ws)
        args.update(bad)
        with pytest.raises(ValueError):
            capi.dsa_dense_mla_decode(**args)
    with pytest.raises(capi.DSAError):
        capi.dsa_dense_mla_decode(f, pool, table, lens, cu, SCALE, out, ws[:64])
    p = torch.zeros(4, 8, device="cuda")
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    u, us, acc = torch.zeros(4, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        capi.dsa_verify_drafts(p, tok, cu, u, us, tok, acc)                    # in place
    with pytest.raises(ValueError):
        capi.dsa_verify_drafts(p, tok, cu, u, us, tok.clone(), acc, draft_probs=p[:, :7])
    x = torch.zeros(4, 584, dtype=torch.bfloat16, device="cuda")
    w, cs = torch.ones(512, device="cuda"), torch.zeros(4, 64, device="cuda")
    i64 = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(capi.DSAError):
        capi.dsa_store_latent_prologue(x[:, 4:580], w, 1e-6, cs, i64, i64, pool)     # rows not 16-byte aligned
    with pytest.raises(ValueError):
        capi.dsa_store_latent_prologue(x[:, :576], w, 1e-6, cs, i64[:3], i64, pool)


def test_device_batch_dense_attention():
    from deepseek_sparse_attention_paged_gb300 import workloads
    from deepseek_sparse_attention_paged_gb300.pipeline import DeviceBatch
    wl = workloads.make("tiny")
    db = DeviceBatch(wl, build_index_cache=False)
    db.dense_mla()
    r = ref.decode(db.mla_q, db.kv_pool, db.block_table, wl.seq_lens.tolist(), wl.q_lens.tolist(), wl.scale)
    ref.check(db.out, db.lse, r)
    assert db.device_error() == (0, 0)


def test_decode_extreme_lengths_and_ranges_outside_the_rows():
    """The smallest int32 as a length sees nothing; a length past the table is cut to it; cu_q outside [0, T] is
    cut to it; each but the first is reported."""
    lens, q_lens = [100, 200, 300], [1, 2, 1]
    q, pool, table = _decode_inputs(lens, q_lens, 16, 71)
    err = _err()
    out, lse = _decode(q, pool, table, [-2 ** 31, 200, -2 ** 31 + 1], q_lens, err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    ref.check(out, lse, ref.decode(q, pool, table, [0, 200, 0], q_lens, SCALE))
    table[1, :] = table[1, 0]
    out, lse = _decode(q, pool, table, [100, 2 ** 31 - 1, 300], q_lens, err)
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_INDEX_RANGE)
    for r in (0, 3):
        one = ref.decode(q[r:r + 1], pool, table[[0 if r == 0 else 2]].contiguous(), [100 if r == 0 else 300], [1], SCALE)
        ref.check(out[r:r + 1], lse[r:r + 1], one)
    err.zero_()
    out = torch.full((4, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    two = table[:2].contiguous()
    capi.dsa_dense_mla_decode(q, pool, two, _i32([100, 300]), _i32([-3, 1, 900]), SCALE, out, dev_err=err)
    assert capi.dsa_read_device_error(err) == (capi.DSA_ERR_DEVICE_BOUNDS, capi.DSA_DEVERR_INDEX_RANGE)
    want = ref.decode(q, pool, two, [100, 300], [1, 3], SCALE)
    assert bool(((out.double() - want[0]).abs() <= want[2]).all())


@pytest.mark.parametrize("H,lens,q_lens", [(16, [9000, 5000, 7777], [5, 1, 7]), (32, [20000, 64], [3, 4]),
                                           (16, [130 * i for i in range(1, 60)], [1 + i % 9 for i in range(59)])])
def test_decode_split_row_tiles_that_are_not_full(H, lens, q_lens):
    """Pieces of row tiles with few rows, next to whole ones: nothing behind their rows is written."""
    q, pool, table = _decode_inputs(lens, q_lens + [2], H, 72 + H)
    out, lse = _decode(q, pool, table, lens, q_lens)
    T = sum(q_lens)
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    ref.check(out[:T], lse[:T], ref.decode(q[:T], pool, table, lens, q_lens, SCALE))


@pytest.mark.parametrize("causal", [True, False])
def test_prefill_items_of_every_shape_after_one_another(causal):
    """Each CTA takes several items in turn: query tiles without rows or without visible keys, single key tiles,
    key tails, requests without keys, in changing order."""
    shapes = [(300, 100), (300, 40), (257, 1), (512, 130), (1, 1), (256, 256), (129, 129), (128, 500), (400, 0), (700, 690),
              (1, 513), (130, 300), (384, 129), (2, 0), (513, 900)]
    order = torch.randperm(3 * len(shapes), generator=_gen(73)).tolist()
    q_lens = [shapes[i % len(shapes)][0] for i in order]
    k_lens = [shapes[i % len(shapes)][1] for i in order]
    q, kv, lat = _prefill_inputs(q_lens, k_lens, 24, 74)
    out, lse = _prefill(q, kv, lat, q_lens, k_lens, causal)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], q_lens, k_lens, SCALE, causal))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,q_lens,k_lens", [
    (2, [40], [3000]), (40, [10], [2500]), (1, [1], [5000]), (1, [4000], [4000]), (2, [1500], [1500]),
    (3, [300, 1, 7], [2000, 6000, 1]),              # parts without a key tile beside long ones
    (2, [500, 3, 0, 2], [400, 9000, 30, 0]),        # rows that see nothing, no rows, no keys
    (16, [1000], [4100]), (9, [257], [2561]),
])
def test_prefill_keys_split_over_a_cluster(H, q_lens, k_lens, causal):
    """Few items with many keys: several CTAs share an item's keys and join their parts."""
    q, kv, lat = _prefill_inputs(q_lens, k_lens, H, 800 + sum(k_lens), extra=5)
    T, S = sum(q_lens), sum(k_lens)
    kv[S:], lat[S:] = math.nan, math.nan
    err = _err()
    out, lse = _prefill(q, kv, lat, q_lens, k_lens, causal, err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    ref.check(out[:T], lse[:T], ref.prefill(q[:T], kv[:S, :, :128], lat[:S, 512:], kv[:S, :, 128:], q_lens, k_lens, SCALE,
                                            causal))


def test_prefill_split_keys_extreme_scores_graph_and_streams():
    """Parts whose maxima are far apart; the same bits again, on two streams at once and from a graph."""
    q_lens, k_lens = [70], [4000]
    q, kv, lat = _prefill_inputs(q_lens, k_lens, 3, 91)
    kv[1000:2000, :, :128] *= 30
    kv[3500:, :, :128] = 0
    lat[3500:, 512:] = 0
    out, lse = _prefill(q, kv, lat, q_lens, k_lens)
    ref.check(out, lse, ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], q_lens, k_lens, SCALE, True))
    cu, ck = _i32(_cum(q_lens)), _i32(_cum(k_lens))

    def call(o, l):
        capi.dsa_dense_mla_prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], cu, ck, SCALE, o, lse=l)

    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [(torch.zeros_like(out), torch.zeros_like(lse)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (o, l) in zip(streams, outs):
            with torch.cuda.stream(s):
                call(o, l)
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, out) and torch.equal(l, lse)
    o, l = torch.zeros_like(out), torch.zeros_like(lse)
    with torch.cuda.stream(streams[0]):
        call(o, l)
        streams[0].synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=streams[0]):
            call(o, l)
    o.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)


@pytest.mark.parametrize("H,per", [(16, 8), (32, 4), (64, 2)])
def test_decode_row_tiles_of_changing_height_after_one_another(H, per):
    """Many short row tiles in turn in each cluster, full ones and ones with few rows in changing order, with one to
    three key tiles: what the scores' CTA sends ahead for the next one stays."""
    g = _gen(95 + H)
    B = 500
    lens = (torch.randint(1, 130, (B,), generator=g) + 128 * (torch.rand(B, generator=g) < 0.2)).tolist()
    q_lens = torch.randint(1, 2 * per, (B,), generator=g).tolist()
    q, pool, table = _decode_inputs(lens, q_lens, H, 96 + H)
    want = ref.decode(q, pool, table, lens, q_lens, SCALE)
    for _ in range(5):
        out, lse = _decode(q, pool, table, lens, q_lens)
        ref.check(out, lse, want)


def test_decode_short_row_tiles_behind_ones_that_see_nothing():
    """Row tiles of one key tile behind low ones and ones without a visible key, whose zeros take the output's CTA
    long: P of the row tile after next is there before it has begun the next."""
    lens = [18, 4116, 6914, 0, 1, 1805, 3, 2657, 13815, 2, 32, 66, 3977]
    q_lens = [2, 37, 2, 38, 31, 30, 28, 21, 26, 39, 4, 24, 8]
    q, pool, table = _decode_inputs(lens, q_lens, 32, 99)
    out, lse = _decode(q, pool, table, lens, q_lens)
    ref.check(out, lse, ref.decode(q, pool, table, lens, q_lens, SCALE))


def test_verify_accepts_at_the_border_down_to_the_smallest_numbers():
    """u q < p without a rounding, also where the product or its error lies below fp32's smallest numbers: p is u q
    rounded, for random u and q of every magnitude, and the neighbours of such a p."""
    g = _gen(63)
    n = 4000
    q = torch.ldexp(1 + torch.rand(n, generator=g), -torch.randint(1, 150, (n,), generator=g).float()).float()
    u = torch.ldexp(torch.randint(1, 2 ** 24, (n,), generator=g).float(), -torch.randint(24, 40, (n,), generator=g).float())
    q[:4] = torch.tensor([2.0 ** -126, 2.0 ** -126, 2.0 ** -126, 3 * 2.0 ** -149])
    u[:4] = torch.tensor([0.5 - 2.0 ** -25, 0.5, 0.5 + 2.0 ** -24, 11184810 * 2.0 ** -25])
    exact = u.double() * q.double()
    p = exact.float()
    step = torch.randint(-1, 2, (n,), generator=g)
    step[:4] = 0
    p = torch.where(step > 0, torch.nextafter(p, torch.tensor(2.0)), torch.where(step < 0, torch.nextafter(p, torch.tensor(0.0)), p))
    V = 4
    target, draft = torch.zeros(2 * n, V), torch.zeros(2 * n, V)
    target[:, 2] = 1.0
    target[0::2, 1], draft[0::2, 1] = p, q
    tok = torch.tensor([1, -1] * n, dtype=torch.int32)
    ua = torch.zeros(2 * n)
    ua[0::2] = u
    got = _verify(target, draft, tok, [2] * n, ua, torch.full((n,), 0.5))
    wrong = torch.nonzero(torch.tensor(got[1]) != (exact < p.double()).int())[:, 0].tolist()
    assert not wrong, f"{len(wrong)} of {n}, the first {wrong[:5]}"
    assert got[1][:4] == [1, 0, 0, 1]


def test_device_batch_dense_attention_on_another_stream():
    """The workspace is the batch's own from the start: a first call on a stream of its own neither waits for the
    current stream nor takes memory that work there still uses."""
    from deepseek_sparse_attention_paged_gb300 import workloads
    from deepseek_sparse_attention_paged_gb300.pipeline import DeviceBatch
    wl = workloads.make_custom("dense_on_a_stream", 262, [700, 90], 1, topk=64, heads=128)
    db = DeviceBatch(wl, build_index_cache=False)
    size = max(16, capi.dsa_dense_mla_decode_workspace_size(wl.T, wl.heads))
    capi.dsa_dense_mla_decode(db.mla_q, db.kv_pool, db.block_table, db.seq_lens, db.cu_q, wl.scale, db.out)   # loaded
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    a = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    b = torch.zeros_like(a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    b.copy_(a)
    del a
    db.dense_mla(stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert bool((b == 255).all())
    r = ref.decode(db.mla_q, db.kv_pool, db.block_table, wl.seq_lens.tolist(), wl.q_lens.tolist(), wl.scale)
    ref.check(db.out, db.lse, r)


def test_device_batch_dense_attention_first_called_in_a_capture():
    """The first dense call is a captured one: the workspace is not the graph's, and outlives it."""
    from deepseek_sparse_attention_paged_gb300 import workloads
    from deepseek_sparse_attention_paged_gb300.pipeline import DeviceBatch
    wl = workloads.make("tiny")
    db = DeviceBatch(wl, build_index_cache=False)
    ws = db.dense_ws.data_ptr()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            db.dense_mla()
    gr.replay()
    torch.cuda.synchronize()
    r = ref.decode(db.mla_q, db.kv_pool, db.block_table, wl.seq_lens.tolist(), wl.q_lens.tolist(), wl.scale)
    ref.check(db.out, db.lse, r)
    del gr
    db.out.zero_()
    db.dense_mla()
    ref.check(db.out, db.lse, r)
    assert db.dense_ws.data_ptr() == ws


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("H,nq,nk,at", [(2, 128, 228, 200), (2, 300, 401, 128), (2, 300, 401, 290), (1, 70, 4000, 3950),
                                        (3, 513, 1000, 600), (40, 400, 1500, 1111)])
def test_prefill_bad_values_within_a_request_reach_what_is_documented(H, nq, nk, at, bad):
    """A value that is not finite reaches a query that does not see its position only where another query of its
    group of 128 sees a key of the same 128; queries that see it get what the formula gives; a key there reaches
    no query that does not see it."""
    q, kv, lat = _prefill_inputs([nq], [nk], H, 900 + nk + at)
    want = ref.prefill(q, kv[..., :128], lat[:, 512:], kv[..., 128:], [nq], [nk], SCALE, True)
    kv[at, :, 128:] = bad
    out, lse = _prefill(q, kv, lat, [nq], [nk])
    seen = nk - nq + 1 + torch.arange(nq)
    last = torch.minimum((torch.arange(nq) // 128 + 1) * 128, torch.tensor(nq)) - 1
    clean = torch.nonzero((seen[last] + 127) // 128 <= at // 128)[:, 0].cuda()
    ref.check(out[clean], lse, tuple(t[clean] if i % 2 == 0 else t for i, t in enumerate(want)))
    sees = torch.nonzero(seen > at)[:, 0].cuda()
    assert not bool(out[sees].isfinite().any())
    kv[at, :, 128:], kv[at, :, :128] = 0.0, bad
    blind = torch.nonzero(seen <= at)[:, 0].cuda()
    out, lse = _prefill(q, kv, lat, [nq], [nk])
    ref.check(out[blind], lse[blind], tuple(t[blind] for t in want))


def test_verify_beside_its_drafts_and_not_over_them():
    """One buffer for drafts and outputs: apart works, half over each other is refused before anything runs."""
    p, d, tok, u, us = _verify_inputs([4, 4], 700, 64)
    buf = torch.full((24,), -7, dtype=torch.int32, device="cuda")
    buf[8:16] = tok.cuda()
    acc = torch.zeros(2, dtype=torch.int32, device="cuda")
    args = (p.cuda(), buf[8:16], _i32([0, 4, 8]), u.cuda(), us.cuda())
    for at in (1, 4, 7, 9, 12, 15):
        with pytest.raises(ValueError):
            capi.dsa_verify_drafts(*args, buf[at:at + 8], acc, draft_probs=d.cuda())
    assert bool((buf[:8] == -7).all()) and bool((buf[16:] == -7).all()) and torch.equal(buf[8:16].cpu(), tok)
    want = ref.verify(p, d, tok.tolist(), [0, 4, 8], u, us)
    for at in (0, 16):
        capi.dsa_verify_drafts(*args, buf[at:at + 8], acc, draft_probs=d.cuda())
        assert (buf[at:at + 8].tolist(), acc.tolist()) == want


def test_binding_refuses_what_the_prefill_does_not_take():
    q = torch.zeros(6, 2, 192, dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(9, 2, 256, dtype=torch.bfloat16, device="cuda")
    lat = torch.zeros(9, 576, dtype=torch.bfloat16, device="cuda")
    out = torch.full((6, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    good = dict(q=q, k_nope=kv[..., :128], k_pe=lat[:, 512:], v=kv[..., 128:], cu_q=_i32([0, 4, 6]), cu_k=_i32([0, 4, 9]),
                scale=SCALE, out=out)
    for bad in (dict(q=q.half()), dict(q=q[..., :128]), dict(q=q[0]), dict(q=q.cpu()), dict(k_nope=kv[:8, :, :128]),
                dict(k_nope=kv[:, :1, :128]), dict(k_nope=kv), dict(v=kv[:8, :, 128:]), dict(v=kv[..., 128:].float()),
                dict(v=kv[:, :1, 128:]), dict(k_pe=lat[:, 504:]), dict(k_pe=lat[:8, 512:]), dict(k_pe=lat),
                dict(k_pe=torch.zeros(64, 9, dtype=torch.bfloat16, device="cuda").t()), dict(cu_q=_i32([0, 6])),
                dict(cu_k=_i32([0, 9])), dict(cu_q=_i32([])), dict(cu_q=torch.tensor([0, 4, 6]).cuda()),
                dict(cu_k=torch.tensor([0, 4, 9], dtype=torch.int32)), dict(out=out[:5]), dict(out=out[:, :1]),
                dict(out=out.float()), dict(out=out.transpose(1, 2)), dict(lse=torch.zeros(6, 3, device="cuda")),
                dict(lse=torch.zeros(6, 2, dtype=torch.float64, device="cuda")), dict(dev_err=torch.zeros(1, device="cuda"))):
        with pytest.raises(ValueError):
            capi.dsa_dense_mla_prefill(**{**good, **bad})
    wide = torch.zeros(6, 2, 200, dtype=torch.bfloat16, device="cuda")
    odd = torch.zeros(9, 2, 260, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=wide[..., 4:196]), dict(k_nope=odd[..., :128]), dict(v=odd[..., 132:]), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(out=out[:1].expand(6, 2, 128)),
                dict(k_pe=lat[:1, 512:].expand(9, 64))):
        with pytest.raises(capi.DSAError):
            capi.dsa_dense_mla_prefill(**{**good, **bad})
    torch.cuda.synchronize()
    assert bool((out == 7.0).all())                              # nothing ran
    capi.dsa_dense_mla_prefill(**good)
    assert bool((out == 0).all())
