"""GPU tests of the calls around a serving step at large sizes and directly behind one another: every page of a long shared
prefix counts once (dense_mla_marked), batches of many units, order on the stream, large batches of rows to sample."""
import math
import threading

import numpy as np
import pytest
import torch

import dense_mla_marked as marked
import dense_mla_ref
from deepseek_sparse_attention_paged_gb300 import capi
from test_gpu_serving_step import SCALE, _check_sample, _check_shared, _cum, _err, _f32, _i32, _logits, _run_sample, _shared_inputs

pytestmark = pytest.mark.gpu

Q_VALUE = 10.0            # times SCALE 0.72 a level


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("H,prefix,own,q_len", [
    (16, 131008, [1 + 37 * i for i in range(40)], 1),            # units of 16 requests, split over many clusters
    (128, 70016, [5, 64, 65, 1000, 12000], 1), (64, 100032, [3, 4, 5], 3), (32, 40000 // 64 * 64, [700] * 9, 2),
    (16, 36 * 14 * 128, [64] * 16, 1), (16, 36 * 14 * 128 - 64, [128] * 17, 1),   # whole shares, and not
])
def test_shared_long_prefixes_count_every_page_once(H, prefix, own, q_len, flat):
    gain = marked.gain_of(Q_VALUE, SCALE)
    B, shared = len(own), prefix // 64
    lens = [prefix + n + q_len - 1 for n in own]
    pages = [(n + 63) // 64 for n in lens]
    total = shared + sum(n - shared for n in pages) + 2
    perm = torch.randperm(total, generator=torch.Generator().manual_seed(prefix + H))
    pool = torch.zeros(total, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((B, max(pages)), -1, dtype=torch.int32)
    most = max(pages)
    marker, level = marked.marker_of(most, 512), marked.levels(most, flat)
    at = shared
    for b, n in enumerate(pages):
        ids = torch.cat([perm[:shared], perm[at:at + n - shared]])
        at += n - shared
        table[b, :n] = ids
        dev = ids.cuda()
        pool[dev, :, marker[:n].cuda()] = 1.0
        pool[dev, :, 520] = level[:n].cuda()[:, None].to(torch.bfloat16)
    T = B * q_len
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 520] = Q_VALUE
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = _err()
    capi.dsa_dense_mla_decode_shared(q, pool, table.cuda(), _i32(lens), _i32(_cum([q_len] * B)), _i32([0, B]), _i32([prefix]),
                                     SCALE, out, lse=lse, dev_err=err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    for b, n in enumerate(lens):
        vis = [n - q_len + j + 1 for j in range(q_len)]
        w, want_lse = marked.weights(vis, level[:pages[b]], gain)
        rows = slice(b * q_len, (b + 1) * q_len)
        marked.check(out[rows], lse[rows], marked.outputs(w, marker[:pages[b]], 512)[:, None], want_lse[:, None])


@pytest.mark.parametrize("H,n", [(16, 1100), (128, 150)])
def test_shared_many_units(H, n):
    """More units than are looked at by a warp each; groups of all sizes, some empty, requests without rows."""
    groups, left, i = [], n, 0
    while left > 0:
        k = min(left, [1, 40, 0, 7, 300, 16, 0, 33][i % 8])
        groups.append((64 * (i % 4), [(1 + (13 * (i + j)) % 150, (j % 5 != 3) + (j % 11 == 0)) for j in range(k)]))
        left -= k
        i += 1
    _check_shared(_shared_inputs(groups, H, 40 + H, alone=5))


def test_calls_back_to_back_keep_stream_order():
    """Each call behind one that makes its inputs, with no other work between them: as with a synchronisation after each,
    bit for bit."""
    H, V, B = 16, 32000, 8
    q, pool0, table, lens, q_lens, cg, sh = _shared_inputs([(16384, [(64 * (i + 1), 1) for i in range(B)])], H, 50)
    n = 60000
    slots = torch.full((n,), -1, dtype=torch.int64)
    flat = (table[0, :256].long()[:, None] * 64 + torch.arange(64)[None]).reshape(-1)
    slots[-flat.numel():] = flat                                 # the last rows of a long store are the prefix
    raw = torch.randn(n, 576, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    ang = torch.rand(300, 32, generator=torch.Generator().manual_seed(2)) * 6.3
    cs, w = torch.cat([ang.cos(), ang.sin()], 1).cuda(), torch.ones(512, device="cuda")
    pos_in = torch.randint(0, 300, (n,), generator=torch.Generator().manual_seed(3)).cuda()
    pool, slots, qd, td = pool0.cuda(), slots.cuda(), q.cuda(), table.cuda()
    u = torch.rand(3, B, generator=torch.Generator().manual_seed(4)).cuda()
    cached, qn, counts = _i32([m - 1 for m in lens]), _i32([1] * B), _i32([(m + 63) // 64 for m in lens])
    stack, top = _i32(list(range(64))), _i32([10])
    seq, cnt, have, cu = _i32([0] * B), _i32([0] * B), _i32([0]), _i32([0] * (B + 1))
    pos, sm = torch.zeros(B, dtype=torch.int64, device="cuda"), torch.zeros(B, dtype=torch.int64, device="cuda")
    out = torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(capi.dsa_dense_mla_decode_shared_workspace_size(B, H), dtype=torch.uint8, device="cuda")
    probs, tokens, res, acc = torch.empty(B, V, device="cuda"), _i32([0] * B), _i32([0] * B), _i32([0] * B)
    logits = _logits(B, V, 5, False).cuda()
    st = torch.full((4096,), -1, dtype=torch.int32, device="cuda")
    st[:64] = stack

    def calls(sync):
        pool.copy_(pool0)
        for t in (seq, cnt, cu, pos, sm, out, probs, tokens, res, acc):
            t.zero_()
        torch.cuda.synchronize()
        capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos_in, slots, pool)
        sync()
        capi.dsa_step_tables(cached, qn, counts, td, 4096, st, top, seq, cnt, have, cu, pos, sm)
        sync()
        capi.dsa_dense_mla_decode_shared(qd, pool, td, seq, cu, _i32(cg), _i32(sh), SCALE, out, ws)
        sync()
        capi.dsa_store_latent_prologue(raw, w, 1e-5, cs, pos_in, slots, pool)   # over rows that may still be read
        sync()
        capi.dsa_sample_tokens(logits, u[0], tokens, top_p=_f32([0.9] * B), probs=probs)
        sync()
        capi.dsa_verify_drafts(probs, tokens, cu, u[1], u[2], res, acc)
        sync()
        capi.dsa_sample_tokens(logits, u[1], tokens, top_k=_i32([20] * B), probs=probs)
        torch.cuda.synchronize()
        return [t.clone() for t in (seq, cnt, have, cu, pos, sm, out, probs, tokens, res, acc, pool)]

    want = calls(torch.cuda.synchronize)
    dense_mla_ref.check(want[6], None, dense_mla_ref.decode(qd, _stored(raw, w, cs, pos_in, slots, pool0), td, lens, q_lens, SCALE))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(calls(lambda: None), want))


def _stored(raw, w, cs, pos, slots, pool0):
    pool = pool0.cuda()
    capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, slots, pool)
    return pool


def test_two_shared_calls_at_once():
    """Two streams, a workspace each: as one after the other, bit for bit."""
    inp = _shared_inputs([(4096, [(30 + i, 1) for i in range(40)])], 16, 60)
    q, pool, table, lens, q_lens, cg, sh = inp
    args = (q.cuda(), pool.cuda(), table.cuda(), _i32(lens), _i32(_cum(q_lens)), _i32(cg), _i32(sh), SCALE)
    size = capi.dsa_dense_mla_decode_shared_workspace_size(q.shape[0], 16)
    outs = [torch.zeros(q.shape[0], 16, 512, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    ws = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    capi.dsa_dense_mla_decode_shared(*args, outs[2], ws[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for s, o, x in zip(streams, outs, ws):
            capi.dsa_dense_mla_decode_shared(*args, o, x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])


@pytest.mark.parametrize("bf16", [False, True])
def test_sample_rows_in_large_batches_as_alone(bf16):
    """The same rows many times over (which are read twice instead of staged): as in a small batch, bit for bit."""
    V, n = 9001, 90
    g = torch.Generator().manual_seed(70)
    x = _logits(8, V, 71, bf16)
    x[0][torch.rand(V, generator=g) < 0.99] = -math.inf
    x[1][torch.rand(V, generator=g) < 0.5] = torch.finfo(x.dtype).min
    x[2][torch.rand(V, generator=g) < 0.5] = math.nan
    x[3] = -math.inf
    x[4, 700] = math.inf
    x[5] = 1.0
    u = [0.1, 0.9, 0.3, 0.5, 0.7, 0.2, 0.6, 0.4]
    for kw in (dict(top_k=[40, 0, 5000, 3, 0, 700, 20, 1]), dict(top_k=[0, 9, 0, 0, 30, 0, 0, 1000], top_p=[0.9, 0.5, 0.99, 0.9, 1.0, 0.5, 0.8, 0.9]),
               dict(top_k=[50] * 8, top_p=[0.95] * 8, min_p=[0.01] * 8, temperature=[0.7, 0.0, 1.3, 1.0, 0.0, 1.0, 2.0, 50.0]),
               dict(top_p=[0.9, 0.5, 0.99, 0.9, 1.0, 0.5, 0.8, 0.9])):
        few = _run_sample(x, V, u, **kw)
        many = _run_sample(x.repeat(n, 1), V, u * n, **{k: v * n for k, v in kw.items()})
        assert many[0] == few[0] * n and few[2] == many[2]
        assert bool((torch.from_numpy(many[1]).view(n, 8, V) == torch.from_numpy(few[1])[None]).all())


@pytest.mark.parametrize("kind", ["usual", "whole", "tiny", "high", "two", "masked"])
def test_sample_top_p_rows_in_large_batches(kind):
    """bf16 rows with top-p alone, as many as make a CTA take each: as in a small batch, bit for bit, odd strides and rows of
    every alignment among them."""
    V, n = 30011, 30
    g = torch.Generator().manual_seed(80 + len(kind))
    x = _logits(8, V, 81, True)
    if kind == "whole":
        x = x.float().round().to(torch.bfloat16)
    elif kind == "tiny":
        x = (x.float() * 1e-4).to(torch.bfloat16)
    elif kind == "high":
        x = (x.float() + 150.0).to(torch.bfloat16)
    elif kind == "two":
        x[:] = -1.0
        x[:, 5::4] = 0.5
    elif kind == "masked":
        x[:, 100:] = torch.where(torch.rand(8, V - 100, generator=g) < 0.9, torch.tensor(-math.inf), x[:, 100:].float()).to(torch.bfloat16)
        x[3] = -math.inf
        x[4, 7:] = math.nan
    u = torch.rand(8, generator=g).tolist()
    for kw in (dict(top_p=[0.9, 0.5, 0.99, 0.1, 0.75, 0.95, 1.0, 0.0]),
               dict(top_p=[0.9, 0.5, 0.99, 0.3, 0.6, 0.95, 0.8, 0.7], temperature=[1.0, 0.0, 0.3, 1.0, 2.0, 8.0, 1.0, 0.9],
                    min_p=[0.0, 0.0, 0.1, 0.5, 0.0, 0.9, 1.0, 0.2])):
        few = _run_sample(x, V, u, **kw)
        for probs in (True, False):
            many = _run_sample(x.repeat(n, 1), V, u * n, probs=probs, **{k: v * n for k, v in kw.items()})
            assert many[0] == few[0] * n and few[2] == many[2]
            if probs:
                assert bool((torch.from_numpy(many[1]).view(n, 8, V) == torch.from_numpy(few[1])[None]).all())


def test_calls_from_two_threads():
    """Two threads with sizes that take different amounts of shared memory, a stream each: no call is refused."""
    sizes = [(3, 200000), (5, 20000)]
    inputs = [(_logits(R, V, 90 + V % 7, False).cuda(), _f32([0.3, 0.6, 0.9, 0.1, 0.5][:R]), _f32([0.9] * R)) for R, V in sizes]
    want = []
    for x, u, p in inputs:
        tokens = _i32([-5] * x.shape[0])
        capi.dsa_sample_tokens(x, u, tokens, top_p=p)
        want.append(tokens.tolist())
    got = [None, None]

    def work(i):
        x, u, p = inputs[i]
        stream = torch.cuda.Stream()
        outs = [_i32([-5] * x.shape[0]) for _ in range(300)]
        torch.cuda.synchronize()
        for out in outs:
            capi.dsa_sample_tokens(x, u, out, top_p=p, stream=stream)
        stream.synchronize()
        got[i] = [o.tolist() for o in outs]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for g, w in zip(got, want):
        assert g == [w] * 300


@pytest.mark.parametrize("V,n,bf16", [(5003, 80, True), (20001, 60, False), (20001, 70, True), (60007, 35, True), (60007, 30, False),
                                      (131072, 25, False), (100003, 40, True)])
def test_sample_top_k_rows_in_large_batches(V, n, bf16):
    """Rows with a top-k in batches that a CTA, or two or four, take a row of: as in a small batch, bit for bit; the largest
    entries all in one place, evenly spread, equal."""
    x = _logits(8, V, 95, False)
    x[0] = x[0].sort(descending=True).values
    x[1] = x[1].sort().values
    x[2, 1000:3100] += 20.0
    x[3] = x[3].round()
    x[4, ::2] = -math.inf
    x[5] = 2.5
    x[6, 600:] = -math.inf
    if bf16:
        x = x.to(torch.bfloat16)
    u = [0.1, 0.9, 0.3, 0.5, 0.7, 0.2, 0.999, 0.4]
    for kw in (dict(top_k=[1024, 1000, 1023, 20, 513, 7, 700, 1]), dict(top_k=[50, 600, 40, 1024, 1, 1024, 50, 1000], top_p=[0.9] * 4 + [1.0] * 4),
               dict(top_k=[0, 1025, 50, 0, 5000, 3, 0, 256], top_p=[0.8, 0.9, 0.99, 0.5, 0.95, 1.0, 0.7, 0.6], min_p=[0.0, 0.1] * 4,
                    temperature=[0.7, 1.0, 0.0, 2.0, 1.0, 1.0, 0.8, 5.0])):
        few = _run_sample(x, V, u, **kw)
        many = _run_sample(x.repeat(n, 1), V, u * n, **{k: v * n for k, v in kw.items()})
        assert many[0] == few[0] * n and few[2] == many[2]
        assert bool((torch.from_numpy(many[1]).view(n, 8, V) == torch.from_numpy(few[1])[None]).all())


@pytest.mark.parametrize("kind", ["distinct", "zeros", "equal"])
def test_sample_top_p_border_among_small_numbers(kind):
    """bf16 rows whose top-p ends within a few hundred numbers next to 0: in the middle of an entry's weight, so that the
    rounding of top_p decides nothing."""
    R, V, n = 8, 20003, 10
    g = torch.Generator().manual_seed(100 + len(kind))
    x = 2.0 * torch.randn(R, V, generator=g)
    x[:, 5::37] = {"distinct": 5e-4, "zeros": 1e-3, "equal": 1e-9}[kind] * torch.randn(R, len(range(5, V, 37)), generator=g)
    if kind == "zeros":
        x[:, 5::74] = 0.0
        x[:, 42::148] = -0.0
    elif kind == "equal":
        x[:, 5::37] = 2.0 ** -12
    x = x.to(torch.bfloat16)
    t = [1.0, 0.7, 1.5, 1.0, 3.0, 20.0, 1.2, 1.0]
    p = []
    for r in range(R):
        z = x[r].double().numpy()
        z = np.sort(z)[::-1]
        w = np.exp((z - z[0]) / np.float32(t[r]).astype(np.float64))
        small = np.flatnonzero(np.abs(z) < 2.0 ** -9)
        at = small[(7 * r + 3) * len(small) // 64]
        p.append(float((w[:at].sum() + 0.5 * w[at]) / w.sum()))
    u = torch.rand(R, generator=g).tolist()
    u[7] = 0.9999999
    for kw in (dict(top_p=p, temperature=t), dict(top_p=p, temperature=t, min_p=[0.0, 1e-9, 0.5, 0.0, 1e-6, 0.0, 0.9, 1e-30])):
        _check_sample(x, V, u, **kw)
        few = _run_sample(x, V, u, **kw)
        for probs in (True, False):
            many = _run_sample(x.repeat(n, 1), V, u * n, probs=probs, **{k: v * n for k, v in kw.items()})
            assert many[0] == few[0] * n and few[2] == many[2]
            if probs:
                assert bool((torch.from_numpy(many[1]).view(n, R, V) == torch.from_numpy(few[1])[None]).all())
