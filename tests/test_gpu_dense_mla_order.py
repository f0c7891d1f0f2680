"""GPU tests of the order of calls: the dense calls launch as programmatic dependents of whatever precedes them on the
stream, so each has to wait on the device for it, and what follows for them."""
import pytest
import torch

from deepseek_sparse_attention_paged_gb300 import capi
from test_gpu_dense_mla import SCALE, _decode_inputs, _gen, _i32

pytestmark = pytest.mark.gpu


def _order_inputs(H, seed):
    g = _gen(seed)
    n, lens = 131072, [60000, 64, 40000, 31007]                 # the store writes every key of the batch, and one more
    q, pool, table = _decode_inputs(lens, [1] * 4, H, seed)
    pos_in = [torch.arange(m) for m in lens]
    slots = torch.cat([table[b].cpu().long()[p // 64] * 64 + p % 64 for b, p in enumerate(pos_in)] +
                      [torch.full((n - sum(lens),), -1)])
    raw = torch.randn(n, 576, generator=g).to(torch.bfloat16)
    ang = torch.rand(300, 32, generator=g, dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, 300, (n,), generator=g)
    return [t.cuda() for t in (raw, torch.ones(512), cs, pos, slots, q, pool, table)] + [lens]


@pytest.mark.parametrize("H", [128, 16])
def test_dense_calls_back_to_back_keep_stream_order(H):
    """Calls that launch as programmatic dependents, one directly behind the other with no other work between them: a
    long store, then the attentions (dense, sparse) that read its rows and queries written just before it, then a
    store over the same rows while they may still be read; then the store's dense rows into the prompt's attention.
    Everything as with a synchronisation after each call, bit for bit."""
    raw, w, cs, pos, slots, q, pool, table, lens = _order_inputs(H, 120 + H)
    T, k = 4, 512
    raw2 = raw.flip(0).contiguous()
    seq, cu = _i32(lens), _i32([0, 1, 2, 3, 4])
    idx = torch.stack([torch.randperm(m, generator=_gen(5))[:k].sort().values if m >= k else
                       torch.cat([torch.arange(m), torch.full((k - m,), -1)]) for m in lens]).int().cuda()
    ws = torch.empty(capi.dsa_dense_mla_decode_workspace_size(T, H), dtype=torch.uint8, device="cuda")
    sws = torch.empty(capi.dsa_sparse_mla_workspace_size(T, H, k) + 16, dtype=torch.uint8, device="cuda")
    dense, sparse = (torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    lse = [torch.empty(T, H, device="cuda") for _ in range(2)]
    lat = torch.empty(raw.shape[0], 576, dtype=torch.bfloat16, device="cuda")
    pq = torch.randn(300, 2, 192, generator=_gen(6)).to(torch.bfloat16).cuda()
    kv = torch.randn(20000, 2, 256, generator=_gen(7)).to(torch.bfloat16).cuda()
    pout = torch.empty(300, 2, 128, dtype=torch.bfloat16, device="cuda")
    pcu, pck = _i32([0, 300]), _i32([0, 20000])
    qbuf, pool0 = torch.empty_like(q), pool.clone()

    def calls(sync, attention):
        qbuf.zero_()
        pool.copy_(pool0)
        for t in (dense, sparse, lat, pout):
            t.fill_(7.0)
        torch.cuda.synchronize()
        store = lambda x: capi.dsa_store_latent_prologue(x, w, 1e-6, cs, pos, slots, pool, latent_out=lat)   # noqa: E731
        torch.mul(q, 1.0, out=qbuf)
        sync()
        store(raw)
        sync()
        if attention == "dense":
            capi.dsa_dense_mla_decode(qbuf, pool, table, seq, cu, SCALE, dense, ws, lse=lse[0])
            sync()
        if attention == "sparse":
            capi.dsa_sparse_mla_decode(qbuf, pool, table, seq, cu, idx, SCALE, sparse, sws, lse=lse[1])
            sync()
        if attention == "prefill":
            capi.dsa_dense_mla_prefill(pq, kv[..., :128], lat[-20000:, 512:], kv[..., 128:], pcu, pck, SCALE, pout)
            sync()
        store(raw2)
        sync()
        capi.dsa_dense_mla_prefill(pq, kv[..., :128], lat[:20000, 512:], kv[..., 128:], pcu, pck, SCALE, pout)
        sync()
        torch.cuda.synchronize()
        return [t.clone() for t in (dense, sparse, lat, pout, pool)]

    for attention in ("dense", "sparse", "prefill"):
        want = calls(torch.cuda.synchronize, attention)
        for _ in range(5):
            for got, t in zip(calls(lambda: None, attention), want):
                assert torch.equal(got, t)
    assert not torch.equal(want[4], pool0)


def test_verify_behind_the_calls_that_make_its_inputs():
    """Verification directly behind a long store and in front of another verification that overwrites its outputs."""
    raw, w, cs, pos, slots, q, pool, table, lens = _order_inputs(16, 140)
    g = _gen(141)
    T, V = 64, 50000
    p, d = (torch.softmax(torch.randn(T, V, generator=g) * 2, 1).cuda() for _ in range(2))
    tok = torch.randint(0, V, (T,), generator=g).int().cuda()
    u, us = torch.rand(T, generator=g).cuda(), torch.rand(16, generator=g).cuda()
    cu = _i32(list(range(0, 65, 4)))
    out = [torch.full((T,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    acc = [torch.full((16,), -7, dtype=torch.int32, device="cuda") for _ in range(2)]
    pbuf = torch.zeros_like(p)

    def calls(sync):
        pbuf.zero_()
        torch.cuda.synchronize()
        capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, slots, pool)
        sync()
        torch.mul(p, 1.0, out=pbuf)
        sync()
        capi.dsa_verify_drafts(pbuf, tok, cu, u, us, out[0], acc[0], draft_probs=d)
        sync()
        capi.dsa_verify_drafts(pbuf, out[0], cu, u, us, out[1], acc[1], draft_probs=d)     # what the first one left
        sync()
        capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, slots, pool)
        torch.cuda.synchronize()
        return [t.clone() for t in out + acc]

    want = calls(torch.cuda.synchronize)
    for _ in range(5):
        for got, t in zip(calls(lambda: None), want):
            assert torch.equal(got, t)


@pytest.mark.parametrize("fork", [False, True])
def test_a_captured_step_replayed_on_other_inputs(fork):
    """Store, decode, prompt and verification in one graph, on one stream or with the prompt on a second one that
    starts behind the store and is waited for by the verification; each replay gives what the calls give one by one."""
    H, n, lens = 16, 40000, [20000, 64, 15000, 4000]
    q, pool, table = _decode_inputs(lens, [1] * 4, H, 150)
    raws = [torch.randn(n, 576, generator=_gen(151 + i)).to(torch.bfloat16).cuda() for i in range(2)]
    slots = torch.cat([table[b].cpu().long()[torch.arange(m) // 64] * 64 + torch.arange(m) % 64 for b, m in enumerate(lens)] +
                      [torch.full((n - sum(lens),), -1)]).cuda()
    pos, w = torch.arange(n).cuda() % 300, torch.ones(512, device="cuda")
    ang = torch.rand(300, 32, generator=_gen(153), dtype=torch.float64) * 6.3
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().cuda()
    raw, lat = torch.empty_like(raws[0]), torch.empty_like(raws[0])
    pq = torch.randn(300, 2, 192, generator=_gen(154)).to(torch.bfloat16).cuda()
    kv = torch.randn(9000, 2, 256, generator=_gen(155)).to(torch.bfloat16).cuda()
    ws = torch.empty(capi.dsa_dense_mla_decode_workspace_size(4, H), dtype=torch.uint8, device="cuda")
    out = torch.empty(4, H, 512, dtype=torch.bfloat16, device="cuda")
    pout = torch.empty(300, 2, 128, dtype=torch.bfloat16, device="cuda")
    lse, probs = torch.empty(4, H, device="cuda"), torch.empty(4, 300 * 2 * 32, device="cuda")
    tok, acc = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    seq, cu, pcu, pck, vcu = _i32(lens), _i32([0, 1, 2, 3, 4]), _i32([0, 300]), _i32([0, 9000]), _i32([0, 3, 4])
    draft = _i32([5, 9, -1, -1])
    u, us = torch.full((4,), 1e-4, device="cuda"), torch.tensor([0.3, 0.8], device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step(sync, forked):
        capi.dsa_store_latent_prologue(raw, w, 1e-6, cs, pos, slots, pool, latent_out=lat)
        sync()
        if forked:
            side.wait_stream(main)
        with torch.cuda.stream(side if forked else torch.cuda.current_stream()):
            capi.dsa_dense_mla_prefill(pq, kv[..., :128], lat[:9000, 512:], kv[..., 128:], pcu, pck, SCALE, pout)
        sync()
        capi.dsa_dense_mla_decode(q, pool, table, seq, cu, SCALE, out, ws, lse=lse)
        sync()
        if forked:
            main.wait_stream(side)
        torch.softmax(pout.view(4, -1).float() * out.float().mean(), 1, out=probs)
        sync()
        capi.dsa_verify_drafts(probs, draft, vcu, u, us, tok, acc)
        sync()

    results = (pool, lat, out, lse, pout, probs, tok, acc)
    want = []
    for r in raws:
        raw.copy_(r)
        step(torch.cuda.synchronize, False)
        want.append([t.clone() for t in results])
    assert not torch.equal(want[0][2], want[1][2])
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=main):
            step(lambda: None, fork)
        for i in (0, 1, 1, 0, 1):
            for t in (out, pout, lat):
                t.fill_(7.0)
            raw.copy_(raws[i])
            gr.replay()
            main.synchronize()
            for got, t in zip(results, want[i]):
                assert torch.equal(got, t)
