"""GPU tests of the dense attention calls at long contexts: every page's weight shows in the output
(dense_mla_marked), so a key tile lost or counted twice where the work is split is seen at any length."""
import pytest
import torch

import dense_mla_marked as marked
from deepseek_sparse_attention_paged_gb300 import capi

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5
Q_VALUE = 10.0            # times SCALE 0.72 a level


def _i32(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _cum(ns):
    c = [0]
    for n in ns:
        c.append(c[-1] + n)
    return c


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("H,lens,q_lens", [
    (128, [131072], [1]), (16, [131073, 131000], [2, 1]),        # over the whole GPU; both halves of it
    (128, [76 * 14 * 128], [1]), (64, [76 * 14 * 128 + 1], [1]), (32, [76 * 14 * 128 - 127], [3]),   # whole shares, +-
    (128, [215001], [1]),                                        # shares of more than 16 tiles
    (16, [100000, 39999, 64, 20000, 0, 65], [2, 1, 1, 4, 1, 1]), (64, [70000 + 1111 * i for i in range(9)], [1] * 9),
])
def test_decode_long_contexts_count_every_page_once(H, lens, q_lens, flat):
    gain = marked.gain_of(Q_VALUE, SCALE)
    g = torch.Generator().manual_seed(1000 + sum(lens) + H)
    pages = [(n + 63) // 64 for n in lens]
    perm = torch.randperm(sum(pages) + 2, generator=g)
    pool = torch.zeros(sum(pages) + 2, 64, 576, dtype=torch.bfloat16, device="cuda")
    table = torch.full((len(lens), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        ids = perm[at:at + n]
        at += n
        table[b, :n] = ids
        ids = ids.cuda()
        pool[ids, :, marked.marker_of(n, 512, b).cuda()] = 1.0
        pool[ids, :, 520] = marked.levels(n, flat).cuda()[:, None].to(torch.bfloat16)
    T = sum(q_lens)
    q = torch.zeros(T, H, 576, dtype=torch.bfloat16, device="cuda")
    q[..., 520] = Q_VALUE
    out = torch.full((T, H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.dsa_dense_mla_decode(q, pool, table.cuda(), _i32(lens), _i32(_cum(q_lens)), SCALE, out, lse=lse, dev_err=err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    r = 0
    for b, (n, m) in enumerate(zip(lens, q_lens)):
        vis = [n - m + j + 1 for j in range(m) if n - m + j + 1 > 0]
        if vis:
            w, want_lse = marked.weights(vis, marked.levels(pages[b], flat), gain)
            want = marked.outputs(w, marked.marker_of(pages[b], 512, b), 512)
            rows = slice(r + m - len(vis), r + m)
            marked.check(out[rows], lse[rows], want[:, None], want_lse[:, None])
        r += m


@pytest.mark.parametrize("flat", [True, False])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,q_lens,k_lens", [
    (2, [300], [40000]), (1, [130], [60001]),                    # the keys split over clusters
    (40, [257], [20001]), (24, [700, 1, 129], [9001, 16000, 12345]),
])
def test_prefill_long_contexts_count_every_page_once(H, q_lens, k_lens, causal, flat):
    gain = marked.gain_of(Q_VALUE, SCALE)
    T, S = sum(q_lens), sum(k_lens)
    q = torch.zeros(T, H, 192, dtype=torch.bfloat16, device="cuda")
    q[..., 130] = Q_VALUE
    kv = torch.zeros(S, H, 256, dtype=torch.bfloat16, device="cuda")
    pe = torch.zeros(S, 64, dtype=torch.bfloat16, device="cuda")
    k0 = 0
    for b, n in enumerate(k_lens):
        page = torch.arange(n) // 64
        pages = int(page[-1]) + 1
        pe[k0:k0 + n, 2] = marked.levels(pages, flat)[page].to(torch.bfloat16).cuda()
        for h in range(H):
            kv[torch.arange(k0, k0 + n).cuda(), h, 128 + marked.marker_of(pages, 128, b + h)[page].cuda()] = 1.0
        k0 += n
    out = torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    capi.dsa_dense_mla_prefill(q, kv[..., :128], pe, kv[..., 128:], _i32(_cum(q_lens)), _i32(_cum(k_lens)), SCALE, out,
                               lse=lse, causal=causal, dev_err=err)
    assert capi.dsa_read_device_error(err) == (0, 0)
    r = 0
    for b, (m, n) in enumerate(zip(q_lens, k_lens)):
        vis = [n - m + j + 1 for j in range(m)] if causal else [n] * m
        pages = (n + 63) // 64
        w, want_lse = marked.weights(vis, marked.levels(pages, flat), gain)
        for h in range(H):
            marked.check(out[r:r + m, h], lse[r:r + m, h], marked.outputs(w, marked.marker_of(pages, 128, b + h), 128), want_lse)
        r += m
