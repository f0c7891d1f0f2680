"""CPU checks of the dense latent-attention calls: refusals of the C entry points (all before any CUDA
call) and of the Python binding, and the plain definitions the GPU tests compare with."""
import ctypes
import math
import os
import re

import pytest
import torch

import dense_mla_ref as ref
from deepseek_sparse_attention_paged_gb300 import build, capi

A, B_, C_, D_ = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000))
ODD = ctypes.c_void_p(0x10008)
F = ctypes.c_float
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def _store(lib, kv=A, stride=576, w=A, eps=1e-6, maxpos=8, n=4, pool=B_, pages=1, out=None, ostride=576, flags=0):
    return lib.dsa_store_latent_prologue(kv, stride, w, F(eps), C_, maxpos, C_, C_, n, pool, pages, out, ostride, flags,
                                         None, None)


def test_store_refusals(lib):
    assert _store(lib, n=0) == OK and _store(lib, n=0, kv=None) == OK
    for kw in ({"kv": None}, {"pool": None}, {"w": None}, {"kv": ODD}, {"pool": ODD}, {"w": ODD}, {"out": ODD}, {"n": -1},
               {"pages": -1}, {"maxpos": -1}, {"stride": 575}, {"stride": 580}, {"stride": 512}, {"flags": 0x2},
               {"eps": -1.0}, {"eps": math.nan}, {"out": D_, "ostride": 572}, {"out": D_, "ostride": 512}):
        assert _store(lib, **kw) == INVALID, kw
    assert _store(lib, pages=1 << 40) == UNSUPPORTED


def _prefill(lib, q=A, qs=(1536, 192), k=B_, ks=(2048, 256), pe=C_, pes=576, v=B_, vs=(2048, 256), cu=D_, b=1, t=4, s=4,
             h=8, scale=0.1, flags=0x40, out=D_, os_=(1024, 128)):
    return lib.dsa_dense_mla_prefill(q, *qs, k, *ks, pe, pes, v, *vs, cu, cu, b, t, s, h, F(scale), flags, out, *os_,
                                     None, None, None)


def test_prefill_refusals(lib):
    assert _prefill(lib, t=0) == OK and _prefill(lib, b=0) == OK and _prefill(lib, h=0) == OK
    for kw in ({"q": None}, {"k": None}, {"pe": None}, {"v": None}, {"cu": None}, {"out": None}, {"q": ODD}, {"k": ODD},
               {"pe": ODD}, {"v": ODD}, {"out": ODD}, {"t": -1}, {"s": -1}, {"b": -1}, {"h": -1}, {"flags": 0x41},
               {"scale": 0.0}, {"scale": -1.0}, {"scale": math.inf}, {"scale": math.nan}, {"qs": (1536, 188)},
               {"qs": (1540, 192)}, {"qs": (1536, 0)}, {"ks": (2048, 64)}, {"vs": (64, 256)}, {"pes": 32}, {"pes": 68},
               {"os_": (1024, 120)}, {"os_": (128, 128)}, {"os_": (512, 128)}):
        assert _prefill(lib, **kw) == INVALID, kw
    assert _prefill(lib, t=1 << 30) in (INVALID, UNSUPPORTED)
    assert _prefill(lib, t=1 << 28, os_=(1024, 128)) == UNSUPPORTED


def _decode(lib, q=A, kv=B_, pages=4, table=C_, maxp=4, lens=C_, cu=C_, b=1, t=1, h=16, scale=0.1, out=D_, ws=A,
            wsb=1 << 30):
    return lib.dsa_dense_mla_decode(q, kv, pages, table, maxp, lens, cu, b, t, h, F(scale), out, None, ws, wsb, None, None)


def test_decode_refusals(lib):
    assert _decode(lib, t=0) == OK and _decode(lib, b=0) == OK
    for h in (0, 1, 8, 24, 96, 256, -16):
        assert _decode(lib, h=h) == UNSUPPORTED
    for kw in ({"q": None}, {"kv": None}, {"table": None}, {"lens": None}, {"cu": None}, {"out": None}, {"q": ODD},
               {"kv": ODD}, {"out": ODD}, {"t": -1}, {"b": -1}, {"maxp": -1}, {"maxp": 0}, {"pages": 0}, {"pages": -1},
               {"scale": 0.0}, {"scale": math.inf}, {"scale": math.nan}):
        assert _decode(lib, **kw) == INVALID, kw
    assert _decode(lib, pages=1 << 26) == UNSUPPORTED
    assert _decode(lib, maxp=1 << 25) == UNSUPPORTED
    assert lib.dsa_dense_mla_decode_workspace_size(0, 128) == 0
    assert lib.dsa_dense_mla_decode_workspace_size(-1, 128) == 0
    if lib.dsa_dense_mla_decode_workspace_size(4, 128) > 0:
        assert _decode(lib, t=4, h=128, ws=None) == INVALID
        assert _decode(lib, t=4, h=128, wsb=16) == INVALID
        assert _decode(lib, t=4, h=128, ws=ODD) == INVALID


def _verify(lib, p=A, ldp=1000, q=B_, ldq=1000, v=1000, tok=C_, cu=C_, b=1, t=2, u=C_, us=C_, out=D_, acc=D_):
    return lib.dsa_verify_drafts(p, ldp, q, ldq, v, tok, cu, b, t, u, us, out, acc, None, None)


def test_verify_refusals(lib):
    assert _verify(lib, b=0) == OK
    for kw in ({"p": None}, {"tok": None}, {"cu": None}, {"u": None}, {"us": None}, {"out": None}, {"acc": None},
               {"ldp": 999}, {"ldq": 999}, {"v": 0}, {"v": -1}, {"b": -1}, {"t": -1}):
        assert _verify(lib, **kw) == INVALID, kw
    assert _verify(lib, v=(1 << 24) + 1, ldp=1 << 25, ldq=1 << 25) == UNSUPPORTED


@pytest.mark.parametrize("at", [-7, -1, 0, 3, 7])
def test_verify_refuses_outputs_over_the_drafts(lib, at):
    """out_tokens apart from draft_tokens in all 8 entries."""
    assert _verify(lib, t=8, out=ctypes.c_void_p(C_.value + 4 * at)) == INVALID


def test_binding_refuses_cpu_tensors():
    bf = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        capi.dsa_dense_mla_decode(bf, torch.zeros(1, 64, 576, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32),
                                  torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0.1,
                                  torch.zeros(2, 16, 512, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        capi.dsa_verify_drafts(torch.zeros(1, 8), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                               torch.zeros(1), torch.zeros(1), torch.zeros(1, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------- the plain definitions

def test_absorbed_and_expanded_definitions_agree():
    """Expanded attention over keys and values up-projected from the latents equals the absorbed one
    followed by the value up-projection (float64 weights: no rounding in between)."""
    g = torch.Generator().manual_seed(5)
    H, n, nq = 2, 90, 5
    pool = torch.randn(2, 64, 576, generator=g).double()
    table = torch.tensor([[1, 0]], dtype=torch.int32)
    c = pool[[1, 0]].reshape(-1, 576)[:n]
    w_uk = torch.randn(H, 128, 512, generator=g).double() / 20
    w_uv = torch.randn(H, 512, 128, generator=g).double() / 20
    q = torch.randn(nq, H, 192, generator=g).double()
    qa = torch.cat([torch.einsum("thp,hpl->thl", q[..., :128], w_uk), q[..., 128:]], 2)
    o_lat, lse_a, _, _ = ref.decode(qa, pool, table, [n], [nq], 0.07)
    o_a = torch.einsum("thl,hlv->thv", o_lat, w_uv)
    k = torch.einsum("sl,hpl->shp", c[:, :512], w_uk)
    v = torch.einsum("sl,hlv->shv", c[:, :512], w_uv)
    o_e, lse_e, _, _ = ref.prefill(q, k, c[:, 512:], v, [nq], [n], 0.07, True)
    assert torch.allclose(o_a, o_e, atol=1e-12) and torch.allclose(lse_a, lse_e, atol=1e-12)


def test_verify_definition_keeps_the_target_distribution():
    """Over a grid of random numbers the first output token is distributed as the target."""
    p = torch.tensor([[0.5, 0.3, 0.2, 0.0], [0.25] * 4])
    q = torch.tensor([[0.2, 0.2, 0.5, 0.1], [0.25] * 4])
    n = 40
    mass = torch.zeros(4, dtype=torch.float64)
    for x in range(4):
        for i in range(n):
            for j in range(n):
                out, acc = ref.verify(p, q, [x, -1], [0, 2], torch.tensor([(i + 0.5) / n, 0.0]),
                                      torch.tensor([(j + 0.5) / n]))
                mass[out[0]] += float(q[0, x]) / (n * n)
                assert acc[0] == (1 if out[1] >= 0 else 0)
    assert torch.allclose(mass, p[0].double(), atol=2.0 / n)


@pytest.mark.parametrize("call,source", [("dsa_store_latent_prologue", "store_latent.cu"), ("dsa_dense_mla_prefill", "dense_mla_prefill.cu"),
                                         ("dsa_dense_mla_decode", "dense_mla_decode.cu"), ("dsa_verify_drafts", "verify_drafts.cu")])
def test_header_names_the_device_errors_that_a_call_raises(call, source):
    """The comment in front of a call's declaration names exactly the error bits that its kernels set."""
    with open(os.path.join(build.CSRC, source)) as f:
        raised = set(re.findall(r"raise_error\([^;]*?(DSA_DEVERR_\w+)\)", f.read()))
    with open(os.path.join(build.INCLUDE, "dsa.h")) as f:
        header = f.read()
    doc = header[header.index(f" * {call} -- "):header.index(f"dsa_status {call}(")]
    assert raised and set(re.findall(r"DSA_DEVERR_\w+", doc)) == raised
