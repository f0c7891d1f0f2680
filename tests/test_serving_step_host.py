"""CPU checks of the calls around a serving step: refusals of the C entry points (all before any CUDA call) and of the
binding, the error bits that the header names, and the plain definitions."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import serving_step_ref as ref
from deepseek_sparse_attention_paged_gb300 import build, capi

A, B_, C_, D_ = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000))
F = ctypes.c_float
OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _tables(lib, cached=0x1000, q=0x2000, counts=0x3000, keep=0x4000, b=4, table=0x5000, maxp=4, pages=16, free=0x6000,
            have=0x7000, seq=0x8000, counts_out=0x9000, have_out=0xa000, cu=0xb000, pos=0xc000, slots=0xd000, t=8):
    return lib.dsa_step_tables(_p(cached), _p(q), _p(counts), _p(keep), b, _p(table), maxp, pages, _p(free), _p(have),
                               _p(seq), _p(counts_out), _p(have_out), _p(cu), _p(pos), _p(slots), t, None, None)


def test_tables_refusals(lib):
    assert _tables(lib, b=0, t=0) == OK
    for kw in ({"cached": None}, {"q": None}, {"counts": None}, {"table": None}, {"free": None}, {"have": None},
               {"seq": None}, {"counts_out": None}, {"have_out": None}, {"cu": None}, {"pos": None}, {"slots": None},
               {"b": -1}, {"t": -1}, {"maxp": 0}, {"maxp": -1}, {"pages": 0}, {"pages": -1}, {"b": 0, "t": 3}):
        assert _tables(lib, **kw) == INVALID, kw
    for kw in ({"b": 16385}, {"maxp": 1 << 29}, {"pages": 1 << 25}):
        assert _tables(lib, **kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("out", ["table", "free", "seq", "counts_out", "have_out", "cu", "pos", "slots"])
def test_tables_refuses_outputs_over_inputs_and_each_other(lib, out):
    for at in (0x1000, 0x2000, 0x3000, 0x4000, 0x7000):
        assert _tables(lib, **{out: at}) == INVALID
    others = {"table": 0x5000, "free": 0x6000, "seq": 0x8000, "counts_out": 0x9000, "have_out": 0xa000, "cu": 0xb000,
              "pos": 0xc000, "slots": 0xd000}
    for name, at in others.items():
        if name != out:
            assert _tables(lib, **{out: at}) == INVALID


def _shared(lib, q=A, kv=B_, pages=4, table=C_, maxp=4, lens=C_, cu=C_, b=1, t=1, h=16, cg=C_, sh=C_, g=1, scale=0.1,
            out=D_, ws=A, wsb=1 << 30):
    return lib.dsa_dense_mla_decode_shared(q, kv, pages, table, maxp, lens, cu, b, t, h, cg, sh, g, F(scale), out, None, ws,
                                           wsb, None, None)


def test_shared_refusals(lib):
    odd = ctypes.c_void_p(0x10008)
    assert _shared(lib, t=0) == OK and _shared(lib, b=0) == OK
    for h in (0, 1, 8, 24, 96, 256, -16):
        assert _shared(lib, h=h) == UNSUPPORTED
    for kw in ({"q": None}, {"kv": None}, {"table": None}, {"lens": None}, {"cu": None}, {"out": None}, {"q": odd},
               {"kv": odd}, {"out": odd}, {"t": -1}, {"b": -1}, {"maxp": -1}, {"maxp": 0}, {"pages": 0}, {"pages": -1},
               {"scale": 0.0}, {"scale": math.inf}, {"scale": math.nan}, {"g": -1}, {"cg": None}, {"sh": None},
               {"ws": None}, {"wsb": 16}, {"ws": odd}):
        assert _shared(lib, **kw) == INVALID, kw
    for kw in ({"pages": 1 << 26}, {"maxp": 1 << 25}, {"g": 8193}, {"b": 16385}, {"t": 1 << 10, "maxp": 1 << 20}, {"t": (1 << 18) + 1}):
        assert _shared(lib, **kw) == UNSUPPORTED, kw
    size = lib.dsa_dense_mla_decode_shared_workspace_size
    assert size(0, 128) == 0 and size(-1, 128) == 0
    assert 0 < size(1, 16) < size(8, 16) == size(1 << 10, 16)          # slots of up to 128 rows


def _sample(lib, lg=0x100000, ld=1000, v=1000, r=2, flags=0, t=0x1000, k=0x1000, p=0x1000, m=0x1000, u=0x1000, tok=0x2000,
            pr=0x900000, ldp=1000):
    return lib.dsa_sample_tokens(_p(lg), ld, v, r, flags, _p(t), _p(k), _p(p), _p(m), _p(u), _p(tok), _p(pr), ldp, None, None)


def test_sample_refusals(lib):
    assert _sample(lib, r=0) == OK
    for kw in ({"lg": None}, {"u": None}, {"tok": None}, {"ld": 999}, {"ldp": 999}, {"v": 0}, {"v": -1}, {"r": -1},
               {"flags": 1}, {"flags": 0x180}, {"lg": 0x100002}, {"lg": 0x100001, "flags": 0x80}, {"pr": 0x900002},
               {"pr": 0x100000}, {"pr": 0x100000 + 7996}, {"pr": 0x100000 - 7996}):
        assert _sample(lib, **kw) == INVALID, kw
    assert _sample(lib, v=(1 << 18) + 1, ld=1 << 20, ldp=1 << 20) == UNSUPPORTED


def test_binding_refuses_cpu_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        capi.dsa_sample_tokens(torch.zeros(1, 8), torch.zeros(1), i32(1))
    with pytest.raises(ValueError):
        capi.dsa_step_tables(i32(1), i32(1), i32(1), i32(1, 2), 4, i32(4), i32(1), i32(1), i32(1), i32(1), i32(2),
                             torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int64))
    bf = torch.zeros(2, 16, 576, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        capi.dsa_dense_mla_decode_shared(bf, torch.zeros(1, 64, 576, dtype=torch.bfloat16), i32(1, 1), i32(1), i32(2), i32(2),
                                         i32(1), 0.1, torch.zeros(2, 16, 512, dtype=torch.bfloat16))


@pytest.mark.parametrize("call,source", [("dsa_step_tables", "step_tables.cu"), ("dsa_sample_tokens", "sample_tokens.cu"),
                                         ("dsa_dense_mla_decode_shared", "dense_mla_shared.cu")])
def test_header_names_the_device_errors_that_a_call_raises(call, source):
    with open(os.path.join(build.CSRC, source)) as f:
        raised = set(re.findall(r"DSA_DEVERR_\w+", f.read()))
    with open(os.path.join(build.INCLUDE, "dsa.h")) as f:
        header = f.read()
    doc = header[header.index(f" * {call} -- "):header.index(f"dsa_status {call}(")]
    assert raised and set(re.findall(r"DSA_DEVERR_\w+", doc)) == raised


# ---------------------------------------------------------------- the plain definitions

def test_sample_definition_draws_with_the_distribution():
    """Over an even grid of random numbers a token comes up as often as its probability says."""
    z = np.array([0.3, -1.0, 2.0, -np.inf, 0.3])
    n = 4001
    for kw in ({}, {"top_k": 2}, {"top_p": 0.8}, {"min_p": 0.1}, {"temperature": 0.5, "top_k": 3, "top_p": 0.9}):
        got = np.zeros(5)
        for i in range(n):
            got[ref.sample(z, u=(i + 0.5) / n, **kw)[0]] += 1.0 / n
        assert np.abs(got - ref.sample(z, **kw)[1]).max() <= 1.0 / n
    assert ref.sample(z, top_k=2)[1].nonzero()[0].tolist() == [0, 2]         # the tie goes to the lower index
    assert ref.sample(z, temperature=0.0)[0] == 2 and ref.sample([-np.inf] * 3)[0] == -1


def test_tables_definition_on_a_case_by_hand():
    table = [[5, 6, -1], [1, 2, 3], [4, -1, -1]]
    stack = [0, 7, -1, -1, -1, -1, -1, -1]
    out = ref.tables([100, 150, 64], [60, -1, 1], [2, 3, 1], [0, 1, 0], table, 8, stack, 2, 64)
    # request 1 gives back 2 and 3; request 0 takes 3, request 2 takes 2
    assert out == ([160, 0, 65], [3, 0, 2], 2, [0, 60, 60, 61], list(range(100, 160)) + [64] + [0] * 3,
                   [6 * 64 + i for i in range(36, 64)] + [3 * 64 + i for i in range(32)] + [2 * 64] + [-1] * 3, 0)
    assert table == [[5, 6, 3], [1, 2, 3], [4, 2, -1]] and stack == [0, 7, 2, 3, -1, -1, -1, -1]
