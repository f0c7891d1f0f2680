"""CPU checks of limits of the calls around a serving step (all before any CUDA call)."""
import pytest

from deepseek_sparse_attention_paged_gb300 import build, capi
from test_serving_step_host import _sample, _shared

INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    build.build()
    return capi.load()


@pytest.mark.parametrize("H", [16, 32, 64, 128])
def test_shared_refuses_units_whose_positions_pass_32_bits(lib, H):
    """A unit's requests (256 / H at most) with their pages one after the other, 2^31 - 128 positions at most."""
    n = 256 // H
    most = ((1 << 31) - 1 - 128 - 1) // (64 * n)                 # pages a request
    too_many = {"b": 20, "t": 20, "h": H, "maxp": most + 1}
    assert _shared(lib, **too_many) == UNSUPPORTED
    # in bounds: it gets to the next check
    for kw in ({"maxp": most}, {"b": n - 1}, {"t": n - 1}):
        assert _shared(lib, **{**too_many, **kw}, ws=None) == INVALID


def test_sample_refuses_outputs_over_inputs_and_each_other(lib):
    """Two rows of 1000: the first and the last bytes of each array."""
    inputs = {"t": 0x51000, "k": 0x51100, "p": 0x51200, "m": 0x51300, "u": 0x51400}
    for at in inputs.values():
        for d in (-4, 0, 4):
            assert _sample(lib, **inputs, tok=at + d) == INVALID
        for d in (-7996, 0, 4):
            assert _sample(lib, **inputs, pr=at + d, lg=0x900000) == INVALID
    for d in (-4, 0, 7996):
        assert _sample(lib, **inputs, tok=0x100000 + d) == INVALID          # logits
        assert _sample(lib, **inputs, tok=0x900000 + d) == INVALID          # probabilities
        assert _sample(lib, **inputs, tok=0x900000 + d, ld=1004, ldp=1004) == INVALID
