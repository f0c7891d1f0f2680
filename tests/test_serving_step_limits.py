"""CPU checks of limits of the calls around a serving step (all before any CUDA call)."""
import pytest

from deepseek_sparse_attention_paged_gb300 import build, capi
from test_serving_step_host import _shared

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
