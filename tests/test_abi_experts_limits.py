"""Sizes at the end of what the 8-bit products accept, through the C ABI (no GPU: every call here
is refused before anything is launched)."""
import pytest

from predictor_gated_channel_b200 import _capi
from predictor_gated_channel_b200 import build as sfn_build

FAKE = 1 << 20   # aligned, never dereferenced by a refused call
UNSUPPORTED = _capi.SFN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def L():
    sfn_build.build()
    return _capi.lib()


@pytest.mark.parametrize("T,N,K", [
    ((1 << 31) - 1, 1, 16),          # the end of a last tile would pass 32 bits
    ((1 << 31) - 256, 16, 16), ((1 << 31) - 4096, 1, 32),
    ((1 << 31) - 4112, 2048, 16),    # 2^27 row tiles of 16 times 16
    (1 << 31, 1, 16), (1 << 20, 1 << 24, 16),
])
def test_products_past_32_bits_are_refused(L, T, N, K):
    assert L.sfn_matmul_i8(FAKE, FAKE, FAKE, FAKE, FAKE, 1, T, N, K, None) == UNSUPPORTED
    assert L.sfn_linear_i8(FAKE, 0, FAKE, FAKE, FAKE, 1, T, N, K, FAKE, 1 << 62,
                           None) == UNSUPPORTED


@pytest.mark.parametrize("T,E,k", [((1 << 31) - 1, 1, 1), ((1 << 31) - 4200, 1024, 1),
                                   ((1 << 30) - 100, 200, 2), (1 << 26, 1024, 32)])
def test_experts_past_32_bits_are_refused(L, T, E, k):
    assert L.sfn_experts_i8_workspace_bytes(T, E, k, 16, 16) == 0
    assert L.sfn_experts_i8_forward(*[FAKE] * 10, T, E, k, 16, 16, FAKE, 1 << 62,
                                    None) == UNSUPPORTED
