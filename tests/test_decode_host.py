"""The decode operators' host side without a GPU: refusals, the cache's handle, the extension module's build."""
import ctypes

import pytest

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def fp4():
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


@pytest.mark.parametrize("inv_t,status", [(0.99e-20, 1), (1e-30, 1), (1.01e-20, 3), (1e6, 3), (1.01e6, 1)])
def test_logprobs_range_of_temperatures(fp4, inv_t, status):
    """Outside the range: refused for it (1), before the misaligned logits are (3)."""
    assert fp4.lib().fp4gemv_token_logprobs(vp((1 << 20) + 1), 100, 0, 1, 100, None, inv_t, 4, None, None, None, None, None,
                                            1, None) == status
