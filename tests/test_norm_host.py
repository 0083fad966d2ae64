"""What add_norm refuses before it looks at a device."""
import pytest
import torch


@pytest.mark.parametrize("same", [False, True])
def test_a_residual_without_a_block(same):
    """With y = None nothing would be written into it."""
    from moe_nvfp4_gemv_gb300 import fp4gemv
    x, w = torch.ones(2, 8, dtype=torch.bfloat16), torch.ones(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="residual needs y"):
        fp4gemv.add_norm(x, None, w, residual=x if same else torch.zeros_like(x))
