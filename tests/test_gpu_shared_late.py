"""attend_shared where a row's maximum comes late: weights that are already made and sums that are already there move to
it.  Against 64 bits; tolerances are those of test_gpu_kv_cache.py (its docstring)."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, fp4, gen, kv, random_cache, scaled  # noqa: F401
from test_gpu_shared import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("where", [20, 63, 100])
@pytest.mark.parametrize("bits", [24, 26, 28])
def test_small_weights_before_the_largest(kv, fmt, dim, where, bits):
    """In 128 common tokens one token scores `bits` (base 2) above the others and holds zeros, the others ones: their weights
    are made first and move with the maximum.  What is lost of them is at most 2^-32 of the largest weight for each, or what
    f16 rounds of the weights; the output rounds once (half a step of bf16)."""
    block, batch = 16, 3
    one, top = (int(ref.encode(torch.tensor([x]), fmt)[0]) for x in (1.0, float(bits)))
    cache = kv.KvCache8.allocate(8 + batch, 1, dim, block, fmt)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    cache.v_codes.fill_(one)
    table = torch.arange(9, dtype=torch.int32, device=DEV).repeat(batch, 1)
    table[:, -1] += torch.arange(batch, dtype=torch.int32, device=DEV)
    value = float(ref.decode(torch.tensor([top], dtype=torch.uint8), fmt))
    cache.k_codes[where // block, 0, where % block, 0] = top
    cache.v_codes[where // block, 0, where % block] = 0
    q = torch.zeros(batch, 1, 2, dim, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    out = cache.attend_shared(q, table, torch.full((batch,), 129, dtype=torch.int32, device=DEV),
                              torch.tensor([128], dtype=torch.int32, device=DEV), sm_scale=math.log(2.0),
                              always=True).double()
    want = 128 * 2.0 ** -value / (1 + 128 * 2.0 ** -value)
    assert ((out - want).abs() <= (2.0 ** -10 + 2.0 ** -9) * want + 128 * 2.0 ** -32).all(), float((out / want).min())
