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


@pytest.mark.parametrize("dim,fmt", [(64, "e4m3"), (96, "int8"), (128, "e4m3"), (128, "int8"), (256, "e4m3"), (256, "int8")])
@pytest.mark.parametrize("batch,heads", [(3, 8), (5, 40), (9, 64)])
def test_maxima_in_later_tiles(kv, dim, fmt, batch, heads):
    """A CTA holds six tiles and more of one KV head: one block of rows (its slots take the tiles by turns), two blocks (a
    slot each), five.  Rows meet the token that takes all in the second, third, a middle or the last tile, in one of a
    beginning's first, middle and last CTAs, some rows several ever larger ones."""
    tile = 64 if dim == 256 else 128
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    items = -(-batch * heads // (128 if dim == 256 else 256))
    n, block = ctas * 6 * tile // items, 64
    n = n // 128 * 128
    g = gen(dim + batch)
    full = n // block
    c = scaled(random_cache(full + batch, 1, block, dim, g, 0.5), fmt)
    c["k_codes"] = ref.encode(20 * torch.randn(c["k_codes"].shape, generator=g), fmt)  # (room for six times as much)
    c["k_scale"] = 0.05 * torch.exp2(0.5 * torch.randn(c["k_scale"].shape, generator=g))
    table = torch.arange(full + 1, dtype=torch.int32).repeat(batch, 1)
    table[:, -1] += torch.arange(batch, dtype=torch.int32)
    q = torch.randn(batch, 1, heads, dim, generator=g).to(torch.bfloat16)
    per = -(-(n // tile) * items // ctas)  # a CTA's tiles
    flat = q.view(-1, dim)
    for j, r in enumerate(range(0, len(flat), 3)):
        for k, size in ((1, 2.0), (2, 3.0), (per // 2, 4.5), (per - 1, 6.0))[j % 4:4 if j % 8 < 4 else j % 4 + 1]:
            cta = (0, ctas // 2, ctas - 1, 7)[(j // 3) % 4]
            at = (cta * per + k) % (n // tile) * tile + (11 * r + 5) % tile
            x = flat[r].float() / flat[r].float().square().mean().sqrt() * size  # its score: about `size` sqrt(dim)
            s = float(c["k_scale"][at // block, 0])
            c["k_codes"][at // block, 0, at % block] = ref.encode((x / s).clamp(-448, 448), fmt)
    check(kv, c, fmt, q.to(DEV), table, [n + 1 + (5 * b) % 60 for b in range(batch)], n)
