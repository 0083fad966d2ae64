"""Pages of V whose scales lie a hundred powers of two apart: a page of zeros has scale 2^-100, its tokens have their part
in the sum of weights.  Attention of the 8-bit cache in all its forms, against 64 bits.

Tolerances are those of test_gpu_kv_cache.py (its docstring)."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, fp4, gen, kv, make_table, on_gpu, random_cache, scaled  # noqa: F401
from test_gpu_sinks import attention64

pytestmark = pytest.mark.gpu

# how a call is made, and the window and first tokens that it stands for (a window of 1 << 24: more than every table holds)
CALLS = {
    "plain": (lambda cache, q, tab, n, **kw: cache.attend(q, tab, n, **kw), 0, 0),
    "window": (lambda cache, q, tab, n, **kw: cache.attend(q, tab, n, window=700, **kw), 700, 0),
    "sinks": (lambda cache, q, tab, n, **kw: cache.attend(q, tab, n, window=700, sinks=64, **kw), 700, 64),
    "all": (lambda cache, q, tab, n, **kw: cache.attend(q, tab, n, window=1 << 24, sinks=4, **kw), 0, 0),
    "apart": (lambda cache, q, tab, n, **kw: cache.attend_shared(q, tab, n, torch.zeros(1, dtype=torch.int32, device=DEV),
                                                                 **kw), 0, 0),
    "together": (lambda cache, q, tab, n, **kw: cache.attend_shared(q, tab, n, n.min().view(1), always=True, **kw), 0, 0),
}


def check(kv, call, c, q, table, lens, fmt, sm_scale=None):
    run, window, sinks = CALLS[call]
    cache = on_gpu(kv, c, fmt)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device=DEV)
    out = run(cache, q, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), lse=lse, sm_scale=sm_scale)
    want, want_lse, mass, peak = attention64(q, c, table, lens, fmt, sm_scale or 1 / math.sqrt(q.shape[-1]), window, sinks)
    n = max(lens)
    tol = 2.0 ** -19 * (1 + peak) + (16 + n / 128) * 2.0 ** -23
    off = (lse.double() - want_lse).abs().max()
    assert off <= tol, f"log of the sums off by {float(off):.3g}, {tol:.3g} allowed"
    vmax = float(ref.decode(c["v_codes"], fmt).abs().amax() * c["v_scale"].amax())
    d = 2.0 ** -10 * mass + n * 2.0 ** -25 * vmax
    assert ((out >= (want - d).to(q.dtype)) & (out <= (want + d).to(q.dtype))).all()


# eight rows and fewer, 16, 32; CTAs of one and of two to an SM; the kernel on the 5th-generation tensor core (24 rows)
SHAPES = [("e4m3", 128, 8), ("int8", 64, 16), ("e4m3", 256, 16), ("int8", 96, 24), ("e4m3", 128, 24)]


@pytest.mark.parametrize("fmt,dim,rows", SHAPES)
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("where", [0, 1, 5])
def test_one_zero_page(kv, call, fmt, dim, rows, where):
    """A page of zeros in the beginning, the middle or the end, others of scale 2^20, random scores."""
    block, lens = 64, [1400, 257, 900]
    g = gen(dim + rows + where)
    table, pages = make_table(lens, block, g)
    if call == "together":  # (the first 257 tokens are common)
        table[1:, :4] = table[0, :4]
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), fmt)
    c["v_scale"][:] = 2.0 ** 20
    for b, n in enumerate(lens):
        page = int(table[b, min(where * 3, (n - 1) // block)])
        c["v_codes"][page] = 0
        c["v_scale"][page] = 2.0 ** -100
    q = 2 * torch.randn(3, 1, 2 * rows, dim, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, call, c, q, table, lens, fmt)


def peaks_among_zeros(n, period, first, bits, batch, fmt, dim, own=16):
    """n tokens on pages of 16, the same for all: every period-th page from `first` on has V of scale 2^20 and a token of
    score 0, its others 40 lower (base 2); the rest are zeros, `bits` lower.  Behind them 16 own tokens like the latter."""
    full = n // 16
    c = dict(k_codes=torch.zeros(full + batch, 1, 16, dim, dtype=torch.uint8), k_scale=torch.ones(full + batch, 1),
             v_codes=torch.zeros(full + batch, 1, 16, dim, dtype=torch.uint8), v_scale=torch.full((full + batch, 1), 2.0 ** -100))
    low, lowest = (int(ref.encode(torch.tensor([x]), fmt)[0]) for x in (-float(bits), -40.0))
    c["k_codes"][..., 0] = low
    peak = torch.arange(first, full, period)
    c["k_codes"][peak, :, :, 0] = lowest
    c["k_codes"][peak, :, 3, 0] = 0
    c["v_codes"][peak] = int(ref.encode(torch.tensor([1.0]), fmt)[0])
    c["v_scale"][peak] = 2.0 ** 20
    table = torch.arange(full + 1, dtype=torch.int32).repeat(batch, 1)
    table[:, -1] += torch.arange(batch, dtype=torch.int32)
    return c, table, [n + own] * batch


@pytest.mark.parametrize("fmt,dim,rows", SHAPES)
@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("bits", [5, 14, 20])
def test_zero_pages_between_peaks(kv, call, fmt, dim, rows, bits):
    """Of 112 tokens one has score 0 and large values, most have no values and lie 5, 14 or 20 powers of two lower: these
    together have 3.5, 2^-7.2 and 2^-13 of it."""
    c, table, lens = peaks_among_zeros(152 * 512 if call == "together" else 4096, 7, 2, bits, 2, fmt, dim)
    q = torch.zeros(2, 1, rows, dim, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    check(kv, call, c, q, table, lens, fmt, sm_scale=math.log(2.0))


@pytest.mark.parametrize("call", ["sinks", "apart", "together"])
@pytest.mark.parametrize("fmt,dim,rows", [("e4m3", 256, 16), ("int8", 96, 24), ("int8", 64, 16)])
def test_zero_pages_of_many_short_items(kv, call, fmt, dim, rows):
    """A warp to an item: 400 sequences of 272 tokens."""
    c, table, lens = peaks_among_zeros(256, 7, 2, 14, 400, fmt, dim)
    q = torch.zeros(400, 1, rows, dim, dtype=torch.bfloat16, device=DEV)
    q[..., 0] = 1.0
    check(kv, call, c, q, table, lens, fmt, sm_scale=math.log(2.0))
