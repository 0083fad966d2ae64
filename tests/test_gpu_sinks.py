"""Attention with a sliding window and first tokens that stay visible
(KvCache8.attend with ``sinks``) on the GPU, against 64 bits.

Tolerances are those of test_gpu_kv_cache.py (its docstring); the mass that the
rounding of weights acts on is that of the tokens seen."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, TYPES, fp4, gen, kv, make_table, on_gpu, random_cache, scaled  # noqa: F401

pytestmark = pytest.mark.gpu


def attention64(q, c, table, lens, fmt, sm_scale, window, sinks):
    """(out, lse, mass, largest score) in 64 bits, as decode_ref.attention, of the tokens that the masks leave."""
    B, n, H, D = q.shape
    kv_heads, block = c["k_codes"].shape[1:3]
    g = H // kv_heads
    out = torch.zeros(B, n, H, D, dtype=torch.float64, device=DEV)
    mass, lse, peak = torch.zeros_like(out), torch.full((B, n, H), -math.inf, dtype=torch.float64, device=DEV), 0.0
    c = {name: t.to(DEV) for name, t in c.items()}
    for b, length in enumerate(lens):
        for i in range(n):
            p = length - n + i
            t = torch.arange(max(0, p + 1))
            if window:
                t = t[(t > p - window) | (t < sinks)]
            if not len(t):
                continue
            page, slot = table[b][t // block].long().to(DEV), (t % block).to(DEV)
            k, v = (ref.decode(c[x + "_codes"][page, :, slot], fmt).double() * c[x + "_scale"][page].double()[..., None]
                    for x in ("k", "v"))
            x = torch.einsum("hgd,thd->hgt", q[b, i].double().view(kv_heads, g, D), k) * sm_scale
            peak = max(peak, float(x.abs().nan_to_num(0).max()))
            w = torch.softmax(x, -1)
            out[b, i] = torch.einsum("hgt,thd->hgd", w, v).reshape(H, D)
            mass[b, i] = torch.einsum("hgt,thd->hgd", w, v.abs()).reshape(H, D)
            lse[b, i] = torch.logsumexp(x, -1).reshape(H)
    return out, lse, mass, peak


def check(kv, q, c, table, lens, fmt, window, sinks, sm_scale=None, nans=False):
    cache = on_gpu(kv, c, fmt)
    tab, n_len = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device=DEV)
    out = cache.attend(q, tab, n_len, window=window, sinks=sinks, lse=lse, sm_scale=sm_scale)
    again = cache.attend(q, tab, n_len, window=window, sinks=sinks, sm_scale=sm_scale)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two calls differ"
    want, want_lse, mass, peak = attention64(q, c, table, lens, fmt, sm_scale or 1 / math.sqrt(q.shape[-1]), window, sinks)
    assert torch.equal(out.isnan(), want.isnan())
    assert bool(want.isnan().any()) == nans
    n = max(max(lens), 1)
    vmax = float(ref.decode(c["v_codes"], fmt).abs().nan_to_num(0).amax() * c["v_scale"].nan_to_num(0, 0, 0).amax())
    d = 2.0 ** -10 * mass + n * 2.0 ** -25 * vmax
    low, high = (want - d).to(q.dtype), (want + d).to(q.dtype)
    outside = ~((out >= low) & (out <= high)) & ~want.isnan()
    assert not outside.any(), f"{int(outside.sum())} values outside"
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty) and (out[empty] == 0).all()
    tol = 2.0 ** -19 * (1 + peak) + (16 + n / 128) * 2.0 ** -23
    assert ((lse.double() - want_lse)[~empty].abs().nan_to_num(0) <= tol).all()


@pytest.mark.parametrize("dim,block,group,fmt,dtype", [
    (64, 16, 1, "e4m3", "bf16"), (96, 32, 3, "int8", "f16"), (128, 64, 4, "e4m3", "f16"), (128, 16, 8, "int8", "bf16"),
    (256, 128, 2, "e4m3", "bf16"), (128, 128, 24, "e4m3", "bf16"), (64, 64, 31, "int8", "bf16")])
@pytest.mark.parametrize("window,sinks", [(1, 1), (1, 16), (16, 4), (20, 17), (100, 4), (64, 130), (300, 33), (2000, 5)])
def test_sinks(kv, dim, block, group, fmt, dtype, window, sinks):
    lens = [0, 1, 2, 5, 16, 17, 33, 100, 129, 333, 700, 1500]
    g = gen(dim + window + sinks)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), fmt)
    for q_len in (1, 5) if group < 24 else (1,):
        q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(TYPES[dtype]).to(DEV)
        check(kv, q, c, table, lens, fmt, window, sinks)


@pytest.mark.parametrize("lens,heads,kv_heads,q_len,window,sinks", [
    ([9000], 8, 8, 1, 1024, 4), ([70000], 4, 1, 1, 30000, 700), ([5000, 4000, 3000], 16, 2, 2, 2500, 64),
    ([3000] * 40, 8, 4, 1, 500, 4), ([257] * 130, 4, 2, 3, 60, 20)])
def test_sinks_of_items_in_pieces(kv, lens, heads, kv_heads, q_len, window, sinks):
    """Items cut by many CTAs, the gap within a share and at its ends."""
    g = gen(len(lens) + heads)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, kv_heads, 64, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, heads, 128, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, "e4m3", window, sinks)


@pytest.mark.parametrize("group,dim,q_len", [(2, 128, 4), (5, 64, 3), (3, 256, 5), (7, 96, 4), (1, 128, 16), (5, 128, 4),
                                             (8, 128, 4), (2, 128, 16), (30, 128, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 3), (20, 18), (130, 5), (150, 140)])
def test_sinks_nan_values(kv, group, dim, q_len, window, sinks):
    """NaN values among the first tokens, behind them, at the window's begin and at the newest tokens: in the rows that see
    them alone.  Short sequences' first tokens are newer than some queries."""
    lens = [1, 3, 5, 17, 40, 133, 300, 1000]
    g = gen(dim + q_len + sinks)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, dim, g, 1.0), "e4m3")
    for b, n in enumerate(lens):
        first = n - q_len + 1 - window
        for i, t in enumerate((n - 1, n - 2, first, first - 1, sinks, sinks + 1, sinks - 1)):
            if 0 <= t < n and (t != sinks - 1 or b % 2):
                code = c["v_codes"][int(table[b, t // 16])]
                code[b % 2, t % 16, 3 + 7 * i] = 0x7F
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.float16).to(DEV)
    check(kv, q, c, table, lens, "e4m3", window, sinks, nans=True)


@pytest.mark.parametrize("fmt,dim,heads", [("e4m3", 64, 4), ("int8", 64, 4), ("e4m3", 128, 24)])
def test_sinks_pages_between_are_not_read(kv, fp4, fmt, dim, heads):
    """Pages of tokens that no query sees may be anyone's: other ids, no ids at all, NaN scales."""
    block, window, sinks, lens = 16, 50, 20, [400, 161, 90]
    g = gen(4)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), fmt)
    q = torch.randn(3, 2, heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    cache, n_len = on_gpu(kv, c, fmt), torch.tensor(lens, dtype=torch.int32, device=DEV)
    want = cache.attend(q, table.to(DEV), n_len, window=window, sinks=sinks)
    for b, n in enumerate(lens):
        for j in range(-(-sinks // block), max(0, n - 2 - window + 1) // block):
            cache.v_scale[int(table[b, j])] = math.nan
            table[b, j] = (-1, 1 << 30)[j % 2]
    got = cache.attend(q, table.to(DEV), n_len, window=window, sinks=sinks)
    assert torch.equal(got, want) and fp4.get_device_error() == 0


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("q_len,group", [(1, 17), (4, 8), (3, 11), (16, 4)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (30, 128), (128, 129), (200, 4), (513, 300)])
def test_sinks_many_rows(kv, block, q_len, group, window, sinks):
    """17 to 64 rows of E4M3 heads of 128: tiles of 128 tokens on both sides of the gap, pages and sets of first tokens that
    end inside a tile."""
    lens = [0, 3, 127, 128, 129, 255, 300, 385, 640, 1000, 2111]
    g = gen(block + window + sinks)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, 128, g, 1.0), "e4m3")
    for b, n in enumerate(lens):  # (what lies past the ends is NaN)
        if n % block:
            for part in ("k_codes", "v_codes"):
                c[part][int(table[b, n // block]), :, n % block:] = 0x7F
    q = torch.randn(len(lens), q_len, 2 * group, 128, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, "e4m3", window, sinks)


@pytest.mark.parametrize("lens,heads,kv_heads,q_len,window,sinks", [
    ([9000], 64, 2, 1, 1024, 4), ([70000], 24, 1, 1, 30000, 700), ([5000, 4000, 3000], 40, 2, 1, 2500, 64),
    ([3000] * 40, 32, 4, 4, 500, 4)])
def test_sinks_many_rows_in_pieces(kv, lens, heads, kv_heads, q_len, window, sinks):
    g = gen(len(lens) + heads)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, kv_heads, 64, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, heads, 128, generator=g).to(torch.float16).to(DEV)
    check(kv, q, c, table, lens, "e4m3", window, sinks)


@pytest.mark.parametrize("fmt,dim,heads", [("e4m3", 128, 24), ("e4m3", 128, 8), ("int8", 64, 24), ("e4m3", 256, 4)])
@pytest.mark.parametrize("where", [0, 1, 5])
def test_sinks_zero_pages(kv, fmt, dim, heads, where):
    """A page of V that is zero, scale 2^-100, beside pages of scale 2^20: its tokens have their part in the sums of weights
    (the factor between the two kinds' largest exponents is about 2^-120, times what scores differ by)."""
    block, lens, window, sinks = 64, [1400, 257, 900], 700, 64
    g = gen(dim + heads + where)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), fmt)
    c["v_scale"][:] = 2.0 ** 20
    for b, n in enumerate(lens):
        page = int(table[b, min(where * 3, (n - 1) // block)])
        c["v_codes"][page] = 0
        c["v_scale"][page] = 2.0 ** -100
    q = 2 * torch.randn(3, 1, 2 * heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, fmt, window, sinks)


@pytest.mark.parametrize("fmt,dim,group,q_len,block", [
    ("e4m3", 64, 1, 1, 16), ("e4m3", 64, 4, 4, 32), ("int8", 64, 24, 1, 64), ("e4m3", 96, 8, 1, 32), ("int8", 96, 5, 3, 16),
    ("e4m3", 96, 6, 4, 16), ("e4m3", 128, 8, 1, 64), ("int8", 128, 4, 4, 16), ("int8", 128, 10, 3, 32), ("e4m3", 256, 3, 2, 16),
    ("int8", 256, 8, 2, 128), ("e4m3", 256, 17, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (20, 17), (60, 100)])
def test_sinks_many_short_items(kv, fmt, dim, group, q_len, block, window, sinks):
    """More items than SMs hold CTAs, of few strips each: a warp takes one by itself."""
    lens = [(37 * i) % 113 if i % 5 else (11 * i) % 900 for i in range(180)]
    g = gen(dim + group + window)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), fmt)
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, fmt, window, sinks)


@pytest.mark.parametrize("fmt,dim,group,q_len", [("e4m3", 64, 3, 1), ("int8", 128, 2, 1), ("int8", 96, 3, 4)])
def test_sinks_many_items_past_a_batch_of_pages(kv, fmt, dim, group, q_len):
    """Enough items for warps to take those of more than 32 strips by themselves (pages are looked up 32 strips at a time)."""
    lens = [620 + (41 * i) % 300 if i % 8 else i for i in range(400)]
    g = gen(dim + group)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 2, 32, dim, g, 1.0), fmt)
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, fmt, 560, 20)


@pytest.mark.parametrize("dim,group,q_len", [(64, 3, 4), (96, 4, 2), (128, 2, 5), (256, 3, 4)])
def test_sinks_many_short_items_nan_values(kv, dim, group, q_len):
    """NaN values in some items of a warp: in their rows that see them and in no others."""
    block, window, sinks = 16, 30, 18
    lens = [3 + (29 * i) % 90 for i in range(200)]
    g = gen(dim)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), "e4m3")
    for b in range(0, 200, 7):
        for t, head, d in ((0, 0, 5), (lens[b] - 1, 1, dim - 1), (max(lens[b] - window - 1, 0), 0, 33), (min(17, lens[b] - 1), 1, 60)):
            c["v_codes"][int(table[b, t // block]), head, t % block, d] = 0x7F
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.float16).to(DEV)
    check(kv, q, c, table, lens, "e4m3", window, sinks, nans=True)


@pytest.mark.parametrize("fmt,dim,group,q_len", [("e4m3", 128, 9, 2), ("e4m3", 256, 4, 4), ("int8", 128, 16, 2),
                                                 ("e4m3", 96, 32, 1), ("int8", 64, 2, 1)])
def test_sinks_largest_batch(kv, fmt, dim, group, q_len):
    """1024 sequences (the plan's tables fill shared memory to its end), idle ones among them."""
    lens = [(11 * i) % 150 for i in range(1024)]
    g = gen(dim)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 1, 32, dim, g, 1.0), fmt)
    q = torch.randn(1024, q_len, group, dim, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, q, c, table, lens, fmt, 40, 20)


@pytest.mark.parametrize("fmt,dim", [("e4m3", 64), ("int8", 256)])
def test_sinks_many_short_items_bad_pages(kv, fp4, fmt, dim):
    """A page id that is none: the error word says so, its sequences read zeros there, the others are untouched."""
    lens = [20 + (7 * i) % 40 for i in range(200)]
    g = gen(dim)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, dim, g, 1.0), fmt)
    q = torch.randn(200, 1, 8, dim, generator=g).to(torch.bfloat16).to(DEV)
    cache, n = on_gpu(kv, c, fmt), torch.tensor(lens, dtype=torch.int32, device=DEV)
    good = cache.attend(q, table.to(DEV), n, window=30, sinks=4)
    assert fp4.get_device_error() == 0
    bad = table.clone()
    bad[50, 0], bad[120, 1] = pages + 5, -7
    got = cache.attend(q, bad.to(DEV), n, window=30, sinks=4)
    assert fp4.get_device_error() == 6
    assert not got.isnan().any()
    same = [b for b in range(200) if b not in (50, 120)]
    assert torch.equal(got[same], good[same])


def test_sinks_leave_other_calls_alone(kv):
    """No window, a window past every length, no sinks: the results of the calls without."""
    lens = [300, 20, 0]
    g = gen(6)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 1, 32, 128, g, 1.0), "e4m3")
    cache, tab, n = on_gpu(kv, c, "e4m3"), table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    for heads in (4, 20):
        q = torch.randn(3, 1, heads, 128, generator=g).to(torch.bfloat16).to(DEV)
        want = cache.attend(q, tab, n)
        for kw in (dict(sinks=5), dict(window=1 << 30, sinks=5), dict(window=400, sinks=3), dict(window=100, sinks=400),
                   dict(window=10, sinks=1 << 30)):
            got = cache.attend(q, tab, n, **kw)
            if kw.get("window", 0) in (0, 400, 1 << 30):
                assert torch.equal(got, want)
            else:  # every token is seen all the same; another kernel's order of sums
                assert (got.float() - want.float()).abs().max() <= 2.0 ** -6
    with pytest.raises(RuntimeError):
        cache.attend(q, tab, n, window=5, sinks=-1)
    with pytest.raises(RuntimeError):
        cache.attend(q, tab, n, window=5, sinks=(1 << 30) + 1)
    with pytest.raises(RuntimeError):
        cache.attend(q, tab, n, window=-1, sinks=2)


def test_sinks_captured(kv):
    """A captured call follows lengths that grow past the window."""
    B, window, sinks = 4, 64, 8
    g = gen(12)
    table, pages = make_table([600] * B, 16, g)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), "int8")
    q = torch.randn(B, 1, 8, 128, generator=g).to(torch.bfloat16).to(DEV)
    cache, tab, n = on_gpu(kv, c, "int8"), table.to(DEV), torch.tensor([1, 60, 72, 100], dtype=torch.int32, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = cache.attend(q, tab, n, window=window, sinks=sinks)
    for lens in ([1, 60, 72, 100], [65, 80, 0, 599], [600, 73, 81, 15]):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, cache.attend(q, tab, n, window=window, sinks=sinks))
        check(kv, q, c, table, lens, "int8", window, sinks)
