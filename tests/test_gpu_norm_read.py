"""The residual stream with its norms (fp4gemv.add_norm) and the cache read back
(KvCache8.read) on the GPU, against 64-bit or exact restatements."""
import pytest
import torch

import decode_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def fp4():
    require_gpu()
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


def rows(m, h, dtype, gen, pad=0, size=1.0):
    """[m, h] with row stride h + pad."""
    return (torch.randn(m, h + pad, generator=gen, device="cuda") * size).to(dtype)[:, :h]


def norm64(x, y, w, post, gate, sigmoid, scale, eps, offset):
    """(out, residual, the block's share of it), and the factor of r in out, in 64 bits."""
    r = x.double()
    delta = torch.zeros_like(r)
    if y is not None:
        u = y.double()
        if post is not None:
            u = u / torch.sqrt((u * u).mean(-1, keepdim=True) + eps) * (offset + post.double())
        if gate is not None:
            g = gate.double()
            u = u * (torch.sigmoid(g) if sigmoid else g)
        delta = scale * u
        r = r + delta
    f = (offset + w.double()) / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    return r * f, r, delta, f


def close(got, want, slack, dtype):
    """Within half a step of the type and the slack of the binary32 arithmetic."""
    info = torch.finfo(dtype)
    tol = info.eps / 2 * want.abs() + slack + info.smallest_normal * info.eps / 2
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), f"{(off - tol).max().item():.3g} past the tolerance of {dtype}"


def check_norm(fp4, x, y, w, post=None, gate=None, sigmoid=False, scale=1.0, eps=1e-6, offset=0.0, **given):
    want, r, delta, f = norm64(x, y, w, post, gate, sigmoid, scale, eps, offset)
    out, residual = fp4.add_norm(x, y, w, post_weight=post, gate=gate, gate_sigmoid=sigmoid, scale=scale, eps=eps,
                                 weight_offset=offset, **given)
    # binary32: sums of squares (at most 32 values in a row, then trees), roots, the logistic function and a few
    # products: together below 2^-19 of the block's share, and below 2^-18 of the norm's result
    close(residual, r, 2.0 ** -19 * delta.abs(), residual.dtype)
    size = r.square().sum(-1, keepdim=True).sqrt().clamp(min=1e-300)
    apart = 2.0 ** -19 * delta.square().sum(-1, keepdim=True).sqrt() / size  # what that does to the norm itself
    close(out, want, 2.0 ** -19 * (delta * f).abs() + want.abs() * (2.0 ** -18 + apart), out.dtype)
    return out, residual


@pytest.mark.parametrize("dtype,res,wt", [(BF16, BF16, BF16), (BF16, F32, F32), (F16, F16, F32), (F16, F32, F16)])
@pytest.mark.parametrize("m,h,pad", [(1, 4096, 0), (3, 1, 0), (5, 7, 0), (9, 129, 0), (2, 256, 8), (33, 257, 0),
                                     (4, 1000, 24), (3, 2048, 1), (2, 5120, 0), (2, 8192, 8), (3, 8191, 0),
                                     (2, 16384, 0), (1, 16390, 0), (2, 32768, 0), (1, 32767, 0), (301, 64, 0),
                                     (5, 2, 0), (7, 66, 0), (33, 258, 2), (5, 1002, 6), (3, 6146, 1), (1300, 514, 0),
                                     (1300, 1026, 4), (700, 2050, 0), (300, 5122, 0), (200, 8194, 0), (700, 4099, 0)])
def test_norm_shapes(fp4, dtype, res, wt, m, h, pad):
    g = torch.Generator(device="cuda").manual_seed(m * 100003 + h)
    x, y = rows(m, h, res, g, pad, 3.0), rows(m, h, dtype, g, pad)
    w, post = (torch.randn(h, generator=g, device="cuda").to(wt) for _ in range(2))
    check_norm(fp4, x, y, w)
    check_norm(fp4, x, y, w, post=post, gate=rows(m, h, dtype, g, pad), sigmoid=True, scale=0.37, offset=1.0)


@pytest.mark.parametrize("res", [BF16, F32])
@pytest.mark.parametrize("which", range(6))
def test_norm_one_off_its_boundary(fp4, res, which):
    """All rows on boundaries of pairs but one tensor's (its first value is its buffer's second)."""
    g = torch.Generator(device="cuda").manual_seed(which)
    m, h = 5, 642
    def make(k, dtype, *shape):
        flat = torch.randn(m * h + 1, generator=g, device="cuda").to(dtype)
        n = 1
        for d in shape:
            n *= d
        return flat[int(k == which):][:n].view(*shape)
    x, y, gate = make(0, res, m, h), make(1, BF16, m, h), make(2, BF16, m, h)
    w, post = make(3, F32, h), make(4, BF16, h) if which == 4 else make(4, F32, h)
    check_norm(fp4, x, y, w.to(post.dtype) if which == 4 else w, post=post, gate=gate, sigmoid=True)


@pytest.mark.parametrize("gate", ["channel", "token", "rows", "expanded"])
@pytest.mark.parametrize("gate_type", [BF16, F32])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("h", [512, 514, 515])
def test_norm_gates(fp4, gate, gate_type, sigmoid, h):
    m = 13
    g = torch.Generator(device="cuda").manual_seed(h + sigmoid)
    x, y = rows(m, h, BF16, g), rows(m, h, BF16, g)
    w = torch.randn(h, generator=g, device="cuda").to(BF16)
    t = torch.randn(h, generator=g, device="cuda").to(gate_type) * 3
    if gate == "token":
        t = rows(m, 1, gate_type, g, 5)
    elif gate == "rows":
        t = rows(m, h, gate_type, g, 8)
    elif gate == "expanded":
        t = t.expand(m, h)
    check_norm(fp4, x, y, w, gate=t, sigmoid=sigmoid, scale=-1.5)
    check_norm(fp4, x, y, w, post=w, gate=t, sigmoid=sigmoid)


def test_norm_alone_and_in_place(fp4):
    g = torch.Generator(device="cuda").manual_seed(5)
    w = torch.randn(1024, generator=g, device="cuda").to(BF16)
    x = rows(7, 1024, BF16, g)
    out, same = check_norm(fp4, x, None, w, offset=1.0)
    assert same is x and out.dtype is BF16
    out, _ = check_norm(fp4, x.float(), None, w)
    assert out.dtype is BF16
    out, _ = check_norm(fp4, x.float(), None, w.to(F16), out=torch.empty(7, 1024, dtype=F16, device="cuda"))
    y = rows(7, 1024, BF16, g)
    want = fp4.add_norm(x, y, w, post_weight=w)
    got = fp4.add_norm(x, y, w, post_weight=w, out=y, residual=x)
    assert got[0].data_ptr() == y.data_ptr() and torch.equal(y, want[0]) and torch.equal(x, want[1])


def test_norm_edges(fp4):
    w = torch.ones(640, dtype=BF16, device="cuda")
    zero = torch.zeros(2, 640, dtype=BF16, device="cuda")
    out, r = fp4.add_norm(zero, zero, w, post_weight=w)
    assert not out.any() and not r.any()
    # a row with NaN or infinities keeps to itself
    x = torch.ones(3, 640, dtype=BF16, device="cuda")
    x[1, 5] = float("nan")
    y = torch.ones(3, 640, dtype=BF16, device="cuda")
    y[2, 600] = float("inf")
    out, r = fp4.add_norm(x, y, w)
    assert out[0].eq(1).all() and out[1].isnan().all() and out[2, 600].isnan() and not out[2, :600].any()
    assert r[1].isnan().sum() == 1 and r[2].isinf().sum() == 1
    # gates far out
    gate = torch.tensor([[200.0], [-200.0], [0.0]], device="cuda")
    _, r = fp4.add_norm(torch.zeros_like(y[:3]), torch.ones_like(y), w, gate=gate, gate_sigmoid=True)
    assert r[0].eq(1).all() and not r[1].any() and r[2].eq(0.5).all()
    # no rows
    out, r = fp4.add_norm(x[:0], y[:0], w)
    assert out.shape == (0, 640) and r.shape == (0, 640)


def test_norm_many_rows(fp4):
    g = torch.Generator(device="cuda").manual_seed(11)
    x, y = rows(70001, 96, BF16, g), rows(70001, 96, BF16, g)
    check_norm(fp4, x, y, torch.randn(96, generator=g, device="cuda").to(BF16), post=torch.ones(96, dtype=BF16, device="cuda"))


def test_norm_is_the_same_again_and_in_a_graph(fp4):
    g = torch.Generator(device="cuda").manual_seed(3)
    x, y = rows(50, 6144, F32, g), rows(50, 6144, BF16, g)
    w = torch.randn(6144, generator=g, device="cuda")
    want = fp4.add_norm(x, y, w, post_weight=w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = fp4.add_norm(x, y, w, post_weight=w)
        again = fp4.add_norm(got[1], got[0], w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    want = fp4.add_norm(want[1], want[0], w)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_norm_refusals(fp4):
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    w = torch.zeros(64, dtype=BF16, device="cuda")
    for bad in (dict(x=x.t()), dict(x=x[0]), dict(x=x.cpu()), dict(x=x.to(F16)), dict(x=x.double()), dict(y=x[:3]),
                dict(y=x.to(F16)), dict(weight=w[:63]), dict(weight=w.to(F16)), dict(weight=w.cpu()),
                dict(weight=x), dict(post_weight=w.float()), dict(gate=w[:63]), dict(gate=x[:, :2]),
                dict(gate=x[:3, :1]), dict(gate=x.cpu()), dict(gate=w.double()), dict(out=x[:, :63]),
                dict(out=x.float(), y=x), dict(residual=x.float()), dict(residual=x[:2]),
                dict(y=None, post_weight=w), dict(y=None, gate=w)):
        args = dict(x=x, y=x, weight=w) | bad
        with pytest.raises((ValueError, TypeError)):
            fp4.add_norm(**args)
    for bad in (dict(scale=float("inf")), dict(eps=-1.0), dict(eps=float("nan")), dict(weight_offset=float("nan"))):
        with pytest.raises(fp4.Fp4GemvError):
            fp4.add_norm(x, x, w, **bad)
    wide = torch.zeros(1, 32769, dtype=BF16, device="cuda")
    with pytest.raises(fp4.Fp4GemvError):
        fp4.add_norm(wide, wide, wide[0])


# ---- the cache read back ----
def filled(pages, heads, dim, block, fmt, seed):
    from moe_nvfp4_gemv_gb300.kvcache import KvCache8
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = KvCache8.allocate(pages, heads, dim, block, fmt)
    for codes, scale in ((c.k_codes, c.k_scale), (c.v_codes, c.v_scale)):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
        scale.copy_(torch.exp2(torch.randint(-12, 6, scale.shape, generator=g, device="cuda")) *
                    (1 if fmt == "e4m3" else 1 + torch.rand(scale.shape, generator=g, device="cuda")))
    return c


def values(cache, table, lens, counts, dtype):
    """Rows of the last counts[b] tokens of every sequence; zeros where there is no token or no page."""
    outs = []
    for codes, scale in ((cache.k_codes, cache.k_scale), (cache.v_codes, cache.v_scale)):
        x = ref.decode(codes.cpu(), cache.fmt) * scale.cpu()[..., None, None]
        rows_ = []
        for b, (n, length) in enumerate(zip(counts, lens)):
            for pos in range(length - n, length):
                page = table[b][pos // cache.block_size] if 0 <= pos < len(table[b]) * cache.block_size else -1
                rows_.append(x[page, :, pos % cache.block_size] if 0 <= page < cache.num_blocks
                             else torch.zeros(cache.kv_heads, cache.head_dim))
        outs.append(torch.stack(rows_).to(dtype) if rows_ else torch.zeros(0, cache.kv_heads, cache.head_dim, dtype=dtype))
    return outs


def same(a, b):
    return torch.equal(a.nan_to_num(nan=-7.0), b.nan_to_num(nan=-7.0)) and torch.equal(a.isnan(), b.isnan())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("heads,dim,block,lens,counts", [
    (1, 64, 16, [1], [1]), (8, 128, 16, [133], [33]), (3, 96, 32, [70, 5, 64], [64, 5, 1]),
    (2, 256, 128, [300, 0, 128], [300, 0, 128]), (5, 128, 64, [65, 129, 1, 200], [1, 66, 1, 0]),
    (16, 64, 16, [40] * 40, [7, 0, 3, 16, 17] * 8)])
def test_read(fp4, fmt, dtype, heads, dim, block, lens, counts):
    width = max(1, max(-(-n // block) for n in lens))
    cache = filled(len(lens) * width + 1, heads, dim, block, fmt, dim + block)
    table = torch.randperm(len(lens) * width, dtype=torch.int32).view(len(lens), width) + 1
    starts = [sum(counts[:i]) for i in range(len(counts) + 1)]
    t, n = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = values(cache, table.tolist(), lens, counts, dtype)
    got = cache.read(t, n, tokens=starts[-1], cu=torch.tensor(starts, dtype=torch.int32, device="cuda"), dtype=dtype)
    for a, b in zip(got, want):
        assert a.dtype is dtype and same(a.cpu(), b)
    even = min(c for c in lens if c) if all(lens) else 0
    got = cache.read(t, n, tokens=even * len(lens), dtype=dtype)
    for a, b in zip(got, values(cache, table.tolist(), lens, [even] * len(lens), dtype)):
        assert same(a.cpu(), b)


def test_read_what_append_wrote(fp4):
    from moe_nvfp4_gemv_gb300.kvcache import KvCache8
    g = torch.Generator(device="cuda").manual_seed(9)
    cache = KvCache8.allocate(6, 4, 128, 32, "e4m3")
    k, v = (torch.randn(90, 4, 128, generator=g, device="cuda").to(BF16) for _ in range(2))
    table = torch.tensor([[4, 2], [0, 5]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([45, 45], dtype=torch.int32, device="cuda")
    cache.append(k, v, table, lens)
    for got, want in zip(cache.read(table, lens, tokens=90), (k, v)):
        # half a step of E4M3's three bits, and of its least step under a scale of at most 2^-6 (magnitudes below 7)
        assert bool(((got - want).float().abs() <= want.float().abs() / 16 + 2.0 ** -16).all())
        again = torch.empty_like(got)
    cache2 = KvCache8.allocate(6, 4, 128, 32, "e4m3")
    got = cache.read(table, lens, tokens=90)
    cache2.append(*got, table, lens)
    again = cache2.read(table, lens, tokens=90)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])  # (values that codes stand for stay)


def test_read_strides_and_rows_left_alone(fp4):
    cache = filled(8, 2, 64, 16, "int8", 1)
    table = torch.arange(8, dtype=torch.int32).view(2, 4)
    lens, counts = [50, 33], [18, 20]
    cu = torch.tensor([3, 21, 41], dtype=torch.int32, device="cuda")
    wide = torch.full((2, 50, 3 * 128), 9.0, dtype=F16, device="cuda")
    k, v = wide[0, :, 128:256].unflatten(1, (2, 64)), wide[1, :, :128].unflatten(1, (2, 64))
    got = cache.read(table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), cu=cu, k=k, v=v)
    assert got[0].data_ptr() == k.data_ptr()
    want = values(cache, table.tolist(), lens, counts, F16)
    for part, columns, w in ((0, slice(128, 256), want[0]), (1, slice(0, 128), want[1])):
        assert same(wide[part, 3:41, columns].cpu(), w.flatten(1))
        wide[part, 3:41, columns] = 9.0
    assert wide.eq(9.0).all()


def test_read_past_what_there_is(fp4):
    cache = filled(4, 2, 64, 16, "e4m3", 2)
    table = [[0, -1, 3], [4, 1, 2]]  # (no such pages: -1, 4)
    lens, counts = [45, 60], [50, 30]  # more than there are; past the table's 48
    cu = torch.tensor([0, 50, 80], dtype=torch.int32, device="cuda")
    got = cache.read(torch.tensor(table, dtype=torch.int32, device="cuda"),
                     torch.tensor(lens, dtype=torch.int32, device="cuda"), tokens=80, cu=cu)
    assert fp4.get_device_error() == 6
    for a, b in zip(got, values(cache, table, lens, counts, BF16)):
        assert same(a.cpu(), b)
    # rows that cu puts outside the output are refused, and nothing is written
    k = torch.full((80, 2, 64), 5.0, dtype=BF16, device="cuda")
    for bad in ([0, 50, 81], [-1, 50, 80], [0, 81, 80]):
        cache.read(torch.zeros(2, 3, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                   cu=torch.tensor(bad, dtype=torch.int32, device="cuda"), k=k, v=torch.empty_like(k))
        assert fp4.get_device_error() == 6


def test_read_refusals(fp4):
    cache = filled(4, 2, 64, 16, "e4m3", 2)
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    k = torch.zeros(4, 2, 64, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        cache.read(table, lens)
    with pytest.raises(ValueError):
        cache.read(table, lens, k=k)
    with pytest.raises(ValueError):
        cache.read(table, lens, tokens=4, k=k, v=k.clone())
    for bad in (dict(k=k.double(), v=k.double()), dict(k=k, v=k.float()), dict(k=k[:3], v=k), dict(k=k.cpu(), v=k),
                dict(k=k[:, :1], v=k[:, :1]), dict(k=k.transpose(1, 2), v=k.transpose(1, 2))):
        with pytest.raises(ValueError):
            cache.read(table, lens, **bad)
    with pytest.raises(ValueError):
        cache.read(table.long(), lens, k=k, v=k.clone())
    with pytest.raises(ValueError):
        cache.read(table, lens[:1], k=k, v=k.clone())
    with pytest.raises(ValueError):
        cache.read(table, lens, k=k, v=k.clone(), cu=lens)
    with pytest.raises(fp4.Fp4GemvError):
        cache.read(table, lens, tokens=3)  # (not the same for both)
    odd = torch.zeros(4, 2 * 64 + 1, dtype=BF16, device="cuda")[:, :128].unflatten(1, (2, 64))
    with pytest.raises(fp4.Fp4GemvError):
        cache.read(table, lens, k=odd, v=k)
    got = cache.read(table, lens, tokens=0)
    assert got[0].shape == (0, 2, 64)
