"""The 8-bit paged cache on the GPU: append bit for bit against a plain
restatement, attention against 64 bits.

Tolerance of attention, per element.  Codes and queries are exact operands, so
what is rounded is: the weights to f16 (2^-11 relative, or 2^-25 of the largest
weight below f16's normal range), fp32 sums and base-2 exponentials (below
2^-18 of a weight at the scores drawn here), and the output once.  With mass =
sum_t p_t |v_t|, the value before the last rounding is within
    d = 2^-10 mass + n 2^-25 max|v|
of the exact one, so the output lies between the roundings of exact - d and
exact + d.  The log of the sums carries the scores' fp32 error and the sums':
    2^-19 (1 + max|score|) + (16 + n / 128) 2^-23.
"""
import math

import numpy as np
import pytest
import torch

import decode_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def kv():
    require_gpu()
    from moe_nvfp4_gemv_gb300 import kvcache
    return kvcache


@pytest.fixture(scope="module")
def fp4():
    require_gpu()
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_table(lens, block, g, spare=3):
    """Shuffled pages; -1 past each sequence's end."""
    need = [-(-n // block) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def random_cache(pages, heads, block, dim, g, spread=2.0):
    """Any finite codes; scales over several powers of two."""
    c = {}
    for part in ("k", "v"):
        codes = torch.randint(0, 256, (pages, heads, block, dim), generator=g, dtype=torch.int32).to(torch.uint8)
        codes[(codes & 0x7F) == 0x7F] = 0x35  # (no E4M3 NaN)
        codes[codes == 0x80] = 0              # (no INT8 -128)
        c[part + "_codes"] = codes
        c[part + "_scale"] = torch.exp2(torch.randn(pages, heads, generator=g) * spread)
    return c


def scaled(c, fmt, k_std=1.0, v_std=1.0):
    """The same with scales that bring the values near the given sizes."""
    for part, std in (("k", k_std), ("v", v_std)):
        rms = ref.decode(c[part + "_codes"], fmt).square().mean().sqrt()
        c[part + "_scale"] = (c[part + "_scale"] / c[part + "_scale"].median() * std / rms).float()
    return c


def on_gpu(kv, c, fmt):
    return kv.KvCache8(*(c[n].to(DEV) for n in ("k_codes", "v_codes", "k_scale", "v_scale")), fmt=fmt)


def check_attention(kv, q, c, table, lens, fmt, dtype, window=0, sm_scale=None):
    cache = on_gpu(kv, c, fmt)
    n_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device=DEV)
    out = cache.attend(q, table.to(DEV), n_len, window=window, lse=lse, sm_scale=sm_scale)
    again = cache.attend(q, table.to(DEV), n_len, window=window, sm_scale=sm_scale)
    dim = q.shape[-1]
    want, want_lse, mass, peak = ref.attention(q, {k: v.to(DEV) for k, v in c.items()}, table, lens, fmt,
                                               sm_scale if sm_scale is not None else 1 / math.sqrt(dim), window)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two calls differ"
    n = max(max(lens), 1)
    vmax = float((ref.decode(c["v_codes"], fmt).abs().nan_to_num(0).amax() * c["v_scale"].amax()))
    d = 2.0 ** -10 * mass + n * 2.0 ** -25 * vmax
    low, high = (want - d).to(q.dtype), (want + d).to(q.dtype)  # (infinite where the type's range ends)
    outside = ~((out >= low) & (out <= high))
    assert not outside.any(), f"{int(outside.sum())} values outside, of {want.abs().max().item():.3g} at most"
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert (out[empty] == 0).all()
    tol_lse = 2.0 ** -19 * (1 + peak) + (16 + n / 128) * 2.0 ** -23
    assert ((lse.double() - want_lse)[~empty].abs() <= tol_lse).all()


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("fmt,dtype", [("e4m3", "bf16"), ("int8", "f16")])
def test_attention_dims_blocks(kv, dim, block, fmt, dtype):
    lens = [0, 1, 15, 16, 17, 31, 100, block, block + 1, 333]
    g = gen(dim + block)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 3, block, dim, g, 1.0), fmt)
    q = torch.randn(len(lens), 1, 6, dim, generator=g).to(TYPES[dtype]).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, dtype)


@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 3), (1, 16), (2, 5), (4, 4), (3, 7), (4, 8), (5, 7), (7, 16),
                                         (16, 4), (1, 64), (16, 1)])
@pytest.mark.parametrize("fmt,dim", [("e4m3", 128), ("int8", 64), ("e4m3", 256), ("int8", 96)])
def test_attention_rows(kv, q_len, group, fmt, dim):
    lens = [0, 1, q_len - 1, q_len, q_len + 15, 200, 61]
    g = gen(q_len * 100 + group)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 2, 32, dim, g, 1.0), fmt)
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16")


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 50, 100000])
@pytest.mark.parametrize("q_len", [1, 5])
def test_attention_window(kv, window, q_len):
    lens = [3, 16, 17, 64, 333, 1000]
    g = gen(window + q_len)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, 8, 128, generator=g).to(torch.float16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "f16", window=window)


@pytest.mark.parametrize("lens,heads,kv_heads,dim,q_len", [
    ([40001], 8, 1, 128, 1), ([40001], 32, 1, 128, 4), ([9000, 0, 20000, 31], 4, 2, 64, 1),
    ([5000] * 3, 16, 8, 256, 2), ([1 + i % 40 for i in range(300)], 4, 4, 96, 1)])
def test_attention_split_items(kv, lens, heads, kv_heads, dim, q_len):
    """Items cut between CTAs, and many items in one CTA."""
    g = gen(sum(lens) % 1000)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, kv_heads, 64, dim, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "bf16")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("k_std,v_std,q_std", [(1e-3, 1e6, 1e3), (30.0, 1e-12, 0.3), (0.0, 1.0, 1.0)])
def test_attention_magnitudes(kv, fmt, k_std, v_std, q_std):
    """Values far from 1, pages whose scales differ by orders of magnitude, zero scales."""
    lens = [700, 65]
    g = gen(17)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 2, 32, 128, g, 2.0), fmt, k_std, v_std)
    if k_std:
        c["v_scale"][::5] = 0.0
    q = (torch.randn(2, 2, 8, 128, generator=g) * q_std).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16")


def test_attention_sharp_scores(kv):
    """One token takes all, at the start, the middle and the end; the running maximum moves late."""
    lens = [512]
    g = gen(5)
    table, pages = make_table(lens, 16, g)
    for where in (0, 250, 511):
        c = scaled(random_cache(pages, 1, 16, 128, g, 0.0), "e4m3")
        q = torch.randn(1, 1, 4, 128, generator=g).to(torch.bfloat16)
        page = int(table[0, where // 16])
        c["k_codes"][page, 0, where % 16] = ref.encode((q[0, 0, 0].float() * 100).clamp(-448, 448), "e4m3")
        check_attention(kv, q.to(DEV), c, table, lens, "e4m3", "bf16")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_garbage_past_the_end(kv, fmt):
    """NaN codes, NaN and infinite scales where no sequence has tokens."""
    lens = [5, 17, 48, 0, 33]
    g = gen(3)
    table, pages = make_table(lens, 16, g, spare=4)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), fmt)
    used = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // 16)):
            page = int(table[b, j])
            used.add(page)
            rest = min(16, n - 16 * j)
            for part in ("k_codes", "v_codes"):
                c[part][page, :, rest:] = 0x7F
                c[part][page, :, rest::2] = 0xFF
    for page in set(range(pages)) - used:
        c["k_codes"][page] = 0x7F
        c["v_codes"][page] = 0x7F
        c["k_scale"][page] = math.nan
        c["v_scale"][page] = math.inf
    q = torch.randn(5, 2, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16")


def test_attention_strided_views_streams_and_graph(kv):
    """q inside a fused projection's rows, out inside a wider buffer; another stream; a captured graph with other lengths."""
    B, heads, kvh, dim, block = 6, 8, 2, 128, 16
    g = gen(8)
    lens = [40, 3, 97, 64, 0, 129]
    table, pages = make_table([160] * B, block, g)
    c = scaled(random_cache(pages, kvh, block, dim, g, 1.0), "e4m3")
    qkv = torch.randn(B, (heads + 2 * kvh) * dim, generator=g).to(torch.bfloat16).to(DEV)
    q = qkv[:, : heads * dim].view(B, 1, heads, dim)
    wide = torch.full((B, heads * dim + 64), 9.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, : heads * dim].view(B, 1, heads, dim)
    cache = on_gpu(kv, c, "e4m3")
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    plain = cache.attend(q.contiguous(), tab, n)
    cache.attend(q, tab, n, out=out)
    assert torch.equal(out, plain) and (wide[:, heads * dim:] == 9).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = cache.attend(q, tab, n)
        graph = torch.cuda.CUDAGraph()
        cache.attend(q, tab, n, out=other)
        with torch.cuda.graph(graph, stream=side):
            cache.attend(q, tab, n, out=other)
            cache.attend(q, tab, n, out=out)
    torch.cuda.current_stream().wait_stream(side)
    n.copy_(torch.tensor([7, 160, 0, 33, 16, 1], dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    want = cache.attend(q, tab, n)
    torch.cuda.synchronize()
    assert torch.equal(other, want) and torch.equal(out, want)


def test_attention_two_streams_at_once(kv):
    lens = [3000, 2000, 4000]
    g = gen(21)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, 2, 64, 128, g, 1.0), "e4m3")
    cache = on_gpu(kv, c, "e4m3")
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    qs = [torch.randn(3, 1, 16, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    want = [cache.attend(q, tab, n) for q in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(cache.attend(qs[i], tab, n))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


def test_attention_bad_pages_and_lengths(kv, fp4):
    """Bad page ids read as zeros, lengths are clamped; both raise the error word and touch nothing else."""
    block, dim = 16, 64
    g = gen(2)
    table, pages = make_table([64, 64], block, g)
    c = scaled(random_cache(pages, 1, block, dim, g, 1.0), "e4m3")
    cache = on_gpu(kv, c, "e4m3")
    q = torch.randn(2, 1, 2, dim, generator=g).to(torch.bfloat16).to(DEV)
    n = torch.tensor([64, 30], dtype=torch.int32, device=DEV)
    good = cache.attend(q, table.to(DEV), n)
    assert fp4.get_device_error() == 0
    for bad in (-1, pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out = cache.attend(q, t.to(DEV), n)
        assert fp4.get_device_error() == 6
        assert torch.isfinite(out).all() and torch.equal(out[1], good[1])
    out = cache.attend(q, table.to(DEV), torch.tensor([65, -3], dtype=torch.int32, device=DEV))
    assert fp4.get_device_error() == 6
    assert torch.equal(out[0], good[0]) and (out[1] == 0).all()


# ---- append ----
def run_append(kv, fmt, dtype, block, heads, dim, pasts, news, seed, ragged, magnitude=1.0, poison=False):
    g = gen(seed)
    lens = [p + n for p, n in zip(pasts, news)]
    table, pages = make_table(lens, block, g)
    c = random_cache(pages, heads, block, dim, g, 1.0)
    for part in ("k", "v"):
        s = c[part + "_scale"] * 2.0 ** -8
        c[part + "_scale"] = torch.exp2(torch.floor(torch.log2(s))) if fmt == "e4m3" else s
    T = sum(news)
    wide = torch.randn(T, 2 * heads * dim + 16, generator=g) * magnitude
    wide *= torch.exp2(torch.randn(T, 1, generator=g) * 2)
    if poison:
        wide[::3, ::7] = math.inf
        wide[1::3, ::11] = -math.inf
        wide[::2, ::13] = math.nan
        wide[:, 16:16 + 4] = 0.0
    wide = wide.to(TYPES[dtype])
    k = wide[:, : heads * dim].view(T, heads, dim) if T else torch.empty(0, heads, dim, dtype=TYPES[dtype])
    v = wide[:, heads * dim: 2 * heads * dim].view(T, heads, dim) if T else k
    gpu = on_gpu(kv, c, fmt)
    wg = wide.to(DEV)
    kg = wg[:, : heads * dim].unflatten(1, (heads, dim))
    vg = wg[:, heads * dim: 2 * heads * dim].unflatten(1, (heads, dim))
    cu = torch.tensor(np.concatenate([[0], np.cumsum(news)]), dtype=torch.int32, device=DEV) if ragged else None
    ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
    gpu.append(kg, vg, table.to(DEV), ln, cu_new=cu)
    want = {n: t.clone() for n, t in c.items()}
    ref.append(want, k, v, table, lens, news, block, fmt)
    for name in ("k_scale", "v_scale", "k_codes", "v_codes"):
        got = getattr(gpu, name).cpu()
        if "codes" in name and fmt == "e4m3":  # (NaN has two codes; -0 and 0 are apart)
            nan = (got & 0x7F) == 0x7F
            assert torch.equal(nan, (want[name] & 0x7F) == 0x7F), name
            got = torch.where(nan, want[name], got)
        assert torch.equal(got, want[name]), f"{name}: {(got != want[name]).sum().item()} differ"
    # again: the pages' scales stand, so the same codes come out
    gpu.append(kg, vg, table.to(DEV), ln, cu_new=cu)
    assert torch.equal(gpu.k_scale.cpu(), want["k_scale"])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (96, "f16"), (128, "bf16"), (256, "f16")])
def test_append(kv, fmt, block, dim, dtype):
    run_append(kv, fmt, dtype, block, 2, dim, [0, 1, block - 1, block, 37], [1] * 5, block + dim, False)
    run_append(kv, fmt, dtype, block, 2, dim, [0, 1, block - 1, block, 37], [block, 1, 2, 0, 3 * block + 5],
               block + dim + 1, True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("magnitude", [1e-30, 1e-4, 3e4])
def test_append_magnitudes_and_non_finite(kv, fmt, magnitude):
    run_append(kv, fmt, "bf16", 16, 3, 128, [5, 0, 30], [9, 40, 3], 11, True, magnitude)
    run_append(kv, fmt, "bf16", 16, 3, 128, [5, 0, 30], [9, 40, 3], 12, True, magnitude, poison=True)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_uniform_many(kv, fmt):
    run_append(kv, fmt, "f16", 16, 4, 64, [i % 50 for i in range(200)], [3] * 200, 4, False)


def test_append_then_attend_steps(kv):
    """Forty decode steps through one page boundary after another, against the plain cache."""
    fmt, block, heads, dim, B = "e4m3", 16, 2, 128, 3
    g = gen(77)
    pasts = [0, 13, 31]
    table, pages = make_table([p + 40 for p in pasts], block, g)
    cache = kv.KvCache8.allocate(pages, heads, dim, block, fmt)
    want = {n: getattr(cache, n).cpu().clone() for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
    x = torch.randn(sum(pasts), 2, heads, dim, generator=g).to(torch.bfloat16)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(pasts)]), dtype=torch.int32, device=DEV)
    cache.append(x[:, 0].to(DEV), x[:, 1].to(DEV), table.to(DEV), torch.tensor(pasts, dtype=torch.int32, device=DEV), cu)
    ref.append(want, x[:, 0], x[:, 1], table, pasts, pasts, block, fmt)
    for step in range(40):
        lens = [p + step + 1 for p in pasts]
        x = (torch.randn(B, 2, heads, dim, generator=g) * (1 + step / 8)).to(torch.bfloat16)
        n = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cache.append(x[:, 0].to(DEV), x[:, 1].to(DEV), table.to(DEV), n)
        ref.append(want, x[:, 0], x[:, 1], table, lens, [1] * B, block, fmt)
        if step % 10 == 9:
            q = torch.randn(B, 1, 6, dim, generator=g).to(torch.bfloat16).to(DEV)
            for name in want:
                assert torch.equal(getattr(cache, name).cpu(), want[name]), name
            check_attention(kv, q, want, table, lens, fmt, "bf16")


def test_append_bad_pages_and_lengths(kv, fp4):
    block, dim = 16, 64
    g = gen(6)
    table, pages = make_table([32, 32], block, g)
    x = torch.randn(4, 2, 1, dim, generator=g).to(torch.bfloat16).to(DEV)

    def attempt(t, lens):
        cache = kv.KvCache8.allocate(pages, 1, dim, block, "e4m3")
        cache.append(x[:, 0], x[:, 1], t.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
        return cache

    good = attempt(table, [18, 20])
    assert fp4.get_device_error() == 0
    t = table.clone()
    t[0, 1] = pages
    bad = attempt(t, [18, 20])
    assert fp4.get_device_error() == 6
    page = int(table[0, 1])
    assert (bad.k_codes[page] == 0).all() and (bad.k_scale[page] == 0).all()
    other = int(table[1, 1])
    assert torch.equal(bad.k_codes[other], good.k_codes[other])
    over = attempt(table, [33, 20])  # the second token lies past the table: the first is stored
    assert fp4.get_device_error() == 6
    last = int(table[0, 1])
    assert (over.v_codes[last, 0, 15] != 0).any() and torch.equal(over.k_codes[other], good.k_codes[other])
    under = attempt(table, [1, 20])  # the first token lies before the sequence
    assert fp4.get_device_error() == 6
    assert (under.k_codes[int(table[0, 0]), 0, 0] != 0).any()


def test_refusals(kv, fp4):
    cache = kv.KvCache8.allocate(4, 2, 128, 16)
    t = torch.zeros(1, 4, dtype=torch.int32, device=DEV)
    n = torch.ones(1, dtype=torch.int32, device=DEV)
    q = torch.zeros(1, 1, 4, 128, dtype=torch.bfloat16, device=DEV)
    k = torch.zeros(1, 2, 128, dtype=torch.bfloat16, device=DEV)
    for bad in (q.float(), q[..., :64], q[0], q.transpose(2, 3).contiguous().transpose(2, 3)):
        with pytest.raises(ValueError):
            cache.attend(bad, t, n)
    for kw in (dict(window=-1), dict(sm_scale=math.inf)):
        with pytest.raises(fp4.Fp4GemvError):
            cache.attend(q, t, n, **kw)
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend(q[:, :, :3].contiguous(), t, n)  # heads not a multiple of the KV heads
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend(q.expand(1, 17, 4, 128).contiguous(), t, n)
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend(q, t, n, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        cache.attend(q, t.long(), n)
    with pytest.raises(ValueError):
        cache.attend(q, t, n.repeat(2))
    with pytest.raises(ValueError):
        cache.attend(q, t, n, out=torch.empty_like(q, dtype=torch.float16))
    with pytest.raises(ValueError):
        cache.append(k.float(), k.float(), t, n)
    with pytest.raises(ValueError):
        cache.append(k, k[:, :1], t, n)
    with pytest.raises(ValueError):
        cache.append(k, k, t, n, cu_new=n)
    with pytest.raises(fp4.Fp4GemvError):
        kv.KvCache8.allocate(4, 2, 80, 16).append(torch.zeros(1, 2, 80, dtype=torch.bfloat16, device=DEV),
                                                  torch.zeros(1, 2, 80, dtype=torch.bfloat16, device=DEV), t, n)
    with pytest.raises(fp4.Fp4GemvError):
        kv.KvCache8.allocate(4, 2, 128, 24).append(k, k, t, n)
    with pytest.raises(ValueError):
        kv.KvCache8.allocate(4, 2, 128, 16, fmt="e5m2")
    # nothing to do is no error
    cache.append(k[:0], k[:0], t, n)
    assert cache.attend(q[:0], t[:0], n[:0]).shape == (0, 1, 4, 128)


@pytest.mark.parametrize("heads", [8, 32])
@pytest.mark.parametrize("lens", [[1 + 17 * i % 90 for i in range(70)], [600 - 8 * i for i in range(45)] + [0] * 5])
def test_attention_more_items_than_sms(kv, heads, lens):
    """head_dim 128 on its two-CTA form (more items than SMs), 2 and 8 rows per KV head; few rounds of 32 sequences."""
    g = gen(len(lens))
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 4, 16, 128, g, 1.0), "int8")
    q = torch.randn(len(lens), 1, heads, 128, generator=g).to(torch.float16).to(DEV)
    check_attention(kv, q, c, table, lens, "int8", "f16")
    q = torch.randn(len(lens), 3, heads, 128, generator=g).to(torch.float16).to(DEV)  # 6 and 24 rows
    check_attention(kv, q, c, table, lens, "int8", "f16")


@pytest.mark.parametrize("B", [31, 32, 33, 64, 65, 200, 1024])
def test_attention_batch_sizes(kv, B):
    lens = [(7 * i) % 50 for i in range(B)]
    g = gen(B)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 1, 16, 64, g, 1.0), "e4m3")
    q = torch.randn(B, 1, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "bf16")


@pytest.mark.parametrize("heads", [1, 5, 8, 11])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_heads(kv, heads, fmt):
    """Several heads per CTA, and a rest of them; the last of 300 sequences (a search of two rounds)."""
    run_append(kv, fmt, "bf16", 16, heads, 128, [3, 16, 29], [1] * 3, heads, False)
    run_append(kv, fmt, "bf16", 32, heads, 64, [0, 31, 64], [70, 1, 5], heads + 1, True)
    run_append(kv, fmt, "f16", 16, heads, 64, [i % 20 for i in range(300)], [i % 4 for i in range(300)], heads + 2, True)


# ---- attention of 17 to 32 rows per KV head and pass (E4M3, head_dim 128: tiles of 128 tokens) ----
@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("q_len,group,dtype", [(1, 17, "bf16"), (4, 8, "f16"), (3, 11, "bf16"), (5, 13, "f16"),
                                               (16, 4, "bf16"), (2, 64, "f16")])
def test_attention_wide_rows(kv, block, q_len, group, dtype):
    """One, two and four passes of 32 rows; lengths around tiles and pages; bf16 and f16 queries (two and three parts)."""
    lens = [0, 1, q_len, 15, 17, 127, 128, 129, 255, 257, 1000, 2050]
    g = gen(block + q_len * group)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, 2 * group, 128, generator=g).to(TYPES[dtype]).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", dtype)


@pytest.mark.parametrize("window", [1, 17, 100, 127, 128, 129, 300, 100000])
@pytest.mark.parametrize("block", [16, 128])
def test_attention_wide_window(kv, fp4, window, block):
    """Pages that lie before every query's window are not looked at: their ids are freed ones."""
    lens = [3, 130, 200, 513, 1000, 1500]
    q_len = 4
    g = gen(window + block)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, 16, 128, generator=g).to(torch.float16).to(DEV)
    assert fp4.get_device_error() == 0
    check_attention(kv, q, c, table, lens, "e4m3", "f16", window=window)
    freed = table.clone()
    for b, n in enumerate(lens):
        freed[b, : max(0, n - q_len - window + 1) // block] = -1
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    cache = on_gpu(kv, c, "e4m3")
    assert torch.equal(cache.attend(q, freed.to(DEV), n, window=window), cache.attend(q, tab, n, window=window))
    assert fp4.get_device_error() == 0


@pytest.mark.parametrize("lens", [[40001], [9000, 0, 20000, 31], [130] * 200, [1 + 37 * i % 700 for i in range(90)],
                                  [16000] + [20] * 40, [128] * 152, [0] * 33 + [700]])
def test_attention_wide_shares(kv, lens):
    """Items cut in many parts, several items in a share, cuts inside items: partials of every kind are joined."""
    g = gen(len(lens))
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, 2, 64, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), 3, 20, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("k_std,v_std,q_std", [(1e-3, 1e6, 1e3), (30.0, 1e-12, 0.3), (0.0, 1.0, 1.0)])
def test_attention_wide_magnitudes(kv, dtype, k_std, v_std, q_std):
    """As above, with a few entries of a query far above its others (what the E4M3 parts of a row have to span)."""
    lens = [700, 65]
    g = gen(18)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 2, 32, 128, g, 2.0), "e4m3", k_std, v_std)
    if k_std:
        c["v_scale"][::5] = 0.0
    q = torch.randn(2, 2, 32, 128, generator=g) * q_std
    q[:, :, ::3, 5] *= 30
    q[:, :, 1::3, 77] *= 1000 if dtype == "bf16" else 10
    q[:, :, 7] = 0
    check_attention(kv, q.to(TYPES[dtype]).to(DEV), c, table, lens, "e4m3", dtype)


def test_attention_wide_sharp_scores(kv):
    """One token takes all, in each group's first and later tiles; the running maximum moves late."""
    lens = [1024]
    g = gen(6)
    table, pages = make_table(lens, 16, g)
    for where in (0, 130, 400, 1023):
        c = scaled(random_cache(pages, 1, 16, 128, g, 0.0), "e4m3")
        q = torch.randn(1, 1, 24, 128, generator=g).to(torch.bfloat16)
        page = int(table[0, where // 16])
        c["k_codes"][page, 0, where % 16] = ref.encode((q[0, 0, 0].float() * 100).clamp(-448, 448), "e4m3")
        check_attention(kv, q.to(DEV), c, table, lens, "e4m3", "bf16")


@pytest.mark.parametrize("block", [16, 64])
def test_attention_wide_garbage_past_the_end(kv, block):
    """NaN codes past the ends, NaN and infinite scales in pages of no sequence, at the tiles' ends too."""
    lens = [5, 127, 130, 0, 333]
    g = gen(block)
    table, pages = make_table(lens, block, g, spare=4)
    c = scaled(random_cache(pages, 2, block, 128, g, 1.0), "e4m3")
    used = set()
    for b, n in enumerate(lens):
        for j in range(-(-n // block)):
            page = int(table[b, j])
            used.add(page)
            for part in ("k_codes", "v_codes"):
                c[part][page, :, min(block, n - block * j):] = 0x7F
    for page in set(range(pages)) - used:
        c["k_codes"][page] = 0x7F
        c["v_codes"][page] = 0xFF
        c["k_scale"][page] = math.nan
        c["v_scale"][page] = math.inf
    q = torch.randn(5, 5, 10, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "bf16")


def test_attention_wide_bad_pages_non_finite_and_streams(kv, fp4):
    """Bad page ids read as zeros and raise the error word; a NaN stays in its rows; strides, streams and a graph."""
    B, q_len, heads, kvh = 3, 2, 24, 2
    g = gen(12)
    lens = [300, 64, 500]
    table, pages = make_table([512] * B, 32, g)
    c = scaled(random_cache(pages, kvh, 32, 128, g, 1.0), "e4m3")
    cache = on_gpu(kv, c, "e4m3")
    rows = torch.randn(B * q_len, (heads + 2 * kvh) * 128, generator=g).to(torch.bfloat16).to(DEV)
    q = rows[:, : heads * 128].view(B, q_len, heads, 128)
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    plain = cache.attend(q.contiguous(), tab, n)
    wide = torch.full((B * q_len, heads * 128 + 64), 9.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, : heads * 128].view(B, q_len, heads, 128)
    cache.attend(q, tab, n, out=out)
    assert torch.equal(out, plain) and (wide[:, heads * 128:] == 9).all()
    assert fp4.get_device_error() == 0
    for bad in (-1, pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        got = cache.attend(q, t.to(DEV), n)
        assert fp4.get_device_error() == 6
        assert torch.isfinite(got).all() and torch.equal(got[1:], plain[1:])
    hot = q.clone()
    hot[1, 0, 3, 9] = math.nan
    hot[2, 1, 20, 100] = math.inf
    got = cache.attend(hot, tab, n)
    assert got[1, 0, 3].isnan().all() and not torch.isfinite(got[2, 1, 20]).any()
    same = torch.ones(B, q_len, heads, dtype=torch.bool, device=DEV)
    same[1, 0, 3] = same[2, 1, 20] = False
    assert torch.equal(got[same], plain[same])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = cache.attend(q, tab, n)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cache.attend(q, tab, n, out=other)
            cache.attend(q, tab, n, out=out)
    torch.cuda.current_stream().wait_stream(side)
    n.copy_(torch.tensor([7, 512, 0], dtype=torch.int32))
    for _ in range(3):
        graph.replay()
    want = cache.attend(q, tab, n)
    torch.cuda.synchronize()
    assert torch.equal(other, want) and torch.equal(out, want) and (want[2] == 0).all()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(cache.attend(q, tab, n))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in got)


@pytest.mark.parametrize("lens,skip,met", [([700, 64], 0, True), ([4000, 300, 2000], 0, True), ([20000], 2, True),
                                           ([4000, 300, 2000], 1, False)])
def test_attention_wide_timeout_then_recovery(kv, fp4, lens, skip, met):
    """A tile's values that never come (a host-side hook; nothing is in flight): the call comes back, the error word
    reads a timeout, outputs are NaN where the tile was missing; the next calls on the same workspace are right.  (The
    last case's 100 tiles are a CTA's first ones each: the hook's second is nobody's.)"""
    g = gen(30)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, 2, 64, 128, g, 1.0), "e4m3")
    cache = on_gpu(kv, c, "e4m3")
    q = torch.randn(len(lens), 3, 16, 128, generator=g).to(torch.bfloat16).to(DEV)
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    good = cache.attend(q, tab, n)
    assert fp4.get_device_error() == 0
    try:
        fp4.set_wait_limit_ns(5_000_000)
        fp4.debug_skip_stage(skip)
        lost = cache.attend(q, tab, n)
        assert fp4.get_device_error() == (5 if met else 0)
    finally:
        fp4.debug_skip_stage(-1)
        fp4.set_wait_limit_ns(0)
    whole = ~lost.isnan().any(-1)
    assert whole.all() != met and torch.equal(lost[whole], good[whole])
    for _ in range(2):
        assert torch.equal(cache.attend(q, tab, n), good)
    assert fp4.get_device_error() == 0


@pytest.mark.parametrize("B", [33, 300, 1024])
def test_attention_wide_batch_sizes(kv, B):
    """Up to the largest batch (the plan's tables fill shared memory to its end), idle sequences among them."""
    lens = [(11 * i) % 150 for i in range(B)]
    g = gen(B)
    table, pages = make_table(lens, 32, g)
    c = scaled(random_cache(pages, 1, 32, 128, g, 1.0), "e4m3")
    q = torch.randn(B, 2, 9, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, "e4m3", "bf16")
