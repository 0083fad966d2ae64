"""Attention over the 8-bit cache where it can go wrong: the ends of its ranges, masked places, captured calls.

Tolerances are those of test_gpu_kv_cache.py (its docstring), with what the range of the weights adds named at the
test that is about it."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, TYPES, check_attention, fp4, gen, kv, make_table, on_gpu, random_cache, scaled  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,fmt", [(2, "e4m3"), (8, "e4m3"), (8, "int8")])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
def test_attention_largest_windows(kv, group, fmt, window):
    """A window past every length is none, on both kernels, for sequences shorter than their queries too."""
    lens = [0, 1, 2, 3, 4, 5, 100, 300]
    g = gen(group)
    table, pages = make_table(lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), fmt)
    q = torch.randn(len(lens), 4, 2 * group, 128, generator=g).to(torch.bfloat16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16", window=window)


@pytest.mark.parametrize("group,dim,fmt", [(2, 128, "e4m3"), (2, 64, "int8"), (8, 96, "e4m3"), (8, 128, "e4m3")])
def test_attention_of_far_negative_scores(kv, group, dim, fmt):
    """Scores of -1e32 and below are scores: their rows are not taken for empty ones.  (Scales and codes of K are alike, and
    no warp has a second strip: next to such a score nothing else has bits left, its own rounding is 2^80.)"""
    lens = [1, 3, 16, 17, 128]
    g = gen(dim + group)
    table, pages = make_table(lens, 32, g)
    c = random_cache(pages, 1, 32, dim, g, 0.0)
    c["k_codes"][:] = int(ref.encode(torch.tensor([1.0]), fmt)[0])
    c["v_scale"][:] = 2.0 ** -6
    q = -torch.ones(len(lens), 4, group, dim, dtype=torch.bfloat16, device=DEV)
    check_attention(kv, q, c, table, lens, fmt, "bf16", sm_scale=1e30)


def tail_output(kv, fmt, heads, q_len, dim, bits, n=32768, B=320):
    """B sequences over the same n tokens: the first scores `bits` (base 2) above all others and holds zeros, the others
    ones.  Returns (out, the exact value)."""
    block = 128
    one, top = (int(ref.encode(torch.tensor([x]), fmt)[0]) for x in (1.0, float(bits)))
    cache = kv.KvCache8.allocate(n // block, 1, dim, block, fmt)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    cache.v_codes.fill_(one)
    table = torch.arange(n // block, dtype=torch.int32, device=DEV).repeat(B, 1)
    cache.k_codes[0, 0, 0, 0] = top
    cache.v_codes[0, 0, 0] = 0
    q = torch.zeros(B, q_len, heads, dim, dtype=torch.float16, device=DEV)
    q[..., 0] = 1.0
    lens = torch.full((B,), n, dtype=torch.int32, device=DEV)
    out = cache.attend(q, table, lens, sm_scale=math.log(2.0))
    seen = torch.arange(n - q_len, n, dtype=torch.float64, device=DEV).view(1, q_len, 1, 1)  # others, for each query
    return out.double(), (seen * 2.0 ** -bits / (1 + seen * 2.0 ** -bits)).expand_as(out)


@pytest.mark.parametrize("heads,q_len,dim,fmt", [(8, 1, 128, "e4m3"), (8, 1, 64, "int8"), (4, 3, 256, "e4m3"),
                                                 (6, 4, 96, "e4m3"), (32, 1, 128, "int8")])
@pytest.mark.parametrize("bits", [24, 26, 28])
def test_attention_small_weights_count(kv, heads, q_len, dim, fmt, bits):
    """Weights of 2^-24 to 2^-28 of the largest, 32767 of them: f16 rounds the weights (2^-11 relative, from 2^-21 of the
    largest down 2^-32 of it), so what is lost is at most 2^-32 for each; f16 outputs."""
    out, want = tail_output(kv, fmt, heads, q_len, dim, bits)
    d = 2.0 ** -10 * want + 32768 * 2.0 ** -32
    assert ((out - want).abs() <= d).all(), float((out / want).min())


@pytest.mark.parametrize("heads,q_len", [(32, 1), (6, 4), (24, 2)])
@pytest.mark.parametrize("bits", [22, 24, 26, 28])
def test_attention_wide_small_weights_count(kv, heads, q_len, bits):
    """The same on the tensor core: three parts of a weight hold what f16 does."""
    out, want = tail_output(kv, "e4m3", heads, q_len, 128, bits)
    d = 2.0 ** -10 * want + 32768 * 2.0 ** -32
    assert ((out - want).abs() <= d).all(), float((out / want).min())


def check_nan_values(kv, q_len, group, dim, block, window):
    """NaN values of tokens that some queries see, some do not, and (before the window) none does: NaN where the formula
    says, the other outputs as if they were not there."""
    lens = [1, 5, 16, 17, 40, 129, 133, 300, 1000]
    g = gen(dim + q_len + block)
    table, pages = make_table(lens, block, g)
    c = scaled(random_cache(pages, 2, block, dim, g, 1.0), "e4m3")
    for b, n in enumerate(lens):
        first = n - q_len + 1 - window if window else n  # the first query's first token
        for i, t in enumerate((n - 1, n - 2, n - q_len, first, first - 1, first - 2)):
            if 0 <= t < n and (i < 3 or window):
                code = c["v_codes"][int(table[b, t // block])]
                code[b % 2, t % block, 3 + 8 * i] = 0x7F
                code[b % 2, t % block, dim - 1 - i] = 0xFF
    q = torch.randn(len(lens), q_len, 2 * group, dim, generator=g).to(torch.float16).to(DEV)
    n_len = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out = on_gpu(kv, c, "e4m3").attend(q, table.to(DEV), n_len, window=window)
    want, _, mass, _ = ref.attention(q, {k: v.to(DEV) for k, v in c.items()}, table, lens, "e4m3", 1 / math.sqrt(dim),
                                     window)
    assert torch.equal(out.isnan(), want.isnan())
    assert 0 < int(want.isnan().sum()) < want.numel() // 8
    vmax = float(ref.decode(c["v_codes"], "e4m3").abs().nan_to_num(0).amax() * c["v_scale"].amax())
    d = 2.0 ** -10 * mass + max(lens) * 2.0 ** -25 * vmax
    low, high = (want - d).to(q.dtype), (want + d).to(q.dtype)
    assert (((out >= low) & (out <= high)) | want.isnan()).all()


@pytest.mark.parametrize("q_len,group,dim,block", [(4, 2, 128, 16), (3, 5, 64, 32), (2, 7, 256, 16), (4, 8, 96, 64),
                                                   (8, 1, 128, 128), (16, 1, 128, 16)])
@pytest.mark.parametrize("window", [0, 1, 20, 130])
def test_attention_nan_values_of_unseen_tokens(kv, q_len, group, dim, block, window):
    check_nan_values(kv, q_len, group, dim, block, window)


@pytest.mark.parametrize("q_len,group,block", [(4, 8, 16), (3, 11, 64), (16, 4, 128), (2, 12, 32)])
@pytest.mark.parametrize("window", [0, 1, 20, 130, 300])
def test_attention_wide_nan_values_of_unseen_tokens(kv, q_len, group, block, window):
    check_nan_values(kv, q_len, group, 128, block, window)


@pytest.mark.parametrize("heads", [8, 24])
def test_first_calls_inside_captures(kv, monkeypatch, heads):
    """Two graphs captured on a stream that attend has never run on, in memory full of ones: each counts on counters that
    it cleared itself, so the second may run before the first; and an eager call there does not meet the graphs'."""
    monkeypatch.setattr(kv, "_workspaces", {})
    lens = [5000, 700]
    g = gen(heads)
    table, pages = make_table(lens, 64, g)
    c = scaled(random_cache(pages, 1, 64, 128, g, 1.0), "e4m3")
    cache, tab = on_gpu(kv, c, "e4m3"), table.to(DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    q = torch.randn(2, 1, heads, 128, generator=g).to(torch.bfloat16).to(DEV)
    want = cache.attend(q, tab, n)
    side, pool = torch.cuda.Stream(), torch.cuda.graph_pool_handle()
    side.wait_stream(torch.cuda.current_stream())
    size = kv.attention_workspace_bytes(128)
    dirty, graphs, outs = torch.cuda.CUDAGraph(), [], []
    with torch.cuda.graph(dirty, pool=pool, stream=side):
        junk = [torch.full((size,), 1, dtype=torch.uint8, device=DEV) for _ in range(3)]
    dirty.replay()
    torch.cuda.synchronize()
    del junk
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        out = torch.full_like(q, 9.0)
        with torch.cuda.graph(graphs[-1], pool=pool, stream=side):
            cache.attend(q, tab, n, out=out)
            cache.attend(q, tab, n, out=out)
        outs.append(out)
    for i in (1, 0, 1):
        outs[i].fill_(9.0)
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i], want)
    with torch.cuda.stream(side):
        eager = cache.attend(q, tab, n)
    torch.cuda.synchronize()
    assert torch.equal(eager, want)


def test_workspace_of_another_stream_is_cleared_there(kv, monkeypatch):
    """The workspace of a stream that is not the current one is cleared on that stream, whatever the current one does."""
    monkeypatch.setattr(kv, "_workspaces", {})
    side, dev = torch.cuda.Stream(), torch.device(DEV, torch.cuda.current_device())
    size = kv.attention_workspace_bytes(64)
    torch.cuda.empty_cache()
    for s in (side, torch.cuda.current_stream()):  # both streams' next block of that size holds ones
        with torch.cuda.stream(s):
            junk = torch.full((size,), 1, dtype=torch.uint8, device=dev)
        torch.cuda.synchronize()
        del junk
    torch.cuda._sleep(400_000_000)  # (some 200 ms of the current stream)
    ws = kv.attention_workspace(dev, 64, side.cuda_stream)
    with torch.cuda.stream(side):
        left = ws.cpu()  # (a copy: a kernel's first launch may wait for all streams)
    assert not left.any()
    assert kv.attention_workspace(dev, 64, side.cuda_stream) is ws


@pytest.mark.parametrize("heads,dim,fmt", [(8, 128, "e4m3"), (24, 128, "e4m3"), (8, 64, "int8"), (4, 256, "e4m3")])
def test_pages_past_four_gibibytes(kv, heads, dim, fmt):
    """Pages at the end of caches whose codes take more than 2^32 bytes: append and attention as on the same pages of a
    small cache."""
    block, n = 128, 700
    g = gen(dim + heads)
    pages = (1 << 32) // (block * dim) + 9
    big = kv.KvCache8.allocate(pages, 1, dim, block, fmt)
    small = kv.KvCache8.allocate(9, 1, dim, block, fmt)
    x = torch.randn(n, 2, 1, dim, generator=g).to(torch.bfloat16).to(DEV)
    q = torch.randn(1, 3, heads, dim, generator=g).to(torch.bfloat16).to(DEV)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    far = torch.tensor([[8, 3, 5, 0, 7, 1]], dtype=torch.int32, device=DEV)
    outs = []
    for cache, table in ((big, far + (pages - 9)), (small, far)):
        cache.append(x[:, 0], x[:, 1], table, lens)
        outs.append(cache.attend(q, table, lens))
    assert torch.equal(big.k_codes[-9:], small.k_codes) and torch.equal(big.v_scale[-9:], small.v_scale)
    assert torch.equal(outs[0], outs[1]) and outs[0].abs().max() > 0
    assert int(big.k_codes[:-9].count_nonzero()) == 0


@pytest.mark.parametrize("heads,q_len,dim,fmt", [(8, 1, 128, "e4m3"), (32, 1, 128, "e4m3"), (8, 2, 64, "int8")])
def test_attention_of_a_very_long_sequence(kv, heads, q_len, dim, fmt):
    """500001 tokens on one KV head: every CTA has a part, joined in two levels."""
    lens = [500001, 3]
    g = gen(dim + heads)
    table, pages = make_table(lens, 128, g)
    c = scaled(random_cache(pages, 1, 128, dim, g, 1.0), fmt)
    q = torch.randn(2, q_len, heads, dim, generator=g).to(torch.float16).to(DEV)
    check_attention(kv, q, c, table, lens, fmt, "f16")
