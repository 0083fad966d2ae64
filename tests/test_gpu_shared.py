"""Attention of sequences that begin alike (KvCache8.attend_shared) on the GPU,
against 64 bits.

Tolerances are those of test_gpu_kv_cache.py (its docstring): the tokens taken
together go through the same roundings as the others."""
import math

import pytest
import torch

import decode_ref as ref
from test_gpu_kv_cache import DEV, TYPES, fp4, gen, kv, on_gpu, random_cache, scaled  # noqa: F401
from test_gpu_sinks import attention64

pytestmark = pytest.mark.gpu


def shared_table(prefix, lens, block, g, spare=3):
    """Shuffled pages, the whole ones of the first ``prefix`` tokens the same for all; -1 past each sequence's end."""
    full = prefix // block
    need = [-(-n // block) for n in lens]
    total = full + sum(max(0, n - full) for n in need) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    at = full
    for b, n in enumerate(need):
        table[b, :min(n, full)] = order[:min(n, full)]
        if n > full:
            table[b, full:n] = order[at:at + n - full]
            at += n - full
    return table, total


def same_beginning(c, table, lens, prefix, block):
    """The page that the common tokens fill in part is each sequence's own, with the same beginning and scales."""
    full, rest = divmod(prefix, block)
    pages = [int(table[b, full]) for b, n in enumerate(lens) if n > full * block] if rest else []
    for page in pages[1:]:
        for part in ("k", "v"):
            c[part + "_scale"][page] = c[part + "_scale"][pages[0]]
            c[part + "_codes"][page, :, :rest] = c[part + "_codes"][pages[0], :, :rest]


def case(prefix, lens, heads, kv_heads, dim, block, fmt, dtype, q_len, seed=0, spread=1.0, k_std=1.0, v_std=1.0, q_std=1.0):
    g = gen(prefix + dim + seed)
    table, pages = shared_table(prefix, lens, block, g)
    c = scaled(random_cache(pages, kv_heads, block, dim, g, spread), fmt, k_std, v_std)
    same_beginning(c, table, lens, prefix, block)
    q = (torch.randn(len(lens), q_len, heads, dim, generator=g) * q_std).to(TYPES[dtype]).to(DEV)
    return c, table, q


def run(kv, c, fmt, q, table, lens, prefix, sm_scale=None, always=True, **kw):
    cache = on_gpu(kv, c, fmt)
    lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device=DEV)
    out = cache.attend_shared(q, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
                              torch.tensor([prefix], dtype=torch.int32, device=DEV), lse=lse, sm_scale=sm_scale, always=always,
                              **kw)
    return out, lse


def check(kv, c, fmt, q, table, lens, prefix, sm_scale=None, nans=False, always=True):
    out, lse = run(kv, c, fmt, q, table, lens, prefix, sm_scale, always=always)
    again, _ = run(kv, c, fmt, q, table, lens, prefix, sm_scale, always=always)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)), "two calls differ"
    scale = sm_scale if sm_scale is not None else 1 / math.sqrt(q.shape[-1])
    want, want_lse, mass, peak = attention64(q, c, table, lens, fmt, scale, 0, 0)
    assert torch.equal(out.isnan(), want.isnan())
    assert bool(want.isnan().any()) == nans
    n = max(max(lens), 1)
    vmax = float(ref.decode(c["v_codes"], fmt).abs().nan_to_num(0).amax() * c["v_scale"].amax())
    d = 2.0 ** -10 * mass + n * 2.0 ** -25 * vmax
    low, high = (want - d).to(q.dtype), (want + d).to(q.dtype)
    outside = ~((out >= low) & (out <= high)) & ~want.isnan()
    assert not outside.any(), f"{int(outside.sum())} of {outside.numel()} values outside"
    empty = torch.isinf(want_lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty) and (out[empty] == 0).all()
    tol = 2.0 ** -19 * (1 + peak) + (16 + n / 128) * 2.0 ** -23
    assert ((lse.double() - want_lse)[~empty].abs().nan_to_num(0) <= tol).all()


def test_shared_smallest(kv):
    """One tile, one block of rows."""
    c, table, q = case(128, [129, 130], 2, 1, 64, 16, "e4m3", "bf16", 1)
    check(kv, c, "e4m3", q, table, [129, 130], 128)


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("fmt,dtype,block", [("e4m3", "bf16", 16), ("int8", "f16", 64), ("e4m3", "f16", 128),
                                             ("int8", "bf16", 32)])
@pytest.mark.parametrize("prefix", [128, 300, 1024])
def test_shared_dims_formats(kv, dim, fmt, dtype, block, prefix):
    lens = [prefix + n for n in (1, 2, 17, 100, 33)]
    c, table, q = case(prefix, lens, 8, 2, dim, block, fmt, dtype, 1)
    check(kv, c, fmt, q, table, lens, prefix)


@pytest.mark.parametrize("batch,q_len,group,kv_heads", [
    (1, 1, 1, 1), (3, 1, 8, 2), (16, 1, 8, 1), (17, 1, 8, 2), (32, 1, 8, 1), (33, 4, 3, 1), (50, 1, 8, 2), (7, 16, 5, 1),
    (100, 2, 2, 3), (5, 3, 64, 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shared_rows(kv, batch, q_len, group, kv_heads, dim):
    """Rows from one to a thousand: one block, two, an odd number of them; rows of a tile of the own part beyond 32."""
    prefix = 700
    lens = [prefix + q_len + (13 * b) % 40 for b in range(batch)]
    c, table, q = case(prefix, lens, kv_heads * group, kv_heads, dim, 32, "e4m3", "bf16", q_len)
    check(kv, c, "e4m3", q, table, lens, prefix)


@pytest.mark.parametrize("prefix,batch,heads,kv_heads,dim,fmt", [
    (20000, 4, 8, 1, 128, "e4m3"), (9999, 40, 8, 1, 128, "int8"), (30000, 2, 4, 2, 256, "e4m3"), (5000, 20, 32, 16, 64, "int8"),
    (2000, 60, 128, 8, 96, "e4m3"), (128, 64, 64, 16, 128, "e4m3"), (256, 300, 32, 4, 128, "int8")])
def test_shared_long(kv, prefix, batch, heads, kv_heads, dim, fmt):
    """Items cut by many CTAs; CTAs that hold several items."""
    lens = [prefix + 1 + (7 * b) % 90 for b in range(batch)]
    c, table, q = case(prefix, lens, heads, kv_heads, dim, 64, fmt, "bf16", 1)
    check(kv, c, fmt, q, table, lens, prefix)


@pytest.mark.parametrize("lens", [[0, 0, 0], [0, 700, 0, 650], [300, 700, 650], [2, 700, 700], [700, 700], [513, 640, 900],
                                  [512, 515, 514]])
@pytest.mark.parametrize("q_len", [1, 4])
@pytest.mark.parametrize("prefix", [-5, 0, 127, 512, 1 << 30])
def test_shared_lengths(kv, lens, q_len, prefix):
    """Empty sequences, the first one among them; sequences shorter than the beginning that they are said to have; that
    end with it; lengths said to be shared beyond all lengths (here all of a sequence's pages are)."""
    g = gen(len(lens) + q_len)
    table, pages = shared_table(max(lens) + 16, lens, 16, g)
    c = scaled(random_cache(pages, 2, 16, 128, g, 1.0), "e4m3")
    q = torch.randn(len(lens), q_len, 6, 128, generator=g).to(torch.bfloat16).to(DEV)
    check(kv, c, "e4m3", q, table, lens, prefix)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("k_std,v_std,q_std", [(1e-3, 1e6, 1e3), (30.0, 1e-12, 0.3), (0.0, 1.0, 1.0)])
@pytest.mark.parametrize("dim", [128, 256])
def test_shared_magnitudes(kv, fmt, k_std, v_std, q_std, dim):
    """Values far from 1, pages whose scales differ by orders of magnitude, zero scales."""
    lens = [600, 577, 640]
    c, table, q = case(512, lens, 8, 2, dim, 32, fmt, "bf16", 2, spread=2.0, k_std=k_std, v_std=v_std, q_std=q_std)
    if k_std:
        c["v_scale"][::5] = 0.0
    check(kv, c, fmt, q, table, lens, 512)


@pytest.mark.parametrize("dim", [64, 256])
def test_shared_sharp_scores(kv, dim):
    """One token takes all, in the first, a middle and the last tile, and in the own part: the maximum moves late."""
    for where in (0, 130, 700, 1023, 1030):
        lens = [1040, 1031]
        c, table, q = case(1024, lens, 4, 1, dim, 16, "e4m3", "bf16", 1, spread=0.0)
        page = int(table[0, where // 16])
        c["k_codes"][page, 0, where % 16] = ref.encode((q[0, 0, 0].float().cpu() * 100).clamp(-448, 448), "e4m3")
        check(kv, c, "e4m3", q, table, lens, 1024)
        check(kv, c, "e4m3", q, table, lens, 1024, sm_scale=-0.3)
        check(kv, c, "e4m3", q, table, lens, 1024, sm_scale=0.0)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("bits", [24, 28])
@pytest.mark.parametrize("dim", [128, 256])
def test_shared_small_weights_count(kv, fmt, bits, dim):
    """32767 weights of 2^-24 and 2^-28 of the largest: f16 rounds weights (2^-11 relative, 2^-32 of the largest)."""
    n, block, batch = 32768, 128, 3
    one, top = (int(ref.encode(torch.tensor([x]), fmt)[0]) for x in (1.0, float(bits)))
    cache = kv.KvCache8.allocate(n // block + batch, 1, dim, block, fmt)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    cache.v_codes.fill_(one)
    table = torch.arange(n // block + 1, dtype=torch.int32, device=DEV).repeat(batch, 1)
    table[:, -1] += torch.arange(batch, device=DEV)
    cache.k_codes[0, 0, 0, 0] = top
    cache.v_codes[0, 0, 0] = 0
    q = torch.zeros(batch, 1, 2, dim, dtype=torch.float16, device=DEV)
    q[..., 0] = 1.0
    out = cache.attend_shared(q, table, torch.full((batch,), n + 1, dtype=torch.int32, device=DEV),
                              torch.tensor([n], dtype=torch.int32, device=DEV), sm_scale=math.log(2.0),
                              always=True).double()
    want = n * 2.0 ** -bits / (1 + n * 2.0 ** -bits)
    assert ((out - want).abs() <= 2.0 ** -10 * want + (n + 1) * 2.0 ** -32).all()


@pytest.mark.parametrize("fmt,dim,heads,q_len,block", [
    ("e4m3", 64, 6, 1, 16), ("int8", 64, 54, 2, 32), ("e4m3", 96, 9, 4, 32), ("int8", 128, 12, 2, 64), ("e4m3", 128, 30, 2, 16),
    ("int8", 128, 24, 4, 128), ("e4m3", 256, 6, 4, 64), ("int8", 256, 51, 1, 32)])
@pytest.mark.parametrize("prefix,always", [(130, True), (500, True), (40, False), (130, False)])
def test_shared_many_short_ends(kv, fmt, dim, heads, q_len, block, prefix, always):
    """More sequences' ends, or whole sequences, than SMs hold CTAs, of few strips each: a warp takes one by itself."""
    lens = [prefix + q_len + (23 * i) % 70 if i % 9 else 0 for i in range(150)]
    c, table, q = case(prefix, lens, heads, 3, dim, block, fmt, "bf16", q_len)
    check(kv, c, fmt, q, table, lens, prefix, always=always)


@pytest.mark.parametrize("fmt,dim,heads,always", [("e4m3", 256, 16, True), ("int8", 128, 32, True), ("e4m3", 96, 12, True),
                                                  ("int8", 256, 16, False), ("e4m3", 128, 16, False)])
def test_shared_largest_batch(kv, fmt, dim, heads, always):
    lens = [130 + (11 * i) % 90 if i % 7 else 0 for i in range(1024)]
    c, table, q = case(128, lens, heads, 1, dim, 32, fmt, "bf16", 1)
    check(kv, c, fmt, q, table, lens, 128, always=always)


def test_shared_many_short_sequences_nan_codes(kv):
    """... their NaN values, each in the rows that see them."""
    prefix, q_len = 40, 4
    lens = [prefix + q_len + (23 * i) % 70 for i in range(200)]
    c, table, q = case(prefix, lens, 6, 3, 64, 16, "e4m3", "bf16", q_len)
    for b in range(0, 200, 9):
        for t, d in ((lens[b] - 1, 3), (lens[b] - 3, 40)):
            c["v_codes"][int(table[b, t // 16]), 1, t % 16, d] = 0x7F
    check(kv, c, "e4m3", q, table, lens, prefix, nans=True, always=False)


def test_shared_nan_codes(kv):
    """A NaN value of the beginning is in every row; one of a sequence's own tokens in that sequence alone; of tokens past
    the ends, and of an idle sequence's pages, in none."""
    lens = [530, 0, 560, 600]
    c, table, q = case(512, lens, 8, 2, 128, 16, "e4m3", "f16", 1)
    c["v_codes"][int(table[0, 3]), 1, 5, 17] = 0x7F
    c["v_codes"][int(table[2, 33]), 0, 4, 90] = 0xFF
    for b, n in enumerate(lens):
        if n % 16:
            c["v_codes"][int(table[b, n // 16]), :, n % 16:] = 0x7F
            c["k_codes"][int(table[b, n // 16]), :, n % 16:] = 0x7F
    check(kv, c, "e4m3", q, table, lens, 512, nans=True)
    c["k_codes"][int(table[0, 7]), 0, 0, 0] = 0x7F
    check(kv, c, "e4m3", q, table, lens, 512, nans=True)


def test_shared_bad_pages(kv, fp4):
    """A page id that is none: its tokens read as zeros, and the error word says so."""
    lens = [520, 530]
    c, table, q = case(512, lens, 4, 1, 128, 16, "int8", "bf16", 1)
    bad = table.clone()
    bad[:, 3], bad[:, 9] = -1, 1 << 20
    got, _ = run(kv, c, "int8", q, bad, lens, 512)
    assert fp4.get_device_error() == 6
    for j in (3, 9):
        page = int(table[0, j])
        c["k_codes"][page] = 0
        c["v_codes"][page] = 0
    want, _, mass, _ = attention64(q, c, table, lens, "int8", 128 ** -0.5, 0, 0)
    assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9 * mass + 1e-6).all()


def share(cache, *args, **kw):
    return cache.attend_shared(*args, always=True, **kw)


def test_shared_strides_streams_and_graph(kv):
    """q and out inside wider rows; another stream; a captured graph whose prefix, lengths and pages change; two graphs."""
    B, heads, dim, block = 5, 8, 128, 16
    lens = [700] * B
    c, table, q0 = case(512, lens, heads, 2, dim, block, "e4m3", "bf16", 1)
    cache = on_gpu(kv, c, "e4m3")
    wide_q = torch.randn(B, (heads + 4) * dim, device=DEV).to(torch.bfloat16)
    q = wide_q[:, 2 * dim:(heads + 2) * dim].view(B, 1, heads, dim)
    wide = torch.full((B, heads * dim + 64), 9.0, dtype=torch.bfloat16, device=DEV)
    out = wide[:, :heads * dim].view(B, 1, heads, dim)
    tab, n = table.to(DEV), torch.tensor([600, 513, 700, 0, 555], dtype=torch.int32, device=DEV)
    prefix = torch.tensor([512], dtype=torch.int32, device=DEV)
    want = share(cache, q.contiguous(), tab, n, prefix)
    share(cache, q, tab, n, prefix, out=out)
    assert torch.equal(out, want) and (wide[:, heads * dim:] == 9).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            first = share(cache, q, tab, n, prefix)
            outs.append((first, share(cache, first, tab, n, prefix, pdl=False)))
        graphs.append(graph)
    torch.cuda.current_stream().wait_stream(side)
    for new_prefix, lens in ((512, [600, 513, 700, 0, 555]), (200, [600, 300, 201, 700, 0]), (0, [1, 2, 3, 4, 5]),
                             (512, [700] * 5)):
        n.copy_(torch.tensor(lens, dtype=torch.int32))
        prefix.fill_(new_prefix)
        want = share(cache, q, tab, n, prefix)
        want = want, share(cache, want, tab, n, prefix)
        for graph, got in zip(graphs, outs):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_shared_two_streams_at_once(kv):
    lens = [3000, 2100, 4000] * 4
    c, table, q = case(2048, lens, 16, 2, 128, 64, "e4m3", "bf16", 1)
    cache = on_gpu(kv, c, "e4m3")
    tab, n = table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    prefix = torch.tensor([2048], dtype=torch.int32, device=DEV)
    qs = [q, q.flip(0).contiguous()]
    want = [share(cache, x, tab, n, prefix) for x in qs]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(share(cache, qs[i], tab, n, prefix))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.parametrize("dim", [64, 128])
def test_shared_right_behind_what_it_reads(kv, dim):
    """Launches that start early: a beginning written again right before every call, queries that are the last call's
    outputs, nothing waited for in between; against the same calls one by one."""
    B, prefix, block = 6, 512, 16
    lens = [prefix + 3 + 5 * b for b in range(B)]
    c, table, q0 = case(prefix, lens, 8, 2, dim, block, "e4m3", "bf16", 1)
    tab, n, start = table.to(DEV), *(torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, [prefix]))
    g = gen(dim)
    new = [(torch.randn(prefix, 2, dim, generator=g).to(torch.bfloat16).to(DEV),
            torch.randn(prefix, 2, dim, generator=g).to(torch.bfloat16).to(DEV)) for _ in range(3)]
    one = torch.tensor([prefix], dtype=torch.int32, device=DEV)
    results = []
    for wait in (True, False):
        cache, q, outs = on_gpu(kv, c, "e4m3"), q0, []
        torch.cuda.synchronize()
        for i in range(30):
            cache.append(*new[i % 3], tab[:1, :prefix // block].contiguous(), one)
            if wait:
                torch.cuda.synchronize()
            q = share(cache, q, tab, n, start)
            if wait:
                torch.cuda.synchronize()
            outs.append(q)
        torch.cuda.synchronize()
        results.append(outs)
    for a, b in zip(*results):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_shared_by_size(kv):
    """Small batches are attended to one by one, with the same results as that call's; large ones together."""
    c, table, q = case(512, [600, 577], 8, 2, 128, 32, "e4m3", "bf16", 1)
    cache, tab = on_gpu(kv, c, "e4m3"), table.to(DEV)
    n, prefix = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([600, 577], [512]))
    from moe_nvfp4_gemv_gb300 import fp4gemv
    count = fp4gemv.launch_count()
    got = cache.attend_shared(q, tab, n, prefix)
    assert fp4gemv.launch_count() == count + 1 and torch.equal(got, cache.attend(q, tab, n))
    wide = torch.full((2, 400000), -1, dtype=torch.int32, device=DEV)  # (the sizes that the host knows: the table's)
    wide[:, :tab.shape[1]] = tab
    count = fp4gemv.launch_count()
    got = cache.attend_shared(q, wide, n, prefix)
    assert fp4gemv.launch_count() == count + 3 and torch.equal(got, cache.attend_shared(q, tab, n, prefix, always=True))


@pytest.mark.parametrize("dim,prefix,skip,met", [(128, 2048, 0, True), (256, 2048, 0, True), (64, 51200, 1, True),
                                                 (96, 51200, 2, True), (128, 2048, 5, False)])
def test_shared_timeout_then_recovery(kv, fp4, dim, prefix, skip, met):
    """A tile's values that are never said to be there (a host-side hook; nothing is in flight): the call comes back, the
    error word reads a timeout, every row is NaN (each has a part in every CTA's sums); the next calls are right.  (2048
    tokens are a tile for each CTA: the hook's sixth is nobody's.)"""
    lens = [prefix + 5 + 7 * b for b in range(20)]
    c, table, q = case(prefix, lens, 8, 1, dim, 64, "e4m3", "bf16", 1)
    cache, tab = on_gpu(kv, c, "e4m3"), table.to(DEV)
    n, start = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (lens, [prefix]))
    good = share(cache, q, tab, n, start)
    assert fp4.get_device_error() == 0
    try:
        fp4.set_wait_limit_ns(5_000_000)
        fp4.debug_skip_stage(skip)
        lost = share(cache, q, tab, n, start)
        assert fp4.get_device_error() == (5 if met else 0)
    finally:
        fp4.debug_skip_stage(-1)
        fp4.set_wait_limit_ns(0)
    assert lost.isnan().all() if met else torch.equal(lost, good)
    for _ in range(2):
        assert torch.equal(share(cache, q, tab, n, start), good)
    assert fp4.get_device_error() == 0


def test_shared_refusals(kv, fp4):
    cache = kv.KvCache8.allocate(4, 2, 64, 16)
    table = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    prefix = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    for args in ((q[0], table, lens, prefix), (q.float(), table, lens, prefix), (q, table.long(), lens, prefix),
                 (q, table, lens[:1], prefix), (q, table, lens, prefix.long()), (q, table, lens, lens),
                 (q, table, lens, prefix.cpu())):
        with pytest.raises(ValueError):
            cache.attend_shared(*args)
    with pytest.raises(TypeError):
        cache.attend_shared(q, table, lens, 5)
    small = torch.empty(cache.shared_scratch_bytes(2, 1, 4) - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend_shared(q, table, lens, prefix, scratch=small)
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend_shared(q[:, :, :3], table, lens, prefix)  # (heads that kv_heads does not divide)
    with pytest.raises(fp4.Fp4GemvError):
        cache.attend_shared(q.expand(2, 17, 4, 64).contiguous(), table, lens, prefix)
    assert cache.shared_scratch_bytes(2, 17, 4) == 0 and cache.shared_scratch_bytes(0, 1, 4) == 0
    none = cache.attend_shared(q[:0], table[:0], lens[:0], prefix)
    assert none.shape == (0, 1, 4, 64)
