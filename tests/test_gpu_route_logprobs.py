"""Routing and token log probabilities on the GPU against 64 bits.

Routing, fixed before the first run: scores are exact to a few fp32 roundings
(exp, a sum carried in 48 bits, one division: 2^-20 relative covers it), so
weights may be 2^-19 |w| off, and ids may differ from the 64-bit order only
between experts whose keys are within 2^-21 (1 + |key|); the inputs below with
exact ties and logits as keys must match exactly.

Log probabilities: x inv_temperature rounds once (2^-24 relative to the largest
|x / T|), the sums' relative error is below 2^-19 for these sizes (fp32 running
sums of at most a few hundred terms per thread, then a tree): log
probabilities may be 2^-19 + 2^-22 max|x / T| off.  The entropy weighs such
differences: log Z's error and, for u = sum e d, the same relative error times
the mean |d|: 2^-18 (1 + max|x / T|)."""
import math

import numpy as np
import pytest
import torch

import decode_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def fp4():
    require_gpu()
    from moe_nvfp4_gemv_gb300 import fp4gemv
    return fp4gemv


def gen(seed):
    return torch.Generator().manual_seed(seed)


def check_route(fp4, x, topk, kind, bias=None, exact=False, **kw):
    """x on the CPU."""
    ids, w = fp4.moe_route(x.to(DEV), topk, scores=kind, bias=None if bias is None else bias.to(DEV), **kw)
    assert fp4.get_device_error() == 0
    ids, w = ids.cpu().numpy(), w.cpu().double().numpy()
    xn = x.double().numpy()
    rid, rw, keys = ref.route(xn, topk, kind, None if bias is None else bias.numpy(), **kw)
    assert ((ids >= 0) & (ids < x.shape[1])).all()
    assert all(len(set(r)) == topk for r in ids.tolist()), "an expert twice"
    if exact:
        assert np.array_equal(ids, rid)
    else:
        differ = ids != rid
        got, want = np.take_along_axis(keys, ids, 1), np.take_along_axis(keys, rid, 1)
        assert not np.isnan(got[differ]).any(), "an expert of a group that takes no part"
        assert (np.abs(got - want)[differ] <= 2.0 ** -21 * (1 + np.abs(want[differ]))).all()
        assert differ.mean() < 0.01
        same = ~differ.any(1)
        w, rw = w[same], rw[same]
    assert (np.abs(w - rw) <= 2.0 ** -19 * np.abs(rw) + 1e-37).all()


@pytest.mark.parametrize("E", [1, 2, 7, 31, 32, 33, 60, 64, 65, 127, 128, 160, 255, 256, 257, 384, 511, 512])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_route_sizes(fp4, E, dtype):
    for i, (M, topk, kind, renorm) in enumerate([(1, min(8, E), "softmax", True), (7, 1, "sigmoid", False),
                                                 (130, min(32, E), "softmax", False)]):
        x = (torch.randn(M, E, generator=gen(E + i)) * 2).to(TYPES[dtype])
        check_route(fp4, x, topk, kind, exact=True, renormalize=renorm, scale=1.7)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,topk", [
    (256, 8, 4, 2, 8), (256, 8, 4, 1, 8), (60, 4, 2, 2, 6), (512, 32, 3, 2, 32), (64, 32, 32, 2, 20), (96, 3, 1, 1, 32),
    (130, 13, 5, 2, 11), (32, 32, 8, 1, 8)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(fp4, kind, E, n_group, topk_group, group_top, topk, with_bias):
    g = gen(E + n_group)
    x = torch.randn(333, E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    check_route(fp4, x, topk, kind, bias, n_group=n_group, topk_group=topk_group, group_top=group_top,
                exact=not with_bias and group_top == 1)


def test_route_bias_large_batch(fp4):
    g = gen(9)
    x = torch.randn(5000, 128, generator=g)
    bias = torch.randn(128, generator=g) * 0.01
    check_route(fp4, x, 8, "softmax", bias, renormalize=False)
    check_route(fp4, x, 8, "sigmoid", bias, scale=2.5)
    check_route(fp4, x[:, :100], 8, "sigmoid", bias[:100])  # a strided view of the rows


def many_tokens():
    """So many that up to 64 experts are routed on 8 lanes per token; not a whole number of CTAs."""
    return 64 * torch.cuda.get_device_properties(0).multi_processor_count + 5


@pytest.mark.parametrize("E,topk,kind,renorm,dtype", [
    (1, 1, "softmax", True, "bf16"), (7, 7, "sigmoid", True, "f16"), (8, 3, "softmax", False, "f32"),
    (33, 32, "softmax", False, "bf16"), (60, 4, "softmax", True, "f32"), (64, 8, "sigmoid", False, "bf16"),
    (64, 32, "softmax", True, "f16")])
def test_route_many_tokens(fp4, E, topk, kind, renorm, dtype):
    x = (torch.randn(many_tokens(), E, generator=gen(E)) * 2).to(TYPES[dtype])
    x[3::7, E // 2] = -math.inf
    x[5::11, 0] = math.nan
    check_route(fp4, x, topk, kind, exact=True, renormalize=renorm, scale=0.6)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,topk", [(60, 4, 2, 2, 6), (64, 32, 31, 2, 20), (64, 8, 3, 1, 8),
                                                                 (30, 10, 4, 2, 9), (32, 4, 1, 2, 8), (64, 4, 2, 2, 8),
                                                                 (64, 2, 1, 1, 12)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_many_tokens_groups(fp4, kind, E, n_group, topk_group, group_top, topk, with_bias):
    g = gen(E * n_group)
    x = torch.randn(many_tokens(), E, generator=g)
    bias = torch.randn(E, generator=g) * 0.1 if with_bias else None
    check_route(fp4, x, topk, kind, bias, n_group=n_group, topk_group=topk_group, group_top=group_top,
                exact=not with_bias and group_top == 1)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_route_ties_and_special_values(fp4, kind):
    E = 96
    rows = [torch.zeros(E), torch.full((E,), -math.inf), torch.full((E,), math.nan), torch.full((E,), -3.0e38)]
    r = torch.zeros(E)
    r[::2] = -0.0
    rows.append(r)
    r = torch.full((E,), -math.inf)
    r[40], r[7] = 2.0, 1.0
    rows.append(r)
    r = torch.randn(E, generator=gen(1))
    r[3::5] = math.nan
    r[50] = -math.inf
    rows.append(r)
    r = torch.full((E,), 80.0)
    r[33] = 90.0
    rows.append(r)
    x = torch.stack(rows)
    check_route(fp4, x, 8, kind, exact=True)
    check_route(fp4, x, 8, kind, exact=True, renormalize=False)
    check_route(fp4, x[:6], 8, kind, exact=True, n_group=4, topk_group=2)
    if kind == "softmax":  # all the weight on infinite logits
        r = torch.zeros(1, E)
        r[0, 90] = r[0, 12] = math.inf
        ids, w = fp4.moe_route(r.to(DEV), 3)
        assert ids.tolist() == [[12, 90, 0]] and w.tolist() == [[0.5, 0.5, 0.0]]


def test_route_outputs_and_streams(fp4):
    x = torch.randn(65, 128, generator=gen(4)).to(DEV)
    ids, w = fp4.moe_route(x, 8)
    i2, w2 = torch.empty_like(ids), torch.empty_like(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, b = fp4.moe_route(x, 8, ids=i2, weights=w2, pdl=False)
    s.synchronize()
    assert a is i2 and b is w2 and torch.equal(ids, i2) and torch.equal(w, w2)
    wide = torch.randn(65, 300, generator=gen(5)).to(DEV)
    wide[:, 100:228] = x
    i3, w3 = fp4.moe_route(wide[:, 100:228], 8)
    assert torch.equal(ids, i3) and torch.equal(w, w3)
    e, f = fp4.moe_route(x[:0], 8)
    assert e.shape == (0, 8) and f.shape == (0, 8)


def test_route_refusals(fp4):
    x = torch.zeros(2, 64, device=DEV)
    for kw in (dict(topk=0), dict(topk=33), dict(topk=8, n_group=5), dict(topk=8, n_group=8, topk_group=9),
               dict(topk=17, n_group=8, topk_group=2), dict(topk=4, n_group=64, topk_group=8, group_top=2),
               dict(topk=4, group_top=3), dict(topk=4, scale=math.inf)):
        with pytest.raises(fp4.Fp4GemvError):
            fp4.moe_route(x, **kw)
    with pytest.raises(fp4.Fp4GemvError):
        fp4.moe_route(torch.zeros(2, 513, device=DEV), 4)
    for bad in (x.double(), x[0], x.t(), x.cpu()):
        with pytest.raises(ValueError):
            fp4.moe_route(bad, 4)
    with pytest.raises(ValueError):
        fp4.moe_route(x, 4, scores="tanh")
    with pytest.raises(ValueError):
        fp4.moe_route(x, 4, bias=torch.zeros(63, device=DEV))
    with pytest.raises(ValueError):
        fp4.moe_route(x, 4, ids=torch.zeros(2, 4, dtype=torch.int64, device=DEV))


# ---- log probabilities ----
def check_logprobs(fp4, x, tokens, top_n, temperature=1.0):
    """x on the CPU, any row stride."""
    base = torch.full((x.shape[0], x.shape[1] + 3), 1e4 if x.dtype == torch.float16 else 1e30, dtype=x.dtype)
    outs = []
    for off in (0, 1):  # rows from an even and from an odd element on
        wide = base.clone()
        wide[:, off:off + x.shape[1]] = x
        got = fp4.token_logprobs(wide.to(DEV)[:, off:off + x.shape[1]], tokens.to(DEV), top_n, temperature)
        outs.append([t.cpu() for t in got])
    assert fp4.get_device_error() == 0
    xn = x.double().numpy()
    lp, rank, ent, ids, tops = ref.logprobs(xn, tokens.numpy(), top_n, temperature)
    big = np.where(xn > -1e30, np.abs(xn), 0).max() / temperature
    for got in outs:
        assert np.array_equal(got[1].numpy(), rank)
        assert np.array_equal(got[3].numpy(), ids)
        for g, r in ((got[0], lp), (got[4], tops)):
            g = g.double().numpy()
            assert np.array_equal(np.isinf(g), np.isinf(r))
            live = np.isfinite(r)
            assert (np.abs(g - r)[live] <= 2.0 ** -19 + 2.0 ** -22 * big).all(), np.abs(g - r)[live].max()
        assert (np.abs(got[2].double().numpy() - ent) <= 2.0 ** -18 * (1 + big)).all()


@pytest.mark.parametrize("V", [1, 2, 5, 31, 100, 1000, 8191, 8193, 32768, 50001, 128003])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_logprobs_sizes(fp4, V, dtype):
    for T, n, temp in ((1, min(20, V), 1.0), (3, min(32, V), 0.6), (9, 0, 1.4)):
        g = gen(V + T)
        x = (torch.randn(T, V, generator=g) * 3).to(TYPES[dtype])
        tokens = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
        tokens[0] = V - 1
        check_logprobs(fp4, x, tokens, n, temp)


@pytest.mark.parametrize("T", [18, 19, 75, 76, 151, 153, 700])
def test_logprobs_batches(fp4, T):
    g = gen(T)
    x = (torch.randn(T, 20011, generator=g) * 2).to(torch.bfloat16)
    check_logprobs(fp4, x, torch.randint(0, 20011, (T,), generator=g, dtype=torch.int32), 7)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [2, 400])
def test_logprobs_masks_and_ties(fp4, dtype, T):
    """Masked tails, equal rows, rising and falling rows, few live tokens: more candidates than the buffer holds."""
    V, g = 30011, gen(3)
    low = torch.finfo(TYPES[dtype]).min
    kinds = [torch.zeros(V), torch.full((V,), -math.inf), torch.full((V,), low),
             torch.arange(V).float() / V * 8, -torch.arange(V).float() / V * 8]
    r = torch.full((V,), -math.inf)
    r[[5, 29000, 777]] = torch.tensor([1.0, 2.0, 1.0])
    kinds.append(r)
    if dtype != "f16":  # (f16's lowest value is an ordinary logit)
        r = torch.full((V,), low)
        r[[5, 29000, 777]] = torch.tensor([1.0, 2.0, 1.0])
        r[100:200] = -math.inf
        kinds.append(r)
    r = torch.randn(V, generator=g)
    r[torch.rand(V, generator=g) < 0.7] = -math.inf
    kinds.append(r)
    r = torch.randn(V, generator=g)
    r[::2] = 3.0
    kinds.append(r)
    r = torch.zeros(V)
    r[torch.arange(V) // 8 % 64 < 20] = 5.0
    kinds.append(r)
    for i in range(0, len(kinds)):
        x = kinds[i].expand(T, V).to(TYPES[dtype]) if T == 2 else kinds[i].repeat(T, 1).to(TYPES[dtype])
        x = x[:, :5003] if T > 2 else x
        tokens = torch.randint(0, x.shape[1], (T,), generator=g, dtype=torch.int32)
        tokens[0] = 777
        check_logprobs(fp4, x, tokens, 20)


def test_logprobs_engineered_candidates(fp4):
    """One group's maximum lies far below the others', with half the row between."""
    V = 65536
    x = torch.zeros(1, V)
    i = torch.arange(V)
    group = i // 4 % 64
    x[0] = torch.where(group < 31, 5 + i / V, torch.where(group == 31, 4.0 + 0 * i, 0.0 * i))
    check_logprobs(fp4, x.float(), torch.tensor([7], dtype=torch.int32), 32)


def test_logprobs_non_finite(fp4):
    x = torch.randn(3, 4000, generator=gen(1))
    x[0, 5], x[1, 6] = math.nan, math.inf
    got = fp4.token_logprobs(x.to(DEV), torch.tensor([1, 1, 1], dtype=torch.int32, device=DEV), 4)
    assert torch.isnan(got.logprob[:2]).all() and torch.isnan(got.entropy[:2]).all()
    assert torch.isfinite(got.logprob[2]) and int(got.top_ids[1, 0]) == 6
    assert 5 not in got.top_ids[0].tolist()


def test_logprobs_bad_tokens(fp4):
    x = torch.randn(3, 500, generator=gen(1)).to(DEV)
    out = fp4.TokenLogprobs(torch.full((3,), 9.0, device=DEV), torch.full((3,), 9, dtype=torch.int32, device=DEV),
                            torch.empty(3, device=DEV), torch.empty(3, 2, dtype=torch.int32, device=DEV),
                            torch.empty(3, 2, device=DEV))
    got = fp4.token_logprobs(x, torch.tensor([-1, 3, 500], dtype=torch.int32, device=DEV), 2, out=out)
    assert fp4.get_device_error() == 6
    assert got.logprob[[0, 2]].tolist() == [9, 9] and got.rank[[0, 2]].tolist() == [9, 9]
    want = torch.log_softmax(x[1].double(), 0)[3]
    assert abs(float(got.logprob[1]) - float(want)) < 1e-5
    assert torch.equal(got.top_ids.long(), x.topk(2).indices)


def test_logprobs_refusals(fp4):
    x = torch.zeros(2, 64, device=DEV)
    t = torch.zeros(2, dtype=torch.int32, device=DEV)
    for kw in (dict(top_n=33), dict(top_n=65), dict(temperature=1e-7)):
        with pytest.raises(fp4.Fp4GemvError):
            fp4.token_logprobs(x, t, **kw)
    for a, b in ((x.double(), t), (x, t.long()), (x, t[:1]), (x.t(), t), (x, t.cpu())):
        with pytest.raises(ValueError):
            fp4.token_logprobs(a, b)
    with pytest.raises(ValueError):
        fp4.token_logprobs(x, t, temperature=0.0)
    assert fp4.token_logprobs(x[:0], t[:0], 3).top_ids.shape == (0, 3)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n_group,topk_group,group_top,topk", [
    (72, 8, 7, 2, 14), (240, 8, 4, 1, 6), (510, 17, 5, 2, 8), (102, 17, 6, 2, 9), (33, 11, 3, 2, 7), (448, 28, 9, 2, 20),
    (300, 2, 1, 1, 32), (62, 31, 20, 1, 16), (291, 3, 2, 2, 7)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_route_uneven_groups(fp4, kind, E, n_group, topk_group, group_top, topk, dtype):
    """Groups that fill their lanes in part, and (17 of 30) groups across lanes."""
    g = gen(E + topk)
    x = torch.randn(200, E, generator=g).to(TYPES[dtype])
    x[::9, 1] = -math.inf
    check_route(fp4, x, topk, kind, n_group=n_group, topk_group=topk_group, group_top=group_top, renormalize=False,
                exact=group_top == 1)
    bias = torch.randn(E, generator=g) * 0.1
    check_route(fp4, x, topk, kind, bias, n_group=n_group, topk_group=topk_group, group_top=group_top)
