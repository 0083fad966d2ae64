"""Token log probabilities over the whole range of temperatures and logits, against 64 bits.

What is rounded, for up to 131072 logits on one CTA: a thread's sums of at most 256 terms each in binary32 (2^-16
relative at worst) and the joins after it (2^-20); every term's exponent (x - m) / T, whose difference, product and
factor round to 2^-24 each, so a term is off by 2^-21 of its exponent, and the exponents' mean is at most the entropy
(ln 131072 < 12); the exponential (2^-22) and the logarithm (2^-21).  Together below 2^-15 in log Z.  Nothing of that
grows with the logits' size or with 1 / T: the largest logit's own term is exactly 1.  So

    |logprob - exact| <= 2^-15 + 2^-21 |exact|,  logprob <= 0,
    |entropy - exact| <= 2^-14 (1 + exact),      entropy >= 0

(the entropy is log Z and the exponents' mean, with the same relative errors)."""
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


def check(fp4, rows, tokens, top_n, temperature, times):
    """The rows (CPU, [k, V]), all of them `times` times over: a cluster per row or, with many, a CTA."""
    got = fp4.token_logprobs(rows.to(DEV).repeat(times, 1), tokens.to(DEV).repeat(times), top_n, temperature)
    assert fp4.get_device_error() == 0
    k = len(rows)
    lp, rank, ent, ids, tops = ref.logprobs(rows.double().numpy(), tokens.numpy(), top_n, temperature)

    def of(t):  # (rows of an odd length begin at other alignments, so their sums differ in the last bits)
        return t.cpu().view(times, k, *t.shape[1:]).numpy()

    assert (of(got.rank) == rank).all()
    assert (of(got.top_ids) == ids).all()
    for g, r in ((of(got.logprob), lp), (of(got.top_logprobs), tops)):
        with np.errstate(over="ignore"):
            r = np.broadcast_to(r.astype(np.float32), g.shape)
        assert np.array_equal(np.isinf(g), np.isinf(r)) and (g <= 0).all()
        live = np.isfinite(r)
        g, r = g[live].astype(np.float64), r[live].astype(np.float64)
        assert (np.abs(g - r) <= 2.0 ** -15 + 2.0 ** -21 * np.abs(r)).all(), np.abs(g - r).max()
    e = of(got.entropy).astype(np.float64)
    assert (e >= 0).all() and (np.abs(e - ent) <= 2.0 ** -14 * (1 + ent)).all(), np.abs(e - ent).max()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [10.0, 1.0, 0.1, 0.01, 1e-3, 1e-5, 1e-6])
@pytest.mark.parametrize("times", [1, 130])
def test_logprobs_at_every_temperature(fp4, dtype, temperature, times):
    """Logits around 20, -500 and (fp32) 10000: log Z must not lose bits with |max| / T."""
    V = 20011
    x = torch.randn(3, V, generator=gen(7)) * 3
    x += torch.tensor([[20.0], [-500.0], [1e4 if dtype == "f32" else 60.0]])
    x = x.to(TYPES[dtype])
    tokens = torch.stack([x[0].argmax(), torch.tensor(77), torch.tensor(V - 1)]).to(torch.int32)
    check(fp4, x, tokens, 5, temperature, times)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [1.0, 1e-3, 1e-5, 1e-6])
@pytest.mark.parametrize("V,times", [(128003, 1), (20011, 100)])
def test_masked_rows_at_low_temperatures(fp4, dtype, temperature, V, times):
    """A few live logits among thousands of masked ones: a thread, a warp or a CTA that has summed masked ones only meets
    a live one later, or never."""
    low = -math.inf if dtype == "f16" else torch.finfo(TYPES[dtype]).min
    g = gen(V)
    few = torch.full((V,), -math.inf)
    few[[5, V // 2, V - 3]] = torch.tensor([1.0, 2.0, 1.5])
    last = torch.full((V,), low)
    last[V - 1] = -30.0
    half = torch.randn(V, generator=g) * 3
    half[torch.rand(V, generator=g) < 0.5] = low
    tail = torch.randn(V, generator=g)
    tail[: V - 700] = -math.inf
    rows = torch.stack([few, last, half, tail]).to(TYPES[dtype])
    check(fp4, rows, torch.tensor([5, V - 1, 17, V - 8], dtype=torch.int32), 3, temperature, times)


@pytest.mark.parametrize("temperature", [1.0, 1e-6])
@pytest.mark.parametrize("times", [1, 200])
def test_logprobs_of_the_largest_numbers(fp4, temperature, times):
    """Differences that overflow once they are divided by T: probability 0, and nothing is NaN."""
    V = 20011
    x = torch.randn(2, V, generator=gen(8))
    x[0, [9, 15000]] = torch.tensor([3.0e38, 3.0e38])
    x[0, [70, 800]] = torch.tensor([1.0e38, -3.0e38])
    x[1, 5] = 3.0e32
    check(fp4, x, torch.tensor([15000, 6], dtype=torch.int32), 4, temperature, times)


@pytest.mark.parametrize("temperature", [1e4, 1e12, 1e20])
def test_masked_rows_at_high_temperatures(fp4, temperature):
    """Up to the highest temperature masked logits (of bf16 and fp32; f16's lowest value is a logit) have no weight."""
    x = torch.randn(2, 5003, generator=gen(9))
    x[0, 100:3000] = -math.inf
    x[1, ::2] = torch.finfo(torch.float32).min
    check(fp4, x, torch.tensor([0, 4], dtype=torch.int32), 2, temperature, 1)
    with pytest.raises(fp4.Fp4GemvError):
        fp4.token_logprobs(x.to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV), temperature=2e20)
