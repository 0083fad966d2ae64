"""The decode path of examples/moe_decode.py: each operator's outputs against
the plain restatements on the inputs that the path gave it, several tokens and
one token per sequence, and captured steps against uncaptured ones."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import decode_ref as ref
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_each_operator_on_the_path(example, fmt):
    B = 3
    model = example.MoeDecoder(B, max_len=40, fmt=fmt, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(2)
    want = [{n: getattr(c, n).cpu().clone() for n in ("k_codes", "v_codes", "k_scale", "v_scale")} for c in model.caches]
    length = 0
    for n in (7, 1, 1, 16, 1):
        tokens = torch.randint(0, model.cfg["vocab"], (B, n), generator=gen, device="cuda")
        trace = []
        logits = model.forward(tokens, trace)
        length += n
        assert torch.isfinite(logits).all()
        for layer, t, w, cache in zip(model.layers, trace, want, model.caches):
            ref.append(w, t["k"].cpu(), t["v"].cpu(), model.block_table.cpu(), [length] * B, [n] * B, 16, fmt)
            for name in w:
                assert torch.equal(getattr(cache, name).cpu(), w[name]), name
            out, _, mass, _ = ref.attention(t["q"], {k: v.cuda() for k, v in w.items()}, model.block_table, [length] * B,
                                            fmt, 1 / math.sqrt(64))
            d = 2.0 ** -10 * mass + length * 2.0 ** -25 * float((w["v_scale"].max() * 448))
            assert (t["att"].double() <= (out + d).to(torch.bfloat16).double()).all()
            assert (t["att"].double() >= (out - d).to(torch.bfloat16).double()).all()
            ids, weights, keys = ref.route(t["router"].double().cpu().numpy(), model.cfg["topk"], "sigmoid",
                                           layer["bias"].cpu().numpy())
            got = t["ids"].cpu().numpy()
            differ = got != ids  # (only between keys that nearly tie)
            gap = np.abs(np.take_along_axis(keys, got, 1) - np.take_along_axis(keys, ids, 1))
            assert (gap[differ] <= 2.0 ** -20).all()
            same = ~differ.any(1)
            assert np.allclose(t["weights"].cpu().numpy()[same], weights[same], rtol=2.0 ** -19, atol=0)


def test_captured_steps_equal_uncaptured(example):
    outs = []
    for graph in (False, True):
        model = example.MoeDecoder(2, max_len=40, seed=9)
        run = example.Generator(model)
        gen = torch.Generator(device="cuda").manual_seed(3)
        prompt = torch.randint(0, model.cfg["vocab"], (2, 5), generator=gen, device="cuda")
        seen = [[t.clone() for t in run.start(prompt, gen)]]
        for _ in range(12):
            seen.append([t.clone() for t in run.step(gen, graph=graph)] + [run.tokens.clone()])
        assert model.seq_lens.tolist() == [17, 17]
        outs.append(seen)
    for a, b in zip(*outs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_log_probabilities_of_the_path(example):
    model = example.MoeDecoder(4, max_len=20, seed=1)
    run = example.Generator(model, top_n=3, temperature=0.8)
    gen = torch.Generator(device="cuda").manual_seed(7)
    prompt = torch.randint(0, model.cfg["vocab"], (4, 3), generator=gen, device="cuda")
    logits = model.forward(prompt)[:, -1]
    model.reset()
    out = run.start(prompt, gen)
    lp, rank, ent, ids, tops = ref.logprobs(logits.double().cpu().numpy(), run.tokens[:, 0].cpu().numpy(), 3, 0.8)
    assert np.array_equal(out.rank.cpu().numpy(), rank) and np.array_equal(out.top_ids.cpu().numpy(), ids)
    big = float(logits.abs().max()) / 0.8
    for got, r in ((out.logprob, lp), (out.top_logprobs, tops)):
        assert np.abs(got.cpu().double().numpy() - r).max() <= 2.0 ** -19 + 2.0 ** -22 * big
    assert np.abs(out.entropy.cpu().double().numpy() - ent).max() <= 2.0 ** -18 * (1 + big)
