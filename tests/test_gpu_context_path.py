"""The decode path of examples/moe_decode.py with windows and first tokens, with a
beginning that the sequences share, and with its norms: each operator's outputs
against the plain restatements on the inputs that the path gave it, captured
steps against uncaptured ones."""
import importlib.util
import math
import os

import pytest
import torch

import decode_ref as ref
from gpu_util import require_gpu
from test_gpu_norm_read import close, norm64
from test_gpu_sinks import attention64

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("moe_decode", os.path.join(ROOT, "examples", "moe_decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def check_step(model, tokens, window=0, sinks=0):
    """One forward pass: the attention of every layer and the norm behind it; the cache read back."""
    n = tokens.shape[1]
    trace = []
    logits = model.forward(tokens, trace)
    assert torch.isfinite(logits).all()
    lens = model.seq_lens.tolist()
    for i, (layer, t, cache) in enumerate(zip(model.layers, trace, model.caches)):
        c = {name: getattr(cache, name).cpu() for name in ("k_codes", "v_codes", "k_scale", "v_scale")}
        want, _, mass, _ = attention64(t["q"], c, model.block_table.cpu(), lens, cache.fmt, 1 / math.sqrt(64), window, sinks)
        top = float(ref.decode(c["v_codes"], cache.fmt).abs().amax() * c["v_scale"].amax())
        d = 2.0 ** -10 * mass + max(lens) * 2.0 ** -25 * top
        assert (t["att"].double() <= (want + d).to(torch.bfloat16).double()).all()
        assert (t["att"].double() >= (want - d).to(torch.bfloat16).double()).all()
        h, r, delta, f = norm64(t["stream"], t["block"], layer["norm2"], None, None, False, 1.0, 1e-6, 0.0)
        close(t["x"], r, 0 * r, torch.bfloat16)
        close(t["h"], h, h.abs() * 2.0 ** -18, torch.bfloat16)
        k, v = model.keys_and_values(i, n)
        page = model.block_table[:, :].cpu()
        for b, length in enumerate(lens):
            pos = torch.arange(length - n, length)
            at, slot = page[b][pos // cache.block_size].long(), pos % cache.block_size
            for got, part in ((k, "k"), (v, "v")):
                values = ref.decode(c[part + "_codes"][at, :, slot], cache.fmt) * c[part + "_scale"][at][..., None]
                assert torch.equal(got[b].cpu(), values.to(torch.bfloat16))
    return logits


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_window_and_first_tokens(example, fmt):
    model = example.MoeDecoder(3, max_len=90, fmt=fmt, seed=4, window=20, sinks=5)
    gen = torch.Generator(device="cuda").manual_seed(2)
    for n in (9, 16, 1, 16, 1, 14, 1, 1, 16, 1):
        check_step(model, torch.randint(0, model.cfg["vocab"], (3, n), generator=gen, device="cuda"), 20, 5)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_shared_beginning(example, fmt):
    """150 common tokens, then steps of one and of several tokens, attended to together; without sharing the same path's
    outputs lie within what the two orders of sums differ by."""
    B = 5
    gen = torch.Generator(device="cuda").manual_seed(6)
    model = example.MoeDecoder(B, max_len=200, fmt=fmt, seed=3)
    common = torch.randint(0, model.cfg["vocab"], (1, 150), generator=gen, device="cuda").expand(B, -1)
    for part in common.split(16, dim=1):
        model.forward(part)
    model.share(150, always=True)
    assert model.block_table[:, :9].eq(model.block_table[0, :9]).all() and model.block_table[1, 9] != model.block_table[0, 9]
    for n in (1, 3, 1, 16, 1):
        check_step(model, torch.randint(0, model.cfg["vocab"], (B, n), generator=gen, device="cuda"))
    model.reset()
    assert model.shared is None and model.block_table.eq(model.own_pages).all()


@pytest.mark.parametrize("shared", [0, 140])
def test_captured_steps_equal_uncaptured(example, shared):
    outs = []
    for graph in (False, True):
        model = example.MoeDecoder(2, max_len=220, seed=9, window=0 if shared else 30, sinks=4)
        run = example.Generator(model)
        gen = torch.Generator(device="cuda").manual_seed(3)
        prompt = torch.randint(0, model.cfg["vocab"], (1, shared + 40), generator=gen, device="cuda").expand(2, -1)
        seen = [[t.clone() for t in run.start(prompt, gen)]]
        if shared:
            model.share(shared, always=True)
        for _ in range(12):
            seen.append([t.clone() for t in run.step(gen, graph=graph)] + [run.tokens.clone()])
        outs.append(seen)
    for a, b in zip(*outs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_example_runs(example, monkeypatch, capsys):
    for extra in ([], ["--window", "16", "--sinks", "2"], ["--shared", "200"]):
        monkeypatch.setattr("sys.argv", ["moe_decode.py", "--batch", "3", "--steps", "6", *extra])
        example.main()
        assert "3 sequences, 6 steps" in capsys.readouterr().out
