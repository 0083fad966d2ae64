"""A small mixture-of-experts decoder on this library, step by step.

Every product is an NVFP4 or BF16 product of ``fp4gemv``, the residual stream and
its norms lie in ``fp4gemv.add_norm``; the cache is held in 8 bits
(``kvcache.KvCache8``: append, attend), the router's logits go through
``fp4gemv.moe_route`` to the expert pair, and the answer's log probabilities
come from ``fp4gemv.token_logprobs``.  Weights are random (seeded), so the text
means nothing; shapes and order of calls are those of a serving program.

A prompt goes through the same calls, up to 16 tokens of every sequence at a
time (the cache takes several new tokens per sequence); after it every step brings one token
per sequence and is one captured CUDA graph: lengths and tokens live on the
device.

With ``--window`` layers see a sliding window and the first ``--sinks`` tokens; with
``--shared`` all sequences begin with the same prompt of that many tokens, whose
pages they share and attend to together.

    python examples/moe_decode.py [--batch 4] [--steps 32] [--window 0] [--sinks 4] [--shared 0]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_nvfp4_gemv_gb300 import fp4gemv, synth  # noqa: E402
from moe_nvfp4_gemv_gb300.kvcache import KvCache8  # noqa: E402

SMALL = dict(layers=2, hidden=1024, heads=16, kv_heads=4, head_dim=64, experts=32, topk=4, inter=512, vocab=4096)


class MoeDecoder:
    """Random-weight decoder: attention over an 8-bit cache, then routed experts with a shared one."""

    def __init__(self, batch: int, max_len: int, cfg: dict = SMALL, block_size: int = 16, fmt: str = "e4m3",
                 seed: int = 0, device: str = "cuda", window: int = 0, sinks: int = 0):
        self.cfg, self.batch, self.device = cfg, batch, device
        self.window, self.sinks = window, sinks
        H, E, I = cfg["hidden"], cfg["experts"], cfg["inter"]
        qkv = (cfg["heads"] + 2 * cfg["kv_heads"]) * cfg["head_dim"]
        self._seed = seed

        def nvfp4(rows: int, cols: int, count: int = 1):
            """codes, scales (128x4 layout), and the global scale that keeps activations near 1"""
            self._seed += 2
            codes = synth.fp4_bytes(rows * count, cols, seed=self._seed, device=device)
            scales = synth.e4m3_bytes(fp4gemv.scale_bytes(rows, cols) * count, seed=self._seed + 1, device=device)
            gain = torch.tensor([1.0 / (8.0 * cols ** 0.5)], dtype=torch.float32, device=device)
            return codes.view(count, rows, cols // 2) if count > 1 else codes, scales, gain

        g = torch.Generator(device=device).manual_seed(seed)
        self.embedding = torch.randn(cfg["vocab"], H, generator=g, device=device).to(torch.bfloat16)
        self.layers = []
        for _ in range(cfg["layers"]):
            w1, w1_sf, g1 = nvfp4(2 * I, H, E)
            w2, w2_sf, g2 = nvfp4(H, I, E)
            self.layers.append(dict(
                qkv=nvfp4(qkv, H), out=nvfp4(H, cfg["heads"] * cfg["head_dim"]),
                router=(torch.randn(E, H, generator=g, device=device) / H ** 0.5).to(torch.bfloat16),
                bias=torch.randn(E, generator=g, device=device) * 0.02,
                w1=w1, w1_sf=w1_sf, alpha1=g1.expand(E).contiguous(), w2=w2, w2_sf=w2_sf,
                alpha2=g2.expand(E).contiguous(), shared_up=nvfp4(2 * I, H), shared_down=nvfp4(H, I),
                norm1=torch.ones(H, dtype=torch.bfloat16, device=device),
                norm2=torch.ones(H, dtype=torch.bfloat16, device=device)))
        self.head = nvfp4(cfg["vocab"], H)
        # one cache per layer; pages are dealt out in advance, one run of them per sequence
        pages = -(-max_len // block_size)
        self.caches = [KvCache8.allocate(batch * pages, cfg["kv_heads"], cfg["head_dim"], block_size, fmt, device)
                       for _ in self.layers]
        self.block_table = torch.arange(batch * pages, dtype=torch.int32, device=device).view(batch, pages)
        self.own_pages = self.block_table.clone()
        self.seq_lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.norm = torch.ones(H, dtype=torch.bfloat16, device=device)
        self.shared, self.always = None, False  # int32 [1]: tokens that all sequences begin with

    def forward(self, tokens: torch.Tensor, trace: list | None = None) -> torch.Tensor:
        """bf16 logits [batch, n, vocab] of n new tokens per sequence (int64 [batch, n], n at most 16 and batch n at
        most 128); the cache and the lengths grow by n.  ``trace`` receives each layer's intermediates."""
        c = self.cfg
        B, n = tokens.shape
        heads, kv, dim, H, I = c["heads"], c["kv_heads"], c["head_dim"], c["hidden"], c["inter"]
        self.seq_lens += n
        x = self.embedding[tokens.reshape(-1)]
        h, x = fp4gemv.add_norm(x, None, self.layers[0]["norm1"])
        M = B * n
        act = torch.empty(M * c["topk"], I, dtype=torch.bfloat16, device=self.device)
        sact = torch.empty(M, I, dtype=torch.bfloat16, device=self.device)
        after = [layer["norm1"] for layer in self.layers[1:]] + [self.norm]  # the norm behind each layer
        for layer, cache, norm in zip(self.layers, self.caches, after):
            qkv = fp4gemv.nvfp4_gemv(h, *layer["qkv"])
            k = qkv[:, heads * dim:(heads + kv) * dim].unflatten(1, (kv, dim))  # (views of the projection's rows)
            v = qkv[:, (heads + kv) * dim:].unflatten(1, (kv, dim))
            cache.append(k, v, self.block_table, self.seq_lens)
            q = qkv.view(B, n, -1)[..., :heads * dim].unflatten(2, (heads, dim))
            if self.shared is not None:
                att = cache.attend_shared(q, self.block_table, self.seq_lens, self.shared, always=self.always)
            else:
                att = cache.attend(q, self.block_table, self.seq_lens, window=self.window, sinks=self.sinks)
            block = fp4gemv.nvfp4_gemv(att.reshape(M, heads * dim), *layer["out"])
            stream = x
            h, x = fp4gemv.add_norm(stream, block, layer["norm2"])
            logits = fp4gemv.bf16_gemv(h, layer["router"])
            ids, weights = fp4gemv.moe_route(logits, c["topk"], scores="sigmoid", bias=layer["bias"])
            fp4gemv.moe_gate_up(h, ids, layer["w1"], layer["w1_sf"], layer["alpha1"], act, *layer["shared_up"], sact)
            y = torch.empty_like(x)
            fp4gemv.moe_down_combine(act, ids, weights, layer["w2"], layer["w2_sf"], layer["alpha2"], sact,
                                     *layer["shared_down"], y)
            if trace is not None:
                trace.append(dict(q=q, k=k, v=v, att=att, router=logits, ids=ids, weights=weights, stream=stream,
                                  block=block, h=h, x=x))
            h, x = fp4gemv.add_norm(x, y, norm)
        return fp4gemv.nvfp4_gemv(h, *self.head).view(B, n, -1)

    def share(self, tokens: int, always: bool = False) -> None:
        """All sequences begin with the same ``tokens`` tokens, already in the cache: from now on the first sequence's
        whole pages of them are everyone's, and steps attend to them together (``always``: however few they are)."""
        if self.window:
            raise ValueError("no window together with a shared beginning")
        full = tokens // self.caches[0].block_size
        self.block_table[:, :full] = self.block_table[0, :full].clone()
        self.shared = torch.tensor([tokens], dtype=torch.int32, device=self.device)
        self.always = always

    def keys_and_values(self, layer: int, tokens: int) -> tuple[torch.Tensor, torch.Tensor]:
        """bf16 [batch, tokens, kv_heads, head_dim]: what a layer's cache holds of every sequence's last tokens."""
        k, v = self.caches[layer].read(self.block_table, self.seq_lens, self.batch * tokens)
        return k.unflatten(0, (self.batch, tokens)), v.unflatten(0, (self.batch, tokens))

    def reset(self) -> None:
        self.seq_lens.zero_()
        self.block_table.copy_(self.own_pages)
        self.shared = None


class Generator:
    """Sampling on top of a decoder: a prompt pass, then one captured graph per step."""

    def __init__(self, model: MoeDecoder, top_n: int = 5, temperature: float = 0.8):
        self.model, self.top_n, self.temperature = model, top_n, temperature
        B, dev = model.batch, model.device
        self.tokens = torch.zeros(B, 1, dtype=torch.int64, device=dev)
        self.noise = torch.zeros(B, model.cfg["vocab"], device=dev)
        self.graph, self.out = None, None

    def _choose(self, logits: torch.Tensor) -> fp4gemv.TokenLogprobs:
        # a sample by the largest of logits / temperature + Gumbel noise
        chosen = (logits.float() / self.temperature + self.noise).argmax(-1)
        self.tokens.copy_(chosen[:, None])
        return fp4gemv.token_logprobs(logits, chosen.to(torch.int32), self.top_n, self.temperature)

    def _draw(self, generator: torch.Generator) -> None:
        u = torch.rand(self.noise.shape, generator=generator, device=self.noise.device)
        self.noise.copy_(-torch.log(-torch.log(u.clamp(1e-7, 1 - 1e-7))))

    def start(self, prompt: torch.Tensor, generator: torch.Generator) -> fp4gemv.TokenLogprobs:
        self.model.reset()
        self._draw(generator)
        n = max(1, min(16, fp4gemv.MAX_M // self.model.batch))  # (what one pass of the products and the cache takes)
        for part in prompt.split(n, dim=1):
            logits = self.model.forward(part)
        return self._choose(logits[:, -1])

    def step(self, generator: torch.Generator, graph: bool = True) -> fp4gemv.TokenLogprobs:
        """One token per sequence after the last; the same tensors come back from every graph step."""
        self._draw(generator)
        if not graph:
            return self._choose(self.model.forward(self.tokens)[:, 0])
        if self.graph is None:
            # an uncaptured step on the capture's stream first, so that its workspaces are there; then as if it had not been
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                lens, tokens = self.model.seq_lens.clone(), self.tokens.clone()
                self._choose(self.model.forward(self.tokens)[:, 0])
                self.model.seq_lens.copy_(lens)
                self.tokens.copy_(tokens)
                self.graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(self.graph, stream=side):
                    self.out = self._choose(self.model.forward(self.tokens)[:, 0])
            torch.cuda.current_stream().wait_stream(side)
        self.graph.replay()
        return self.out


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=4)
    ap.add_argument("--shared", type=int, default=0)
    args = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = MoeDecoder(args.batch, max_len=12 + args.shared + args.steps + 1, window=args.window, sinks=args.sinks)
    run = Generator(model)
    prompt = torch.randint(0, model.cfg["vocab"], (args.batch, 12), generator=gen, device="cuda")
    if args.shared:
        common = torch.randint(0, model.cfg["vocab"], (1, args.shared), generator=gen, device="cuda")
        prompt = torch.cat([common.expand(args.batch, -1), prompt], 1)
    out = run.start(prompt, gen)
    if args.shared:
        model.share(args.shared)
    run.step(gen)  # (captures)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(args.steps - 1):
        out = run.step(gen)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t0) / max(1, args.steps - 1)
    print(f"{args.batch} sequences, {args.steps} steps of {dt * 1e6:.0f} us; lengths {model.seq_lens.tolist()}")
    for b in range(min(args.batch, 4)):
        top = ", ".join(f"{i} {lp:.2f}" for i, lp in zip(out.top_ids[b].tolist(), out.top_logprobs[b].tolist()))
        print(f"  sequence {b}: token {int(run.tokens[b])}, log probability {float(out.logprob[b]):.2f} (rank "
              f"{int(out.rank[b])}), entropy {float(out.entropy[b]):.2f}; most likely {top}")
    if fp4gemv.get_device_error() != 0:
        raise SystemExit("device error word set")


if __name__ == "__main__":
    main()
