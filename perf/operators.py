"""The decode-step operators around the expert products, as measured cases.

Four operators of a serving step, each in two forms: elementary torch
operations in 32 bits (``own = False``), and the calls of this package
(``own = True``):

* ``append``: new keys and values into a paged cache of 8-bit codes with one
  scale for each page and head (``KvCache8.append``);
* ``attend``: attention of the newest tokens over that cache
  (``KvCache8.attend``);
* ``route``: routing of tokens to experts (``fp4gemv.moe_route``);
* ``logprobs``: log probabilities of given tokens, their rank, the entropy and
  the top alternatives (``fp4gemv.token_logprobs``).

The cache's format.  A page holds ``block_size`` tokens of every KV head:
codes ``[pages, heads, block_size, dim]`` and scales ``[pages, heads]``, keys
and values apart; ``value = code * scale``.  Codes are E4M3 (the scale is the
least power of two for which the page's largest magnitude is at most 448) or
INT8 (the scale is that magnitude / 127); no scale is below 2^-100.  Appending
to a page that already holds tokens never lowers its scale; where the scale
grows, the codes already there are rounded again to the new scale.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
MIN_SCALE = 2.0 ** -100


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one user's chat turn: a short context, latency alone counts
        dict(name="attend_1x777", op="attend", batch=1, len=777, ragged=False, q_len=1, heads=32, kv_heads=8, dim=128,
             block=16, fmt="e4m3", dtype="bf16", window=0),
        # a serving batch of mixed lengths, one slot idle, wide head groups
        dict(name="attend_24x8191_ragged", op="attend", batch=24, len=8191, ragged=True, q_len=1, heads=64, kv_heads=8,
             dim=128, block=64, fmt="e4m3", dtype="bf16", window=0),
        # one very long document: few rows, the work lies along the context
        dict(name="attend_1x131071_int8", op="attend", batch=1, len=131071, ragged=False, q_len=1, heads=32, kv_heads=8,
             dim=128, block=64, fmt="int8", dtype="f16", window=0),
        # verification of four drafted tokens for a full batch: the largest
        dict(name="attend_32x16384_q4", op="attend", batch=32, len=16384, ragged=False, q_len=4, heads=64, kv_heads=8,
             dim=128, block=64, fmt="e4m3", dtype="bf16", window=0),
        # the decode step's own append: one token for each of 64 sequences
        dict(name="append_64x1", op="append", batch=64, new=1, past=50, ragged=False, kv_heads=8, dim=128, block=16,
             fmt="e4m3", dtype="bf16"),
        # prompts of uneven lengths entering the cache in one call
        dict(name="append_5_prompts", op="append", batch=5, new=16001, past=0, ragged=True, kv_heads=8, dim=128,
             block=64, fmt="int8", dtype="bf16"),
        # one token through the routed layer of the package's MoE shape
        dict(name="route_1x128", op="route", tokens=1, experts=128, topk=8, scores="softmax", bias=False, groups=1,
             topk_groups=1, group_top=1, renormalize=True, scale=1.0, dtype="bf16"),
        # a batch with balance bias and expert groups
        dict(name="route_96x256_groups", op="route", tokens=96, experts=256, topk=8, scores="sigmoid", bias=True,
             groups=8, topk_groups=4, group_top=2, renormalize=True, scale=2.5, dtype="f32"),
        # a prompt's tokens over an uneven number of experts
        dict(name="route_20011x60", op="route", tokens=20011, experts=60, topk=4, scores="softmax", bias=True, groups=1,
             topk_groups=1, group_top=1, renormalize=False, scale=1.0, dtype="f32"),
        # the sampled token's log probability with twenty alternatives
        dict(name="logprobs_1x128003", op="logprobs", tokens=1, vocab=128003, top_n=20, dtype="bf16", temperature=1.0),
        # a batch's tokens at a sampling temperature, fp32 logits
        dict(name="logprobs_64x100001", op="logprobs", tokens=64, vocab=100001, top_n=5, dtype="f32", temperature=0.7),
        # scoring of a whole prompt
        dict(name="logprobs_2048x131072", op="logprobs", tokens=2048, vocab=131072, top_n=1, dtype="bf16",
             temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; from 100 on of the form 3k + 1: even and odd ones, few on a tile's edge."""
    n = int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n if n < 100 or n - (n - 1) % 3 < lo else n - (n - 1) % 3


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "route", "logprobs"])
    if op == "attend":
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        dim = rng.choice([64, 96, 128, 256])
        batch = _log_int(rng, 1, 64)
        most = min(131072, (1 << 30) // (batch * kv_heads * dim * 2))  # at most the largest listed cache
        length = _log_int(rng, 1, most)
        q_len = rng.choice([1, 1, 1, 2, 4, 7])
        group = rng.choice([1, 2, 3, 4, 6, 8, 16])
        while q_len * group > 32:  # ... and its rows
            group //= 2
        return dict(op="attend", batch=batch, len=length, ragged=rng.random() < 0.6, q_len=q_len,
                    heads=kv_heads * group, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32, 64, 128]),
                    fmt=rng.choice(["e4m3", "int8"]), dtype=rng.choice(["bf16", "f16"]),
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, length)]))
    if op == "append":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 96, 128, 256])
        if rng.random() < 0.5:
            batch, new, past = _log_int(rng, 1, 256), rng.choice([1, 1, 2, 5]), _log_int(rng, 1, 200)
        else:
            batch = _log_int(rng, 1, 16)
            new, past = _log_int(rng, 8, (1 << 24) // (kv_heads * dim * batch)), rng.choice([0, 0, 37])
        ragged = rng.random() < 0.4
        if ragged:  # tokens in all, of the form that _log_int gives
            new = new * batch - (new * batch - 1) % 3
        return dict(op="append", batch=batch, new=new, past=past, ragged=ragged,
                    kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                    dtype=rng.choice(["bf16", "f16"]))
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.randint(2, 512 // groups)
        topk_groups = 1 if groups == 1 else rng.randint(1, groups)
        topk = rng.randint(1, min(16, topk_groups * (experts // groups)))
        return dict(op="route", tokens=_log_int(rng, 1, 30000 * 64 // max(64, experts)), experts=experts, topk=topk,
                    scores=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=topk_groups, group_top=1 if groups == 1 else rng.choice([1, 2]),
                    renormalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    dtype = rng.choice(["bf16", "f16", "f32"])
    vocab = _log_int(rng, 1000, 262144)
    most = max(1, 2048 * 131072 * 2 // (vocab * (4 if dtype == "f32" else 2)))
    return dict(op="logprobs", tokens=_log_int(rng, 1, min(8192, most)), vocab=vocab, top_n=rng.randint(0, 20),
                dtype=dtype, temperature=rng.choice([1.0, 1.0, 0.6, 1.3]))


def _lens(case):
    """Context lengths of the batch: all ``len``, or an even spread up to it with one idle slot."""
    b, n = case["batch"], case["len"]
    if not case["ragged"]:
        return [n] * b
    lens = [max(1, n * ((37 * i) % b + 1) // b) for i in range(b)] if b % 37 else [max(1, n * (i + 1) // b) for i in range(b)]
    if b >= 8:
        lens[lens.index(min(lens))] = 0
    return lens


def _news(case):
    """New tokens of each sequence: ``new`` for all, or ``new`` in all, shared out unevenly."""
    b, n = case["batch"], case["new"]
    if not case["ragged"]:
        return [n] * b
    parts = [i % 4 + 1 for i in range(b)]
    out = [n * p // sum(parts) for p in parts]
    out[0] += n - sum(out)
    return out


def _pasts(case):
    """Tokens already cached for each sequence."""
    return [case["past"] and (case["past"] + 7 * i) % (2 * case["past"]) for i in range(case["batch"])]


def _seen(case, length):
    """Cached tokens that the queries of one sequence read between them."""
    first = max(0, length - case["q_len"])
    return length if not case["window"] else length - max(0, first - case["window"] + 1)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _pow2(e):
    """2^e in 32 bits, exactly, for whole e of normal numbers."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantise(x, fmt):
    """Codes (bytes) and scales of whole pages x [..., tokens, dim] with a scale for each leading index."""
    amax = x.abs().amax(dim=(-1, -2))
    if fmt == "int8":
        scale = (amax / 127.0).clamp(min=MIN_SCALE)
        return (x / scale[..., None, None]).round().to(torch.int8).view(torch.uint8), scale
    m, e = torch.frexp(amax)
    scale = _pow2((e - 9 + (m > 0.875)).clamp(min=-100))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _filled_cache(pages, heads, block, dim, fmt, gen):
    """Codes and scales of pages full of normal values, page by page of differing size."""
    codes = torch.empty(pages, heads, block, dim, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, heads, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (heads * block * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        size = 0.5 + torch.rand(n, heads, 1, 1, generator=gen, device=DEV)
        x = torch.randn(n, heads, block, dim, generator=gen, device=DEV) * size
        codes[p:p + n], scales[p:p + n] = _quantise(x, fmt)
    return codes, scales


def _pages_for(lens, block, gen):
    """A block table over shuffled pages (-1 past each sequence's end) and the number of pages."""
    need = [-(-n // block) for n in lens]
    total = max(1, sum(need))
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def _package_cache(state):
    """The package's cache object over the state's tensors."""
    if state.get("cache") is None:
        from moe_nvfp4_gemv_gb300.kvcache import KvCache8
        state["cache"] = KvCache8(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"],
                                  fmt=state["case"]["fmt"])
    return state["cache"]


def prepare(case, seed):
    gen = _gen(seed)
    op = case["op"]
    dt = DTYPES[case["dtype"]]
    s = {"op": op, "case": case}
    if op == "attend":
        lens = _lens(case)
        block, kv, dim = case["block"], case["kv_heads"], case["dim"]
        s["table"], pages = _pages_for(lens, block, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["k_codes"], s["k_scale"] = _filled_cache(pages, kv, block, dim, case["fmt"], gen)
        s["v_codes"], s["v_scale"] = _filled_cache(pages, kv, block, dim, case["fmt"], gen)
        for b, n in enumerate(lens):  # what lies past a sequence's end is of no sequence: NaN codes, where there are such
            if n % block:
                page = int(s["table"][b, n // block])
                s["k_codes"][page, :, n % block:] = 0x7F
                s["v_codes"][page, :, n % block:] = 0x7F
        shape = (case["batch"], case["q_len"], case["heads"], dim)
        s["q"] = (torch.randn(shape, generator=gen, device=DEV) * 1.5).to(dt)
        s["out"] = torch.empty(shape, dtype=dt, device=DEV)
        s["lse"] = torch.empty(shape[:3], dtype=torch.float32, device=DEV)
    elif op == "append":
        news, pasts = _news(case), _pasts(case)
        block, kv, dim = case["block"], case["kv_heads"], case["dim"]
        lens = [p + n for p, n in zip(pasts, news)]
        s["table"], pages = _pages_for(lens, block, gen)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        cu = np.concatenate([[0], np.cumsum(news)])
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
        s["pos"] = torch.tensor(np.concatenate([np.arange(p, p + n) for p, n in zip(pasts, news)]), device=DEV)
        s["seq"] = torch.tensor(np.repeat(np.arange(len(news)), news), device=DEV)
        for part in ("k", "v"):
            s[part + "_codes"], s[part + "_scale"] = _filled_cache(pages, kv, block, dim, case["fmt"], gen)
            size = 0.3 + 2 * torch.rand(int(cu[-1]), kv, 1, generator=gen, device=DEV)
            s[part] = (torch.randn(int(cu[-1]), kv, dim, generator=gen, device=DEV) * size).to(dt)
    elif op == "route":
        s["logits"] = torch.randn(case["tokens"], case["experts"], generator=gen, device=DEV).to(dt)
        s["bias"] = torch.randn(case["experts"], generator=gen, device=DEV) * 0.05 if case["bias"] else None
        s["ids"] = torch.empty(case["tokens"], case["topk"], dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty(case["tokens"], case["topk"], dtype=torch.float32, device=DEV)
    else:
        t, v, n = case["tokens"], case["vocab"], case["top_n"]
        s["logits"] = torch.empty(t, v, dtype=dt, device=DEV)
        step = max(1, (1 << 26) // v)
        for i in range(0, t, step):
            s["logits"][i:i + step] = torch.randn(min(step, t - i), v, generator=gen, device=DEV) * 2.5
        s["logits"][:, ::17] -= 8.0
        s["tokens"] = torch.randint(0, v, (t,), generator=gen, device=DEV, dtype=torch.int32)
        s["logits"].scatter_add_(1, s["tokens"][:, None].long(),  # given tokens are mostly likely ones
                                 (torch.rand(t, 1, generator=gen, device=DEV) * 14).to(dt))
        s["out"] = (torch.empty(t, dtype=torch.float32, device=DEV), torch.empty(t, dtype=torch.int32, device=DEV),
                    torch.empty(t, dtype=torch.float32, device=DEV), torch.empty(t, n, dtype=torch.int32, device=DEV),
                    torch.empty(t, n, dtype=torch.float32, device=DEV))
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"attend": _attend, "append": _append, "route": _route, "logprobs": _logprobs}[state["op"]](state)


def _run_own(s):
    from moe_nvfp4_gemv_gb300 import fp4gemv
    c = s["case"]
    if s["op"] == "attend":
        _package_cache(s).attend(s["q"], s["table"], s["lens"], window=c["window"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if s["op"] == "append":
        _package_cache(s).append(s["k"], s["v"], s["table"], s["lens"], cu_new=s["cu"] if c["ragged"] else None)
        return _cache_out(s)
    if s["op"] == "route":
        fp4gemv.moe_route(s["logits"], c["topk"], scores=c["scores"], bias=s["bias"], n_group=c["groups"],
                          topk_group=c["topk_groups"], group_top=c["group_top"], renormalize=c["renormalize"],
                          scale=c["scale"], ids=s["ids"], weights=s["weights"])
        return s["ids"], s["weights"]
    return tuple(fp4gemv.token_logprobs(s["logits"], s["tokens"], top_n=c["top_n"], temperature=c["temperature"],
                                        out=s["out"]))


def _as_codes(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def _cache_out(s):
    fmt = s["case"]["fmt"]
    return _as_codes(s["k_codes"], fmt), s["k_scale"], _as_codes(s["v_codes"], fmt), s["v_scale"]


def _attend(s):
    """softmax(q k / sqrt(dim)) v over the tokens that each query may see; no such token: zeros, and lse -inf."""
    c, q = s["case"], s["q"].float()
    b, n, h, d = q.shape
    kv, block = c["kv_heads"], c["block"]
    table = s["table"].clamp(min=0).long()
    span = table.shape[1] * block
    pos = torch.arange(span, device=DEV)
    at = s["lens"][:, None] - n + torch.arange(n, device=DEV)  # the queries' positions
    seen = (pos <= at[..., None]) & (pos < s["lens"][:, None, None])
    if c["window"]:
        seen = seen & (pos > at[..., None] - c["window"])
    held = (pos < s["lens"][:, None]).view(b, 1, span, 1)

    def values(codes, scale):
        x = _as_codes(codes, c["fmt"])[table].float() * scale[table][..., None, None]  # [b, pages, kv, block, d]
        return torch.where(held, x.transpose(1, 2).reshape(b, kv, span, d), 0.0)

    q = q.view(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, d)
    x = torch.matmul(q, values(s["k_codes"], s["k_scale"]).transpose(2, 3)) * (1.0 / math.sqrt(d))
    mask = seen[:, None, None].expand(b, 1, h // kv, n, span).reshape(b, 1, -1, span)
    x = torch.where(mask, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values(s["v_codes"], s["v_scale"])) / torch.where(total == 0, 1.0, total)
    lse = torch.log(total) + top

    def back(y):
        return y.view(b, kv, h // kv, n, -1).permute(0, 3, 1, 2, 4).reshape(b, n, h, -1)

    return back(out).to(s["q"].dtype), back(lse).squeeze(-1)


def _append(s):
    """Rescales the pages that new tokens join, then writes the tokens' codes; see the format above."""
    c = s["case"]
    block, fmt = c["block"], c["fmt"]
    page = s["table"][s["seq"], s["pos"] // block].long()
    slot = s["pos"] % block
    pages = s["k_scale"].shape[0]
    first = torch.full((pages,), block, device=DEV).index_reduce_(0, page, slot, "amin")  # first new slot of a page
    old = torch.arange(block, device=DEV) < first[:, None]
    for part in ("k", "v"):
        codes, scale, x = s[part + "_codes"], s[part + "_scale"], s[part].float()
        amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(-1), "amax")
        if fmt == "int8":
            want = (amax / 127.0).clamp(min=MIN_SCALE)
        else:
            m, e = torch.frexp(amax)
            want = _pow2((e - 9 + (m > 0.875)).clamp(min=-100))
        kept = torch.where((first > 0)[:, None], scale, 0.0)
        new = torch.where((first < block)[:, None], torch.maximum(kept, want), scale)
        grown = ((new > scale) & (first < block)[:, None])[..., None, None] & old[:, None, :, None]
        again = _as_codes(codes, fmt).float() * scale[..., None, None] / new[..., None, None]
        fresh = x / new[page][..., None]
        if fmt == "int8":
            again, fresh = again.round().to(torch.int8), fresh.round().to(torch.int8)
        else:
            again, fresh = again.to(torch.float8_e4m3fn), fresh.to(torch.float8_e4m3fn)
        codes.copy_(torch.where(grown, again.view(torch.uint8), codes))
        codes[page, :, slot] = fresh.view(torch.uint8)
        scale.copy_(new)
    return _cache_out(s)


def _route(s):
    """Scores, the groups with the best scores, the experts with the best scores in them, and their weights.

    Experts are ordered by score + bias; with no bias, and where a group counts by its best expert, by the logits
    (the scores are monotone in them).  Ties go to the lower index.  The softmax's sum is taken in 64 bits, so that
    its rounding to 32 is the same in any order."""
    c, x = s["case"], s["logits"].float()
    t, n = x.shape
    if c["scores"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True, dtype=torch.float64).float()
    key = score + s["bias"] if c["bias"] else score if c["group_top"] > 1 else x
    if c["groups"] > 1:
        per = key.view(t, c["groups"], -1)
        best = per.sort(dim=-1, descending=True).values[..., :c["group_top"]].sum(-1)
        chosen = best.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, chosen, True)
        key = torch.where(allowed[..., None], per, -math.inf).view(t, n)
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk"]]
    w = score.gather(1, ids)
    if c["renormalize"]:
        total = w.sum(-1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    return ids.to(torch.int32), w * c["scale"]


def _logprobs(s):
    """Log probabilities of the given tokens, their ranks, entropies, and the top tokens (ties: the lower id)."""
    c, raw = s["case"], s["logits"].float()
    t, v = raw.shape
    x = raw * (1.0 / c["temperature"])
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    at = s["tokens"][:, None].long()
    lse = torch.log(total)
    entropy = lse.squeeze(1) - torch.where(e > 0, e * x, 0.0).sum(-1) / total.squeeze(1)
    rank = 1 + (raw > raw.gather(1, at)).sum(-1)
    bits = (raw + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() * v + torch.arange(v - 1, -1, -1, device=DEV)
    ids = order.topk(c["top_n"], dim=-1).indices
    return ((x.gather(1, at) - lse).squeeze(1), rank.to(torch.int32), entropy, ids.to(torch.int32),
            x.gather(1, ids) - lse)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]]
    if op == "attend":
        seen = sum(_seen(case, n) for n in _lens(case))
        rows = case["batch"] * case["q_len"] * case["heads"]
        pages = -(-seen // case["block"])
        cache = 2 * case["kv_heads"] * (seen * case["dim"] + pages * 4)
        pairs = 0  # (query, token) pairs
        for n in _lens(case):
            for i in range(case["q_len"]):
                p = max(0, n - case["q_len"] + 1 + i)
                pairs += min(p, case["window"]) if case["window"] else p
        return {"bytes": cache + rows * (2 * case["dim"] * size + 4) + 4 * (pages + case["batch"]),
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if op == "append":
        tokens = sum(_news(case))
        values = 2 * tokens * case["kv_heads"] * case["dim"]
        pages = sum(-(-(p + n) // case["block"]) - p // case["block"] for p, n in zip(_pasts(case), _news(case)) if n)
        return {"bytes": values * (size + 1) + pages * (2 * 8 * case["kv_heads"] + 4), "flops": 4 * values}
    if op == "route":
        cells = case["tokens"] * case["experts"]
        return {"bytes": cells * size + 8 * case["tokens"] * case["topk"] + (4 * case["experts"] if case["bias"] else 0),
                "flops": 4 * cells}
    cells = case["tokens"] * case["vocab"]
    return {"bytes": cells * size + case["tokens"] * (16 + 8 * case["top_n"]), "flops": 6 * cells}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "append": _exact_append, "route": _exact_route,
            "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_attend(s):
    c = s["case"]
    b, n, h, d = s["q"].shape
    kv, block = c["kv_heads"], c["block"]
    g = h // kv
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, n, h), -math.inf, dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :-(-length // block)].long()
        if not length:
            continue
        for j in range(kv):
            k = _as_codes(s["k_codes"][pages, j], c["fmt"]).double() * s["k_scale"][pages, j].double()[:, None, None]
            v = _as_codes(s["v_codes"][pages, j], c["fmt"]).double() * s["v_scale"][pages, j].double()[:, None, None]
            k, v = k.reshape(-1, d)[:length], v.reshape(-1, d)[:length]
            for r in range(n):
                end = length - n + r + 1
                begin = max(0, end - c["window"]) if c["window"] else 0
                if end <= begin:
                    continue
                x = s["q"][i, r, j * g:(j + 1) * g].double() @ k[begin:end].T / math.sqrt(d)
                lse[i, r, j * g:(j + 1) * g] = torch.logsumexp(x, -1)
                out[i, r, j * g:(j + 1) * g] = torch.softmax(x, -1) @ v[begin:end]
    return out, lse


def _pow2_64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(x):
    """The nearest E4M3 value of |x| <= 448 (ties to the even code)."""
    _, e = torch.frexp(x)
    step = _pow2_64((e - 4).clamp(min=-9))  # three mantissa bits; the least exponent is -6
    return torch.round(x / step) * step


def _exact_append(s):
    c = s["case"]
    block, limit = c["block"], 127.0 if c["fmt"] == "int8" else 448.0
    result = []
    pos, seq = s["pos"].cpu().numpy(), s["seq"].cpu().numpy()
    page = s["table"].cpu().numpy()[seq, pos // block]
    starts = np.flatnonzero(np.diff(np.concatenate([[-1], page]))) if len(page) else []
    for part in ("k", "v"):
        codes = _as_codes(s[part + "_codes"], c["fmt"]).double()
        scale = s[part + "_scale"].double()
        x = s[part].double()
        for i, t0 in enumerate(starts):
            t1 = starts[i + 1] if i + 1 < len(starts) else len(page)
            p, first = int(page[t0]), int(pos[t0]) % block
            want = x[t0:t1].abs().amax((0, 2)) / limit
            if c["fmt"] == "e4m3":
                m, e = torch.frexp(want)
                want = _pow2_64(e - (m == 0.5).int())
            want = want.clamp(min=MIN_SCALE)
            new = torch.maximum(want, scale[p]) if first else want
            ratio = (scale[p] / new)[:, None, None]
            codes[p, :, :first] = torch.where(ratio < 1, codes[p, :, :first] * ratio, codes[p, :, :first])
            codes[p, :, first:first + t1 - t0] = (x[t0:t1] / new[None, :, None]).transpose(0, 1)
            scale[p] = new
        result += [_round_e4m3(codes) if c["fmt"] == "e4m3" else None, scale]
    return result


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    if c["scores"] == "sigmoid":
        score = 1 / (1 + np.exp(-x))
    else:
        score = np.exp(x - x.max(1, keepdims=True))
        score /= score.sum(1, keepdims=True)
    order = score + (s["bias"].double().cpu().numpy() if c["bias"] else 0.0)
    if not c["bias"] and c["group_top"] == 1:
        order = x
    if c["groups"] > 1:
        split = order.reshape(len(x), c["groups"], -1)
        strength = np.sort(split, -1)[..., ::-1][..., :c["group_top"]].sum(-1)
        ranking = np.argsort(-strength, 1, kind="stable")
        out = np.ones_like(strength, dtype=bool)
        np.put_along_axis(out, ranking[:, :c["topk_groups"]], False, 1)
        order = np.where(out[..., None], -np.inf, split).reshape(x.shape)
    ids = np.argsort(-order, 1, kind="stable")[:, :c["topk"]]
    w = np.take_along_axis(score, ids, 1)
    if c["renormalize"]:
        w = w / w.sum(1, keepdims=True)
    return None, w * c["scale"]


def _exact_logprobs(s):
    c, n = s["case"], s["case"]["top_n"]
    lp, ent, tops = [], [], []
    rows = max(1, (1 << 26) // c["vocab"])
    for i in range(0, c["tokens"], rows):
        y = torch.log_softmax(s["logits"][i:i + rows].double() / c["temperature"], -1)
        lp.append(y.gather(1, s["tokens"][i:i + rows, None].long())[:, 0])
        ent.append(-torch.special.xlogy(y.exp(), y.exp()).sum(-1))
        tops.append(y.topk(n, -1).values)
    return torch.cat(lp), None, torch.cat(ent), None, torch.cat(tops)
