"""Operators of a decode step over long and shared contexts, as measured cases.

Four operators of a serving step, each in two forms: elementary torch
operations in 32 bits (``own = False``), and the calls of this package
(``own = True``):

* ``shared``: attention of a batch whose sequences begin with the same tokens,
  that beginning computed once for all (``KvCache8.attend_shared``);
* ``sinks``: attention with a sliding window and a few first tokens that stay
  visible (``KvCache8.attend`` with ``window`` and ``sinks``);
* ``read``: the last tokens of sequences out of the cache again
  (``KvCache8.read``);
* ``norm``: a block's output into the residual stream, with the norm behind the
  block, a gate and a scale, and the next block's norm (``fp4gemv.add_norm``).

The cache's format.  A page holds ``block`` tokens of every KV head: codes
``[pages, heads, block, dim]`` and scales ``[pages, heads]``, keys and values
apart; ``value = code * scale``.  Codes are E4M3 or INT8.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # a system prompt shared by four short chats: latency counts
        dict(name="shared_4x1000", op="shared", batch=4, prefix=1000, own=77, ragged=False, q_len=1, heads=32,
             kv_heads=8, dim=128, block=16, fmt="e4m3", dtype="bf16"),
        # a full batch of chats on a long common document, own parts of mixed lengths, one slot idle
        dict(name="shared_64x32768", op="shared", batch=64, prefix=32768, own=701, ragged=True, q_len=1, heads=64,
             kv_heads=8, dim=128, block=64, fmt="e4m3", dtype="bf16"),
        # verification of four drafted tokens of samples of one prompt, INT8, small heads
        dict(name="shared_24x8191_q4", op="shared", batch=24, prefix=8191, own=210, ragged=True, q_len=4, heads=32,
             kv_heads=8, dim=64, block=32, fmt="int8", dtype="f16"),
        # a few samples of a very long prompt with large heads: few rows, bound by the cache
        dict(name="shared_7x65536_d256", op="shared", batch=7, prefix=65536, own=50, ragged=False, q_len=1, heads=16,
             kv_heads=4, dim=256, block=128, fmt="e4m3", dtype="bf16"),
        # one chat turn on a windowed layer
        dict(name="sinks_1x5000", op="sinks", batch=1, len=5000, ragged=False, q_len=1, heads=32, kv_heads=8, dim=128,
             block=16, fmt="e4m3", dtype="bf16", window=1024, sinks=4),
        # a serving batch of long streams, the window long past the first tokens
        dict(name="sinks_32x32768", op="sinks", batch=32, len=32768, ragged=False, q_len=1, heads=64, kv_heads=8,
             dim=128, block=64, fmt="e4m3", dtype="bf16", window=4096, sinks=4),
        # drafted tokens, lengths around the window, a wide set of first tokens
        dict(name="sinks_48x3001_q4_int8", op="sinks", batch=48, len=3001, ragged=True, q_len=4, heads=32, kv_heads=8,
             dim=96, block=32, fmt="int8", dtype="f16", window=777, sinks=130),
        # one sequence's last tokens: the smallest
        dict(name="read_1x33", op="read", batch=1, new=33, past=100, ragged=False, kv_heads=8, dim=128, block=16,
             fmt="e4m3", dtype="bf16"),
        # prompts of uneven lengths for an attention over wide types
        dict(name="read_5_prompts_int8", op="read", batch=5, new=40001, past=37, ragged=True, kv_heads=8, dim=128,
             block=64, fmt="int8", dtype="bf16"),
        # one token between two blocks
        dict(name="norm_1x4096", op="norm", tokens=1, width=4096, dtype="bf16", residual="bf16", weights="bf16",
             post=False, gate="none", sigmoid=False, scale=1.0, offset=0.0),
        # a batch with norms on both sides of the block, a gate for each channel, the stream kept in fp32
        dict(name="norm_37x6144_both", op="norm", tokens=37, width=6144, dtype="bf16", residual="f32", weights="f32",
             post=True, gate="channel", sigmoid=False, scale=0.5, offset=1.0),
        # a prompt's tokens, gates of their own
        dict(name="norm_20011x4096_gated", op="norm", tokens=20011, width=4096, dtype="bf16", residual="bf16",
             weights="bf16", post=True, gate="token", sigmoid=True, scale=1.0, offset=0.0),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm; from 100 on of the form 3k + 1: even and odd ones, few on a tile's edge."""
    n = int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))
    return n if n < 100 or n - (n - 1) % 3 < lo else n - (n - 1) % 3


def draw(rng):
    op = rng.choice(["shared", "shared", "sinks", "read", "norm"])
    if op in ("shared", "sinks"):
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        dim = rng.choice([64, 96, 128, 256])
        q_len = rng.choice([1, 1, 1, 2, 4, 7])
        group = rng.choice([1, 2, 3, 4, 6, 8, 16])
        common = dict(q_len=q_len, kv_heads=kv_heads, dim=dim, block=rng.choice([16, 32, 64, 128]),
                      fmt=rng.choice(["e4m3", "int8"]), dtype=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.5)
    if op == "shared":
        batch = _log_int(rng, 2, 64)
        rows = batch * q_len * group
        # at most the largest listed one's products, and a cache of 2^28 values
        most = min(65536, (1 << 34) // (rows * kv_heads * dim), (1 << 28) // (kv_heads * dim))
        return dict(op=op, batch=batch, prefix=_log_int(rng, 16, max(17, most)), own=q_len + _log_int(rng, 1, 800),
                    heads=kv_heads * group, **common)
    if op == "sinks":
        while q_len * group > 32:
            group //= 2
        batch = _log_int(rng, 1, 64)
        most = min(65536, (1 << 30) // (batch * kv_heads * dim * 2))
        length = _log_int(rng, 1, most)
        window = _log_int(rng, 1, length)
        # at most the tokens of the largest listed one
        window = min(window, max(1, (1 << 28) // (batch * kv_heads * dim * 2)))
        return dict(op=op, batch=batch, len=length, window=window, sinks=rng.choice([1, 4, 4, 16, 100]),
                    heads=kv_heads * group, **common)
    if op == "read":
        kv_heads, dim = rng.choice([1, 2, 4, 8, 16]), rng.choice([64, 96, 128, 256])
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(2, (1 << 24) // (kv_heads * dim * batch)))
        ragged = rng.random() < 0.5
        if ragged:  # tokens in all
            new = new * batch - (new * batch - 1) % 3
        return dict(op=op, batch=batch, new=new, past=rng.choice([0, 0, 37, 500]), ragged=ragged, kv_heads=kv_heads,
                    dim=dim, block=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                    dtype=rng.choice(["bf16", "f16", "f32"]))
    width = 8 * rng.randint(8, 80) * rng.choice([1, 2, 8, 16]) if rng.random() < 0.75 else _log_int(rng, 16, 10000)
    dtype = rng.choice(["bf16", "bf16", "f16"])
    return dict(op=op, tokens=_log_int(rng, 1, max(2, 14000 * 4096 // width)), width=width, dtype=dtype,
                residual=rng.choice([dtype, dtype, "f32"]), weights=rng.choice([dtype, "f32"]),
                post=rng.random() < 0.5, gate=rng.choice(["none", "none", "channel", "token", "scalar"]),
                sigmoid=rng.random() < 0.5, scale=rng.choice([1.0, 1.0, 0.22]), offset=rng.choice([0.0, 0.0, 1.0]))


def _spread(b, n):
    """An even spread of b lengths up to n, in mixed order; an idle one in a batch of eight or more."""
    lens = [max(1, n * ((37 * i) % b + 1) // b) for i in range(b)] if b % 37 else [max(1, n * (i + 1) // b) for i in range(b)]
    if b >= 8:
        lens[lens.index(min(lens))] = 0
    return lens


def _lens(case):
    """Context lengths of the batch."""
    b = case["batch"]
    if case["op"] == "sinks":
        return _spread(b, case["len"]) if case["ragged"] else [case["len"]] * b
    if not case["ragged"]:
        return [case["prefix"] + case["own"]] * b
    return [case["prefix"] + max(case["q_len"], n) if n else 0 for n in _spread(b, case["own"])]


def _news(case):
    """Tokens of each sequence to read: ``new`` for all, or ``new`` in all, shared out unevenly."""
    b, n = case["batch"], case["new"]
    if not case["ragged"]:
        return [n] * b
    parts = [i % 4 + 1 for i in range(b)]
    out = [n * p // sum(parts) for p in parts]
    out[0] += n - sum(out)
    return out


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _filled_cache(pages, heads, block, dim, fmt, gen):
    """Codes and scales of pages full of normal values, page by page of differing size."""
    codes = torch.empty(pages, heads, block, dim, dtype=torch.uint8, device=DEV)
    scales = torch.empty(pages, heads, dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (heads * block * dim))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, heads, block, dim, generator=gen, device=DEV)
        x *= 0.5 + torch.rand(n, heads, 1, 1, generator=gen, device=DEV)
        amax = x.abs().amax(dim=(-1, -2))
        if fmt == "int8":
            scale = amax / 127.0
            codes[p:p + n] = (x / scale[..., None, None]).round().to(torch.int8).view(torch.uint8)
        else:
            scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
            codes[p:p + n] = (x / scale[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + n] = scale
    return codes, scales


def _pages_for(lens, block, gen, shared=0):
    """A block table over shuffled pages (-1 past each sequence's end) and the number of pages; the first ``shared``
    pages are the same for all sequences."""
    need = [-(-n // block) for n in lens]
    total = max(1, shared + sum(max(0, n - shared) for n in need))
    order = torch.randperm(total, generator=gen, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32, device=DEV)
    at = shared
    for b, n in enumerate(need):
        if n:
            table[b, :shared] = order[:shared]
            table[b, shared:n] = order[at:at + n - shared]
            at += max(0, n - shared)
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
    if op == "norm":
        t, n, wt = case["tokens"], case["width"], DTYPES[case["weights"]]
        near = 0.0 if case["offset"] else 1.0
        s["x"] = (torch.randn(t, n, generator=gen, device=DEV) * 3).to(DTYPES[case["residual"]])
        s["y"] = (torch.randn(t, n, generator=gen, device=DEV) * 0.8).to(dt)
        s["weight"] = (near + 0.2 * torch.randn(n, generator=gen, device=DEV)).to(wt)
        s["post"] = (near + 0.2 * torch.randn(n, generator=gen, device=DEV)).to(wt) if case["post"] else None
        shape = {"none": None, "channel": (n,), "token": (t, n), "scalar": (t, 1)}[case["gate"]]
        s["gate"] = torch.randn(shape, generator=gen, device=DEV).to(dt) if shape else None
        s["residual"], s["out"] = torch.empty_like(s["x"]), torch.empty_like(s["y"])
        return s
    block, kv, dim = case["block"], case["kv_heads"], case["dim"]
    if op == "read":
        news = _news(case)
        lens = [case["past"] + n for n in news]
        starts = [sum(news[:i]) for i in range(len(news) + 1)]
        s["cu"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["k"], s["v"] = (torch.empty(starts[-1], kv, dim, dtype=dt, device=DEV) for _ in range(2))
        s["table"], pages = _pages_for(lens, block, gen)
    else:
        lens = _lens(case)
        # (a page that the common beginning fills in part is each sequence's own, with the same beginning)
        s["table"], pages = _pages_for(lens, block, gen, case["prefix"] // block if op == "shared" else 0)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["k_codes"], s["k_scale"] = _filled_cache(pages, kv, block, dim, case["fmt"], gen)
    s["v_codes"], s["v_scale"] = _filled_cache(pages, kv, block, dim, case["fmt"], gen)
    if op == "read":
        return s
    if op == "shared":
        s["prefix"] = torch.tensor([case["prefix"]], dtype=torch.int32, device=DEV)
        full, rest = divmod(case["prefix"], block)
        if rest:
            copies = torch.tensor([p for p, n in zip(s["table"][:, full].tolist(), lens) if n], device=DEV)
            for part in ("k", "v"):
                s[part + "_scale"][copies] = s[part + "_scale"][copies[0]].clone()
                s[part + "_codes"][copies, :, :rest] = s[part + "_codes"][copies[0], :, :rest].clone()
    for b, n in enumerate(lens):  # what lies past a sequence's end is of no sequence: NaN codes, where there are such
        if n % block:
            page = int(s["table"][b, n // block])
            s["k_codes"][page, :, n % block:] = 0x7F
            s["v_codes"][page, :, n % block:] = 0x7F
    shape = (case["batch"], case["q_len"], case["heads"], dim)
    s["q"] = (torch.randn(shape, generator=gen, device=DEV) * 1.5).to(dt)
    s["out"] = torch.empty(shape, dtype=dt, device=DEV)
    s["lse"] = torch.empty(shape[:3], dtype=torch.float32, device=DEV)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        return _run_own(state)
    return {"shared": _shared, "sinks": _sinks, "read": _read, "norm": _norm}[state["op"]](state)


def _run_own(s):
    c = s["case"]
    if s["op"] == "norm":
        from moe_nvfp4_gemv_gb300 import fp4gemv
        return fp4gemv.add_norm(s["x"], s["y"], s["weight"], post_weight=s["post"], gate=s["gate"],
                                gate_sigmoid=c["sigmoid"], scale=c["scale"], eps=EPS, weight_offset=c["offset"],
                                out=s["out"], residual=s["residual"])
    cache = _package_cache(s)
    if s["op"] == "read":
        return cache.read(s["table"], s["lens"], cu=s["cu"], k=s["k"], v=s["v"])
    if s["op"] == "shared":
        cache.attend_shared(s["q"], s["table"], s["lens"], s["prefix"], out=s["out"], lse=s["lse"])
    else:
        cache.attend(s["q"], s["table"], s["lens"], window=c["window"], sinks=c["sinks"], out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _as_codes(codes, fmt):
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def _values(s, part, pages):
    """fp32 values [..., kv, tokens, dim] of the pages [..., n]."""
    x = _as_codes(s[part + "_codes"], s["case"]["fmt"])[pages].float() * s[part + "_scale"][pages][..., None, None]
    return x.transpose(-4, -3).flatten(-3, -2)


def _softmax_parts(x):
    """exp(x - max) and the max of the last dimension, 0 where nothing is seen."""
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    return torch.exp(x - top), top


def _rows(s):
    """Queries as [b, kv, group * q_len, dim] in fp32, and the way back."""
    q = s["q"].float()
    b, n, h, d = q.shape
    kv = s["case"]["kv_heads"]

    def back(y):
        return y.view(b, kv, h // kv, n, -1).permute(0, 3, 1, 2, 4).reshape(b, n, h, -1)

    return q.view(b, n, kv, h // kv, d).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, d), back


def _shared(s):
    """Scores of all rows on the common pages at once, of each sequence's on its own ones, and one softmax over both."""
    c = s["case"]
    q, back = _rows(s)
    b, kv, rows, d = q.shape
    n, block, group = c["q_len"], c["block"], c["heads"] // c["kv_heads"]
    full = c["prefix"] // block
    table = s["table"].clamp(min=0).long()
    first = (s["lens"] > 0).long().argmax()  # (a sequence that is not idle)
    scale = 1.0 / math.sqrt(d)
    q = q * scale
    flat = q.transpose(0, 1).reshape(kv, b * rows, d)
    k0, v0 = (_values(s, part, table[first, :full]) for part in ("k", "v"))
    x0 = torch.matmul(flat, k0.transpose(1, 2)).view(kv, b, rows, -1).transpose(0, 1)
    pos = full * block + torch.arange((table.shape[1] - full) * block, device=DEV)
    at = s["lens"][:, None] - n + torch.arange(n, device=DEV)
    seen = pos <= at[..., None]
    held = (pos < s["lens"][:, None])[:, None, :, None]
    k1, v1 = (torch.where(held, _values(s, part, table[:, full:]), 0.0) for part in ("k", "v"))
    x1 = torch.matmul(q, k1.transpose(2, 3))
    mask = seen[:, None, None].expand(b, 1, group, n, -1).reshape(b, 1, rows, -1)
    x1 = torch.where(mask, x1, -math.inf)
    x0 = torch.where((s["lens"] > 0)[:, None, None, None], x0, -math.inf)
    p, top = _softmax_parts(torch.cat([x0, x1], -1))
    split = x0.shape[-1]
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p[..., :split].transpose(0, 1).reshape(kv, b * rows, split), v0)
    out = out.view(kv, b, rows, d).transpose(0, 1) + torch.matmul(p[..., split:], v1)
    out = out / torch.where(total == 0, 1.0, total)
    return back(out).to(s["q"].dtype), back(torch.log(total) + top).squeeze(-1)


def _sinks(s):
    """softmax(q k / sqrt(dim)) v over the tokens of the window and the first ones."""
    c = s["case"]
    q, back = _rows(s)
    b, kv, rows, d = q.shape
    n, block, group = c["q_len"], c["block"], c["heads"] // c["kv_heads"]
    table = s["table"].clamp(min=0).long()
    # pages of the first tokens, and of each sequence's window: all that is gathered
    most = table.shape[1]
    lead = min(most, -(-c["sinks"] // block))
    width = min(most, (c["window"] + n - 2) // block + 2)
    start = ((s["lens"] - n - c["window"] + 1).clamp(min=0) // block).clamp(max=most - width)
    page = torch.cat([torch.arange(lead, device=DEV).expand(b, lead),
                      start[:, None] + torch.arange(width, device=DEV)], 1)
    pos = (page[..., None] * block + torch.arange(block, device=DEV)).flatten(1)[:, None]
    again = (torch.arange(page.shape[1], device=DEV) >= lead) & (page < lead)  # (pages of both kinds count once)
    pages = table.gather(1, page)
    at = (s["lens"][:, None] - n + torch.arange(n, device=DEV))[..., None]
    seen = (pos <= at) & ((pos > at - c["window"]) | (pos < c["sinks"])) & ~again.repeat_interleave(block, 1)[:, None]
    held = (pos < s["lens"][:, None, None]).unsqueeze(-1)
    k, v = (torch.where(held, _values(s, part, pages), 0.0) for part in ("k", "v"))
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    mask = seen[:, None, None].expand(b, 1, group, n, -1).reshape(b, 1, rows, -1)
    p, top = _softmax_parts(torch.where(mask, x, -math.inf))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return back(out).to(s["q"].dtype), back(torch.log(total) + top).squeeze(-1)


def _read(s):
    """The codes of each token times its page's scale."""
    c = s["case"]
    row = torch.arange(s["k"].shape[0], device=DEV)
    seq = torch.searchsorted(s["cu"], row, right=True) - 1
    pos = s["lens"][seq] - s["cu"][seq + 1] + row
    page = s["table"][seq, pos // c["block"]].long()
    slot = pos % c["block"]
    return tuple((_as_codes(s[p + "_codes"], c["fmt"])[page, :, slot].float() *
                  s[p + "_scale"][page][..., None]).to(s[p].dtype) for p in ("k", "v"))


def _norm(s):
    """The block's output, normalised, gated and scaled, into the stream; the stream normalised."""
    c = s["case"]
    u = s["y"].float()
    if c["post"]:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + EPS) * (s["post"].float() + c["offset"])
    if s["gate"] is not None:
        g = s["gate"].float()
        u = u * (1.0 / (1.0 + torch.exp(-g)) if c["sigmoid"] else g)
    r = s["x"].float() + c["scale"] * u
    h = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + EPS) * (s["weight"].float() + c["offset"])
    return h.to(s["y"].dtype), r.to(s["x"].dtype)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def _seen_tokens(case, length):
    """Cached tokens that the queries of one sequence read between them."""
    first = max(0, length - case["q_len"])  # the first query's position
    low = max(0, first - case["window"] + 1)
    return length - low + min(low, case["sinks"])


def work(case):
    op = case["op"]
    size = SIZES[case["dtype"]]
    if op == "norm":
        cells, width = case["tokens"] * case["width"], case["width"]
        gate = {"none": 0, "channel": width, "token": cells, "scalar": case["tokens"]}[case["gate"]]
        return {"bytes": cells * (2 * SIZES[case["residual"]] + 2 * size) + gate * size +
                width * SIZES[case["weights"]] * (2 if case["post"] else 1),
                "flops": cells * (12 if case["post"] else 8)}
    if op == "read":
        tokens = sum(_news(case))
        values = 2 * tokens * case["kv_heads"] * case["dim"]
        pages = sum(-(-(case["past"] + n) // case["block"]) - case["past"] // case["block"] for n in _news(case) if n)
        return {"bytes": values * (1 + size) + pages * (8 * case["kv_heads"] + 4), "flops": values}
    lens = _lens(case)
    n = case["q_len"]
    pairs = 0  # (query, token) pairs
    for length in lens:
        for i in range(n if length else 0):
            p = length - n + 1 + i  # tokens up to the query's own
            if op == "sinks":
                low = max(0, p - case["window"])
                p = max(0, p - low + min(low, case["sinks"]))
            pairs += max(0, p)
    if op == "shared":
        seen = case["prefix"] + sum(length - case["prefix"] for length in lens if length)
    else:
        seen = sum(_seen_tokens(case, length) for length in lens if length)
    rows = case["batch"] * n * case["heads"]
    pages = -(-seen // case["block"])
    cache = 2 * case["kv_heads"] * (seen * case["dim"] + pages * 4)
    return {"bytes": cache + rows * (2 * case["dim"] * size + 4) + 4 * (pages + case["batch"]),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"shared": _exact_attention, "sinks": _exact_attention, "read": _exact_read, "norm": _exact_norm}[case["op"]](s)


def _exact_attention(s):
    """Every sequence by itself, over the pages of its own row of the table."""
    c = s["case"]
    b, n, h, d = s["q"].shape
    kv, block = c["kv_heads"], c["block"]
    g = h // kv
    out = torch.zeros(b, n, h, d, dtype=torch.float64, device=DEV)
    lse = torch.full((b, n, h), -math.inf, dtype=torch.float64, device=DEV)
    for i, length in enumerate(s["lens"].tolist()):
        if not length:
            continue
        token = torch.arange(length, device=DEV)
        if c["op"] == "sinks":
            low = max(0, length - n - c["window"] + 1)
            token = token[(token >= low) | (token < c["sinks"])]
        page, slot = s["table"][i].long()[token // block], token % block
        k, v = (_as_codes(s[p + "_codes"], c["fmt"])[page, :, slot].double() * s[p + "_scale"][page].double()[..., None]
                for p in ("k", "v"))  # [tokens, kv, d]
        at = length - n + torch.arange(n, device=DEV)[:, None]
        hidden = token > at
        if c["op"] == "sinks":
            hidden |= (token <= at - c["window"]) & (token >= c["sinks"])
        for j in range(kv):
            x = torch.einsum("ngd,td->gnt", s["q"][i, :, j * g:(j + 1) * g].double(), k[:, j]) / math.sqrt(d)
            x.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(x, -1, keepdim=True)
            w = torch.exp(x - torch.where(z == -math.inf, 0.0, z))
            out[i, :, j * g:(j + 1) * g] = torch.matmul(w, v[:, j]).transpose(0, 1)
            lse[i, :, j * g:(j + 1) * g] = z[..., 0].T
    return out, lse


def _exact_read(s):
    c = s["case"]
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    result = []
    for part in ("k", "v"):
        rows = []
        for b, length in enumerate(lens):
            pages = s["table"][b, :-(-length // c["block"])].long()
            x = _as_codes(s[part + "_codes"], c["fmt"])[pages].double() * s[part + "_scale"][pages].double()[..., None, None]
            rows.append(x.transpose(1, 2).reshape(-1, c["kv_heads"], c["dim"])[length - (cu[b + 1] - cu[b]):length])
        result.append(torch.cat(rows))
    return tuple(result)


def _exact_norm(s):
    c = s["case"]
    outs = []
    step = max(1, (1 << 25) // c["width"])
    for i in range(0, c["tokens"], step):
        r = s["y"][i:i + step].double()
        if c["post"]:
            r = r / torch.sqrt(torch.sum(r ** 2, -1, keepdim=True) / c["width"] + EPS) * (c["offset"] + s["post"].double())
        if c["gate"] != "none":
            g = (s["gate"] if c["gate"] == "channel" else s["gate"][i:i + step]).double()
            r = r * (torch.sigmoid(g) if c["sigmoid"] else g)
        r = r * c["scale"] + s["x"][i:i + step].double()
        h = r / torch.sqrt(torch.sum(r ** 2, -1, keepdim=True) / c["width"] + EPS) * (c["offset"] + s["weight"].double())
        outs.append((h, r))
    return torch.cat([h for h, _ in outs]), torch.cat([r for _, r in outs])
