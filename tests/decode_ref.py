"""Plain 64-bit restatements of the decode step's operators, for the tests:
the paged 8-bit cache, attention over it, routing, log probabilities.  They
share nothing with the kernels but the definitions in
include/fp4gemv_decode.h."""
import math

import numpy as np
import torch

MIN_SCALE = np.float32(2.0 ** -100)


# ---- the 8-bit cache ----
def page_scale(amax: np.ndarray, fmt: str) -> np.ndarray:
    """fp32 scales of fp32 magnitudes."""
    amax = np.asarray(amax, np.float32)
    if fmt == "int8":
        return np.maximum(amax * np.float32(1 / 127), MIN_SCALE).astype(np.float32)
    e = np.full(amax.shape, -100.0)
    live = amax > 0
    m, x = np.frexp(amax[live].astype(np.float64) / 448.0)  # exact enough: a 24-bit number over 7 * 2^6
    e[live] = np.maximum(np.where(m == 0.5, x - 1, x), -100)
    return np.exp2(e).astype(np.float32)


def encode(x: torch.Tensor, fmt: str) -> torch.Tensor:
    """uint8 codes of fp32 values already divided by their scale (CPU)."""
    if fmt == "int8":
        q = torch.nan_to_num(x, nan=0.0).clamp(-127, 127).round().to(torch.int8)
        return q.view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def decode(codes: torch.Tensor, fmt: str) -> torch.Tensor:
    """fp32 values of uint8 codes."""
    return codes.view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).float()


def append(cache: dict, k, v, table, lens, news, block, fmt):
    """Appends on CPU copies of the cache's tensors, page by page."""
    t0 = 0
    for b, n in enumerate(news):
        start = int(lens[b]) - n
        pos = start
        while pos < start + n:
            page, slot = int(table[b][pos // block]), pos % block
            m = min(block - slot, start + n - pos)
            for part, x in (("k", k), ("v", v)):
                new = x[t0 + pos - start: t0 + pos - start + m].float()  # [m, heads, dim]
                mag = new.abs()
                amax = torch.where(torch.isfinite(mag), mag, 0.0).amax(dim=(0, 2)).numpy()
                want = page_scale(amax, fmt)
                codes, scale = cache[part + "_codes"], cache[part + "_scale"]
                for h in range(new.shape[1]):
                    old = np.float32(scale[page, h]) if slot else np.float32(0)
                    s = max(old, want[h])
                    if slot and s > old:
                        again = decode(codes[page, h, :slot], fmt) * torch.tensor(old) / torch.tensor(s)
                        codes[page, h, :slot] = encode(again, fmt)
                    codes[page, h, slot:slot + m] = encode(new[:, h] / torch.tensor(s), fmt)
                    scale[page, h] = float(s)
            pos += m
        t0 += n


def attention(q, cache, table, lens, fmt, sm_scale, window=0):
    """(out, lse, mass) in float64 on q's device: mass[...] = sum_t p_t |v_t|,
    which bounds what rounding the probabilities does."""
    B, n, H, D = q.shape
    block = cache["k_codes"].shape[2]
    kv = cache["k_codes"].shape[1]
    g = H // kv
    dev = q.device
    out = torch.zeros(B, n, H, D, dtype=torch.float64, device=dev)
    mass = torch.zeros_like(out)
    lse = torch.full((B, n, H), -math.inf, dtype=torch.float64, device=dev)
    peak = 0.0
    for b in range(B):
        length = int(lens[b])
        if length <= 0:
            continue
        pages = torch.as_tensor(table[b][: -(-length // block)].tolist(), device=dev, dtype=torch.long)
        k = (decode(cache["k_codes"][pages], fmt).double() * cache["k_scale"][pages].double()[:, :, None, None])
        v = (decode(cache["v_codes"][pages], fmt).double() * cache["v_scale"][pages].double()[:, :, None, None])
        k = k.permute(1, 0, 2, 3).reshape(kv, -1, D)[:, :length]
        v = v.permute(1, 0, 2, 3).reshape(kv, -1, D)[:, :length]
        for i in range(n):
            end = length - n + i + 1
            begin = max(0, end - window) if window else 0
            if end <= begin:
                continue
            x = torch.einsum("hgd,htd->hgt", q[b, i].double().view(kv, g, D), k[:, begin:end]) * sm_scale
            peak = max(peak, float(x.abs().max()))
            p = torch.softmax(x, -1)
            out[b, i] = torch.einsum("hgt,htd->hgd", p, v[:, begin:end]).reshape(H, D)
            mass[b, i] = torch.einsum("hgt,htd->hgd", p, v[:, begin:end].abs()).reshape(H, D)
            lse[b, i] = torch.logsumexp(x, -1).reshape(H)
    return out, lse, mass, peak


# ---- routing ----
def route_scores(x: np.ndarray, kind: str) -> np.ndarray:
    """float64 scores of float64 logits (NaN as -inf)."""
    x = np.where(np.isnan(x), -np.inf, x)
    with np.errstate(invalid="ignore", over="ignore"):
        if kind == "sigmoid":
            return 1 / (1 + np.exp(-x))
        top = x.max(-1, keepdims=True)
        e = np.where(x == -np.inf, 0.0, np.where(x == top, 1.0, np.exp(x - top)))
        total = e.sum(-1, keepdims=True)
        return np.where(total > 0, e / np.where(total > 0, total, 1), 0.0)


def route(x, topk, kind, bias=None, n_group=1, topk_group=1, group_top=1, renormalize=True, scale=1.0):
    """(ids, weights, keys) with float64 keys; ties to the lower index."""
    x = np.asarray(x, np.float64)
    score = route_scores(x, kind)
    key = score + (0 if bias is None else np.asarray(bias, np.float64))
    if bias is None and (group_top == 1 or n_group == 1):
        key = np.where(np.isnan(x), -np.inf, x)
    allowed = key
    if n_group > 1:
        per = key.reshape(len(x), n_group, -1)
        with np.errstate(invalid="ignore"):
            strength = np.sort(per, -1)[..., ::-1][..., :group_top].sum(-1)
        order = np.argsort(-strength, 1, kind="stable")[:, :topk_group]
        keep = np.zeros_like(strength, bool)
        np.put_along_axis(keep, order, True, 1)
        allowed = np.where(keep[..., None], per, np.nan).reshape(x.shape)  # NaN: not allowed at all
    # excluded experts sort last, behind allowed ones at -inf
    ids = np.argsort(np.where(np.isnan(allowed), np.inf, -allowed), 1, kind="stable")
    if n_group > 1:
        out = []
        for r, row in enumerate(ids):
            ok = row[~np.isnan(allowed[r, row])]
            out.append(ok[:topk])
        ids = np.stack(out)
    else:
        ids = ids[:, :topk]
    w = np.take_along_axis(score, ids, 1)
    if renormalize:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1), 0.0)
    return ids, w * scale, allowed


# ---- log probabilities ----
def logprobs(x, tokens, top_n, temperature):
    """(logprob, rank, entropy, top_ids, top_logprobs) of float64 logits [T, V]
    (numpy); logits at or below -2^100 are masked."""
    x = np.asarray(x, np.float64)
    T, V = x.shape
    masked = x <= -(2.0 ** 100)
    y = np.where(masked, -np.inf, x) / temperature
    lp = np.full((T, V), -np.inf)
    entropy = np.zeros(T)
    for t in range(T):
        if masked[t].all():
            continue
        top = y[t].max()
        e = np.exp(y[t] - top)
        lp[t] = y[t] - top - np.log(e.sum())
        p = np.exp(lp[t])
        entropy[t] = -(p[p > 0] * lp[t][p > 0]).sum()
    rows = np.arange(T)
    rank = 1 + (x > x[rows, tokens][:, None]).sum(1)
    ids = np.argsort(-x, 1, kind="stable")[:, :top_n]
    return lp[rows, tokens], rank, entropy, ids, np.take_along_axis(lp, ids, 1)
