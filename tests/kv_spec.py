"""The paged KV cache operators from their definitions, in float64 / integers on the CPU: one request, one head after another."""
import math

import torch


def plan(ctx, new, pt, table, free, head, max_tokens):
    """(table, next head, cu, kv_len, positions, slots) as lists; table is a list of rows and is not changed."""
    table = [list(r) for r in table]
    cu, positions, slots = [0], [], []
    for r, (c, n) in enumerate(zip(ctx, new)):
        for b in range(-(-c // pt), -(-(c + n) // pt)):
            table[r][b] = free[head]
            head += 1
        for t in range(c, c + n):
            positions.append(t)
            slots.append(table[r][t // pt] * pt + t % pt)
        cu.append(cu[-1] + n)
    pad = max_tokens - len(slots)
    return table, head, cu, [c + n for c, n in zip(ctx, new)], positions + [0] * pad, slots + [-1] * pad


def normed_rotated(x, w, eps, cos_sin, positions, pairs):
    """x [tokens, heads, dim] float64 through the RMS norm (w or None) and the rotation (cos_sin or None)."""
    x = x.double().clone()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        half = rot // 2
        out = x.clone()
        for i in range(half):
            c = cos_sin[positions.long(), i].double()[:, None]
            s = cos_sin[positions.long(), half + i].double()[:, None]
            ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + half)
            out[..., ia] = x[..., ia] * c - x[..., ib] * s
            out[..., ib] = x[..., ib] * c + x[..., ia] * s
        x = out
    return x


def rows_of(cache, slots, name):
    """float64 values of the rows at these slots: [tokens, kv_heads, dim]."""
    pt = cache.page_tokens
    x, s = getattr(cache, name), getattr(cache, name + "_scale")
    p, t = slots.long() // pt, slots.long() % pt
    return x[p, :, t].double() * s[p, :, t].double()[..., None]


def token_slots(pages, pt, n):
    t = torch.arange(n, device=pages.device)
    return pages.long()[t // pt] * pt + t % pt


def attention(q, k, v, seen, scale):
    """q [rows, dim], k and v [tokens, dim] float64; row i sees the first seen[i] tokens. Returns (out, bound): the
    result and, for each value, how far it may be off with float32 scores and sums, weights and values rounded once to
    fp16 or bfloat16 and the result once to bfloat16.

    The bound: a weight and a value are rounded by at most 2^-8 of themselves together (bfloat16 weights: eps/2 = 2^-8; fp16
    weights and values: 2^-11 each). fp16 has a floor besides, half its smallest step, 2^-25: a weight p <= 2^8 enters as
    p 2^(e - E), where 2^e is the size of its tile's value scales and 2^E that of the range the sum is held in, and its value as
    v 2^-e, below 254. So one key's product is off by at most 2^-25 254 2^E, and 2^E is at most the largest value scale, which is
    vmax / 127 with vmax the largest value an INT8 127 can stand for: 2^-24 vmax a key, against a sum of weights of at least 1. The
    largest value of the tokens given stands for vmax; twice that covers a largest INT8 of only 64.
    A score is a float32 sum of dim products (error at most (dim + 8) 2^-24 times the sum of their magnitudes, the scalings
    included), which changes a weight's share by at most 2 max(error); the sums over n tokens add at most (2 n + 64) 2^-24,
    which covers the exponential's 2^-22; the result is rounded by 2^-8 of itself."""
    s = q @ k.T * scale
    mask = torch.arange(k.shape[0], device=k.device)[None, :] >= seen[:, None]
    s = s.masked_fill(mask, -math.inf)
    w = torch.nan_to_num(torch.softmax(s, -1), nan=0.0)
    w = torch.where((seen > 0)[:, None], w, torch.zeros_like(w))
    out = w @ v
    mass = w @ v.abs()
    size = (q.abs() @ k.abs().T * abs(scale)).masked_fill(mask, 0.0).amax(-1, keepdim=True) if k.shape[0] else q.new_zeros(q.shape[0], 1)
    err = 2 * (q.shape[1] + 8) * 2.0**-24 * size + (2 * k.shape[0] + 64) * 2.0**-24 + 2.0**-8
    floor = 2.0**-23 * (w > 0).sum(-1, keepdim=True) * v.abs().max() if k.shape[0] else 0.0
    return out, err * mass + floor + 2.0**-8 * out.abs() + 1e-30


def cache_attention(q, cache, pages_of, kv_len, cu, scale, prefix=None):
    """q [tokens, heads, dim]; pages_of(r): the pages of request r's tokens in order; causal, the queries of r last.
    prefix: (pages, n), where the first n tokens of every request lie instead."""
    n, h, d = q.shape
    hk = cache.kv_heads
    out = torch.zeros(n, h, d, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    for r, length in enumerate(kv_len):
        a, b = cu[r], cu[r + 1]
        if a == b:
            continue
        sl = token_slots(pages_of(r), cache.page_tokens, length)
        if prefix is not None:
            m = min(prefix[1], length)
            sl[:m] = token_slots(prefix[0], cache.page_tokens, m)
        k, v = rows_of(cache, sl, "k"), rows_of(cache, sl, "v")
        seen = (length - (b - a) + torch.arange(b - a, device=q.device) + 1).clamp_min(0)
        for j in range(h):
            out[a:b, j], tol[a:b, j] = attention(q[a:b, j].double(), k[:, j * hk // h], v[:, j * hk // h], seen, scale)
    return out, tol
