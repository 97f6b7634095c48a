"""Attention over the paged Q4_0 cache in 64 bits, with what each way of computing it may
err by and no more.

Which way a sequence takes goes by its rows (rows of q times heads per kv head) and q's type,
as the public header states it:
  row    fp32 q: nothing is rounded to fewer than 32 bits;
  few    16-bit q, no offsets or up to 32 rows: keys' codes exact, their scales fp32;
  many   16-bit q, more rows: decoded keys rounded to fp16.
Both matrix-core ways round decoded values to fp16, and weights: to one fp16, or (few rows,
fp16 q, 16 rows to a product) to two.

Errors, with u = 2^-24, w_t the softmax weights, n the positions:
  - a score s = scale q.k: d + 8 roundings of sum |scale q k|; many: |scale q| |fp16(k) - k|
    as it is; bf16 q below 2^-32 of their row's largest magnitude: 2^-40 of that times |k|;
  - the capped score f = c tanh(s / c), whose slope is at most 1: s's error and 16 u |f|.
    (|s / c| up to 5/8: s P(z^2), z two roundings, the polynomial's terms below 0.08 of the
    whole, a product, a sum, the fit 2^-27: 5 u.  Above: z two, its exponent's factor one,
    exp 2 u: (6 |z| + 2) u / sinh 2 |z| <= 3.6 u; 2 t / (1 + t) three and the reciprocal 2 u of
    at most 0.445 of 0.555: 4 u; the last sum, factor and unit 4 u: 12 u.);
  - an exponent s - m: 8 u |f| (factor and unit) + 4 u (|f| + |m|);
  - exp 8 u; in fp16 parts 2^-11 or 2^-21 more of the sum over values alone, at least half
    fp16's smallest step, 2^-25, of weights that are lifted by 2^12 (few) or 2^8 (many);
  - y: numerator sum w |v| e + |fp16(v) - v| w, denominator |y| sum w e, n + 40 roundings of
    sum w |v|, and one rounding to y's type.  lse: sum w e, n + 40 u, 4 u |lse|.

`fault` plants a mistake in the values, for tests of the bounds themselves:
  keys     few: decoded keys rounded to fp16 as in the way of many rows;
  weights  weights in one fp16 part everywhere;
  cap      c - 2 c / (exp(2 s / c) + 1) in fp32.
"""

import math

import numpy as np
import torch

from _cache import HALF, TINY, U, Batch, random_cache, rows, sequence

FEW_ROWS = 32


def way_of(batch, s, group, dtype):
    if dtype == torch.float32:
        return "row"
    return "few" if batch.offsets is None or batch.counts[s] * group <= FEW_ROWS else "many"


def two_parts(batch, way, group, d, dtype):
    wide = d <= 192 and (batch.offsets is None or d > 64) and batch.tokens * group > 16 * batch.seqs
    return way == "few" and dtype == torch.float16 and not wide


# Batches of few rows over few positions, where what a score or a weight is rounded to shows:
# lse of one position is its score, and a weight is a good part of all.
FEW = {
    "single": (Batch([1] * 60, [1] * 60, 16, single=True), 4, 2, 64),
    "tokens": (Batch([2, 3, 5, 9, 17, 40], [1] * 6, 16, seed=1, single=True), 4, 2, 64),
    "drafts": (Batch([2, 9, 17, 40], [2, 3, 1, 4], 16, seed=2), 4, 2, 128),
}


def few_example(name, dtype, seed=1):
    """A batch, its cache, whose values fp16 holds exactly, and q."""
    b, heads, kv, d = FEW[name]
    cache = random_cache(seed, b.pages, kv, b.page, d)
    scales = np.ascontiguousarray(cache[:, :, 1, :, 8 * d:]).view(np.uint16)
    cache[:, :, 1, :, 8 * d:] = (scales & 0xFC00).view(np.uint8)  # powers of two
    return b, cache, rows(seed + 1, dtype, b.tokens, heads, d, scale=0.5)


def to_half(x):
    return x.half().double()


def capped(s, c, fault):
    if fault == "cap":
        s, c = s.numpy().astype(np.float32), np.float32(c)
        with np.errstate(all="ignore"):
            return torch.from_numpy((c - 2 * c / (np.exp(2 * s / c) + np.float32(1))).astype(np.float64))
    return c * torch.tanh(s / c)


def attention_bounds(q, cache, batch, scale=None, causal=True, window=0, softcap=0.0, dtype=None, fault=None):
    """(y, bound, lse, bound) in 64 bits; rows of no sequence NaN with an infinite bound."""
    tokens, heads, d = q.shape
    kv = cache.shape[1]
    group = heads // kv
    dtype = dtype or q.dtype
    scale = d ** -0.5 if scale is None else scale
    softcap = float(np.float32(softcap))
    y = torch.full((tokens, heads, d), math.nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), math.nan, dtype=torch.float64)
    eb, el = torch.full_like(y, math.inf), torch.full_like(lse, math.inf)
    start = 0 if batch.offsets is None else int(batch.offsets[0])
    for s in range(batch.seqs):
        n, length = batch.counts[s], batch.lengths[s]
        mine = slice(start, start + n)
        start += n
        if n == 0:
            continue
        way = way_of(batch, s, group, q.dtype)
        two = two_parts(batch, way, group, d, q.dtype)
        k, v, live = sequence(cache, batch, s)
        if fault == "keys" and way == "few":
            k = to_half(k)
        t = torch.arange(length)
        p = (length - n + torch.arange(n))[:, None]
        seen = live[None, :].expand(n, length)
        if causal:
            seen = seen & (t[None, :] <= p)
        if window:
            seen = seen & (t[None, :] > p - window)
        for h in range(heads):
            qh, kh, vh = q[mine, h].double(), k[:, h // group], v[:, h // group]
            raw, mag = scale * (qh @ kh.T), abs(scale) * (qh.abs() @ kh.abs().T)
            es = mag * U * (d + 8)
            if way == "many":
                es = es + abs(scale) * (qh.abs() @ (to_half(kh) - kh).abs().T)
            if q.dtype == torch.bfloat16:
                top = qh.abs().amax(1, keepdim=True)
                small = (qh.abs() < 2.0 ** -32 * top).double()
                es = es + abs(scale) * 2.0 ** -40 * top * (small @ kh.abs().T)
            f = raw
            if softcap:
                f = capped(raw, softcap, fault)
                es = es + 16 * U * f.abs()
            f = f.masked_fill(~seen, -math.inf)
            m = f.amax(-1, keepdim=True) if length else torch.full((n, 1), -math.inf, dtype=torch.float64)
            some = m > -math.inf
            m0 = torch.where(some, m, torch.zeros_like(m))
            size = torch.where(seen, f.abs(), torch.zeros_like(f))
            es = es + U * (12 * size + 4 * m0.abs())
            e = torch.exp(f - m0) * seen
            total = e.sum(-1, keepdim=True)
            whole = torch.where(total > 0, total, torch.ones_like(total))
            w = e / whole
            given = w
            if fault == "weights" and way != "row":  # (lifted by 2^12 in units of log2, as the kernel holds them)
                given = to_half(e * 4096) / 4096 / whole
            yh = given @ vh
            ep = (torch.expm1(es).clamp_max(1.0) + 8 * U) * seen
            parts, floor = 0.0, 2.0 ** -120
            if way != "row":
                parts, floor = 2.0 ** -21 if two else 2.0 ** -11, 2.0 ** -37 if way == "few" else 2.0 ** -33
            over = w * (ep + parts) + floor * seen / whole
            under = (w * ep).sum(-1, keepdim=True) + length * 2.0 ** -120
            b = over @ vh.abs() + under * yh.abs() + (length + 40) * U * (w @ vh.abs())
            if way != "row":
                b = b + w @ (to_half(vh) - vh).abs()
            y[mine, h] = yh
            eb[mine, h] = b + HALF[dtype] * (yh.abs() + b) + TINY[dtype]
            big = torch.where(some, m0 + whole.log(), torch.full_like(m0, -math.inf))[:, 0]
            lse[mine, h] = big
            el[mine, h] = under[:, 0] + (length + 40) * U + 4 * U * torch.where(some[:, 0], big.abs(), torch.zeros_like(big))
    return y, eb, lse, el
