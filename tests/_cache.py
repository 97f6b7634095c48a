"""The paged Q4_0 cache byte by byte, attention over it in 64 bits, and the error an
output may have.

`Batch` holds a batch on the host: the page of every position and the position of
every row.  `written` is the cache after q4_cache_write, from the oracle's quantiser
and the layout that the public header states.

Errors of attention (`attention64`), with u = 2^-24 and w_t the softmax weights:
  - a score: fp32 sums of d exact products, d u sum |q k|; with `rounded` (sequences of
    many rows) each decoded key is rounded to fp16, 2^-11 |q k|; bf16 q below 2^-32 of
    their row's largest magnitude are rounded to multiples of 2^-39 of it, half a step
    each; the factors and the cap 8 roundings of the score and, capped, of the cap, the
    exponent's argument 4 of the score and of the maximum;
  - a weight: relatively its score's error, 8 u for exp and, on matrix cores, 2^-11 for
    fp16 (2^-22 in two parts, of which the lower one's own grain is 2^-24 too), with a
    floor of 2^-33 of the largest weight where fp16 has no more bits (half its subnormal
    step, 2^-25, of weights that are lifted by 2^8 or more), in fp32 of 2^-126: a
    weight below 2^-126 of the largest (which is exp(0) = 1) is below fp32's normal
    range, and whether it is kept on the subnormal grid or flushed, it moves by at most itself;
  - y: sum w_t (|v_t| + |y|) times the weights' errors, (n + 40) u sum w |v| for the
    sums (n positions), 2^-11 sum w |v| where decoded values are rounded to fp16, and one
    rounding to y's type.  lse: sum w_t times the scores' errors, (n + 40) u and 4 u |lse|.
"""

import math

import numpy as np
import torch

import oracle
from _fused import HALF, TINY, TYPES, rows  # noqa: F401

U = 2.0 ** -24
PLACE = (0, 2, 1, 3)


class Batch:
    """lengths and rows per sequence; pages in random order, spare ones at random places."""

    def __init__(self, lengths, counts, page, seed=0, before=0, behind=0, spare=2, single=False):
        rng = np.random.default_rng(seed)
        self.lengths, self.counts, self.page = list(lengths), list(counts), page
        self.seqs = len(self.lengths)
        each = [max(0, -(-n // page)) for n in self.lengths]
        self.max_pages = max(1, max(each))
        self.pages = sum(each) + spare
        order = rng.permutation(self.pages)
        self.tables = np.full((self.seqs, self.max_pages), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(each):
            self.tables[s, :n] = order[at:at + n]
            at += n
        self.offsets = None if single else np.cumsum([before] + self.counts).astype(np.int32)
        self.tokens = before + sum(self.counts) + behind
        self.places = []  # (row, sequence, position)
        row = before
        for s, (length, n) in enumerate(zip(self.lengths, self.counts)):
            for i in range(n):
                self.places.append((row, s, length - n + i))
                row += 1

    def device(self, dev):
        t = [torch.from_numpy(self.tables).to(dev), torch.tensor(self.lengths, dtype=torch.int32, device=dev),
             None if self.offsets is None else torch.from_numpy(self.offsets).to(dev)]
        return t

    def page_of(self, s, t):
        """The page of position t, -1 where none is named."""
        slot = t // self.page
        if t < 0 or slot >= self.max_pages:
            return -1
        p = int(self.tables[s, slot])
        return p if 0 <= p < self.pages else -1


def storable(x):
    x = x.double().numpy()
    return np.where(np.isnan(x), 0.0, np.clip(x, -65504.0, 65504.0)).astype(np.float32)


def blocks(x):
    """Q4_0 of rows [n, d]: scales [n, d / 32] (bits) and code bytes [n, d / 32, 16]."""
    x = np.ascontiguousarray(storable(x))
    n, d = x.shape
    b = oracle.quantize(x).reshape(n, d // 32, 18)
    return b[:, :, :2].copy().view(np.uint16)[..., 0], b[:, :, 2:].copy()


def index(d, value, t):
    """Bytes of position t of a granule: code bytes [d / 32, 16], scales [d / 32] (each its first byte)."""
    nb = d // 32
    b, i = np.arange(nb)[:, None], np.arange(16)[None, :]
    if value:
        return (b * 16 + i) * 16 + t, 8 * d + 2 * (np.arange(nb) * 16 + t // 4 * 4 + PLACE[t % 4])
    return t * (d // 2) + (i // 4 * nb + b) * 4 + i % 4, 8 * d + 2 * ((t // 4 * nb + np.arange(nb)) * 4 + t % 4)


def written(cache, batch, k, v):
    """cache [pages, kv, 2, page / 16, 9 d] (numpy) with k, v [tokens, kv, d] written."""
    out = cache.copy()
    kv, d = k.shape[1], k.shape[2]
    for value, x in ((0, k), (1, v)):
        scales, codes = blocks(x.reshape(-1, d))
        scales, codes = scales.reshape(-1, kv, d // 32), codes.reshape(-1, kv, d // 32, 16)
        for row, s, t in batch.places:
            p = batch.page_of(s, t)
            if t < 0 or t >= batch.lengths[s] or p < 0:
                continue
            code_at, scale_at = index(d, value, t % 16)
            for h in range(kv):
                g = out[p, h, value, t % batch.page // 16]
                g[code_at] = codes[row, h]
                g[scale_at] = scales[row, h] & 255
                g[scale_at + 1] = scales[row, h] >> 8
    return out


def decoded(cache, batch, s, t, value):
    """[kv, d] float64 of position t of sequence s; None without a page."""
    p = batch.page_of(s, t)
    if p < 0:
        return None
    d = cache.shape[-1] // 9
    g = cache[p, :, value, t % batch.page // 16]
    code_at, scale_at = index(d, value, t % 16)
    bits = g[:, scale_at].astype(np.uint16) | (g[:, scale_at + 1].astype(np.uint16) << 8)
    sc = bits.view(np.float16).astype(np.float64)
    c = g[:, code_at.reshape(-1)].reshape(-1, d // 32, 16)
    q = np.concatenate([c & 15, c >> 4], -1).astype(np.float64) - 8
    return (q * sc[..., None]).reshape(-1, d)


def random_cache(seed, pages, kv, page, d, scale=1.0):
    """A cache of random codes and scales whose values are of about `scale`."""
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 256, (pages, kv, 2, page // 16, 9 * d), dtype=np.uint8)
    sc = (rng.uniform(0.05, 0.4, (pages, kv, 2, page // 16, d // 2)) * scale * rng.choice([-1, 1], (
        pages, kv, 2, page // 16, d // 2))).astype(np.float16)
    c[..., 8 * d:] = sc.view(np.uint8)
    return c


def sequence(cache, batch, s):
    """(k, v [length, kv, d] float64, live [length]) of a sequence."""
    d, kv, n = cache.shape[-1] // 9, cache.shape[1], batch.lengths[s]
    k, v = np.zeros((n, kv, d)), np.zeros((n, kv, d))
    live = np.zeros(n, dtype=bool)
    p = batch.tables[s][np.arange(n) // batch.page] if n else np.zeros(0, np.int32)
    ok = (p >= 0) & (p < batch.pages)
    for t0 in range(16):  # sixteen places of a granule, all granules at once
        t = np.arange(t0, n, 16)
        t = t[ok[t]]
        live[t] = True
        for value, out in ((0, k), (1, v)):
            g = cache[p[t], :, value, t % batch.page // 16]  # [m, kv, 9 d]
            code_at, scale_at = index(d, value, t0)
            bits = g[..., scale_at].astype(np.uint16) | (g[..., scale_at + 1].astype(np.uint16) << 8)
            sc = bits.view(np.float16).astype(np.float64)
            c = g[..., code_at.reshape(-1)].reshape(len(t), kv, d // 32, 16)
            q = np.concatenate([c & 15, c >> 4], -1).astype(np.float64) - 8
            out[t] = (q * sc[..., None]).reshape(len(t), kv, d)
    return torch.from_numpy(k), torch.from_numpy(v), torch.from_numpy(live)


def attention64(q, cache, batch, scale=None, causal=True, window=0, softcap=0.0, dtype=None, matrix=None,
                rounded=True):
    """(y, bound, lse, bound) in 64 bits; rows of no sequence NaN with an infinite bound.
    matrix: products on matrix cores (default: q of 16 bits)."""
    tokens, heads, d = q.shape
    kv = cache.shape[1]
    dtype = dtype or q.dtype
    matrix = q.dtype != torch.float32 if matrix is None else matrix
    scale = d ** -0.5 if scale is None else scale
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
        k, v, live = sequence(cache, batch, s)
        t = torch.arange(length)
        p = (length - n + torch.arange(n))[:, None]
        seen = live[None, :] & (t[None, :] < length)
        if causal:
            seen = seen & (t[None, :] <= p)
        if window:
            seen = seen & (t[None, :] > p - window)
        if not causal and not window:
            seen = seen.expand(n, length)
        for h in range(heads):
            qh = q[mine, h].double()
            kh, vh = k[:, h // (heads // kv)], v[:, h // (heads // kv)]
            raw, mag = scale * (qh @ kh.T), abs(scale) * (qh.abs() @ kh.abs().T)
            es = mag * (U * (d + 8) + (2.0 ** -11 if matrix and rounded else 0.0))
            if q.dtype == torch.bfloat16:
                top = qh.abs().amax(1, keepdim=True)
                small = (qh.abs() < 2.0 ** -32 * top).double()
                es = es + abs(scale) * 2.0 ** -40 * top * (small @ kh.abs().T)
            z = softcap * torch.tanh(raw / softcap) if softcap else raw
            es = es + 8 * U * (raw.abs() + softcap)
            z = z.masked_fill(~seen, -math.inf)
            m = z.amax(-1, keepdim=True) if length else torch.full((n, 1), -math.inf, dtype=torch.float64)
            some = m > -math.inf
            m0 = torch.where(some, m, torch.zeros_like(m))
            es = es + 4 * U * (raw.abs() + m0.abs())
            e = torch.exp(z - m0) * seen
            total = e.sum(-1, keepdim=True)
            w = e / torch.where(total > 0, total, torch.ones_like(total))
            yh = w @ vh
            ep = (es.exp() - 1).clamp_max(1.0) + 8 * U
            if matrix:
                ep = ep + 2.0 ** -11
            ew = w * ep + (2.0 ** -33 if matrix else 2.0 ** -126) * seen / total.clamp_min(1e-300)
            size = w @ vh.abs()
            b = ew @ vh.abs() + ew.sum(-1, keepdim=True) * yh.abs()
            b = b + size * ((length + 40) * U + (2.0 ** -11 if matrix else 0.0))
            y[mine, h] = yh
            eb[mine, h] = b + HALF[dtype] * (yh.abs() + b) + TINY[dtype]
            big = torch.where(some, m0 + total.clamp_min(1e-300).log(), torch.full_like(m0, -math.inf))[:, 0]
            lse[mine, h] = big
            size = torch.where(some[:, 0], big.abs(), torch.zeros_like(big))
            el[mine, h] = (w * (ep - (2.0 ** -11 if matrix else 0))).sum(-1) + (length + 40) * U + 4 * U * size + (
                length * 2.0 ** -33 if matrix else 0.0)
    return y, eb, lse, el


def check(got, want, bound, what=""):
    """Every output within its bound; infinities equal; NaN (rows of no sequence) skipped."""
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    skip = want.isnan()
    same = (got == want) | ((got - want).abs() <= bound)
    bad = ~(skip | same)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        over = ((got - want).abs() / bound).masked_fill(skip, 0).nan_to_num(nan=math.inf).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {float(over):.3g} x bound; "
                             f"at {i}: got {got[i]!r}, is {want[i]!r}, bound {bound[i]!r}")
