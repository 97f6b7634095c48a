"""64-bit forms of the fused layers and the error each output may have.

Every form returns (value, bound).  The bound adds up, per output:
  - the fp32 sums of a product: every product is formed exactly and a sum of
    t terms errs by at most t 2^-24 of the sum of magnitudes S = sum |x w|;
  - with `rounded` (more than 32 rows per product, 16-bit x): each dequantised
    weight is rounded to fp16 once, 2^-11 of |x w| each;
  - with `scaled` (bf16 x): activations below 2^-32 of their row's largest are
    rounded to multiples of 2^-39 of it, half a step each, times |w|;
  - the activation: a slope of at most 1.13 (silu, gelu) on that error, and 16
    roundings of 2^-24 in its evaluation;
  - one rounding to the output type: half a step.
"""

import math

import numpy as np
import torch

import oracle

U32 = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def weights(seed, *shape, scale=0.05):
    """(packed uint8 [..., n, k/32*18], decoded float64) of seeded Q4_0 weights."""
    rng = np.random.default_rng(seed)
    w = (rng.standard_normal(shape) * scale).astype(np.float32)
    flat = w.reshape(-1, shape[-1])
    packed = oracle.quantize(flat)
    dec = decode(packed, flat.shape[0], shape[-1])
    return (torch.from_numpy(packed).view(*shape[:-1], -1), torch.from_numpy(dec).view(*shape))


def decode(packed, n, k):
    b = np.ascontiguousarray(packed).reshape(n, k // 32, 18)
    d = b[:, :, :2].copy().view(np.float16).astype(np.float64)
    lo, hi = (b[:, :, 2:] & 15).astype(np.float64), (b[:, :, 2:] >> 4).astype(np.float64)
    return ((np.concatenate([lo, hi], -1) - 8) * d).reshape(n, k)


def rows(seed, dtype, *shape, scale=1.0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TYPES[dtype])


def act64(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "gelu_erf":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    return z


def product64(x, w, bias, act, gated, rounded=False, scaled=False):
    """(v, bound) of the rows before residual and rounding; x [m, k], w [n, k] float64."""
    x = x.double()
    k = x.shape[1]
    z, S = x @ w.T, x.abs() @ w.abs().T
    err = S * (U32 * (k + 8) + (2.0 ** -11 if rounded else 0.0))
    if scaled:
        top = x.abs().amax(1, keepdim=True)
        small = (x.abs() < 2.0 ** -32 * top).double()
        err = err + 2.0 ** -40 * top * (small @ w.abs().T)
    if bias is not None:
        z = z + bias.double()
        err = err + U32 * (S + bias.double().abs())
    half = z.shape[1] // 2
    z0, e0 = (z[:, :half], err[:, :half]) if gated else (z, err)
    a = act64(z0, act)
    ea = e0 * (1.13 if act != "none" else 1.0) + (16 * U32 * a.abs() if act != "none" else 0.0)
    if act in ("silu", "gelu"):  # exp's argument carries |z| roundings of itself
        ea = ea + 4 * U32 * z0.abs() * a.abs()
    if act == "gelu":
        ea = ea + 16 * U32 * (z0.abs() ** 3).clamp_max(1e3) * a.abs()
    if not gated:
        return a, ea
    u, eu = z[:, half:], err[:, half:]
    return a * u, a.abs() * eu + u.abs() * ea + ea * eu + U32 * (a * u).abs()


def finish64(v, err, residual, dtype):
    if residual is not None:
        v = v + residual.double()
        err = err + U32 * v.abs()
    return v, err + HALF[dtype] * (v.abs() + err) + TINY[dtype]


def check(y, v, bound, what=""):
    y = y.detach().cpu().double()
    assert y.shape == v.shape, (what, y.shape, v.shape)
    bad = ~((y - v).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        worst = ((y - v).abs() / bound).nan_to_num(nan=math.inf).max()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {worst:.3g} x bound; "
                             f"at {i}: got {y[i]!r}, is {v[i]!r}, bound {bound[i]!r}")


# ------------------------------------------------------------------ routing

def route64(logits, topk, score="softmax", bias=None, groups=1, group_topk=1, group_score="max",
            renormalise=True, scale=1.0):
    """(ids, weights float64), one token after the other."""
    m, E = logits.shape
    ids = torch.full((m, topk), -1, dtype=torch.int32)
    out = torch.zeros((m, topk), dtype=torch.float64)
    big = float(torch.finfo(torch.float32).max)
    for t in range(m):
        l = [float(v) for v in logits[t].double()]
        live = [v > -math.inf for v in l]
        l = [min(v, big) if ok else 0.0 for v, ok in zip(l, live)]
        if score == "softmax":
            top = max([v for v, ok in zip(l, live) if ok], default=0.0)
            p = [math.exp(max(v - top, -800.0)) if ok and v - top > -745 else 0.0 for v, ok in zip(l, live)]
            total = sum(p)
            s = [v / total if total > 0 else 0.0 for v in p]
        else:
            s = [(1 / (1 + math.exp(-v)) if v > -700 else 0.0) if ok else 0.0 for v, ok in zip(l, live)]
        additive = bias is not None or (groups > 1 and group_score == "top2")
        key = []
        for e in range(E):
            v = (s[e] if additive else l[e]) + (float(bias[e]) if bias is not None else 0.0)
            key.append(v if live[e] and v > -math.inf else -math.inf)
        if groups > 1:
            per = E // groups
            value = []
            for g in range(groups):
                two = sorted(key[g * per:(g + 1) * per], reverse=True)[:2]
                v = two[0]
                if group_score == "top2" and len(two) > 1 and two[1] > -math.inf:
                    v = two[0] + two[1]
                value.append(v)
            best = sorted(range(groups), key=lambda g: (-value[g], g))[:group_topk]
            key = [v if e // per in best else -math.inf for e, v in enumerate(key)]
        chosen = [e for e in sorted(range(E), key=lambda e: (-key[e], e))[:topk] if key[e] > -math.inf]
        total = sum(s[e] for e in chosen)
        for j, e in enumerate(chosen):
            ids[t, j] = e
            w = s[e]
            if renormalise:
                w = w / total if total > 0 else 0.0
            out[t, j] = w * scale
    return ids, out


def plan64(ids, experts):
    flat = [int(v) for v in ids.flatten()]
    order, offsets = [], [0]
    for e in range(experts):
        order += [p for p, v in enumerate(flat) if v == e]
        offsets.append(len(order))
    return offsets, order + [-1] * (len(flat) - len(order))


def experts64(x, w, ids, bias, act, gated, dtype, weights=None, residual=None, y0=None, rounded=False,
              scaled=False):
    """(value, bound) of q4_experts: x [m or m topk, k], w [E, n, k] float64, ids [m, topk]."""
    m, topk = ids.shape
    flat = ids.flatten()
    per = topk if x.shape[0] == m else 1
    nout = w.shape[1] // 2 if gated else w.shape[1]
    v = torch.zeros((m * topk, nout), dtype=torch.float64)
    err = torch.zeros_like(v)
    for e in range(w.shape[0]):
        at = (flat == e).nonzero().flatten()
        if len(at):
            v[at], err[at] = product64(x[at // per], w[e], None if bias is None else bias[e], act, gated,
                                       rounded, scaled)
    live = (flat >= 0) & (flat < w.shape[0])
    if weights is None:
        v, err = finish64(v, err, residual, dtype)
        if y0 is not None:  # rows without an expert stay as they were
            v[~live], err[~live] = y0.double()[~live], 0.0
        return v, err
    g = (weights.double().flatten() * live).view(m, topk, 1)
    v3, e3 = v.view(m, topk, -1), err.view(m, topk, -1)
    total = (g.abs() * v3.abs()).sum(1)
    return finish64((g * v3).sum(1), (g.abs() * e3).sum(1) + (topk + 1) * U32 * total, residual, dtype)
