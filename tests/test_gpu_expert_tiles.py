"""The experts' products at every tile height a plan may choose, each at the error
its own kernels may have, and weights beyond fp16 in one expert."""

import numpy as np
import pytest
import torch

import oracle
from _fused import TYPES, check, decode, experts64, rows, weights

pytestmark = pytest.mark.gpu


def tile_rows(m, topk, E):
    """Rows per tile of a plan: by the mean number of rows per expert."""
    mean = m * topk / E
    return 16 if mean <= 12 or m <= 16 else 32 if mean <= 40 or m <= 32 else 128 if mean <= 80 else 192


def draw_ids(rng, m, topk, E, skew):
    """Every token's experts, distinct; with a skew expert E - 1 is in nearly all rows,
    and some pairs have none."""
    ids = np.stack([rng.permutation(E)[:topk] for _ in range(m)]).astype(np.int32)
    if skew:
        for i in range(m):
            if rng.random() < 0.9 and E - 1 not in ids[i]:
                ids[i, 0] = E - 1
        ids[rng.random((m, topk)) < 0.05] = -1
    return torch.from_numpy(ids)


def run(q4lib, gpu, m, topk, E, n, k, xt, packed, w, ids, act="none", gated=False, bias=False, combine=False,
        per_pair=False, inplace=False, seed=0):
    """One call against the 64-bit form.  16- and 32-row tiles multiply exact codes and
    apply fp32 scales; fp16 weights, rounded once, are the higher tiles' alone (and the
    exact route's never)."""
    yt = torch.float32
    x = rows(seed + 2, xt, m * topk if per_pair else m, k)
    b = rows(seed + 3, xt, E, n, scale=0.3) if bias else None
    nout, nrows = n // 2 if gated else n, m if combine else m * topk
    g = rows(seed + 5, "f32", m, topk).abs() if combine else None
    r = rows(seed + 4, "f32", nrows, nout)
    d = lambda t: None if t is None else t.to(gpu)  # noqa: E731
    plan = q4lib.q4_route_plan(d(ids), E)
    y = d(r).clone() if inplace else torch.full((nrows, nout), 7.5, dtype=yt, device=gpu)
    y0 = r if inplace else y.cpu()
    q4lib.q4_experts(d(x), d(packed), plan, bias=d(b), activation=act, gated=gated, weights=d(g),
                     residual=y if inplace else d(r), y=y)
    v, err = experts64(x, w, ids, b, act, gated, yt, weights=g, residual=r, y0=y0,
                       rounded=tile_rows(m, topk, E) > 32 and xt != "f32", scaled=xt == "bf16")
    check(y, v, err, f"m{m} topk{topk} E{E} n{n} k{k} {xt} tiles of {tile_rows(m, topk, E)}")


# Tiles of 16 (mean of 8 and 12 rows; 16 tokens on two experts), 32 (13, 25, 40), 128
# (41, 60, 80; two and three column tiles, several tiles of one expert) and 192 rows
# (81, 130, 300), of k in whole 64-wide steps and not.
SIZES = [(32, 2, 8, 200, 1024), (48, 2, 8, 136, 704), (16, 2, 2, 264, 512), (26, 4, 8, 130, 512), (100, 2, 8, 300, 1024),
         (80, 4, 8, 96, 1088), (17, 2, 4, 34, 544), (82, 4, 8, 300, 512), (120, 4, 8, 272, 1024), (160, 4, 8, 136, 320),
         (160, 4, 8, 132, 96), (162, 4, 8, 300, 512), (260, 4, 8, 516, 256), (300, 4, 4, 264, 544)]


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,topk,E,n,k", SIZES)
@pytest.mark.parametrize("skew", [False, True])
def test_experts_at_every_tile_height(q4lib, gpu, m, topk, E, n, k, xt, skew):
    packed, w = weights(m + n, E, n, k)
    ids = draw_ids(np.random.default_rng(m), m, topk, E, skew)
    run(q4lib, gpu, m, topk, E, n, k, xt, packed, w, ids, act="silu", gated=True, bias=True, seed=m)
    run(q4lib, gpu, m, topk, E, n, k, xt, packed, w, ids, inplace=True, per_pair=True, seed=m + 1)
    run(q4lib, gpu, m, topk, E, n, k, xt, packed, w, ids, combine=True, per_pair=True, bias=True, seed=m + 2)


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,topk,E,n,k", [(12, 2, 8, 96, 512), (60, 2, 6, 132, 704), (120, 3, 6, 300, 512),
                                          (100, 4, 6, 140, 96), (260, 3, 6, 264, 512), (270, 3, 6, 300, 1088)])
@pytest.mark.parametrize("gated", [False, True])
def test_experts_with_scales_beyond_fp16(q4lib, gpu, m, topk, E, n, k, xt, gated):
    """Block scales whose largest weight is beyond fp16 (80000) in one expert, not the
    first: the tiles of its rows that meet them run again from the original rows, the
    residual is y itself, and other tiles and experts know nothing of it."""
    rng = np.random.default_rng(m)
    w = (rng.standard_normal((E, n, k)) * 0.05).astype(np.float32)
    w[3, n // 2 + 3, 5] = 80000.0
    w[3, 1, k - 3] = -90000.0
    w[E - 1, n - 1, k // 2] = 70000.0
    flat = oracle.quantize(w.reshape(-1, k))
    packed = torch.from_numpy(flat).view(E, n, -1)
    dec = torch.from_numpy(decode(flat, E * n, k)).view(E, n, k)
    for skew in (False, True):
        ids = draw_ids(rng, m, topk, E, skew)
        run(q4lib, gpu, m, topk, E, n, k, xt, packed, dec, ids, act="relu", gated=gated, inplace=True, seed=m)
        run(q4lib, gpu, m, topk, E, n, k, xt, packed, dec, ids, act="relu", gated=gated, combine=True, per_pair=True,
            inplace=True, bias=True, seed=m)
