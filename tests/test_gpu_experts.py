"""Routing and the experts' products against 64-bit forms: ties, masks, groups,
experts without rows and rows without an expert, one token to many."""

import math

import numpy as np
import pytest
import torch

from _fused import TYPES, U32, check, experts64, plan64, route64, rows, weights

pytestmark = pytest.mark.gpu


def dev(t, gpu):
    return None if t is None else t.to(gpu)


def run_route(q4lib, gpu, logits, topk, bias=None, **kw):
    ids, w, plan = q4lib.q4_route(dev(logits, gpu), topk, bias=dev(bias, gpu), **kw)
    rid, rw = route64(logits, topk, bias=bias, **kw)
    assert torch.equal(ids.cpu(), rid), (ids.cpu()[(ids.cpu() != rid).any(1)], rid[(ids.cpu() != rid).any(1)])
    # computed in 64 bits and rounded once
    assert torch.all((w.cpu().double() - rw).abs() <= 2 * U32 * rw.abs() + 2.0 ** -149)
    offsets, order = plan64(rid, logits.shape[1])
    assert plan.offsets.cpu().tolist() == offsets
    assert plan.order.cpu().tolist() == order


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("m,experts,topk", [(1, 1, 1), (1, 8, 2), (3, 60, 8), (5, 64, 6), (16, 128, 8),
                                            (7, 160, 6), (130, 256, 8), (9, 384, 32), (4, 1024, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_sizes(q4lib, gpu, dtype, m, experts, topk, score):
    logits = rows(m + experts, dtype, m, experts, scale=2.0)
    run_route(q4lib, gpu, logits, topk, score=score)


@pytest.mark.parametrize("groups,group_topk", [(2, 1), (4, 2), (8, 4), (32, 5), (64, 64)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_groups(q4lib, gpu, groups, group_topk, group_score, score, with_bias):
    logits = rows(groups, "bf16", 37, 64, scale=1.5)
    bias = rows(groups + 1, "f32", 64, scale=0.05) if with_bias else None
    run_route(q4lib, gpu, logits, 6, bias=bias, score=score, groups=groups, group_topk=group_topk,
              group_score=group_score, renormalise=group_topk != 2, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups", [1, 8])
def test_route_masks_ties_and_extremes(q4lib, gpu, score, with_bias, groups):
    E, big = 72, 3.0e38
    l = rows(5, "f32", 12, E)
    l[0] = -math.inf                    # nothing left
    l[1] = -math.inf
    l[1, 70] = -5.0                     # one left
    l[2] = 0.25                         # all equal: lowest indices
    l[3, ::2] = math.nan                # NaN counts as masked
    l[4, 10] = math.inf
    l[4, 20] = math.inf                 # two infinities: equal
    l[5] = -big                         # the type's lowest values are not masks
    l[6, 5] = big
    l[7] = torch.arange(E) * 1e-7 + 1.0  # near ties
    l[8] = torch.arange(E, 0, -1).float() * 40 - 1400  # scores that underflow fp32
    l[9, 1:] = -math.inf
    bias = None
    if with_bias:
        bias = rows(6, "f32", E, scale=0.1)
        bias[3], bias[4] = -math.inf, math.nan  # never chosen
        bias[30] = 10.0
    run_route(q4lib, gpu, l, 8, bias=bias, score=score, groups=groups, group_topk=min(3, groups),
              group_score="top2")


@pytest.mark.parametrize("m,topk,experts", [(1, 1, 1), (3, 4, 5), (100, 8, 64), (700, 3, 130), (33, 2, 1024)])
def test_plan_of_given_ids(q4lib, gpu, m, topk, experts):
    rng = np.random.default_rng(m)
    ids = torch.from_numpy(rng.integers(-1, experts + 1, (m, topk)).astype(np.int32))  # both ends name none
    if m > 50:
        ids[10:40] = 2  # the same expert again and again
    plan = q4lib.q4_route_plan(dev(ids, gpu), experts)
    clean = ids.clone()
    offsets, order = plan64(clean, experts)
    assert plan.offsets.cpu().tolist() == offsets
    assert plan.order.cpu().tolist() == order


def run_experts(q4lib, gpu, m, topk, E, n, k, xt, yt=None, act="none", gated=False, bias=False,
                combine=False, residual=False, per_pair=None, ids=None, seed=0):
    yt = yt or xt
    rng = np.random.default_rng(seed)
    packed, w = weights(seed + 1, E, n, k)
    if ids is None:
        ids = torch.from_numpy(np.stack([rng.permutation(E)[:topk] for _ in range(m)]).astype(np.int32))
    per_pair = combine if per_pair is None else per_pair
    x = rows(seed + 2, xt, m * topk if per_pair else m, k)
    b = rows(seed + 3, xt, E, n, scale=0.3) if bias else None
    nout = n // 2 if gated else n
    nrows = m if combine else m * topk
    r = rows(seed + 4, yt, nrows, nout) if residual else None
    g = rows(seed + 5, "f32", m, topk).abs() if combine else None
    y0 = torch.full((nrows, nout), 7.5, dtype=TYPES[yt])
    plan = q4lib.q4_route_plan(dev(ids, gpu), E)
    y = dev(y0, gpu).clone()
    q4lib.q4_experts(dev(x, gpu), dev(packed, gpu), plan, bias=dev(b, gpu), activation=act, gated=gated,
                     weights=dev(g, gpu), residual=dev(r, gpu), y=y)
    v, err = experts64(x, w, ids, b, act, gated, TYPES[yt], weights=g, residual=r, y0=y0,
                       rounded=m > 16 and xt != "f32", scaled=xt == "bf16")
    check(y, v, err, f"m{m} topk{topk} E{E} n{n} k{k} {xt}")


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,topk,E,n,k", [
    (1, 1, 1, 2, 32), (1, 2, 8, 66, 128), (1, 8, 16, 96, 512), (3, 2, 5, 130, 704), (9, 4, 8, 40, 1408),
    (16, 6, 64, 72, 256), (17, 2, 4, 34, 544), (40, 8, 16, 96, 512), (100, 2, 8, 200, 1024),
    (64, 8, 8, 64, 96), (300, 4, 6, 260, 512)])
@pytest.mark.parametrize("form", ["gate_up", "down", "rows"])
def test_experts_sizes(q4lib, gpu, m, topk, E, n, k, xt, form):
    kw = {"gate_up": dict(act="silu", gated=True), "down": dict(combine=True, residual=True, bias=True),
          "rows": dict(act="gelu", bias=True, residual=True, per_pair=True)}[form]
    run_experts(q4lib, gpu, m, topk, E, n, k, xt, seed=m + n, **kw)


@pytest.mark.parametrize("m", [6, 30, 200])
@pytest.mark.parametrize("combine", [False, True])
def test_experts_without_rows_and_rows_without_experts(q4lib, gpu, m, combine):
    """All rows on one expert, the other experts empty; some pairs, and whole
    tokens, with no expert at all; an expert named twice by a token."""
    ids = torch.full((m, 4), 2, dtype=torch.int32)
    ids[1] = -1
    ids[2, 1:] = 9
    ids[3, 0] = -7
    ids[4] = torch.tensor([5, 5, 0, 5])
    for gated in (False, True):
        run_experts(q4lib, gpu, m, 4, 9, 130, 512, "f16", combine=combine, gated=gated, act="silu", ids=ids,
                    seed=m)
    run_experts(q4lib, gpu, m, 4, 9, 130, 512, "bf16", combine=combine, ids=torch.full_like(ids, -1), seed=m)


@pytest.mark.parametrize("yt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m", [4, 90])
def test_experts_output_types(q4lib, gpu, m, yt):
    run_experts(q4lib, gpu, m, 2, 4, 96, 256, "f16", yt, combine=True, residual=True)
    run_experts(q4lib, gpu, m, 2, 4, 96, 256, "bf16", yt, gated=True, act="silu", residual=True)


def run_moe(q4lib, gpu, m, topk, E, hidden, inter, xt, seed=0, score="softmax", stream=None):
    """q4_moe against its own three operators called one by one: the same bits."""
    up, _ = weights(seed + 1, E, 2 * inter, hidden)
    down, _ = weights(seed + 2, E, hidden, inter)
    x, logits = rows(seed + 3, xt, m, hidden), rows(seed + 4, "f32", m, E, scale=2.0)
    ub, db = rows(seed + 5, xt, E, 2 * inter, scale=0.2), rows(seed + 6, xt, E, hidden, scale=0.2)
    r = rows(seed + 7, xt, m, hidden)
    rb = rows(seed + 8, "f32", E, scale=0.1)
    a = [dev(t, gpu) for t in (x, logits, up, down, ub, db, r, rb)]
    ids, w, plan = q4lib.q4_route(a[1], topk, score=score, bias=a[7])
    h = q4lib.q4_experts(a[0], a[2], plan, bias=a[4], activation="silu", gated=True)
    want = q4lib.q4_experts(h, a[3], plan, bias=a[5], weights=w, residual=a[6])
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    y = q4lib.q4_moe(a[0], a[1], a[2], a[3], topk, up_bias=a[4], down_bias=a[5], residual=a[6], score=score,
                     route_bias=a[7], ids=ids2, weights=w2)
    assert torch.equal(y, want) and torch.equal(ids, ids2) and torch.equal(w, w2)
    # and the operators' run as a whole against 64 bits
    rid, rw = route64(logits, topk, score=score, bias=rb)
    assert torch.equal(ids.cpu(), rid)


@pytest.mark.parametrize("m,topk,E,hidden,inter,xt", [
    (1, 2, 8, 512, 256, "f16"), (1, 4, 16, 512, 704, "bf16"), (7, 8, 64, 256, 128, "f16"),
    (64, 4, 8, 512, 352, "bf16"), (200, 2, 4, 256, 512, "f16"), (3, 2, 4, 96, 32, "f32"), (40, 1, 3, 544, 96, "bf16")])
def test_moe_is_its_operators_in_a_row(q4lib, gpu, m, topk, E, hidden, inter, xt):
    run_moe(q4lib, gpu, m, topk, E, hidden, inter, xt)


@pytest.mark.parametrize("m,topk,E,n,k", [(2, 2, 3, 3000, 256), (16, 2, 12, 1000, 448), (60, 1, 6, 520, 320),
                                          (30, 2, 4, 900, 1088), (5, 8, 32, 200, 2048), (8, 3, 64, 24, 4096)])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_experts_decode_row_tiles(q4lib, gpu, m, topk, E, n, k, xt):
    run_experts(q4lib, gpu, m, topk, E, n, k, xt, gated=True, act="silu", residual=True, seed=m)
    run_experts(q4lib, gpu, m, topk, E, n, k, xt, combine=True, bias=True, seed=m)


@pytest.mark.parametrize("m,topk,E,n,k", [(9, 4, 64, 130, 512), (2, 8, 16, 72, 448), (24, 2, 16, 264, 1024)])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_experts_named_often_by_a_token(q4lib, gpu, m, topk, E, n, k, xt):
    """Tokens that name one expert in all their places: more rows in its tiles
    than there are tokens."""
    ids = torch.full((m, topk), 3, dtype=torch.int32)
    ids[m // 2] = torch.arange(topk, dtype=torch.int32)
    run_experts(q4lib, gpu, m, topk, E, n, k, xt, gated=True, act="silu", ids=ids, seed=m)
    run_experts(q4lib, gpu, m, topk, E, n, k, xt, combine=True, residual=True, ids=ids, seed=m)


@pytest.mark.parametrize("m,topk,experts", [(1025, 1, 3), (257, 4, 1), (1366, 3, 7), (2000, 8, 1024), (300001, 1, 64),
                                            (70000, 8, 200)])
@pytest.mark.parametrize("skew", [False, True])
def test_plan_of_many_pairs(q4lib, gpu, m, topk, experts, skew):
    """Any number of workgroups and of pairs per workgroup, odd ends, nearly all
    pairs on one expert; against a stable sort."""
    g = torch.Generator().manual_seed(m)
    ids = torch.randint(-2, experts + 2, (m, topk), generator=g, dtype=torch.int32)
    if skew:
        ids[torch.rand((m, topk), generator=g) < 0.9] = experts // 2
    plan = q4lib.q4_route_plan(ids.to(gpu), experts)
    key = torch.where((ids < 0) | (ids >= experts), experts, ids).flatten()
    counts = torch.bincount(key, minlength=experts + 1)[:experts]
    offsets = torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)])
    order = torch.sort(key, dim=0, stable=True).indices
    order[offsets[-1]:] = -1
    assert torch.equal(plan.offsets.cpu().long(), offsets)
    assert torch.equal(plan.order.cpu().long(), order)
