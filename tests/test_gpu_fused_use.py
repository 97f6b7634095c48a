"""The fused layers as they are used: one token, a captured and replayed layer,
two streams at once, rows with an infinity or NaN, tensors of more than 4 GiB."""

import math

import pytest
import torch

from _fused import TYPES, check, finish64, product64, route64, rows, weights

pytestmark = pytest.mark.gpu


def dev(t, gpu):
    return None if t is None else t.to(gpu)


class Layer:
    """An expert layer on the device, run whole or operator by operator."""

    def __init__(self, gpu, E, hidden, inter, xt, seed, gated=True, bias=True):
        n = 2 * inter if gated else inter
        self.up, _ = weights(seed + 1, E, n, hidden)
        self.down, _ = weights(seed + 2, E, hidden, inter)
        self.up, self.down = self.up.to(gpu), self.down.to(gpu)
        self.ub = rows(seed + 3, xt, E, n, scale=0.2).to(gpu) if bias else None
        self.db = rows(seed + 4, xt, E, hidden, scale=0.2).to(gpu) if bias else None
        self.gated = gated

    def whole(self, q4, x, logits, topk, act="silu", residual=None, y=None, ids=None, weights=None, y_dtype=None,
              bias=None, stream=None, **routing):
        return q4.q4_moe(x, logits, self.up, self.down, topk, activation=act, gated=self.gated, up_bias=self.ub,
                         down_bias=self.db, residual=residual, y=y, ids=ids, weights=weights, y_dtype=y_dtype,
                         route_bias=bias, stream=stream, **routing)

    def parts(self, q4, x, logits, topk, act="silu", residual=None, y_dtype=None, bias=None, **routing):
        ids, w, plan = q4.q4_route(logits, topk, bias=bias, **routing)
        h = q4.q4_experts(x, self.up, plan, bias=self.ub, activation=act, gated=self.gated)
        y = q4.q4_experts(h, self.down, plan, bias=self.db, weights=w, residual=residual, y_dtype=y_dtype)
        return y, ids, w


def bits(t):
    return t.contiguous().view(torch.uint8)


# ------------------------------------------------------------------ one token

@pytest.mark.parametrize("topk,E,hidden,inter", [
    (1, 1, 64, 64), (1, 2, 256, 64), (2, 3, 192, 320), (3, 60, 256, 448), (8, 12, 2048, 768), (16, 20, 448, 704),
    (16, 16, 512, 2048), (17, 24, 256, 256), (4, 257, 256, 128), (8, 9, 4160, 192), (2, 4, 512, 6144)])
@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("gated,act", [(True, "silu"), (False, "gelu")])
def test_one_token_is_its_operators_in_a_row(q4lib, gpu, topk, E, hidden, inter, xt, gated, act):
    L = Layer(gpu, E, hidden, inter, xt, seed=topk + hidden, gated=gated, bias=E % 2 == 0)
    x, logits = rows(5, xt, 1, hidden).to(gpu), rows(6, "f32", 1, E, scale=2.0).to(gpu)
    r = rows(7, xt, 1, hidden).to(gpu)
    bias = rows(8, "f32", E, scale=0.1).to(gpu) if E % 3 == 0 else None
    for kw in ({}, dict(score="sigmoid", renormalise=False, scale=2.5)):
        want, ids, w = L.parts(q4lib, x, logits, topk, act=act, residual=r, bias=bias, **kw)
        ids2, w2 = torch.full_like(ids, 99), torch.full_like(w, 99.0)
        y = L.whole(q4lib, x, logits, topk, act=act, residual=r, bias=bias, ids=ids2, weights=w2, **kw)
        assert torch.equal(bits(y), bits(want)) and torch.equal(ids, ids2) and torch.equal(w, w2)
        yin = r.clone()  # in place
        L.whole(q4lib, x, logits, topk, act=act, residual=yin, y=yin, bias=bias, **kw)
        assert torch.equal(bits(yin), bits(want))


@pytest.mark.parametrize("xt,yt", [("f16", "f32"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("groups,kw", [(1, {}), (4, dict(group_topk=2)),
                                       (4, dict(group_topk=2, group_score="top2", score="sigmoid"))])
def test_one_token_masks_and_groups(q4lib, gpu, xt, yt, groups, kw):
    """Experts masked by -inf and NaN, fewer left than are asked for, none at all."""
    E, topk = 32, 6
    L = Layer(gpu, E, 512, 192, xt, seed=3)
    x = rows(5, xt, 1, 512).to(gpu)
    base = rows(6, "f32", 1, E, scale=2.0)
    few = torch.full((1, E), -math.inf)
    few[0, 9], few[0, 20], few[0, 21] = 1.0, math.nan, -torch.finfo(torch.float32).max
    odd = base.clone()
    odd[0, ::3], odd[0, 1::5], odd[0, 7] = -math.inf, math.nan, math.inf
    for logits in (base, few, odd, torch.full((1, E), -math.inf), torch.full((1, E), math.nan)):
        l = logits.to(gpu)
        want, ids, w = L.parts(q4lib, x, l, topk, groups=groups, y_dtype=TYPES[yt], **kw)
        assert torch.equal(ids.cpu(), route64(logits, topk, groups=groups, **kw)[0])
        y = L.whole(q4lib, x, l, topk, groups=groups, y_dtype=TYPES[yt], **kw)
        assert torch.equal(bits(y), bits(want))
        if (ids < 0).all():
            assert not y.any()


# ------------------------------------------------------------------ graphs, streams

@pytest.mark.parametrize("m,xt", [(1, "f16"), (6, "bf16"), (48, "f16"), (300, "bf16")])
def test_layer_captured_and_replayed(q4lib, gpu, m, xt):
    """Fused projections and expert layers in one graph,
    replayed on new inputs with eager work in between: the eager calls' bits."""
    E, topk, hidden, inter = 16, 4, 512, 320
    L = Layer(gpu, E, hidden, inter, xt, seed=11)
    wq, _ = weights(21, 3 * hidden, hidden)
    wo, _ = weights(22, hidden, 3 * hidden)
    router, _ = weights(23, E, hidden)
    wq, wo, router = wq.to(gpu), wo.to(gpu), router.to(gpu)

    def step(x):
        q = q4lib.q4_linear(x, wq, activation="silu")
        x = q4lib.q4_linear(q, wo, residual=x)
        logits = q4lib.q4_linear(x, router, y_dtype=torch.float32)
        ids, w, plan = q4lib.q4_route(logits, topk)
        h = q4lib.q4_experts(x, L.up, plan, bias=L.ub, activation="silu", gated=True)
        y = q4lib.q4_experts(h, L.down, plan, weights=w, residual=x)
        return L.whole(q4lib, y, logits, topk, residual=y), ids

    xs = [rows(30 + i, xt, m, hidden).to(gpu) for i in range(4)]
    want = [tuple(t.clone() for t in step(x)) for x in xs]
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(static)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, ids = step(static)
    for i in (1, 0, 3, 2, 2):
        static.copy_(xs[i])
        g.replay()
        step(xs[(i + 1) % 4])  # eager work over other memory
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want[i][0])) and torch.equal(ids, want[i][1])


def test_two_streams_at_once(q4lib, gpu):
    """The same layer on two streams, given as a stream and as a handle, and on the
    current one: every call has its own workspace."""
    E, topk, hidden, inter = 16, 2, 512, 256
    L = Layer(gpu, E, hidden, inter, "bf16", seed=41)
    wl, _ = weights(42, 1024, hidden)
    wl = wl.to(gpu)
    xs = {m: rows(50 + m, "bf16", m, hidden).to(gpu) for m in (1, 5, 40, 300)}
    ls = {m: rows(60 + m, "f32", m, E).to(gpu) for m in xs}
    lin = {m: q4lib.q4_linear(xs[m], wl, activation="gelu", gated=True) for m in xs}
    moe = {m: L.whole(q4lib, xs[m], ls[m], topk, residual=xs[m]) for m in xs}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(3):
        got = []
        for turn in range(4):
            for s in (streams[0], streams[1].cuda_stream, None):
                for m in xs:
                    got.append((lin[m], q4lib.q4_linear(xs[m], wl, activation="gelu", gated=True, stream=s)))
                    got.append((moe[m], L.whole(q4lib, xs[m], ls[m], topk, residual=xs[m], stream=s)))
        torch.cuda.synchronize()
        for want, y in got:
            assert torch.equal(bits(y), bits(want))
    ids, w, plan = q4lib.q4_route(ls[5], topk, stream=streams[0])
    plan2 = q4lib.q4_route_plan(ids, E, stream=streams[0])
    y = q4lib.q4_experts(xs[5], L.up, plan2, activation="silu", gated=True, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(plan.offsets, plan2.offsets) and torch.equal(plan.order, plan2.order)
    assert torch.equal(bits(y), bits(q4lib.q4_experts(xs[5], L.up, plan, activation="silu", gated=True)))


# ------------------------------------------------------------------ infinities

@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(1, 40, 96), (4, 130, 512), (20, 64, 1024), (60, 140, 320), (130, 300, 1024)])
def test_rows_with_an_infinity_or_nan(q4lib, gpu, m, n, k, xt):
    """An infinity gives every output its own infinity (NaN where the weight is 0),
    whatever finite values stand beside it; a NaN gives NaN; other rows are as ever."""
    packed, w = weights(m, n, k)
    x = rows(m + 1, xt, m, k)
    x[0, 7] = math.inf
    if xt != "f16":
        x[0, 20:30] = 1e30
    if m > 3:
        x[2, k - 1] = -math.inf
        x[3, 5] = math.nan
    with_inf = x.double() @ w.T
    y = q4lib.q4_linear(dev(x, gpu), dev(packed, gpu), y_dtype=torch.float32).cpu()
    for i in (0, 2, 3) if m > 3 else (0,):
        assert torch.equal(y[i].isnan(), with_inf[i].isnan()), i
        ok = ~with_inf[i].isnan()
        assert torch.equal(y[i][ok].double(), with_inf[i][ok]), i
    rest = [i for i in range(m) if i not in (0, 2, 3)]
    if rest:
        v, err = finish64(*product64(x[rest], w, None, "none", False, rounded=m > 32 and xt != "f32",
                                     scaled=xt == "bf16"), None, torch.float32)
        check(y[rest], v, err)
    # the same rows as an expert's
    ids = torch.zeros((m, 1), dtype=torch.int32, device=gpu)
    e = q4lib.q4_experts(dev(x, gpu), dev(packed, gpu)[None], q4lib.q4_route_plan(ids, 1),
                         y_dtype=torch.float32).cpu()
    for i in (0, 2, 3) if m > 3 else (0,):
        assert torch.equal(e[i].isnan(), with_inf[i].isnan()), i
        assert torch.equal(e[i].nan_to_num(0, 1, -1), y[i].nan_to_num(0, 1, -1)), i


# ------------------------------------------------------------------ large

@pytest.mark.parametrize("m,xt", [(3, "f16"), (40, "bf16"), (70, "f16")])
@pytest.mark.parametrize("gated", [False, True])
def test_weights_of_more_than_4_gib(q4lib, gpu, m, xt, gated):
    """Rows at both ends of a layer whose packed weights pass 32-bit offsets."""
    n, k, part = 1 << 20, 7680, 1024
    some, w = weights(71, part, k)
    packed = torch.empty((n, k // 32 * 18), dtype=torch.uint8, device=gpu)
    assert packed.numel() > 1 << 32
    packed.view(n // part, part, -1).copy_(some.to(gpu)[None])
    x = rows(72, xt, m, k)
    y = q4lib.q4_linear(dev(x, gpu), packed, activation="silu", gated=gated)
    # rows repeat every `part` columns, and so do the outputs
    ww = torch.cat([w, w]) if gated else w
    v, err = finish64(*product64(x, ww, None, "silu", gated, rounded=m > 32, scaled=xt == "bf16"), None, TYPES[xt])
    check(y[:, :part], v, err)
    first = y[:, :part]
    for c in range(0, y.shape[1], part):
        got = y[:, c:c + part]
        if not torch.equal(got, first):  # another tile's split of k: other sums
            check(got, v, err, f"columns {c}")


def test_rows_of_more_than_4_gib(q4lib, gpu):
    """Expert rows gathered and written beyond 32-bit offsets."""
    E, n, k, m, topk = 2, 64, 4096, 263168, 2
    packed, w = weights(81, E, n, k)
    some = rows(82, "f16", 512, k)
    x = some.to(gpu).repeat(m * topk // 512, 1)
    assert x.numel() * 2 > 1 << 32
    ids = torch.tensor([[0, 1], [1, 0], [1, 1], [0, -1]], dtype=torch.int32).repeat(m // 4, 1)
    plan = q4lib.q4_route_plan(ids.to(gpu), E)
    y = torch.zeros((m * topk, n), dtype=torch.float16, device=gpu)
    q4lib.q4_experts(x, packed.to(gpu), plan, y=y)
    for at in (0, m * topk // 512 // 2 * 512, m * topk - 512):
        e = ids.flatten()[at:at + 512]
        both = [finish64(*product64(some, w[i], None, "none", False, rounded=True), None, torch.float16)
                for i in range(E)]
        v = torch.where((e == 0)[:, None], both[0][0], both[1][0]) * (e >= 0)[:, None]
        err = torch.where((e == 0)[:, None], both[0][1], both[1][1]) * (e >= 0)[:, None]
        check(y[at:at + 512], v, err, f"rows {at}")
    assert torch.equal(y[:512], y[-512:])
