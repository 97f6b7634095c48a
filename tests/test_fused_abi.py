"""Refusals of the fused layers, the routing and the experts, and their sizes:
all of it on the host, before anything is launched."""

import ctypes
import math

import pytest

OK, INVALID, SHAPE, DTYPE, ALIGN, HIP, WORKSPACE = range(7)
F32, F16, BF16 = 0, 1, 2
A, B, C, D, W = 0x100000000, 0x200000000, 0x300000000, 0x400000000, 0x500000000
E_, F_, G_ = 0x600000000, 0x700000000, 0x800000000
BIG = 1 << 62


def ep(q4, bias=None, bias_dtype=F16, act=0, gated=0, residual=None):
    return ctypes.byref(q4.Epilogue(bias, bias_dtype, act, gated, residual))


def test_linear_refusals(q4lib):
    L = q4lib.lib()

    def f(x=A, xt=F16, w=B, e=None, y=C, yt=F16, m=4, n=64, k=64, ws=W, wb=BIG):
        return L.q4_linear(x, xt, w, e, y, yt, m, n, k, ws, wb, None)

    assert f(x=None) == INVALID and f(w=None) == INVALID and f(y=None) == INVALID
    for kw in (dict(m=0), dict(m=-1), dict(n=0), dict(k=0), dict(k=48), dict(k=(1 << 24) + 32),
               dict(m=1 << 31), dict(n=1 << 31)):
        assert f(**kw) == SHAPE, kw
    assert f(xt=3) == DTYPE and f(yt=-1) == DTYPE and f(e=ep(q4lib, D, 7)) == DTYPE
    assert f(e=ep(q4lib, None, 7, residual=None), x=A + 8) == ALIGN   # the type of no bias is not read
    assert f(e=ep(q4lib, act=5)) == INVALID and f(e=ep(q4lib, act=-1)) == INVALID
    assert f(e=ep(q4lib, gated=2)) == INVALID
    assert f(e=ep(q4lib, gated=1), n=65) == SHAPE
    for kw in (dict(x=A + 2), dict(w=B + 8), dict(y=C + 4), dict(e=ep(q4lib, D + 8)),
               dict(e=ep(q4lib, residual=D + 4))):
        assert f(**kw) == ALIGN, kw
    assert f(y=A) == INVALID and f(y=B) == INVALID and f(y=A + 16) == INVALID
    assert f(e=ep(q4lib, C)) == INVALID                          # bias inside y
    assert f(e=ep(q4lib, residual=C + 16)) == INVALID            # a residual may be y, not overlap it
    assert f(e=ep(q4lib, residual=C), x=A + 2) == ALIGN          # (in place passes that check)


def test_linear_workspace(q4lib):
    size = q4lib.q4_linear_workspace_size
    L = q4lib.lib()
    for m, n, k, dt, gated in ((300, 512, 1024, BF16, False), (64, 1024, 17408, F16, False),
                               (2048, 34816, 5120, BF16, True)):
        need = size(m, n, k, dt, gated)
        if not need:
            continue
        e = ep(q4lib, gated=int(gated))
        assert L.q4_linear(A, dt, B, e, C, dt, m, n, k, None, 0, None) == WORKSPACE
        assert L.q4_linear(A, dt, B, e, C, dt, m, n, k, W, need - 1, None) == WORKSPACE
        assert L.q4_linear(A, dt, B, e, C, dt, m, n, k, W + 8, need, None) == ALIGN
        for over in (A, B, C):
            assert L.q4_linear(A, dt, B, e, C, dt, m, n, k, over, need, None) == INVALID
    for bad in ((0, 64, 64, F16), (4, 64, 40, F16), (4, 64, 64, 9)):
        assert size(*bad) == 0
    assert size(4, 65, 64, F16, True) == 0


def routing(q4, score=0, bias=None, groups=1, group_topk=1, group_score=0, renormalise=1, scale=1.0):
    return ctypes.byref(q4.Routing(score, bias, groups, group_topk, group_score, renormalise, scale))


def test_route_refusals(q4lib):
    L = q4lib.lib()

    def f(l=A, dt=F32, m=4, E=64, topk=4, r=None, ids=B, w=C, plan=D, **kw):
        return L.q4_route(l, dt, m, E, topk, r or routing(q4lib, **kw), ids, w, plan, None)

    assert f(l=None) == INVALID and f(ids=None) == INVALID and f(w=None) == INVALID
    assert L.q4_route(A, F32, 4, 64, 4, None, B, C, D, None) == INVALID
    for kw in (dict(m=0), dict(E=0), dict(E=1025), dict(topk=0), dict(topk=33), dict(topk=65), dict(E=3),
               dict(m=(1 << 24) + 1), dict(m=1 << 23), dict(groups=0), dict(groups=3), dict(groups=128),
               dict(groups=8, group_topk=9), dict(groups=8, group_topk=0)):
        assert f(**kw) == SHAPE, kw
    assert f(dt=3) == DTYPE
    for kw in (dict(score=2), dict(score=-1), dict(group_score=2), dict(renormalise=2), dict(scale=math.nan),
               dict(scale=math.inf)):
        assert f(**kw) == INVALID, kw
    assert f(l=A + 4) == ALIGN and f(ids=B + 4) == ALIGN and f(w=C + 8) == ALIGN and f(plan=D + 4) == ALIGN
    assert f(bias=E_ + 2) == ALIGN
    assert f(ids=A) == INVALID and f(w=B) == INVALID and f(plan=C) == INVALID and f(plan=A) == INVALID
    assert f(bias=D) == INVALID                                 # bias inside the plan


def test_plan_refusals_and_sizes(q4lib):
    L = q4lib.lib()
    assert L.q4_route_plan(None, 4, 2, 8, B, None) == INVALID
    assert L.q4_route_plan(A, 4, 2, 8, None, None) == INVALID
    for m, topk, E in ((0, 2, 8), (4, 0, 8), (4, 33, 64), (4, 2, 0), (4, 2, 1025), (1 << 24, 2, 8)):
        assert L.q4_route_plan(A, m, topk, E, B, None) == SHAPE
        assert q4lib.q4_route_plan_size(m, topk, E) == 0
    assert L.q4_route_plan(A + 4, 4, 2, 8, B, None) == ALIGN
    assert L.q4_route_plan(A, 4, 2, 8, A, None) == INVALID
    for m, topk, E in ((1, 1, 1), (16, 8, 128), (4096, 8, 256)):
        # at least the offsets and the order, in whole words
        size = q4lib.q4_route_plan_size(m, topk, E)
        assert size % 4 == 0 and size >= 4 * (E + 1 + m * topk)


def test_experts_refusals(q4lib):
    L = q4lib.lib()

    def f(x=A, xt=F16, xr=4, w=B, e=None, plan=D, g=None, y=C, yt=F16, m=4, topk=2, E=8, n=64, k=64, ws=W,
          wb=BIG):
        return L.q4_experts(x, xt, xr, w, e, plan, g, y, yt, m, topk, E, n, k, ws, wb, None)

    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(plan=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(xr=5), dict(m=0), dict(topk=0), dict(topk=33), dict(E=0), dict(E=2000), dict(n=0),
               dict(k=40), dict(e=ep(q4lib, gated=1), n=63)):
        assert f(**kw) == SHAPE, kw
    assert f(xt=4) == DTYPE and f(yt=4) == DTYPE
    for kw in (dict(x=A + 2), dict(w=B + 4), dict(y=C + 8), dict(plan=D + 8), dict(g=E_ + 4)):
        assert f(**kw) == ALIGN, kw
    for kw in (dict(y=D), dict(y=A), dict(y=B + 64), dict(g=C)):
        assert f(**kw) == INVALID, kw
    need = q4lib.q4_experts_workspace_size(4, 2, 8, 64, 64, 8, F16, combine=True)
    assert need >= 4 * 2 * 64 * 4 or need == 0
    if need:
        assert f(xr=8, g=E_, ws=None, wb=0) == WORKSPACE
        assert f(xr=8, g=E_, wb=need - 1) == WORKSPACE
        assert f(xr=8, g=E_, ws=E_) == INVALID


def test_moe_refusals(q4lib):
    L = q4lib.lib()

    def f(x=A, xt=F16, l=B, lt=F32, r=None, up=C, ue=True, down=D, de=None, y=E_, yt=F16, m=4, topk=2, E=8,
          hidden=64, inter=32, ids=None, w=None, ws=W, wb=BIG):
        ue = ep(q4lib, act=4, gated=1) if ue is True else ue
        return L.q4_moe(x, xt, l, lt, r or routing(q4lib), up, ue, down, de, y, yt, m, topk, E, hidden, inter,
                        ids, w, ws, wb, None)

    for kw in (dict(x=None), dict(l=None), dict(up=None), dict(down=None), dict(y=None), dict(ue=None)):
        assert f(**kw) == INVALID, kw
    for kw in (dict(inter=48), dict(hidden=40), dict(topk=9), dict(m=0), dict(inter=0)):
        assert f(**kw) == SHAPE, kw
    assert f(xt=3) == DTYPE and f(lt=3) == DTYPE and f(yt=3) == DTYPE
    assert f(ue=ep(q4lib, gated=1, residual=F_)) == INVALID     # nothing to add between the products
    assert f(de=ep(q4lib, act=4)) == INVALID and f(de=ep(q4lib, gated=1)) == INVALID
    assert f(ws=None, wb=0) == WORKSPACE
    need = q4lib.q4_moe_workspace_size(4, 2, 8, 64, 32, F16)
    assert need > 0 and f(wb=need - 1) == WORKSPACE
    for kw in (dict(ws=A), dict(ws=B), dict(ws=C), dict(ws=D), dict(ws=E_), dict(y=A), dict(y=C), dict(y=D),
               dict(ids=E_), dict(w=A), dict(ids=F_, w=F_), dict(de=ep(q4lib, residual=W)),
               dict(de=ep(q4lib, residual=E_ + 16))):
        assert f(**kw) == INVALID, kw
    for kw in (dict(x=A + 4), dict(l=B + 4), dict(ids=F_ + 4), dict(w=F_ + 8), dict(ws=W + 4), dict(y=E_ + 2)):
        assert f(**kw) == ALIGN, kw
    for bad in ((0, 2, 8, 64, 32, F16), (4, 9, 8, 64, 32, F16), (4, 2, 8, 64, 40, F16), (4, 2, 8, 64, 32, 5)):
        assert q4lib.q4_moe_workspace_size(*bad) == 0


def test_python_refusals(q4lib):
    """The binding's own checks: shapes, types and places, before any pointer is read."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.float16)
    packed = torch.zeros(8, 36, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_linear(x, packed)
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_route(torch.zeros(2, 8), 2)
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_route_plan(torch.zeros(2, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="activation"):
        q4lib._code(q4lib.ACTIVATIONS, "tanh", "activation")
    with pytest.raises(TypeError, match="uint8"):
        q4lib._need_packed(x)


def test_options_of_the_binding_match_the_header():
    import re
    from pathlib import Path
    import bit_block_quantized_q4_amd as q4
    text = (Path(__file__).resolve().parent.parent / "include" / "q4.h").read_text()
    for table, prefix in ((q4.ACTIVATIONS, "Q4_ACT_"), (q4.SCORES, "Q4_SCORE_"), (q4.GROUP_SCORES, "Q4_GROUP_")):
        named = {k.lower(): int(v) for k, v in re.findall(prefix + r"([A-Z0-9_]+) = (\d+)", text)}
        assert named == table
    assert f"#define Q4_MAX_EXPERTS {q4.MAX_EXPERTS}" in text and f"#define Q4_MAX_TOPK {q4.MAX_TOPK}" in text


def test_native_binding_leaves_what_it_does_not_take_to_python(q4lib):
    """The short way answers None (and the Python function raises) for host
    tensors, wrong shapes and options; nothing is launched."""
    torch = pytest.importorskip("torch")
    fast = q4lib._fast()
    assert fast is not None, "the native binding is built with the library"
    x, packed = torch.zeros(4, 64, dtype=torch.float16), torch.zeros(8, 36, dtype=torch.uint8)
    assert fast.linear(x, packed, None, 0, False, None) is None
    assert fast.linear(x, packed, None, None, False, None) is None
    assert fast.linear(None, packed, None, 0, False, None) is None
    assert fast.linear(x, 3, None, 0, False, None) is None
    assert fast.linear(x) is None
    assert fast.route(torch.zeros(2, 8), 2, None, 0, 1, 1, 0, True, 1.0) is None
    assert fast.route_plan(torch.zeros(2, 2, dtype=torch.int32), 8) is None
    assert fast.experts(x, packed, x, 4, 1, 2, None, 0, False, None, None) is None
    assert fast.moe(*([None] * 17)) is None
    with pytest.raises(TypeError):
        fast.bind()
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_linear(x, packed)


def test_more_workgroups_than_a_launch_holds(q4lib):
    """Refused by the launch rule itself, not cut to 32 bits."""
    L = q4lib.lib()
    far = ctypes.c_void_p
    rows_, base = 65536 * 128, 1 << 40
    x, w, y = far(base), far(base * 2), far(base * 3)
    assert L.q4_linear(x, F32, w, ep(q4lib), y, F32, rows_, 1, 32, None, 0, None) == SHAPE
    assert q4lib.q4_experts_workspace_size(1024, 32, 1024, 1 << 23, 32, 1024, F32) == 0
    plan = far(base * 4)
    assert L.q4_experts(x, F32, 1024, w, ep(q4lib), plan, None, y, F32, 1024, 32, 1024, 1 << 23, 32, None, 0,
                        None) == SHAPE
