"""The fused linear layer and the experts against 64-bit forms, at the sizes,
types and masks where they can go wrong."""

import numpy as np
import pytest
import torch

from _fused import (TYPES, check, experts64, finish64, plan64, product64, route64, rows, weights)

pytestmark = pytest.mark.gpu


def dev(t, gpu):
    return None if t is None else t.to(gpu)


def run_linear(q4lib, gpu, m, n, k, xt, yt=None, act="none", gated=False, bias=None, residual=False,
               inplace=False, seed=0, scale=1.0):
    yt = yt or xt
    packed, w = weights(seed + 1, n, k)
    x = rows(seed + 2, xt, m, k, scale=scale)
    nout = n // 2 if gated else n
    b = rows(seed + 3, bias, n, scale=0.3) if bias else None
    r = rows(seed + 4, yt, m, nout) if residual else None
    kw = {}
    if inplace:
        kw["y"] = kw["residual"] = dev(r, gpu).clone()
    else:
        kw["residual"] = dev(r, gpu)
    y = q4lib.q4_linear(dev(x, gpu), dev(packed, gpu), bias=dev(b, gpu), activation=act, gated=gated,
                        y_dtype=TYPES[yt], **kw)
    assert y.dtype == TYPES[yt]
    v, err = product64(x, w, b, act, gated, rounded=m > 32 and xt != "f32", scaled=xt == "bf16")
    v, err = finish64(v, err, r, TYPES[yt])
    check(y, v, err, f"m{m} n{n} k{k} {xt}->{yt} {act} gated={gated}")
    return y


SIZES = [(1, 1, 32), (1, 7, 96), (1, 512, 512), (2, 66, 64), (3, 130, 128), (5, 34, 1056), (8, 96, 256),
         (10, 516, 512), (16, 260, 1408), (17, 200, 1024), (31, 1028, 512), (32, 70, 704), (33, 130, 512),
         (40, 258, 96), (64, 96, 544), (127, 300, 1024), (128, 128, 256), (257, 516, 1088), (300, 260, 2048)]


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_plain_sizes(q4lib, gpu, m, n, k, xt):
    run_linear(q4lib, gpu, m, n, k, xt, seed=m + n + k)


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(m, n + n % 2, k) for m, n, k in SIZES])
def test_linear_gated_sizes(q4lib, gpu, m, n, k, xt):
    run_linear(q4lib, gpu, m, n, k, xt, act="silu", gated=True, bias=xt, residual=True, seed=m + n + k + 7)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_erf", "silu"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [1, 6, 20, 150])
def test_linear_activations(q4lib, gpu, m, act, gated):
    run_linear(q4lib, gpu, m, 136, 512, "f16", act=act, gated=gated, bias="f16", seed=m, scale=3.0)


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("yt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("bt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m", [2, 70])
def test_linear_types(q4lib, gpu, m, xt, yt, bt):
    run_linear(q4lib, gpu, m, 96, 256, xt, yt, act="gelu", bias=bt, residual=True, seed=11)


@pytest.mark.parametrize("m", [1, 12, 32, 64, 200])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_in_place_residual(q4lib, gpu, m, gated):
    run_linear(q4lib, gpu, m, 264, 512, "bf16", act="silu", gated=gated, residual=True, inplace=True, seed=m)


@pytest.mark.parametrize("xt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n,k", [(3, 70, 512), (70, 200, 96), (150, 300, 512), (300, 516, 1024), (1030, 260, 320)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_scales_beyond_fp16(q4lib, gpu, m, n, k, xt, gated):
    """Block scales whose largest weight is beyond fp16 (80000): only some tiles
    meet them, and the residual is y itself, which those must find unchanged."""
    import oracle
    from _fused import decode
    rng = np.random.default_rng(m)
    w = (rng.standard_normal((n, k)) * 0.05).astype(np.float32)
    w[n // 2 + 3, 5] = 80000.0
    w[1, k - 3] = -90000.0
    packed = oracle.quantize(w)
    x = rows(1, xt, m, k)
    nout = n // 2 if gated else n
    r = rows(2, "f32", m, nout)
    y = dev(r, gpu).clone()
    q4lib.q4_linear(dev(x, gpu), dev(torch.from_numpy(packed), gpu), activation="relu", gated=gated, residual=y, y=y)
    v, err = product64(x, torch.from_numpy(decode(packed, n, k)), None, "relu", gated, rounded=m > 32, scaled=xt == "bf16")
    v, err = finish64(v, err, r, torch.float32)
    check(y, v, err, f"m{m} n{n} k{k} {xt}")


@pytest.mark.parametrize("m", [4, 200])
@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e25])
def test_linear_bf16_rows_of_any_magnitude(q4lib, gpu, m, scale):
    """bf16 rows far beyond fp16's range, rows of zeros, and rows that mix
    magnitudes: every row to its own precision."""
    n, k = 130, 512
    packed, w = weights(3, n, k)
    x = rows(4, "f32", m, k, scale=scale)
    x[1] = 0
    x[2] = 0
    x[2, 7] = scale
    x[3, ::2] *= 1e-4
    x[3, 5] = 1e-13 * scale  # below 2^-32 of the row's largest
    x = x.to(torch.bfloat16)
    y = q4lib.q4_linear(dev(x, gpu), dev(packed, gpu), y_dtype=torch.float32)
    v, err = product64(x, w, None, "none", False, rounded=m > 32, scaled=True)
    v, err = finish64(v, err, None, torch.float32)
    check(y, v, err + 1e-42, f"m{m} scale {scale}")


@pytest.mark.parametrize("m,n,k", [(10, 33290, 512), (9, 45000, 256), (16, 28004, 320), (14, 40000, 128),
                                   (32, 17000, 512), (20, 30000, 128), (4, 9000, 1024), (2, 5120, 2048),
                                   (12, 20480, 192), (7, 12288, 4160), (10, 34816, 64)])
@pytest.mark.parametrize("gated", [False, True])
def test_linear_decode_row_tiles(q4lib, gpu, m, n, k, gated):
    """Wide layers: every number of row tiles per workgroup, both ring depths,
    two workgroups per compute unit, several rounds; short last phases."""
    run_linear(q4lib, gpu, m, n, k, "f16" if m % 2 else "bf16", act="silu", gated=gated, residual=True, seed=m)


def test_both_ways_from_python_agree_and_refuse_alike(q4lib, gpu):
    """A call with an output of the caller's takes the full way, one without the
    native way: the same bits.  Calls that neither may take raise."""
    packed, _ = weights(1, 96, 256)
    x, b, r = rows(2, "f16", 5, 256), rows(3, "f16", 96), rows(4, "f16", 5, 48)
    pd, xd, bd, rd = dev(packed, gpu), dev(x, gpu), dev(b, gpu), dev(r, gpu)
    kw = dict(bias=bd, activation="silu", gated=True, residual=rd)
    want = q4lib.q4_linear(xd, pd, y=torch.empty_like(rd), **kw)
    assert torch.equal(q4lib.q4_linear(xd, pd, **kw), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        on_side = q4lib.q4_linear(xd, pd, **kw)
    torch.cuda.synchronize()
    assert torch.equal(on_side, want)
    for bad, err in ((dict(bias=bd[:-1]), ValueError), (dict(activation="tanh"), ValueError),
                     (dict(residual=rd.float()), ValueError), (dict(residual=rd.t()), ValueError),
                     (dict(bias=b), ValueError)):
        with pytest.raises(err):
            q4lib.q4_linear(xd, pd, **{**kw, **bad})
    with pytest.raises(ValueError):
        q4lib.q4_linear(xd[:, ::2], pd, **kw)
    with pytest.raises(TypeError):
        q4lib.q4_linear(xd, pd.view(torch.int8), **kw)
    with pytest.raises(q4lib.Q4Error):
        q4lib.q4_route(dev(rows(5, "f32", 3, 8), gpu), 9)
    with pytest.raises(q4lib.Q4Error):
        q4lib.q4_route(dev(rows(5, "f32", 3, 9), gpu), 2, groups=2)


@pytest.mark.parametrize("m,n,k", [(1, 4112, 2112), (2, 8192, 320), (8, 514, 2048), (4, 4096, 4160), (3, 8180, 704),
                                   (1, 16, 16384), (7, 100, 8192), (5, 2050, 1088), (1, 8194, 576), (6, 34, 2304)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("xt", ["f16", "bf16"])
def test_linear_rows_split_over_wavefronts(q4lib, gpu, m, n, k, gated, xt):
    """Narrow layers: parts of k of unequal length, a short last chunk, fewer chunks
    than wavefronts, one and two row tiles per compute unit and just more."""
    run_linear(q4lib, gpu, m, n, k, xt, act="silu", gated=gated, bias=xt, residual=True, seed=m + k)
    run_linear(q4lib, gpu, m, n, k, xt, "f32", gated=gated, inplace=True, residual=True, seed=m)


@pytest.mark.parametrize("m", [1, 4, 10, 32])
@pytest.mark.parametrize("yt", ["f16", "f32"])
def test_plain_products_are_the_decode_gemv(q4lib, gpu, m, yt):
    packed, _ = weights(m, 130, 608)
    x, pd = rows(m + 1, "f16", m, 608).to(gpu), packed.to(gpu)
    want = q4lib.q4_gemv(x, pd, y_dtype=TYPES[yt])
    assert torch.equal(q4lib.q4_linear(x, pd, y_dtype=TYPES[yt]), want)
