"""The fused layers at calls that once went wrong or slow."""

import pytest
import torch

from _fused import rows, weights

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ plain products

@pytest.mark.parametrize("m,n,k", [(10, 300, 1408), (3, 2048, 896), (32, 132, 704), (17, 64, 768), (4, 4864, 896),
                                   (1, 8192, 1280), (2, 4112, 2112)])
def test_plain_products_that_the_decode_gemv_takes_slowly(q4lib, gpu, m, n, k):
    """Where q4_gemv has no matrix-core kernel (k % 512 != 0) a plain product runs as
    one with an epilogue does: the same sums (10 rows of 2048 x 1408: 9.2 -> 4.8 us)."""
    packed, _ = weights(m, n, k)
    x, pd = rows(m + 1, "f16", m, k).to(gpu), packed.to(gpu)
    none = torch.zeros(n, dtype=torch.float32, device=gpu)
    y = q4lib.q4_linear(x, pd, y_dtype=torch.float32)
    assert torch.equal(y, q4lib.q4_linear(x, pd, bias=none, y_dtype=torch.float32))


@pytest.mark.parametrize("m,n,k", [(1, 130, 512), (10, 300, 1024), (32, 64, 1536), (1, 2048, 1408), (2, 1000, 8640),
                                   (16, 4096, 768), (5, 130, 96)])
def test_plain_products_that_stay_the_decode_gemvs(q4lib, gpu, m, n, k):
    packed, _ = weights(m, n, k)
    x, pd = rows(m + 1, "f16", m, k).to(gpu), packed.to(gpu)
    for yt in (torch.float16, torch.float32):
        assert torch.equal(q4lib.q4_linear(x, pd, y_dtype=yt), q4lib.q4_gemv(x, pd, y_dtype=yt))


# ------------------------------------------------------------------ gradients

def test_device_tensors_that_need_a_gradient_are_refused(q4lib, gpu):
    """By the native way from Python too; under no_grad the result is the same as ever."""
    packed, _ = weights(1, 64, 256)
    x, pd, r = rows(2, "f16", 5, 256).to(gpu), packed.to(gpu), rows(3, "f16", 5, 64).to(gpu)
    want = q4lib.q4_linear(x, pd, residual=r)
    xg, rg = x.clone().requires_grad_(), r.clone().requires_grad_()
    for a, b in ((xg, r), (x, rg)):
        with pytest.raises(RuntimeError, match="part in a gradient"):
            q4lib.q4_linear(a, pd, residual=b)
        with torch.no_grad():
            y = q4lib.q4_linear(a, pd, residual=b)
        assert torch.equal(y, want) and not y.requires_grad
        with torch.inference_mode():
            assert torch.equal(q4lib.q4_linear(a, pd, residual=b), want)
    logits = rows(4, "f32", 3, 8).to(gpu).requires_grad_()
    with pytest.raises(RuntimeError, match="part in a gradient"):
        q4lib.q4_route(logits, 2)
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="part in a gradient"):
            q4lib.q4_linear(dual, pd, residual=r)
