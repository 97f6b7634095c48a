"""CPU checks of the fused layers at calls that once went wrong."""

import shutil
import subprocess

import pytest

from test_fused_abi import A, B, BIG, C, D, E_, F16, F32, BF16, SHAPE, W, ep, routing


# ------------------------------------------------------------------ grids

def test_products_that_no_grid_holds_are_refused_before_any_launch(q4lib):
    """Where a later launch of the call does not fit, the earlier ones (staging, the
    products before their sum) are not made either: SHAPE, not a failed launch, and
    no workspace size."""
    L = q4lib.lib()
    tall = 1 << 25  # 131072 tiles of 256 rows
    for dt in (F16, BF16):
        assert q4lib.q4_linear_workspace_size(tall, 64, 64, dt) == 0
        assert L.q4_linear(A << 8, dt, B << 8, ep(q4lib), C << 8, dt, tall, 64, 64, W << 8, BIG, None) == SHAPE
    # 2^24 pairs: 87389 tiles of 192; 2^23 sums of 2560 columns: 3 2^31 threads
    for m, topk, E, n, combine in ((1 << 21, 8, 8, 64, False), (1 << 21, 8, 8, 64, True), (1 << 23, 1, 1, 2560, True)):
        for dt in (F16, BF16):
            rows = m * topk
            assert q4lib.q4_route_plan_size(m, topk, E) > 0
            assert q4lib.q4_experts_workspace_size(m, topk, E, n, 64, rows, dt, combine=combine) == 0
            x, w, p, g, y, ws = (v << 12 for v in (A, B, C, D, E_, W))
            assert L.q4_experts(x, dt, rows, w, ep(q4lib), p, g if combine else None, y, dt, m, topk, E, n, 64, ws,
                                BIG, None) == SHAPE


@pytest.mark.parametrize("m,topk,hidden,inter", [(1 << 21, 8, 64, 64), (1 << 23, 1, 2560, 64)])
def test_layers_that_no_grid_holds_are_refused_before_the_routing(q4lib, m, topk, hidden, inter):
    L, E = q4lib.lib(), 8
    assert q4lib.q4_moe_workspace_size(m, topk, E, hidden, inter, BF16) == 0
    x, l, u, d, y, ws = (v << 12 for v in (A, B, C, D, E_, W))
    args = (x, BF16, l, F32, routing(q4lib), u, ep(q4lib, act=4, gated=1), d, None, y, BF16, m, topk, E, hidden, inter)
    assert L.q4_moe(*args, None, None, ws, BIG, None) == SHAPE
    assert L.q4_moe(*args, None, None, None, 0, None) == SHAPE


def test_products_that_grids_hold_keep_their_sizes(q4lib):
    assert q4lib.q4_linear_workspace_size(1 << 23, 64, 64, BF16) >= (1 << 23) * 128
    assert q4lib.q4_experts_workspace_size(1 << 20, 8, 8, 64, 64, 1 << 20, BF16) >= (1 << 20) * 128
    assert q4lib.q4_moe_workspace_size(1 << 20, 8, 8, 64, 64, F16) > 0
    assert q4lib.q4_moe_workspace_size(1, 8, 64, 2048, 768, F16) > 0


# ------------------------------------------------------------------ 32-bit offsets

def test_matrices_that_end_at_4_gib_leave_the_32_bit_offsets(q4lib):
    """Rows that fill 2^32 - 4 bytes: an expert that starts 12 bytes into a 16-byte
    piece reaches its last row by offsets of 2^32 and more from that piece.  The
    decode kernels, whose offsets have 32 bits, stage bf16 rows; the row kernel, with
    64, takes them as they are."""
    n, k = 349867, 21824
    assert n * (k // 32 * 18) == (1 << 32) - 4
    size = q4lib.q4_experts_workspace_size
    assert size(64, 1, 4, n - 1, k, 64, BF16) >= 64 * k * 2
    assert size(64, 1, 4, n, k, 64, BF16) == 0


# ------------------------------------------------------------------ plans

def test_words_that_are_no_plan_of_those_sizes_are_refused(q4lib):
    """The full way from Python (an output of the caller's) took any words."""
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.float16)
    packed, y = torch.zeros(8, 32, 36, dtype=torch.uint8), torch.zeros(8, 32, dtype=torch.float16)
    words = q4lib.q4_route_plan_size(4, 2, 8) // 4
    for plan in (q4lib.Plan(torch.zeros(3, dtype=torch.int32), 4, 2, 8),
                 q4lib.Plan(torch.zeros(words, dtype=torch.int64), 4, 2, 8),
                 q4lib.Plan(torch.zeros(words, dtype=torch.int32), 400, 2, 8),
                 q4lib.Plan(torch.zeros(0, dtype=torch.int32), 0, 2, 8)):
        with pytest.raises(ValueError, match="plan of"):
            q4lib.q4_experts(x, packed, plan, y=y)
        with pytest.raises(ValueError, match="plan of"):
            q4lib.q4_experts(x, packed, plan)
    with pytest.raises(ValueError, match="device tensor"):
        q4lib.q4_experts(x, packed, q4lib.Plan(torch.zeros(words, dtype=torch.int32), 4, 2, 8), y=y)


# ------------------------------------------------------------------ older libraries

@pytest.mark.skipif(shutil.which("gcc") is None, reason="gcc not available")
def test_a_library_older_than_the_binding_is_named_as_such(q4lib, monkeypatch, tmp_path):
    """One of the same ABI version without the fused calls, and one of another version."""
    def library(name, functions, version):
        text = f"int q4_abi_version(void) {{ return {version}; }}\n" + "".join(
            f"int {f}(void) {{ return 0; }}\n" for f in functions if f != "q4_abi_version")
        (tmp_path / (name + ".c")).write_text(text)
        so = tmp_path / (name + ".so")
        subprocess.run(["gcc", "-shared", "-fPIC", str(tmp_path / (name + ".c")), "-o", str(so)], check=True)
        return so

    every = list(q4lib._SIGS)
    monkeypatch.setattr(q4lib, "_LIB", None)
    for so, match in ((library("old", [f for f in every if f != "q4_moe"], 1), "no q4_moe.*rebuild"),
                      (library("other", every, 99), "ABI version mismatch")):
        monkeypatch.setattr(q4lib, "LIB_PATH", so)
        with pytest.raises(q4lib.Q4LibraryMissing, match=match):
            q4lib.lib()


# ------------------------------------------------------------------ gradients

def test_tensors_that_need_a_gradient_are_refused(q4lib):
    torch = pytest.importorskip("torch")
    x, r = torch.zeros(4, 64), torch.zeros(4, 8)
    packed, up, down = (torch.zeros(*s, dtype=torch.uint8) for s in ((8, 36), (8, 64, 36), (8, 64, 18)))
    logits, plan = torch.zeros(4, 8), q4lib.Plan(torch.zeros(q4lib.q4_route_plan_size(4, 2, 8) // 4,
                                                             dtype=torch.int32), 4, 2, 8)
    needs = {n: t.clone().requires_grad_() for n, t in dict(x=x, r=r, logits=logits, bias=torch.zeros(8)).items()}
    calls = {"x linear": lambda: q4lib.q4_linear(needs["x"], packed),
             "x full way": lambda: q4lib.q4_linear(needs["x"], packed, y_dtype=torch.float32),
             "residual": lambda: q4lib.q4_linear(x, packed, residual=needs["r"]),
             "bias": lambda: q4lib.q4_linear(x, packed, bias=needs["bias"]),
             "logits": lambda: q4lib.q4_route(needs["logits"], 2),
             "weights": lambda: q4lib.q4_experts(x, up, plan, weights=torch.zeros(4, 2, requires_grad=True)),
             "x experts": lambda: q4lib.q4_experts(needs["x"], up, plan),
             "moe": lambda: q4lib.q4_moe(x, needs["logits"], up, down, 2)}
    for name, f in calls.items():
        with pytest.raises(RuntimeError, match="part in a gradient"):
            f()
        with torch.no_grad(), pytest.raises(ValueError, match="device tensor"):  # as ever
            f()
    with torch.autograd.forward_ad.dual_level():
        dual = torch.autograd.forward_ad.make_dual(x, torch.ones_like(x))
        with pytest.raises(RuntimeError, match="part in a gradient"):
            q4lib.q4_linear(dual, packed)
