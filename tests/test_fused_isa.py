"""CPU checks on the compiled kernels of the fused layers: those launched with
dynamic LDS have none of their own beside it, and no register is used before the
load that writes it has been waited for."""

import pytest

from isa_check import kernels, load_hazards, metadata
from test_isa import HIPCC, asm, pytestmark  # noqa: F401


@pytest.mark.parametrize("src,pattern", [("q4_fused_gemv.hip", "fused_gemv_kernel"),
                                         ("q4_fused_wave.hip", "fused_"),
                                         ("q4_moe_one.hip", "moe_one_")])
def test_dynamic_lds_kernels_have_no_static_lds(src, pattern):
    """They may ask for all 160 KB of a compute unit."""
    meta = metadata(asm(src))
    names = [nm for nm in meta if pattern in nm]
    assert names, pattern
    for nm in names:
        assert meta[nm]["group_segment_fixed_size"] == 0, nm


def test_static_lds_fits():
    """The routing's single workgroup and the prefill tiles, within 160 KB."""
    for src in ("q4_route.hip", "q4_fused_gemm.hip"):
        for name, m in metadata(asm(src)).items():
            assert m["group_segment_fixed_size"] <= 160 * 1024, name


def own_loads(body):
    """The loads of inline assembly, which the compiler does not wait for."""
    inside, out = False, set()
    for line in body:
        if "#ASMSTART" in line:
            inside = True
        elif "#ASMEND" in line:
            inside = False
        elif inside and "global_load" in line and "_lds_" not in line:
            out.add(line.split(";")[0].strip())
    return out


def test_no_register_used_before_its_load_lands():
    """(Loads in branches of which one runs, one per type, are the compiler's own;
    joining them the pass cannot tell that only one is in flight.)"""
    ks = kernels(asm("q4_fused_gemm.hip"), "fused_")
    assert any(own_loads(body) for _, body in ks)
    for name, body in ks:
        assert not own_loads(body) & {str(h) for h in load_hazards(body)}, name


@pytest.mark.parametrize("src", ["q4_fused_wave.hip", "q4_moe_one.hip", "q4_fused_gemv.hip", "q4_route.hip"])
def test_own_loads_go_to_lds_alone(src):
    for name, body in kernels(asm(src), "kernel"):
        assert not own_loads(body), name
