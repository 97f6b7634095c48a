"""CPU checks on the compiled kernels of the fused layers: those launched with
dynamic LDS have none of their own beside it, and no register is used before the
load that writes it has been waited for."""

import re

import pytest

from isa_check import kernels, load_hazards, metadata
from test_isa import CSRC, HIPCC, asm, pytestmark  # noqa: F401


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


def scalar_address_hazards(body):
    """Vector memory instructions that take their scalar address from a register
    that a vector instruction wrote fewer than five wait states before: hardware
    does not wait, and the compiler does not either for inline assembly."""
    out, recent = [], []
    for line in body:
        t = line.split(";")[0].strip()
        if not t or t.startswith(".") or t.endswith(":"):
            continue
        if t.startswith("global_"):
            need = {r for a, b in re.findall(r"s\[(\d+):(\d+)\]", t) for r in range(int(a), int(b) + 1)}
            states = 0
            for p in reversed(recent):
                w = re.match(r"v_read(?:first)?lane_b32 s(\d+)", p)
                if states < 5 and w and int(w.group(1)) in need:
                    out.append((p, t))
                n = re.match(r"s_nop (\d+)", p)
                states += int(n.group(1)) + 1 if n else 1
        recent = (recent + [t])[-8:]
    return out


def test_the_scan_finds_a_scalar_address_hazard():
    load = "global_load_lds_dwordx4 v2, s[6:7]"
    assert scalar_address_hazards(["v_readlane_b32 s7, v69, 1", load])
    assert scalar_address_hazards(["v_readfirstlane_b32 s6, v1", "s_nop 3", load])
    assert not scalar_address_hazards(["v_readlane_b32 s7, v69, 1", "s_nop 4", load])
    assert not scalar_address_hazards(["v_readlane_b32 s8, v69, 1", load])


@pytest.mark.parametrize("src", sorted(p.name for p in CSRC.glob("*.hip") if p.name != "q4_api.hip"))
def test_scalar_addresses_have_settled(src):
    for name, body in kernels(asm(src), ""):
        assert not scalar_address_hazards(body), name
