"""CPU check on the compiled kernels: every copy into LDS lies its wait states behind
the instructions that wrote M0 and its scalar address."""

import pytest

from _wait_states import copies_too_early, kernels
from test_isa import CSRC, asm, pytestmark  # noqa: F401

COPY = "global_load_lds_dwordx4 v2, s[6:7]"
FLAT = "global_load_lds_dwordx4 v[2:3], off"


@pytest.mark.parametrize("src", sorted(p.name for p in CSRC.glob("*.hip") if p.name != "q4_api.hip"))
def test_copies_keep_their_wait_states(src):
    for name, body in kernels(asm(src), ""):
        assert not copies_too_early(body), name


def test_the_check_knows_a_write_of_m0():
    assert copies_too_early(["s_mov_b32 m0, s4", FLAT])
    assert copies_too_early(["s_add_i32 m0, s4, 0x400", COPY])
    assert not copies_too_early(["s_mov_b32 m0, s4", "s_nop 0", FLAT])
    assert not copies_too_early(["s_mov_b32 m0, s4", "s_mov_b64 s[6:7], s[8:9]", COPY])
    assert copies_too_early(["v_readfirstlane_b32 m0, v4", "s_nop 3", FLAT])
    assert not copies_too_early(["v_readfirstlane_b32 m0, v4", "s_nop 4", FLAT])


def test_the_check_knows_a_vector_write_of_the_address():
    for write in ("v_readlane_b32 s7, v69, 1", "v_readfirstlane_b32 s6, v1", "v_cmp_lt_u32_e64 s[6:7], v1, v2",
                  "v_add_co_u32_e64 v1, s[6:7], v2, v3"):
        assert copies_too_early([write, COPY]), write
        assert copies_too_early([write, "s_nop 3", COPY]), write
        assert not copies_too_early([write, "s_nop 4", COPY]), write
        assert not copies_too_early([write, "s_mov_b64 s[6:7], s[6:7]", COPY]), write
    assert not copies_too_early(["v_readlane_b32 s8, v69, 1", COPY])
    assert not copies_too_early(["v_readlane_b32 s7, v69, 1", FLAT])


def test_the_check_follows_loops_and_branches():
    loop = ["s_mov_b32 m0, s4", "s_nop 0", ".LBB0_1:", FLAT, "s_add_i32 s4, s4, 16", "s_mov_b32 m0, s4",
            "s_cbranch_scc1 .LBB0_1", "s_endpgm"]
    assert not copies_too_early(loop)  # the branch is a wait state
    loop[5:6] = ["v_readfirstlane_b32 m0, v4"]
    assert copies_too_early(loop)
    write, end = "v_readlane_b32 s6, v9, 0", [".LBB0_2:", COPY, "s_endpgm"]
    assert copies_too_early([write, "s_cbranch_scc0 .LBB0_2", "s_nop 4"] + end)  # the branch skips the wait
    assert not copies_too_early([write, "s_nop 3", "s_cbranch_scc0 .LBB0_2", "s_nop 4"] + end)
