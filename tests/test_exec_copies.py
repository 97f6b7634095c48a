"""CPU check on the compiled kernels: where the lanes of a branch come together again, no
vector register is written before they all take part.

A value that all lanes hold and that the compiler moves to another register in that place
(in a kernel short of registers) is moved for the branch's own lanes only, and the others
find something else there later: an address, in the worst case."""

import re

import pytest

from isa_check import kernels
from test_isa import CSRC, asm, pytestmark  # noqa: F401

JOIN = re.compile(r"s_or_b64 exec, exec, |s_(or|andn2)_saveexec_b64 ")  # (the latter: where an else begins)


def blocks(body):
    """(label, instructions) of basic blocks; those that are only fallen into are `%bb.`."""
    out = [("", [])]
    for line in body:
        m = re.match(r"(\.LBB\w+):", line.strip()) or re.match(r"; (%bb\.\d+):", line.strip())
        if m:
            out.append((m.group(1), []))
            continue
        t = line.split(";")[0].strip()
        if t:
            out[-1][1].append(t)
    return out


def writes_vector(t):
    op = t.split()[0]
    if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp", "v_writelane")):
        return False  # (scalar results; lanes whatever takes part)
    return op.startswith(("v_", "ds_read", "ds_bpermute")) or "_load_" in op and op.startswith(("global", "flat", "buffer"))


def writes_before_joins(body):
    """Vector writes between the place where a branch's lanes come together (the target of its
    s_cbranch_execz, or what follows a loop's s_cbranch_execnz) and the instruction that
    makes them take part."""
    found, before = [], []
    targets = {m.group(1) for line in body for m in [re.search(r"s_cbranch_execz (\S+)", line)] if m}
    for label, ins in blocks(body):
        here = label in targets or bool(before) and before[-1].startswith("s_cbranch_execnz")
        before = ins
        joins = [i for i, t in enumerate(ins) if JOIN.match(t)]
        if here and joins:
            found += [(label, t) for t in ins[:joins[0]] if writes_vector(t)]
    return found


@pytest.mark.parametrize("src", sorted(p.name for p in CSRC.glob("*.hip") if p.name != "q4_api.hip"))
def test_no_register_is_written_for_some_lanes_where_all_go_on(src):
    for name, body in kernels(asm(src), ""):
        assert not writes_before_joins(body), name


BRANCH = ["s_and_saveexec_b64 s[4:5], vcc", "s_cbranch_execz .LBB0_2", "; %bb.1:", "global_load_dword v3, v[4:5], off"]


def test_the_check_knows_a_move_before_the_join():
    for move in ("v_accvgpr_write_b32 a3, v9", "v_mov_b32_e32 v7, v9", "v_accvgpr_read_b32 v7, a3"):
        assert writes_before_joins(BRANCH + [".LBB0_2:", move, "s_mov_b64 s[8:9], s[2:3]", "s_or_b64 exec, exec, s[4:5]"])
        assert not writes_before_joins(BRANCH + [".LBB0_2:", "s_or_b64 exec, exec, s[4:5]", move])
        assert not writes_before_joins(BRANCH + [move, ".LBB0_2:", "s_or_b64 exec, exec, s[4:5]"])
    loop = [".LBB0_1:", "s_andn2_b64 exec, exec, s[4:5]", "s_cbranch_execnz .LBB0_1", "; %bb.2:"]
    assert writes_before_joins(loop + ["v_mov_b32_e32 v7, v9", "s_or_b64 exec, exec, s[4:5]"])
    assert not writes_before_joins(loop + ["s_or_b64 exec, exec, s[4:5]", "v_mov_b32_e32 v7, v9"])


def test_the_check_leaves_scalars_alone():
    assert not writes_before_joins(BRANCH + [".LBB0_2:", "s_mov_b64 s[8:9], s[2:3]", "v_readlane_b32 s3, v255, 4",
                                             "v_cmp_gt_i32_e32 vcc, 4, v1", "s_or_b64 exec, exec, s[4:5]"])
