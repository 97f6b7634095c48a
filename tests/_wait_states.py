"""Wait states before the copies into LDS, on a kernel's gfx950 assembly (test support).

A `global_load_lds_*` reads M0 and, in the scalar-base form, an address in scalar
registers.  Hardware does not wait for either where a vector instruction wrote
it (five wait states must lie between) nor for a scalar instruction's write of
M0 (one), and the compiler does not before inline assembly.  The pass follows
every path through the kernel, loops and branches included.
"""

import re

from isa_check import kernels  # noqa: F401

VECTOR, SCALAR = 5, 1  # wait states that must lie between


def blocks_of(body):
    """(instructions, successors) of every basic block."""
    instrs = [t for t in (ln.split(";")[0].strip() for ln in body) if t]
    instrs = [t for t in instrs if t.endswith(":") or not t.startswith(".")] + ["s_endpgm"]
    blocks, cur = [], []
    for t in instrs:
        if t.endswith(":") and cur:
            blocks.append(cur)
            cur = []
        cur.append(t)
        if t.startswith(("s_branch", "s_cbranch", "s_endpgm", "s_setpc")):
            blocks.append(cur)
            cur = []
    if cur:
        blocks.append(cur)
    at = {b[0][:-1]: i for i, b in enumerate(blocks) if b[0].endswith(":")}
    succ = []
    for i, b in enumerate(blocks):
        last = b[-1]
        to = [] if last.startswith(("s_endpgm", "s_setpc", "s_branch")) else [i + 1]
        if last.startswith(("s_branch", "s_cbranch")):
            to.append(at[last.split()[1]])
        succ.append([j for j in to if j < len(blocks)])
    return blocks, succ


def scalars(token):
    """Scalar registers of an operand ('m0', 's5', 's[4:5]', 'vcc')."""
    m = re.match(r"s\[(\d+):(\d+)\]$", token)
    if m:
        return {f"s{r}" for r in range(int(m.group(1)), int(m.group(2)) + 1)}
    if re.match(r"s\d+$", token) or token == "m0":
        return {token}
    return {"vcc_lo", "vcc_hi"} if token == "vcc" else {token} if token.startswith("vcc_") else set()


def step(state, t, found):
    """Registers written less than their wait states ago -> states still missing."""
    parts = [p for p in re.split(r"[\s,]+", t) if p]
    op = parts[0]
    if op.startswith("global_load_lds"):
        reads = {"m0"}.union(*(scalars(p) for p in parts[1:]))
        for r in sorted(reads & set(state)):
            found.add((t, r, state[r][1]))
    passed = int(parts[1]) + 1 if op == "s_nop" else 1
    state = {r: (n - passed, w) for r, (n, w) in state.items() if n > passed}
    if op.startswith("v_"):  # (every scalar destination comes first or, for carries and compares, second)
        for p in parts[1:3]:
            if scalars(p) and (p == parts[1] or re.match(r"v_(add|sub|subrev|addc|subb|div_scale|mad_[ui]64)", op)):
                for r in scalars(p):
                    state[r] = (VECTOR, t)
    elif op.startswith("s_") and len(parts) > 1 and not op.startswith(("s_nop", "s_wait", "s_cmp", "s_bitcmp")):
        for r in scalars(parts[1]):
            state.pop(r, None)  # an address from a scalar instruction is waited for
            if r == "m0":
                state[r] = (SCALAR, t)
    return state


def copies_too_early(body):
    """(copy, register, the write it is too close behind), over all paths."""
    blocks, succ = blocks_of(body)
    into = [None] * len(blocks)
    into[0] = {}
    work, found = [0], set()
    while work:
        i = work.pop()
        state = into[i]
        for t in blocks[i]:
            if not t.endswith(":"):
                state = step(state, t, found)
        for j in succ[i]:
            old = into[j]
            new = dict(state) if old is None else dict(old)
            for r, (n, w) in state.items():
                if r not in new or new[r][0] < n:
                    new[r] = (n, w)
            if new != old:
                into[j] = new
                work.append(j)
    return sorted(found)
