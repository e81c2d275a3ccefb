"""Wait states of the loads to LDS that lds_fetch.h writes as inline assembly, where
the compiler adds none. On gfx950 a VMEM instruction reads a scalar register
five wait states at the earliest behind the vector instruction (v_readfirstlane, which
makes the address the same in all lanes) that wrote it, and a load to LDS reads
M0 one behind its write. Nothing is known of what comes before an assembly's text, so
it has to hold all of them itself."""

import os
import re

import pytest

from agent_handoff_amd import build

SGPR_TO_VMEM, M0_TO_LDS_LOAD = 5, 1


def assemblies(text):
    """(instructions, constraints of the operands, clobbers) of each statement with loads to LDS."""
    for m in re.finditer(r"asm volatile\((.*?)\);", text, re.S):
        # text, outputs, inputs, clobbers: a colon outside of strings lies between them
        parts = re.split(r':(?=(?:[^"]*"[^"]*")*[^"]*$)', m.group(1))
        lines = "".join(re.findall(r'"([^"]*)"', parts[0])).replace("\\t", "").split("\\n")
        if any("_lds_" in x for x in lines):
            yield lines, re.findall(r'"([^"]+)"\s*\(', ":".join(parts[1:3])), re.findall(r'"([^"]+)"', parts[3])


def wait_states(lines, constraints):
    """(of the first read of a scalar register by a load, of the least distance from a write of M0 to a load)."""
    passed, m0, scalar, least = 0, 0, None, None
    for x in lines:
        op, _, rest = x.strip().partition(" ")
        if op == "s_nop":
            passed += int(rest, 0) + 1
            continue
        if "_lds_" in op:
            least = passed - m0 if least is None else min(least, passed - m0)
            if scalar is None and any(constraints[int(i)] == "s" for i in re.findall(r"%(\d+)", rest)):
                scalar = passed
        passed += 1
        if op == "s_mov_b32" and rest.startswith("m0"):
            m0 = passed
    return scalar, least


def found():
    out = []
    for path in build.sources() + [os.path.join(build.CSRC, f) for f in os.listdir(build.CSRC) if f.endswith(".h")]:
        with open(path) as f:
            out += [(os.path.basename(path), *a) for a in assemblies(f.read())]
    return out


FOUND = found()


def test_there_are_some():
    assert [name for name, *_ in FOUND] == ["lds_fetch.h"] * 4
    assert sum(wait_states(lines, c)[0] is not None for _, lines, c, _ in FOUND) == 3


@pytest.mark.parametrize("at", range(len(FOUND)))
def test_waits_for_addresses_and_m0(at):
    _, lines, constraints, clobbers = FOUND[at]
    scalar, m0 = wait_states(lines, constraints)
    assert scalar is None or scalar >= SGPR_TO_VMEM, lines
    assert m0 >= M0_TO_LDS_LOAD, lines
    assert clobbers == ["memory"], clobbers   # (M0 is the compiler's own, and cannot be declared)


def test_counting():
    lines = ["s_mov_b32 m0, %0", "s_nop 0", "global_load_lds_dwordx4 %2, %1", "global_load_lds_dwordx4 %3, %1 offset:0x400"]
    assert wait_states(lines, ["s", "s", "v", "v"]) == (2, 1)
    assert wait_states(["s_mov_b32 m0, %0", "global_load_lds_dword %1, off"], ["s", "v"]) == (None, 0)
    lines[1] = "s_nop 3"
    assert wait_states(lines, ["s", "s", "v", "v"]) == (5, 4)
