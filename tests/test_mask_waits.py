"""Wait states around the vector instructions that kernels_common.h writes as inline assembly and that read or write lane
masks in scalar registers. On gfx950 a vector instruction reads a scalar register two wait states at the earliest behind the
vector instruction that wrote it, carry and mask included; the compiler adds none inside of such a text, nor behind it for
what the text wrote."""

import os
import re

from agent_handoff_amd import build

WAIT = 2


def text_of(function):
    """(instructions, constraints of the operands) of the assembly in a function of kernels_common.h."""
    with open(os.path.join(build.CSRC, "kernels_common.h")) as f:
        s = f.read()
    s = s[s.index(function + "("):]
    m = re.search(r"asm\((.*?)\);", s, re.S).group(1)
    parts = re.split(r':(?=(?:[^"]*"[^"]*")*[^"]*$)', m)
    lines = "".join(re.findall(r'"([^"]*)"', parts[0])).replace("\\t", "").split("\\n")
    return [x.strip() for x in lines], re.findall(r'"([^"]+)"\s*\(', ":".join(parts[1:]))


def places(lines):
    """(wait states before it, operands written, operands read) of each instruction; and the wait states of all."""
    passed, found = 0, []
    for x in lines:
        op, _, rest = x.partition(" ")
        if op == "s_nop":
            passed += int(rest, 0) + 1
            continue
        args = [int(i) for i in re.findall(r"%(\d+)", rest)]
        written = 2 if "_co_" in op else 1   # a vector and, with a carry, a mask
        found.append((passed, args[:written], args[written:]))
        passed += 1
    return found, passed


def test_masks_that_go_in():
    lines, constraints = text_of("shift_in_bits")
    found, _ = places(lines)
    reads = [(at, i) for at, _, read in found for i in read if constraints[i] == "s"]
    assert len(reads) == 3 and min(at for at, _ in reads) >= WAIT, lines
    # what is written in it is read by none of the others
    written = {i for _, w, _ in found for i in w if "s" in constraints[i]}
    assert written and not written & {i for _, i in reads}


def test_masks_that_come_out():
    lines, constraints = text_of("shift_out_bits")
    found, end = places(lines)
    masks = [i for i, c in enumerate(constraints) if "s" in c]
    at = {i: p for p, w, _ in found for i in w}
    assert end - at[masks[2]] - 1 >= WAIT, lines
    # the others are read by scalar instructions alone, which wait by themselves
    with open(os.path.join(build.CSRC, "pool_kernels.hip")) as f:
        s = f.read()
    s = s[s.index("shift_out_bits(pw, w0, w1, w2);"):]
    s = s[:s.index("fwht_quad")]
    assert re.findall(r"w[01]\b", s[s.index(";"):]) == ["w1", "w0"] and "m1 = ~(w1 ^ w2), m0 = ~(w0 ^ w2)" in s


def test_counting():
    assert places(["s_nop 1", "v_addc_co_u32_e64 %0, %1, %0, %0, %2"]) == ([(2, [0, 1], [0, 0, 2])], 3)
    assert places(["v_add_co_u32_e64 %0, %2, %0, %0", "v_add_co_u32_e64 %1, %3, %1, %1"])[0][1] == (1, [1, 3], [1, 1])
