"""Attention of many new tokens notes in LDS (`odd`) which tiles hold values that are not finite:
wave 0 clears the notes of a block, and whichever wave puts a tile there sets its
own. Every order in which the waves may run, by the barriers that the source
has between these steps, has to keep what was set."""

import os
import re
from functools import lru_cache

from agent_handoff_amd import build

WAVES = 4


def steps():
    """What a wave does, in order: "clear", "set" (a tile is put into LDS) and "barrier", from the clearing of the notes to
    the first turn, with the condition of the format where there is one."""
    with open(os.path.join(build.CSRC, "prompt_kernels.hip")) as f:
        text = f.read()
    text = text[text.index("if (thread < 8) sh.odd[thread] = 0;"):]
    text = re.sub(r"//[^\n]*", "", text[:text.index("s0 = mfma<FMT>")])
    # what lies inside of the lambdas that are defined there is not run there
    found = re.findall(r"sh\.odd\[thread\] = 0|\bput\(|__syncthreads\(\)", text[:text.index("const auto take_out")])
    found += re.findall(r"\bput\(|__syncthreads\(\)", text[text.index("if (j0 < j1) {"):])
    return [{"put(": "set", "__syncthreads()": "barrier"}.get(x, "clear") for x in found]


def kept(program):
    """Whether every order of the waves ends with every note that was set."""
    @lru_cache(None)
    def run(at, noted):
        ends = True
        moved = False
        for w in range(WAVES):
            i = at[w]
            if i == len(program):
                continue
            if program[i] == "barrier":
                if any(j < i for j in at):   # some wave has not come to it
                    continue
                now = noted
            elif program[i] == "clear":
                now = frozenset() if w == 0 else noted
            else:
                now = noted | {(w, i)}
            moved = True
            ends &= run(at[:w] + (i + 1,) + at[w + 1:], now)
        return ends if moved else noted == {(w, i) for w in range(WAVES) for i, x in enumerate(program) if x == "set"}

    return run((0,) * WAVES, frozenset())


def test_the_model_sees_a_race():
    assert not kept(("clear", "set", "barrier"))
    assert not kept(("barrier", "clear", "set", "barrier"))
    assert kept(("clear", "barrier", "set", "barrier"))


def test_no_note_is_lost():
    program = steps()
    assert program[0] == "clear" and program.count("clear") == 1
    assert program.count("set") == 4 and program[-1] == "barrier"   # (two of them in one format, one in the others, and one)
    sets = program.index("set")
    # (each of the four stands for itself: what holds with one holds with fewer)
    assert kept(tuple(x for i, x in enumerate(program) if x != "set" or i == sets))
