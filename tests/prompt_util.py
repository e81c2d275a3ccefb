"""Which plan a call of kvpage_attend_prompt takes, asked of the library itself, and the error bound of each row by what that
row sees alone."""

import ctypes

import numpy as np

from agent_handoff_amd import kvcodec as kv
from oracle import attend as oa
from serving_util import check_rows, half


class Plan(ctypes.Structure):
    """kvc::PromptPlan."""
    _fields_ = [("few", ctypes.c_bool), ("shares", ctypes.c_uint32), ("blocks", ctypes.c_uint64), ("bytes", ctypes.c_uint64),
                ("room", ctypes.c_uint64)]


_u32, _u64 = ctypes.c_uint32, ctypes.c_uint64
_prompt = getattr(kv.library(), "_ZN3kvc11prompt_planEjjjjjmjj")
_prompt.restype, _prompt.argtypes = Plan, [_u32, _u32, _u32, _u32, _u32, _u64, _u32, _u32]


def prompt_plan(spec, seqs, tokens, q_heads, cols, window=0, sinks=0):
    return _prompt(seqs, tokens, spec[1], q_heads, spec[3], cols * spec[2], window, sinks)


def plan_name(plan):
    return "few" if plan.few else "shared" if plan.shares else "blocks"


def value_steps(host, spec, slots):
    """The 8-bit steps of the values of `slots`: [heads, n]; None for formats without."""
    num, heads, page, d, fmt = spec
    if not half(fmt):
        return None
    steps, each = oa.page_layout(spec)[1:]
    s = np.ascontiguousarray(host.reshape(num, each)[:, steps:steps + 8 * heads * page]).view(np.float32)
    return s.reshape(num, 2, heads, page)[slots // page, 1, :, slots % page].T


def check_each_row(got, lse, q, keys, values, steps, scale, fmt, see, what=""):
    """check_rows, one row and kv head at a time, each with the steps of the values that it sees alone: what a binary16 weight
    loses goes by the largest step that its own row has met. steps: [kv_heads, T] or None."""
    group = q.shape[1] // keys.shape[0]
    for h in range(keys.shape[0]):
        hs = slice(h * group, (h + 1) * group)
        for i in range(len(q)):
            at = slice(i, i + 1)
            own = None if steps is None else steps[h][see[i]]
            # without what it does not see, whose size would count for the bound
            k, v = keys[h:h + 1][:, see[i]], values[h:h + 1][:, see[i]]
            check_rows(got[at, hs], None if lse is None else lse[at, hs], q[at, hs], k, v, scale, fmt, own,
                       np.ones((1, k.shape[1]), bool), (what, "row", i, "kv head", h))


def growing_values(rng, n, d, low, high):
    """bf16 bits [n, 1, d] whose sizes go from 2^low to 2^high along the tokens."""
    from attend_util import bits
    v = bits(rng, (n, 1, d))
    e = (v >> 7 & 255).astype(int) + np.round(np.linspace(low, high, n)).astype(int)[:, None, None]
    return ((v & 0x807F) | (e << 7)).astype(np.uint16)
