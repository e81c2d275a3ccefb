"""Which plan a call of kvpage_attend or kvpool_attend takes, asked of the
library itself, so that a test can say which kernel it is meant for; and a
store written in one go, for tests of many tokens."""

import ctypes

import numpy as np

from agent_handoff_amd import kvcodec as kv
from oracle import attend as oa


class Plan(ctypes.Structure):
    """kvc::AttendPlan."""
    _fields_ = [("rows", ctypes.c_uint32), ("rt", ctypes.c_uint32), ("row_blocks", ctypes.c_uint32), ("whole", ctypes.c_bool),
                ("units", ctypes.c_uint64), ("W", ctypes.c_uint64), ("blocks", ctypes.c_uint64), ("slots", ctypes.c_uint64),
                ("room", ctypes.c_uint64)]


_u32, _u64, _bool = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_bool
_page = getattr(kv.library(), "_ZN3kvc16page_attend_planEjjjjmb")
_page.restype, _page.argtypes = Plan, [_u32, _u32, _u32, _u32, _u64, _bool]
_pool = getattr(kv.library(), "_ZN3kvc16pool_attend_planEjjjjjb")
_pool.restype, _pool.argtypes = Plan, [_u32, _u32, _u32, _u32, _u32, _bool]


def page_plan(spec, seqs, q_heads, cols, tail=False):
    return _page(seqs, spec[1], q_heads, spec[3], cols * spec[2], tail)


def pool_plan(shape, agents, q_heads, tail=False):
    return _pool(shape[1], agents, q_heads, shape[3], shape[2], tail)


def one_wave_joins(plan):
    """Whether one wave joins a row (else four do)."""
    return plan.whole or plan.W <= 6 * plan.units


def put_all(host, spec, k, v, slots):
    """oracle.attend.page_write of distinct slots (negative ones and those outside left out), vectorised."""
    num, heads, page, d, fmt = spec
    size, steps, each = oa.page_layout(spec)
    live = (slots >= 0) & (slots < num * page)
    s = slots[live]
    store = host.reshape(num, each)
    codes = store[:, :steps].reshape(num, 2, heads, page, d * size)
    for j, x in enumerate((k[live], v[live])):
        if fmt == oa.BF16:
            codes[s // page, j, :, s % page] = np.ascontiguousarray(x).view(np.uint8).reshape(len(s), heads, 2 * d)
            continue
        c, st = oa.quantise(x, fmt)
        codes[s // page, j, :, s % page] = c.view(np.uint8)
        at = steps + 4 * ((j * heads + np.arange(heads)) * page + (s % page)[:, None])           # [n, heads]
        raw = np.ascontiguousarray(st, np.float32).view(np.uint8).reshape(len(s), heads, 4)
        for i in range(4):
            store[(s // page)[:, None], at + i] = raw[..., i]
