"""The largest sizes that the entry points of kvattend.h take, and what they
refuse beyond, all before any device work."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv

fake_addresses = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only host")

L = kv.library()
A = 1 << 44   # addresses far enough apart for the largest rows


def _rotate(n, base=A, rows=None, heads=1):
    f = np.ones(32, np.float32)
    q = ka.kvc_rows(base, heads * 64, 64) if rows is None else rows
    return L.kvc_norm_rotate(n, heads, 0, 64, q, None, None, None, 1e-6, 2 * A, f.ctypes.data, 32, 0, q, None, None)


@fake_addresses
def test_rotation_launches_stay_below_2_32_threads():
    """Four tokens a workgroup of 256 threads: 2^26 - 4 tokens are the most that fit below 2^32 threads. The rows'
    wrong alignment, looked at behind the size, keeps the calls from launching."""
    most = (1 << 26) - 4
    for n in (most - 1, most):
        assert _rotate(n, A + 8) == kv.KVC_E_ALIGN
    for n in (most + 1, most + 2, most + 3, 1 << 26, (1 << 32) - 1):
        assert _rotate(n) == kv.KVC_E_SHAPE and _rotate(n, A + 8) == kv.KVC_E_SHAPE


# ---------------------------------------------------------------- outputs inside one another's rows
# [tokens][heads][q, k, v][d], as a fused projection of one key head a query head gives it, its heads-first
# counterpart, and single tokens of either: every vector has elements of its own.

def _in_place(n, heads, q, k, shift=0, d=64):
    """kvc_norm_rotate in place on rows (offset in vectors, token stride, head stride), in vectors."""
    f = np.ones(32, np.float32)
    q, k = (ka.kvc_rows(A + 2 * d * r[0] + s, r[1] * d, r[2] * d) for r, s in ((q, 0), (k, shift)))
    return L.kvc_norm_rotate(n, heads, heads, d, q, k, None, None, 1e-6, 2 * A, f.ctypes.data, 32, 0, q, k, None)


def _read(n, heads, k, v, d=64):
    spec = ka.kvc_pages(4, heads, 16, d, 1)
    k, v = (ka.kvc_rows(A + 2 * d * r[0], r[1] * d, r[2] * d) for r in (k, v))
    return L.kvpage_read(spec, 2 * A, ka.kvpage_bytes(spec), n, 3 * A, k, v, None, None)


APART = [  # tokens, heads, rows of two outputs
    (5, 8, (0, 24, 3), (1, 24, 3)), (5, 8, (1, 24, 3), (0, 24, 3)), (5, 8, (0, 24, 3), (2, 24, 3)),
    (1, 8, (0, 24, 3), (1, 24, 3)), (5, 1, (0, 3, 3), (2, 3, 3)),
    (5, 8, (0, 3, 15), (1, 3, 15)),                                   # heads first, tokens interleaved
    (5, 4, (0, 1, 15), (5, 1, 15)), (5, 4, (5, 1, 15), (0, 1, 15)),   # heads first, a plane of each in turn
    (5, 4, (0, 30, 2), (8, 30, 2)), (5, 4, (0, 30, 2), (9, 30, 2)),
]
MEET = [
    (5, 8, (0, 24, 3), (0, 24, 3)), (5, 8, (0, 24, 3), (3, 24, 3)), (5, 8, (0, 24, 3), (6, 25, 3)),
    (1, 8, (0, 24, 3), (3, 24, 3)), (5, 8, (0, 3, 15), (3, 3, 15)), (5, 4, (0, 1, 15), (3, 1, 15)),
    (5, 4, (0, 1, 15), (11, 1, 15)), (5, 4, (0, 30, 2), (2, 30, 2)), (5, 4, (0, 30, 2), (30, 30, 2)),
    (5, 4, (0, 30, 2), (4, 31, 2)),
]


def _vectors(n, heads, r):
    return {r[0] + i * r[1] + h * r[2] for i in range(n) for h in range(heads)}


def test_the_cases_are_what_they_say():
    for n, heads, a, b in APART:
        assert len(_vectors(n, heads, a) | _vectors(n, heads, b)) == 2 * n * heads, (n, heads, a, b)
    for n, heads, a, b in MEET:
        assert len(_vectors(n, heads, a) | _vectors(n, heads, b)) < 2 * n * heads, (n, heads, a, b)


@fake_addresses
@pytest.mark.parametrize("n, heads, a, b", APART)
def test_outputs_between_one_anothers_heads_are_taken(n, heads, a, b):
    """Past every check, the launch fails for want of a GPU."""
    assert _in_place(n, heads, a, b) == kv.KVC_E_HIP
    assert _read(n, heads, a, b) == kv.KVC_E_HIP


@fake_addresses
@pytest.mark.parametrize("n, heads, a, b", MEET)
def test_outputs_that_share_elements_are_refused(n, heads, a, b):
    assert _in_place(n, heads, a, b) == kv.KVC_E_ALIAS
    assert _read(n, heads, a, b) == kv.KVC_E_ALIAS


@fake_addresses
def test_outputs_that_share_part_of_a_vector_are_refused():
    for shift, rc in ((0, kv.KVC_E_HIP), (16, kv.KVC_E_ALIAS), (112, kv.KVC_E_ALIAS), (-16, kv.KVC_E_HIP),
                      (-128, kv.KVC_E_HIP), (-144, kv.KVC_E_ALIAS)):
        assert _in_place(5, 8, (0, 24, 3), (2, 24, 3), shift) == rc, shift   # the gap is of vectors 1 and 2
