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
