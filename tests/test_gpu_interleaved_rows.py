"""Rows of several outputs between one another in one buffer, as a projection
with one key head for each query head gives them: [tokens][heads][q, k, v][d]."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import FORMATS, bits
from gpu_util import DEV, to_dev, to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 37])
@pytest.mark.parametrize("heads_first", [False, True])
def test_turned_in_place_and_read_back_between_one_another(n, heads_first):
    rng = np.random.default_rng(n)
    heads, d = 5, 64
    raw = bits(rng, (n, heads, 3, d))
    f = (10000.0 ** (-np.arange(32) / 32)).astype(np.float32)
    pos = torch.arange(n, device=DEV) + 3
    w = to_dev(bits(rng, d))

    def rows():
        if heads_first:
            return to_dev(raw.transpose(1, 0, 2, 3)).permute(1, 0, 2, 3)
        return to_dev(raw)

    x = rows()
    alone = [x[:, :, i].contiguous() for i in (0, 1)]
    ka.kvc_norm_rotate(*alone, pos, f, *alone, q_weight=w)
    q, k, v = (x[:, :, i] for i in range(3))
    ka.kvc_norm_rotate(q, k, pos, f, q, k, q_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(q, alone[0]) and torch.equal(k, alone[1])
    assert np.array_equal(to_host(v), raw[:, :, 2])
    for fmt in FORMATS:
        cache = ka.PagedKV(3, heads, 16, d, fmt)
        slots = torch.from_numpy(rng.permutation(48)[:n].astype(np.int64)).to(DEV)
        cache.write(k, v, slots)
        want = cache.read(slots)
        y = rows()
        before = to_host(y[:, :, 1])
        cache.read(slots, y[:, :, 0], y[:, :, 2])
        torch.cuda.synchronize()
        assert torch.equal(y[:, :, 0], want[0]) and torch.equal(y[:, :, 2], want[1])
        assert np.array_equal(to_host(y[:, :, 1]), before)
