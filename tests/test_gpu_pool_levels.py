"""How exactly kvpool_attend takes a pool's value levels.

One token has weight 1, so a row's output is that token's value: the inverse
transform of levels times size, rounded to bf16. Transformed back, each
channel is its level plus the outputs' roundings, which are independent of
one another: at most 2^-8 of an output each, so a variance of at most
(2^-8 x)^2 / 3 (a uniform error; the outputs' mean square is the levels',
since the transform keeps it). Their mean over N channels of one level is off by
2^-8 rms / sqrt(3 N) (one standard deviation); six of those and 2^-17 of the level
(binary32 sums of d, and the level's own rounding) is the tolerance. Levels
rounded to binary16 as they are would be 0.5 to 0.8 of 2^-12 off."""

import math

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv
from agent_handoff_amd import synth
from attend_util import host_f64
from gpu_util import DEV, say
from oracle import attend as oa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_levels_are_not_rounded_to_binary16(d):
    L, H = 16, 512
    shape = (L, H, 1, d)
    gen = torch.Generator(device=DEV).manual_seed(d)
    k, v = (torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for _ in range(2))
    pool = kv.SharedKVPool.encode(k, v)
    q = torch.zeros(1, H, d, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(ka.kvpool_attend_workspace_bytes(shape, 1, H), dtype=torch.uint8, device=DEV)
    outs = torch.empty(L, 1, H, d, dtype=torch.bfloat16, device=DEV)
    for layer in range(L):
        ka.kvpool_attend(shape, pool.pool, layer, q, outs[layer], ws)
    torch.cuda.synchronize()
    host, levels, got = pool.pool.cpu().numpy(), [], []
    for layer in range(L):
        rot = oa.pool_rotated(host, shape, layer)[1][:, 0]                    # [H, d]: level times size
        back = host_f64(outs[layer])[0] @ oa.hadamard(d) / math.sqrt(d)
        size = np.sqrt(np.mean(rot * rot, -1, keepdims=True))                 # any factor of the vector serves
        levels.append(rot / size)
        got.append(back / size)
    levels, got = np.concatenate(levels).ravel(), np.concatenate(got).ravel()
    # the same level in units of its vector's size differs from vector to vector: relative errors, weighted by level
    mags = np.abs(np.concatenate([oa.pool_rotated(host, shape, layer)[1][:, 0] for layer in range(L)]).ravel())
    sizes = np.repeat(host[kv_scale(shape)].view(np.float16).astype(np.float64), d)
    index = np.rint(mags / sizes * 2 ** 15).astype(np.int64)                  # units of 2^-15, the table's own
    assert set(np.unique(index)) == {8031, 24773, 44037, 70515}
    for unit in (8031, 24773, 44037, 70515):
        at = index == unit
        x, y = levels[at], got[at]
        slope = np.sum((y - x) * x) / np.sum(x * x)
        # sum of errors (variance 2^-16 / 3 each, in units of the vector's rms) times x, over the sum of x^2
        sigma = 2.0 ** -8 / math.sqrt(3) / math.sqrt(np.sum(x * x))
        say("level", unit, "relative error in 2^-12:", slope * 2 ** 12, "tolerance", (6 * sigma + 2.0 ** -17) * 2 ** 12)
        assert abs(slope) <= 6 * sigma + 2.0 ** -17, unit


def kv_scale(shape):
    """The bytes of a pool that hold its value sizes."""
    import oracle
    L, H, T, _ = shape
    at = oracle.pool_layout(*shape)[2]
    return slice(at, at + 2 * L * H * T)
