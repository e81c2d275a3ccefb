"""Attention over keys and queries at the ends of bf16's range whose logits are
ordinary: no step between the stored codes and a logit may leave binary32's
range when the logit itself does not."""

import math

import numpy as np
import pytest
import torch

import oracle
from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import synth
from attend_util import FORMATS, bits, check_attend, host_f64, random_sequences, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _outputs(n, hq, d):
    return torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV), torch.empty(n, hq, device=DEV)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("e, n", [(-122, 150), (-122, 1500), (116, 150), (116, 1500)])
def test_keys_at_the_ends_of_the_range(fmt, e, n):
    """Keys of about 2^e and queries of about 2^-e, whole tiles and a part of one. One query head of each is of ordinary
    size where the keys are small (its logits are about 0), so both orders of the factors meet in one wave."""
    rng = np.random.default_rng(e + 200 + n)
    say("range", fmt, e, n)
    d, page, heads = 128, 32, 2
    spec = (-(-n // page) + 1, heads, page, d, fmt)
    store, table = random_sequences(rng, spec, [n])
    t = np.arange(n)
    store.put(bits(rng, (n, heads, d), 2.0 ** e), bits(rng, (n, heads, d)), table[0, t // page] * page + t % page)
    q = bits(rng, (1, 3 * heads, d), 2.0 ** -e)
    if e < 0:
        q[0, ::3] = bits(rng, (heads, d))
    out, lse = _outputs(1, 3 * heads, d)
    ws = torch.empty(ka.kvpage_attend_workspace_bytes(spec, 1, 3 * heads, table.shape[1] * page), dtype=torch.uint8, device=DEV)
    ka.kvpage_attend(spec, store.dev(), to_dev(q), _i32(table), _i32([n]), out, ws, lse=lse)
    torch.cuda.synchronize()
    k, v = sequence(store, table, 0, n)
    steps = None if fmt == ka.KVC_PAGE_BF16 else np.array([0.1])   # values of N(0, 1): steps below 6 / 127
    check_attend(host_f64(out)[0], host_f64(lse)[0], oa.f64(q)[0], k, v, 1 / math.sqrt(d), fmt != 0, steps, (fmt, e, n))


@pytest.mark.parametrize("d", [64, 128])
def test_a_pool_head_of_zeros_beside_a_head_of_large_keys(d):
    """A pool has one key step for all heads of a layer. Queries of 2^100 over a head whose keys are all zero have
    logits of 0 (the mean of the values), whatever the step that another head's keys set."""
    rng = np.random.default_rng(d)
    T = 70
    shape = (1, 2, T, d)
    k, v = bits(rng, shape, 2.0 ** 60), bits(rng, shape)
    k[0, 1] = 0
    pool = oracle.pool_encode(k, v)
    q = bits(rng, (2, 4, d), 2.0 ** 100)
    q[:, :2] = bits(rng, (2, 2, d), 2.0 ** -60)
    out, lse = _outputs(2, 4, d)
    ws = torch.empty(ka.kvpool_attend_workspace_bytes(shape, 2, 4), dtype=torch.uint8, device=DEV)
    ka.kvpool_attend(shape, torch.from_numpy(pool).to(DEV), 0, to_dev(q), out, ws, lse=lse)
    torch.cuda.synchronize()
    rot = oa.pool_rotated(pool, shape, 0)[1]
    want = np.mean(rot[1], 0) @ oa.hadamard(d) / math.sqrt(d)
    # weights and levels rounded to binary16, the transform spreads their errors over all channels
    b = np.sum(np.mean(np.abs(rot[1]), 0)) / math.sqrt(d) * (2.01 * 2.0 ** -11 + 2.0 ** -18)
    assert np.all(np.abs(host_f64(out)[:, 2:] - want) <= b + (np.abs(want) + b) * 2.0 ** -8)
    assert np.all(np.abs(host_f64(lse)[:, 2:] - math.log(T)) <= 2.0 ** -18)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
