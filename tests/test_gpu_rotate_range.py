"""Norms at the ends of the range that the header gives: mean(x^2) + eps a
normal binary32 number. The bound is that of test_gpu_rotate."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import synth
from attend_util import bits, host_f64
from gpu_util import DEV, to_dev
from oracle import attend as oa
from test_gpu_rotate import _check, _freqs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("e, eps", [(60, 1e-6), (60, 0.0), (-59, 0.0), (-59, 1e-6), (0, 0.0), (-20, 1e-12)])
def test_norms_of_large_and_small_vectors(d, e, eps):
    """Vectors whose largest value is 2^e, all of that size among them, and one of that size alone."""
    rng = np.random.default_rng(d + 100 + e)
    x = rng.uniform(0.5, 1.0, (6, 3, d)) * np.where(rng.random((6, 3, d)) < 0.5, -1, 1) * 2.0 ** e
    x[1] = 2.0 ** e
    x[2, :, 1:] *= 2.0 ** -12
    x[..., 0] = 2.0 ** e
    b = synth.f32_to_bf16_bits(x.astype(np.float32))
    w = bits(rng, d)
    pos = np.arange(6) * 100
    out = torch.empty(6, 3, d, dtype=torch.bfloat16, device=DEV)
    ka.kvc_norm_rotate(to_dev(b), None, torch.from_numpy(pos).to(DEV), _freqs(d // 2), out, None, q_weight=to_dev(w), eps=eps)
    torch.cuda.synchronize()
    _check(host_f64(out), oa.f64(b), oa.f64(w), float(np.float32(eps)), pos, _freqs(d // 2), 0, (d, e, eps))


def test_zero_vectors_without_eps_have_no_norm():
    out = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    ka.kvc_norm_rotate(torch.zeros_like(out), None, None, np.empty(0, np.float32), out, None, q_weight=w, eps=0.0)
    torch.cuda.synchronize()
    assert bool(torch.isnan(out).all())
