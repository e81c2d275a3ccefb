"""GPU parity of the head norms with the position rotation (kvc_norm_rotate)
against the binary64 oracle.

Bound of a value: the result's rounding to bf16 (2^-8 of it), and binary32
roundings before it: the sum of squares (d additions and products, halved by
the root), root, quotient, two products, cos and sin (2^-22 with the
reduced angle's own rounding), two products and a sum; (d / 2 + 16) * 2^-24 of
the pair's size."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import U_BF16, bits, host_f64, place
from gpu_util import DEV, say, to_dev, to_host
from oracle import attend as oa

pytestmark = pytest.mark.gpu


def _freqs(pairs):
    return (500000.0 ** (-np.arange(pairs) / max(pairs, 1))).astype(np.float32)


def _check(got, x, w, eps, pos, f, pairing, what):
    want = oa.norm_rotate(x, w, eps, pos, f, pairing)
    flat = oa.norm_rotate(x, w, eps, pos, [], pairing)   # without the turn: sizes of pairs
    size = np.abs(flat).copy()
    n = len(f)
    if n:
        a, b = (slice(0, n), slice(n, 2 * n)) if pairing == 0 else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
        s = np.abs(flat[..., a]) + np.abs(flat[..., b])
        size[..., a] = size[..., b] = s
    inner = size * (x.shape[-1] / 2 + 16) * 2.0 ** -24
    bound = inner + U_BF16 * (np.abs(want) + inner) + 2.0 ** -134
    err = np.abs(got - want)
    assert np.all(err <= bound), f"{what}: {np.max(err / np.maximum(bound, 1e-300))}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n, hq, hk", [(1, 1, 1), (1, 32, 8), (3, 5, 3), (15, 28, 4), (257, 2, 0), (130, 0, 7), (4099, 3, 1)])
def test_norm_rotate(d, n, hq, hk):
    rng = np.random.default_rng(d + n)
    pos = rng.integers(0, 1 << 20, n)
    pos[0] = 0
    w = [bits(rng, d, 0.3) for _ in range(2)]
    eps = 1e-6
    for pairing in (ka.KVC_ROPE_HALVES, ka.KVC_ROPE_ADJACENT):
        for pairs in (d // 2, d // 4, 8, 0):
            for norm in (True, False):
                layout = ["tokens", "heads", "fused"][(pairs // 8 + norm + pairing) % 3]
                say("rotate", d, n, hq, hk, pairing, pairs, norm, layout)
                x = [bits(rng, (n, h, d), 2.0) for h in (hq, hk)]
                t = [place(b, layout) if b.size else None for b in x]
                o = [None if i is None else torch.full_like(i, float("nan")) for i in t]
                f = _freqs(pairs)
                ka.kvc_norm_rotate(t[0], t[1], torch.from_numpy(pos).to(DEV) if pairs else None, f, o[0], o[1],
                                   q_weight=to_dev(w[0]) if norm else None, k_weight=to_dev(w[1]) if norm else None,
                                   eps=eps, pairing=pairing)
                torch.cuda.synchronize()
                for i in range(2):
                    if t[i] is None:
                        continue
                    _check(host_f64(o[i]), oa.f64(x[i]), oa.f64(w[i]) if norm else None, eps, pos, f, pairing,
                           (i, layout))
                    if not norm and pairs == 0:
                        assert np.array_equal(to_host(o[i]), x[i])


def test_in_place_on_a_fused_projection():
    """Queries and keys turned inside the projection's rows; values and what lies behind stay as they were."""
    rng = np.random.default_rng(1)
    n, hq, hk, d = 37, 8, 2, 128
    b = bits(rng, (n, (hq + 2 * hk) * d + 64), 2.0)
    wide = to_dev(b)
    q, k = wide[:, :hq * d].view(n, hq, d), wide[:, hq * d:(hq + hk) * d].view(n, hk, d)
    pos = torch.arange(n, device=DEV) * 1000
    w = bits(rng, d)
    ka.kvc_norm_rotate(q, k, pos, _freqs(64), q, k, q_weight=to_dev(w))
    torch.cuda.synchronize()
    f = _freqs(64)
    _check(host_f64(q), oa.f64(b[:, :hq * d]).reshape(n, hq, d), oa.f64(w), 1e-6, pos.cpu().numpy(), f, 0, "q")
    _check(host_f64(k), oa.f64(b[:, hq * d:(hq + hk) * d]).reshape(n, hk, d), None, 0, pos.cpu().numpy(), f, 0, "k")
    assert np.array_equal(to_host(wide)[:, (hq + hk) * d:], b[:, (hq + hk) * d:])


def test_far_and_negative_positions_match_the_turn():
    rng = np.random.default_rng(2)
    pos = np.array([-1, -4097, 1 << 24, (1 << 31) + 5, 1 << 40, -(1 << 33)], np.int64)
    b = bits(rng, (6, 2, 64))
    f = _freqs(32)
    out = torch.empty(6, 2, 64, dtype=torch.bfloat16, device=DEV)
    ka.kvc_norm_rotate(to_dev(b), None, torch.from_numpy(pos).to(DEV), f, out, None)
    torch.cuda.synchronize()
    # the binary64 product itself: |angle| * 2^-53, far below binary32 up to 2^24; above it adds up to 2^40 * 2^-52
    _check(host_f64(out)[:3], oa.f64(b)[:3], None, 0, pos[:3], f, 0, "near")
    got, want = host_f64(out), oa.norm_rotate(oa.f64(b), None, 0, pos, f, 0)
    size = np.abs(oa.f64(b)[..., :32]) + np.abs(oa.f64(b)[..., 32:])
    assert np.all(np.abs(got - want)[..., :32] <= size * (2.0 ** -8 + 2.0 ** -11))


def test_zero_vectors_and_non_finite_values():
    b = np.zeros((3, 1, 64), np.uint16)
    b[1, 0, 5] = 0x7F80
    b[2, 0, 9] = 0x7FC0
    w = np.full(64, 0x3F80, np.uint16)
    out = torch.empty(3, 1, 64, dtype=torch.bfloat16, device=DEV)
    ka.kvc_norm_rotate(to_dev(b), None, torch.zeros(3, dtype=torch.int64, device=DEV), _freqs(32), out, None,
                       q_weight=to_dev(w))
    torch.cuda.synchronize()
    got = host_f64(out)
    assert not got[0].any()                     # eps keeps a zero vector zero
    assert np.all(np.isnan(got[2])) and np.isnan(got[1, 0, 5])
    # without a norm, a NaN stays in its pair
    ka.kvc_norm_rotate(to_dev(b), None, torch.ones(3, dtype=torch.int64, device=DEV), _freqs(32), out, None)
    torch.cuda.synchronize()
    got = host_f64(out)
    assert np.all(np.isnan(got[2, 0, [9, 41]])) and np.isfinite(np.delete(got[2, 0], [9, 41])).all()


def test_captured_and_replayed_on_a_side_stream():
    rng = np.random.default_rng(4)
    q, k = to_dev(bits(rng, (15, 32, 128))), to_dev(bits(rng, (15, 8, 128)))
    pos = torch.arange(15, device=DEV)
    f = _freqs(64)
    want_q, want_k = torch.empty_like(q), torch.empty_like(k)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ka.kvc_norm_rotate(q, k, pos, f, qo, ko)
    for step in range(4):
        q.copy_(to_dev(bits(rng, (15, 32, 128))))
        pos.add_(17)
        g.replay()
        torch.cuda.synchronize()
        ka.kvc_norm_rotate(q, k, pos, f, want_q, want_k, stream=s)
        s.synchronize()
        assert torch.equal(qo, want_q) and torch.equal(ko, want_k), step


def test_empty_calls():
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    ka.kvc_norm_rotate(e, e.clone(), torch.empty(0, dtype=torch.int64, device=DEV), _freqs(32), e, e.clone())
