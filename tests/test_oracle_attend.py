"""The binary64 oracle of the attention-side operators against independent
statements of the same definitions: exact rational arithmetic for the codes,
complex turns for the rotation, the C oracle's decode for the pool's values,
plain loops for attention."""

import math
from fractions import Fraction

import numpy as np
import pytest

import oracle
from agent_handoff_amd import synth
from oracle import attend as oa


def _bits(rng, shape, size=1.0):
    return synth.f32_to_bf16_bits((rng.standard_normal(shape) * size).astype(np.float32))


def test_e4m3_table():
    assert oa.E4M3[0x7E] == 448.0 and np.isnan(oa.E4M3[0x7F]) and np.isnan(oa.E4M3[0xFF])
    assert oa.E4M3[1] == 2.0 ** -9 and oa.E4M3[8] == 2.0 ** -6 and oa.E4M3[0x38] == 1.0 and oa.E4M3[0xB8] == -1.0
    assert np.all(np.diff(oa.E4M3[:127]) > 0)


@pytest.mark.parametrize("fmt", [oa.INT8, oa.FP8])
@pytest.mark.parametrize("size", [1.0, 1e-38, 1e30])
def test_codes_are_nearest_ties_to_even(fmt, size):
    rng = np.random.default_rng(fmt)
    x = _bits(rng, (6, 64), size)
    # ties of int8: multiples of half a step (m = 127 and 254, values k + 1/2)
    x[0] = synth.f32_to_bf16_bits((np.arange(64, dtype=np.float32) - 31.5))
    x[0, 0] = synth.f32_to_bf16_bits(np.float32([127.0]))[0]
    # ties of e4m3: odd multiples of half a unit, m = 448
    x[1] = synth.f32_to_bf16_bits((2 * np.arange(64, dtype=np.float32) + 1) / 2 ** 10)
    x[1, 0] = synth.f32_to_bf16_bits(np.float32([448.0]))[0]
    codes, step = oa.quantise(x, fmt)
    most = 127 if fmt == oa.INT8 else 448
    table = [Fraction(i) for i in range(-127, 128)] if fmt == oa.INT8 else [Fraction(float(v)) for v in oa.E4M3[:127]]
    v = oa.f64(x)
    for i in range(x.shape[0]):
        m = Fraction(float(np.max(np.abs(v[i]))))
        assert step[i] == np.float32(float(m) / most)
        for j in range(x.shape[1]):
            y = Fraction(float(v[i, j])) * most / m
            if fmt == oa.INT8:
                got = Fraction(int(codes[i, j].astype(np.int8)))
                even = got % 2 == 0
            else:
                got = Fraction(float(oa.E4M3[codes[i, j]]))
                y, got = abs(y), abs(got)
                even = (int(codes[i, j]) & 1) == 0
            best = min(abs(t - y) for t in table)
            assert abs(got - y) == best
            if sum(abs(t - y) == best for t in table) == 2:
                assert even


def test_zero_and_non_finite_vectors():
    x = np.zeros((4, 64), np.uint16)
    x[1, 3] = 0x7F80
    x[2, 5] = 0x7FC1
    x[3, 7] = 0xFF80
    for fmt in (oa.INT8, oa.FP8):
        codes, step = oa.quantise(x, fmt)
        assert step[0] == 0 and np.all(np.isnan(step[1:])) and not codes.any()


@pytest.mark.parametrize("fmt", [oa.BF16, oa.INT8, oa.FP8])
def test_pages_round_trip_and_padding(fmt):
    rng = np.random.default_rng(3)
    spec = (5, 3, 16, 64, fmt)
    pages = np.full(oa.page_bytes(spec), 0xFF, np.uint8)
    slots = np.array([79, -1, 0, 17, 33, 80, 5], np.int64)
    k, v = _bits(rng, (7, 3, 64)), _bits(rng, (7, 3, 64), 0.1)
    oa.page_write(pages, spec, k, v, slots)
    ok = np.array([0, 2, 3, 4, 6])
    kk, vv = oa.page_values(pages, spec, slots[ok])
    most = {oa.BF16: 1, oa.INT8: 127, oa.FP8: 448}[fmt]
    for got, want in ((kk, oa.f64(k[ok])), (vv, oa.f64(v[ok]))):
        m = np.max(np.abs(want), -1, keepdims=True)
        # half a step: m / 254, or 2^-4 of the value (e4m3's three mantissa bits) and half its smallest unit
        bound = 0 if fmt == oa.BF16 else m / 254 if fmt == oa.INT8 else np.abs(want) / 16 + m / 448 * 2.0 ** -10
        # the step itself is rounded to binary32: 2^-24 of it, so of the value too
        assert np.all(np.abs(got - want) <= bound + (np.abs(want) + m / most) * 2.0 ** -24)
    other, _ = oa.page_values(pages, spec, [1])
    assert np.all(np.isnan(other))  # a slot that nobody wrote


def test_rotation_is_a_complex_turn():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 2, 64))
    f = (500000.0 ** (-np.arange(16) / 16)).astype(np.float32)
    pos = np.array([0, 1, 977, 131071])
    for pairing in (oa.HALVES, oa.ADJACENT):
        y = oa.norm_rotate(x, None, 0.0, pos, f, pairing)
        for t in range(4):
            for j in range(16):
                a, b = (j, j + 16) if pairing == oa.HALVES else (2 * j, 2 * j + 1)
                z = complex(x[t, 1, a], x[t, 1, b]) * np.exp(1j * float(pos[t]) * float(f[j]))
                assert abs(complex(y[t, 1, a], y[t, 1, b]) - z) < 1e-12 * (1 + abs(z))
        assert np.array_equal(y[..., 32:], x[..., 32:])
    w = rng.standard_normal(64)
    y = oa.norm_rotate(x, w, 1e-6, pos, [], 0)
    r = math.sqrt(sum(float(a) ** 2 for a in x[1, 0]) / 64 + 1e-6)
    np.testing.assert_allclose(y[1, 0], x[1, 0] / r * w, rtol=1e-13)


@pytest.mark.parametrize("shape", [(2, 2, 21, 128), (1, 3, 9, 64)])
def test_pool_values_agree_with_the_decode(shape):
    """The rotated values, transformed back and rounded to bf16, are the C oracle's decode within one step."""
    k, v = synth.kv_bits(synth.WORKLOADS[3], 1, shape=shape)
    pool = oracle.pool_encode(k, v)
    kd, vd = oracle.pool_decode(pool, shape)
    for layer in range(shape[0]):
        keys, y = oa.pool_rotated(pool, shape, layer)
        vals = y @ oa.hadamard(shape[3]) / math.sqrt(shape[3])
        for got, want in ((keys, oa.f64(kd[layer])), (vals, oa.f64(vd[layer]))):
            assert np.all(np.abs(got - want) <= np.abs(got) * 2.0 ** -8 + 1e-30)


def test_attention_by_loops():
    rng = np.random.default_rng(9)
    q, k, v = rng.standard_normal((4, 64)), rng.standard_normal((2, 11, 64)), rng.standard_normal((2, 11, 64))
    out, lse, p = oa.attend(q, k, v, 0.3)
    for h in range(4):
        w = [math.exp(0.3 * sum(q[h, c] * k[h // 2, t, c] for c in range(64))) for t in range(11)]
        assert abs(lse[h] - math.log(sum(w))) < 1e-12
        for c in range(64):
            assert abs(out[h, c] - sum(w[t] * v[h // 2, t, c] for t in range(11)) / sum(w)) < 1e-12
    out, lse, _ = oa.attend(q, k[:, :0], v[:, :0], 0.3)
    assert not out.any() and np.all(lse == -np.inf)
