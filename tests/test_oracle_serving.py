"""The oracle's 4-bit pages and visibility rule, against direct formulas."""

import numpy as np
import pytest

from agent_handoff_amd import synth
from oracle import attend as oa


def _bits(x):
    return synth.f32_to_bf16_bits(np.asarray(x, np.float32))


def test_codes_are_the_nearest_ones():
    """Every bf16 number beside a largest one that makes the power 1: the code is the nearest value, ties to the even code."""
    every = np.arange(1 << 16).astype(np.uint16)
    v = oa.f64(every)
    every = every[np.isfinite(v) & (np.abs(v) <= 7)]
    x = np.zeros((every.size, 32), np.uint16)
    x[:, 0], x[:, 5] = _bits([7.0])[0], every
    codes, powers = oa.quantise4(x)
    assert np.all(powers == 127)
    got = codes[:, 2] >> 4
    a = oa.f64(every)
    for code, y in zip(got, a):
        d = np.abs(np.minimum(abs(y), 6.0) - oa.E2M1[:8])
        best = np.nonzero(d == d.min())[0]
        assert (code & 7) in best and (len(best) == 1 or code % 2 == 0), (code, y)
    assert np.array_equal(got >> 3, np.signbit(a))


def test_powers():
    """The largest value of a block lies at 3.5 (not reached) to 7 times the power; ends of the range; zeros and non-finite."""
    for big, want in ((1.0, 125), (1.75, 125), (1.7578125, 126), (2.0, 126), (2.0 ** -123, 2), (2.0 ** -133, 2), (0.0, 2),
                      (3.0e38, 252), (np.inf, 255), (-np.nan, 255)):
        x = np.zeros((1, 64), np.uint16)
        x[0, 40] = _bits([big])[0]
        x[0, 3] = _bits([1.0])[0]
        codes, powers = oa.quantise4(x)
        assert powers[0, 1] == want and powers[0, 0] == 125, (big, powers)
        v = oa.values4(codes, powers)
        assert np.isnan(v[0, 32:]).all() == (want == 255) and v[0, 3] == 1.0 and not v[0, 4:32].any()


def test_error_of_a_code():
    """Within one power for what lies between 4 and 7 powers, half of one between 2 and 4, a quarter below."""
    rng = np.random.default_rng(3)
    x = _bits(rng.standard_normal((500, 128)) * np.exp(rng.standard_normal((500, 1)) * 5))
    codes, powers = oa.quantise4(x)
    p = np.repeat(np.exp2(powers.astype(float) - 127), 32, -1)
    y = oa.f64(x) / p
    err = np.abs(oa.values4(codes, powers) / p - y)
    assert np.all(np.abs(y) <= 7) and np.all(np.abs(y).reshape(500, 4, 32).max(-1) > 3.5)
    assert np.all(err <= np.where(np.abs(y) > 4, 1.0, np.where(np.abs(y) > 2, 0.5, 0.25)))


@pytest.mark.parametrize("fmt", [oa.BF16, oa.INT8, oa.FP8, oa.FP4])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_hold_what_is_written(fmt, d):
    rng = np.random.default_rng(4)
    spec = (5, 3, 16, d, fmt)
    pages = np.full(oa.page_bytes(spec), 0xFF, np.uint8)
    k, v = (_bits(rng.standard_normal((20, 3, d))) for _ in range(2))
    slots = rng.permutation(80)[:20]
    oa.page_write(pages, spec, k, v, slots)
    for got, x in zip(oa.page_values(pages, spec, slots), (k, v)):
        if fmt == oa.FP4:
            want = oa.values4(*oa.quantise4(x))
        elif fmt == oa.BF16:
            want = oa.f64(x)
        else:
            c, s = oa.quantise(x, fmt)
            want = (c.view(np.int8).astype(float) if fmt == oa.INT8 else oa.E4M3[c]) * s.astype(float)[..., None]
        assert np.array_equal(got, want)


def test_what_a_token_sees():
    for length in (0, 1, 5, 40):
        for at in range(-2, length):
            for window in (0, 1, 3, 50):
                for sinks in (0, 2, 100):
                    want = [t for t in range(length) if t <= at and (window == 0 or t < sinks or at - t < window)]
                    assert np.nonzero(oa.seen(length, at, window, sinks))[0].tolist() == want


def test_no_tokens():
    for fmt in (oa.INT8, oa.FP4):
        spec = (2, 3, 16, 64, fmt)
        k, v = oa.page_values(np.zeros(oa.page_bytes(spec), np.uint8), spec, np.zeros(0, np.int64))
        assert k.shape == v.shape == (0, 3, 64)
    assert oa.quantise4(np.zeros((0, 64), np.uint16))[0].shape == (0, 32)
