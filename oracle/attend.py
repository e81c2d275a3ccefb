"""Oracle of the operators of include/kvattend.h, in numpy binary64.

TEST INFRASTRUCTURE, as the rest of this package. bf16 arrays are uint16 bit
patterns; results are binary64 values before their last rounding, and the paged
cache is the exact bytes.
"""

import numpy as np

from . import codebook, pool_layout

HALVES, ADJACENT = 0, 1
BF16, INT8, FP8, FP4 = 0, 1, 2, 4
BLOCK4 = 32  # channels that share a power of two (FP4)


def f64(bits):
    """bf16 bits -> binary64 values."""
    return (np.asarray(bits, np.uint16).astype(np.uint32) << np.uint32(16)).view(np.float32).astype(np.float64)


def norm_rotate(x, weight, eps, positions, inv_freq, pairing):
    """x: binary64 [n, heads, d]; weight: binary64 [d] or None."""
    x = np.array(x, np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) * weight
    f = np.asarray(inv_freq, np.float32).astype(np.float64)
    n = f.size
    if n == 0:
        return x
    angle = np.asarray(positions, np.int64).astype(np.float64)[:, None] * f
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = (slice(0, n), slice(n, 2 * n)) if pairing == HALVES else (slice(0, 2 * n, 2), slice(1, 2 * n, 2))
    u, v = x[..., a].copy(), x[..., b].copy()
    x[..., a], x[..., b] = u * c - v * s, u * s + v * c
    return x


# ------------------------------------------------------------------ paged cache

def _e4m3_values():
    """The value of each e4m3 code (OCP: no infinities, 0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * np.exp2(e.astype(np.float64) - 7))
    v = np.where(c & 127 == 127, np.nan, v)
    return np.where(c & 128, -v, v)


E4M3 = _e4m3_values()


#: The value of each e2m1 code.
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def page_layout(spec):
    """(bytes of a code, offset of the steps in a page, bytes of a page)."""
    _, heads, page, d, fmt = spec
    size = {BF16: 2, FP4: 0.5}.get(fmt, 1)
    steps = int(2 * heads * page * d * size)
    return size, steps, -(-(steps + 2 * heads * page * step_bytes(fmt, d)) // 256) * 256


def step_bytes(fmt, d):
    """Bytes of a vector's step or steps."""
    return {BF16: 0, FP4: d // BLOCK4}.get(fmt, 4)


def page_bytes(spec):
    return spec[0] * page_layout(spec)[2]


def quantise(bits, fmt):
    """Codes (uint8) and steps (float32) of bf16 vectors [..., d], by exact arithmetic."""
    x = f64(bits)
    m = np.max(np.abs(x), -1)
    most = 127 if fmt == INT8 else 448
    bad = ~np.isfinite(np.sum(x, -1)) | np.any(~np.isfinite(x), -1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        step = np.where(bad, np.nan, m / most).astype(np.float32)
        safe = np.where(bad | (m == 0), 1.0, m)[..., None]
        # both factors are integers below 2^8 and 2^9 times powers of two: the
        # product is exact, and the binary64 quotient cannot cross a tie
        y = np.where((bad | (m == 0))[..., None], 0.0, x / 2.0 ** np.floor(np.log2(safe)) * most / (
            safe / 2.0 ** np.floor(np.log2(safe))))
    if fmt == INT8:
        return np.rint(y).astype(np.int8).view(np.uint8), step
    pos = E4M3[:127]
    a = np.abs(y)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    sign = np.where((np.asarray(bits) & 0x8000).astype(bool) & ~(bad | (m == 0))[..., None], 128, 0).astype(np.uint8)
    return code | sign, step


def quantise4(bits):
    """Codes (uint8, two to a byte) and powers (uint8) of bf16 vectors [..., d], by exact arithmetic."""
    x = f64(bits).reshape(*np.shape(bits)[:-1], np.shape(bits)[-1] // BLOCK4, BLOCK4)
    m = np.max(np.abs(x), -1)
    bad = ~np.isfinite(x).all(-1)
    m = np.where(bad | (m == 0), 2.0 ** -133, m)
    fraction, exponent = np.frexp(m)                       # fraction in [1/2, 1)
    e = np.clip(exponent - 3 + (fraction > 0.875), -125, 125)
    y = np.where(bad[..., None], 0.0, x) * np.exp2(-e.astype(np.float64))[..., None]
    a = np.minimum(np.abs(y), 6.0)
    hi = np.clip(np.searchsorted(E2M1[:8], a), 1, 7)
    lo = hi - 1
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    none = (bad | (np.max(np.abs(np.where(bad[..., None], 0, x)), -1) == 0))[..., None]
    code = np.where(none, 0, code | np.where(np.signbit(y), 8, 0)).astype(np.uint8).reshape(np.shape(bits))
    return code[..., 0::2] | code[..., 1::2] << 4, np.where(bad, 255, e + 127).astype(np.uint8)


def values4(codes, powers):
    """binary64 values [..., d] of codes [..., d / 2] and powers [..., d / 32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*powers.shape, BLOCK4)
    s = np.where(powers == 255, np.nan, np.exp2(powers.astype(np.float64) - 127))
    return (E2M1[c] * s[..., None]).reshape(*codes.shape[:-1], 2 * codes.shape[-1])


def page_write(pages, spec, k, v, slots):
    """Writes k, v (bits [n, heads, d]) into the uint8 array `pages`."""
    num, heads, page, d, fmt = spec
    size, steps, each = page_layout(spec)
    for i, slot in enumerate(slots):
        if slot < 0 or slot >= num * page:
            continue
        base = (slot // page) * each
        for j, x in enumerate((k[i], v[i])):
            for h in range(heads):
                line = (j * heads + h) * page + slot % page
                at = int(base + line * d * size)
                if fmt == FP4:
                    code, power = quantise4(x[h])
                    pages[at:at + d // 2] = code
                    st = base + steps + line * (d // BLOCK4)
                    pages[st:st + d // BLOCK4] = power
                elif fmt == BF16:
                    pages[at:at + 2 * d] = np.ascontiguousarray(x[h], np.uint16).view(np.uint8)
                else:
                    code, step = quantise(x[h], fmt)
                    pages[at:at + d] = code
                    st = base + steps + 4 * line
                    pages[st:st + 4] = np.array([step], np.float32).view(np.uint8)


def page_values(pages, spec, slots):
    """binary64 keys and values [n, heads, d] of the slots: code * step."""
    num, heads, page, d, fmt = spec
    size, steps, each = page_layout(spec)
    slots = np.asarray(slots, np.int64)
    store = pages.reshape(num, each)
    rows = store[:, :steps].reshape(num, 2, heads, page, int(d * size))
    x = rows[slots // page, :, :, slots % page]
    if fmt == FP4:
        n = d // BLOCK4
        s = store[:, steps:steps + 2 * heads * page * n].reshape(num, 2, heads, page, n)
        x = values4(x, s[slots // page, :, :, slots % page])
    elif fmt == BF16:
        x = f64(np.ascontiguousarray(x).view(np.uint16))
    else:
        s = np.ascontiguousarray(store[:, steps:steps + 8 * heads * page]).view(np.float32).reshape(num, 2, heads, page)
        s = s[slots // page, :, :, slots % page].astype(np.float64)[..., None]
        x = (x.view(np.int8).astype(np.float64) if fmt == INT8 else E4M3[x]) * s
    return x[:, 0], x[:, 1]


# ------------------------------------------------------------------ attention

def hadamard(d):
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h


def pool_rotated(pool, shape, layer):
    """binary64 keys [H, T, d], and rotated values (level times size) [H, T, d], of one layer of pool bytes."""
    L, H, T, d = shape
    k_scale, k_codes, v_scale, v_codes = pool_layout(*shape)[:4]
    first, n = layer * H * T, H * T
    step = float(pool[k_scale:k_scale + 4 * L].view(np.float32)[layer])
    k = pool[k_codes + first * d:k_codes + (first + n) * d].view(np.int8).astype(np.float64) * step
    size = pool[v_scale + 2 * first:v_scale + 2 * (first + n)].view(np.float16).astype(np.float64)
    w = 3 * d // 8
    planes = pool[v_codes + first * w:v_codes + (first + n) * w].reshape(n, 3, d // 8)
    bits = np.unpackbits(planes, axis=-1, bitorder="little").astype(np.int64)
    levels = np.asarray(codebook.codec_table()[0], np.float64)
    y = levels[bits[:, 0] + 2 * bits[:, 1] + 4 * bits[:, 2]] * size[:, None]
    return k.reshape(H, T, d), y.reshape(H, T, d)


def seen(length, position, window=0, sinks=0):
    """Which of `length` tokens the one at `position` sees."""
    t = np.arange(length)
    s = t <= position
    return s & ((t < sinks) | (t > position - window)) if window else s


def attend(q, keys, values, scale):
    """q: binary64 [heads, d]; keys, values: [kv_heads, T, d]. Returns (out
    [heads, d], lse [heads], p [heads, T])."""
    heads, d = q.shape
    group = heads // keys.shape[0]
    out, lse, ps = np.zeros((heads, d)), np.full(heads, -np.inf), np.zeros((heads, keys.shape[1]))
    if keys.shape[1] == 0:
        return out, lse, ps
    for h in range(heads):
        with np.errstate(invalid="ignore"):
            x = keys[h // group] @ q[h] * scale
            m = np.max(x)
            p = np.exp(x - m)
            lse[h] = m + np.log(np.sum(p))
            ps[h] = p / np.sum(p)
            out[h] = ps[h] @ values[h // group]
    return out, lse, ps
