"""Helpers of the tests of appending, 4-bit pages, windows and prompts: stores
written in one go, and the error bounds of the documented roundings."""

import math

import numpy as np
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import FORMATS, U_BF16, U_HALF, Store, bits, logit_bound, lse_bound
from gpu_util import DEV
from oracle import attend as oa

ALL_FORMATS = FORMATS + [ka.KVC_PAGE_FP4]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def half(fmt):
    """Whether a format's weights are rounded to binary16 (times the step)."""
    return fmt in (ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8)


def put_all(host, spec, k, v, slots):
    """oracle.attend.page_write of distinct slots inside the cache, vectorised."""
    num, heads, page, d, fmt = spec
    size, steps, each = oa.page_layout(spec)
    store = host.reshape(num, each)
    codes = store[:, :steps].reshape(num, 2, heads, page, int(d * size))
    n = oa.step_bytes(fmt, d)
    for j, x in enumerate((k, v)):
        if fmt == oa.BF16:
            codes[slots // page, j, :, slots % page] = np.ascontiguousarray(x).view(np.uint8).reshape(len(slots), heads, 2 * d)
            continue
        c, st = oa.quantise4(x) if fmt == oa.FP4 else oa.quantise(x, fmt)
        codes[slots // page, j, :, slots % page] = c.view(np.uint8)
        at = steps + n * ((j * heads + np.arange(heads)) * page + (slots % page)[:, None])
        raw = np.ascontiguousarray(st).view(np.uint8).reshape(len(slots), heads, n)
        for i in range(n):
            store[(slots // page)[:, None], at + i] = raw[..., i]


def store_of(rng, spec, lens, size_v=0.5, cols=None):
    """A store with `lens` tokens for each sequence in pages of random order, all other bytes 0xFF (NaN in each format);
    returns (store, table). holes(b): tokens of sequence b whose pages, if they hold no others, are given away."""
    num, heads, page, d, fmt = spec
    need = [-(-n // page) for n in lens]
    cols = max([1] + need) if cols is None else cols
    order = rng.permutation(num)
    assert sum(need) <= num
    table = np.full((len(lens), cols), -7, np.int32)
    store, at = Store(spec), 0
    for b, n in enumerate(lens):
        pages = order[at:at + need[b]]
        at += need[b]
        table[b, :need[b]] = pages
        if n:
            t = np.arange(n)
            put_all(store.host, spec, bits(rng, (n, heads, d)), bits(rng, (n, heads, d), size_v),
                    pages[t // page].astype(np.int64) * page + t % page)
    return store, table


def largest_steps(store):
    """The 8-bit steps of a store's written tokens (for out_bound's lost weights)."""
    spec = store.spec
    if not half(spec[4]):
        return None
    num, heads, page, d, fmt = spec
    steps, each = oa.page_layout(spec)[1:]
    s = np.ascontiguousarray(store.host.reshape(num, each)[:, steps:steps + 8 * heads * page]).view(np.float32)
    return s[np.isfinite(s)]


def check_rows(got, lse, q, keys, values, scale, fmt, steps, see, what=""):
    """Rows of one sequence. got [m, heads, d] and lse [m, heads] against the formula; q [m, heads, d] binary64; keys,
    values [kv_heads, T, d]; see [m, T]: what each row sees.

    Per row: the weights' rounding (bf16 or binary16), twice the weight's own error from its logit (numerator and
    sum) and exp2 (2^-20), the lane's sum of weights (32 of a tile, one after another, half a step each), the matrix
    cores' sums (four a tile, truncating) and 64 joins; binary16 weights below 2^-26 of the largest step lose up to
    2^-36 of that step each, times the largest code (448); the output's rounding. A weight below 2^-126, binary32's
    smallest normal number, becomes 0: the weights' sum is at least 1, that of the row's largest logit, whose own is
    never below the running maximum; so each of T tokens may cost 2^-126 of its value, which is all there is of a
    channel whose other values are 0 (logits 87 apart or more)."""
    m, heads, d = q.shape
    group = heads // keys.shape[0]
    T = keys.shape[1]
    rel = (U_HALF if half(fmt) else U_BF16) + 2.0 ** -20 + (T / 2 + 64) * 2.0 ** -24 + (T / 16 + 64) * 2.0 ** -23
    for h in range(heads):
        K, V = keys[h // group], values[h // group]
        # what no row sees may be NaN
        used = see.any(0)
        K, V = np.where(used[:, None], K, 0), np.where(used[:, None], V, 0)
        x = np.where(see, q[:, h] @ K.T * scale, -np.inf)
        top = np.max(x, -1, initial=-np.inf)
        base = np.where(np.isfinite(top), top, 0)
        p = np.exp(x - base[:, None])
        total = p.sum(-1)
        empty = total == 0
        p /= np.where(empty, 1, total)[:, None]
        want = p @ V
        dl = (np.abs(q[:, h]) @ np.abs(K).T).max(-1, initial=0) * abs(scale) * (2 * d + 8) * 2.0 ** -24 + np.abs(K).sum(
            -1).max(initial=0) * np.abs(q[:, h]).max(-1, initial=0) * abs(scale) * 2.0 ** -38
        b = p @ np.abs(V) * (rel + 2 * dl)[:, None]
        if steps is not None:
            b += T * np.max(steps, initial=0.0) * 448 * 2.0 ** -36
        b += T * 2.0 ** -126 * np.abs(V).max(0, initial=0)
        b += U_BF16 * (np.abs(want) + b)
        err = np.abs(got[:, h] - want)
        assert np.all(err <= b), f"{what} head {h}: off by {np.nanmax(err / np.maximum(b, 1e-300))} bounds"
        if lse is not None:
            assert np.all(lse[empty, h] == -np.inf), what
            wl = base[~empty] + np.log(total[~empty])
            lb = dl[~empty] + (T / 2 + 64) * 2.0 ** -24 + (T / 32 + 64) * 2.0 ** -23 + np.abs(wl) * 2.0 ** -22 + 2.0 ** -20
            assert np.all(np.abs(lse[~empty, h] - wl) <= lb), (what, np.max(np.abs(lse[~empty, h] - wl) / lb))


def rows_see(m, n, window=0, sinks=0):
    """What each of the m last of n tokens sees: [m, n]."""
    return np.stack([oa.seen(n, n - m + i, window, sinks) for i in range(m)]) if m else np.zeros((0, n), bool)


def default_scale(d):
    return 1 / math.sqrt(d)


__all__ = ["ALL_FORMATS", "Store", "bits", "check_rows", "default_scale", "half", "i32", "largest_steps", "logit_bound",
           "lse_bound", "put_all", "rows_see", "status", "store_of"]
