"""GPU parity of single-token attention with a sliding window and sinks
(kvpage_attend_window) against the oracle."""

import math

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import bits, check_attend, host_f64, place, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from serving_util import ALL_FORMATS, half, i32, largest_steps, status, store_of

pytestmark = pytest.mark.gpu


def _attend(spec, dev, q, table, lens, window, sinks, st=None, layout="tokens", scale=None):
    n, hq, d = q.shape
    out = place(np.full((n, hq, d), 0x7FC0, np.uint16), layout)
    lse = torch.full((n, hq), 7.0, device=DEV)
    need = ka.kvpage_attend_window_workspace_bytes(spec, n, hq, table.shape[1] * spec[2], window, sinks)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ka.kvpage_attend_window(spec, dev, place(q, layout), i32(table), i32(lens), window, sinks, out, ws, lse=lse, scale=scale,
                            dev_status=st)
    torch.cuda.synchronize()
    return out, lse


def _check(spec, store, table, q, lens, window, sinks, out, lse, scale=None, only=None):
    d, fmt = spec[3], spec[4]
    o, l = host_f64(out), host_f64(lse)
    for b, n in enumerate(lens):
        if only is not None and b not in only:
            continue
        k, v = sequence(store, table, b, n) if n else (np.zeros((spec[1], 0, d)),) * 2
        see = oa.seen(n, n - 1, window, sinks)
        check_attend(o[b], l[b], oa.f64(q)[b], k[:, see], v[:, see], 1 / math.sqrt(d) if scale is None else scale, half(fmt),
                     largest_steps(store), (spec, b, n, window, sinks))


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d, heads, group, page, lens", [
    (64, 2, 4, 16, [0, 1, 5, 40, 129, 700]), (128, 3, 7, 32, [33, 1000, 64]), (128, 1, 1, 256, [3000, 255, 257]),
    (64, 1, 40, 64, [500, 128, 127]), (128, 8, 4, 16, [2500])])
@pytest.mark.parametrize("window, sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 16), (33, 17), (640, 33), (5, 300)])
def test_window_and_sinks(fmt, d, heads, group, page, lens, window, sinks):
    rng = np.random.default_rng(sum(lens) + window)
    spec = (sum(-(-n // page) for n in lens) + 3, heads, page, d, fmt)
    say("window", spec, lens, window, sinks)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (len(lens), heads * group, d), 1.5)
    st = status()
    out, lse = _attend(spec, store.dev(), q, table, lens, window, sinks, st, "heads" if group == 4 else "tokens")
    assert int(st) == 0
    _check(spec, store, table, q, lens, window, sinks, out, lse)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_pages_between_sinks_and_window_may_be_gone(fmt):
    """Table entries of pages without a token that counts are no pages, and tokens that do not count are NaN."""
    rng = np.random.default_rng(20)
    lens, window, sinks, page = [900, 333, 4000], 70, 5, 16
    spec = (sum(-(-n // page) for n in lens), 2, page, 64, fmt)
    store, table = store_of(rng, spec, lens)
    dev = store.dev()
    q = bits(rng, (3, 4, 64))
    want = _attend(spec, dev, q, table, lens, window, sinks)
    gone = table.copy()
    for b, n in enumerate(lens):
        cols = np.arange(table.shape[1])
        gone[b, (cols * page >= sinks) & ((cols + 1) * page <= n - window)] = 1 << 30
        hidden = np.arange(sinks, n - window)
        x = np.full((len(hidden), 2, 64), 0x7FC0, np.uint16)
        slots = torch.from_numpy(table[b, hidden // page].astype(np.int64) * page + hidden % page).to(DEV)
        ka.kvpage_write(spec, dev, to_dev(x), to_dev(x), slots)
    st = status()
    got = _attend(spec, dev, q, gone, lens, window, sinks, st)
    assert int(st) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    _check(spec, store, table, q, lens, window, sinks, *got)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_no_window_and_wide_windows_are_plain_attention(fmt):
    rng = np.random.default_rng(21)
    lens = [70, 1, 2000, 0]
    spec = (140, 2, 16, 128, fmt)
    store, table = store_of(rng, spec, lens)
    dev, q = store.dev(), bits(rng, (4, 8, 128))
    out = torch.empty(4, 8, 128, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(4, 8, device=DEV)
    most = table.shape[1] * 16
    ws = torch.empty(ka.kvpage_attend_workspace_bytes(spec, 4, 8, most), dtype=torch.uint8, device=DEV)
    ka.kvpage_attend(spec, dev, to_dev(q), i32(table), i32(lens), out, ws, lse=lse)
    for window, sinks in ((0, 0), (0, 9), (most, 4), (1 << 31, 0), (0xFFFFFFFF, 0xFFFFFFFF), (most - 1, 0xFFFFFFFF)):
        got = _attend(spec, dev, q, table, lens, window, sinks)
        assert torch.equal(got[0], out) or window == most - 1, (window, sinks)
        _check(spec, store, table, q, lens, window, sinks, *got)


def test_many_sequences_and_bad_tables():
    """More sequences than a wave has lanes; bad pages among those that count, and bad lengths, are reported."""
    rng = np.random.default_rng(22)
    lens = [int(x) for x in rng.integers(0, 1500, 70)]
    spec = (sum(-(-n // 32) for n in lens) + 1, 1, 32, 64, ka.KVC_PAGE_INT8)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (70, 2, 64))
    dev = store.dev()
    for window, sinks in ((600, 4), (64, 0)):
        got = _attend(spec, dev, q, table, lens, window, sinks)
        _check(spec, store, table, q, lens, window, sinks, *got)
    big = int(np.argmax(lens))
    wrong = table.copy()
    wrong[big, (lens[big] - 1) // 32] = spec[0]
    st = status()
    got = _attend(spec, dev, q, wrong, lens, 64, 0, st)
    assert int(st) == ka.KVC_DEV_BAD_PAGE
    _check(spec, store, table, q, lens, 64, 0, *got, only=[b for b in range(70) if b != big])
    full = np.where(table < 0, 0, table)
    more = list(lens)
    more[3] = table.shape[1] * 32 + 1
    st = status()
    got = _attend(spec, dev, q, full, more, 64, 0, st)
    assert int(st) == ka.KVC_DEV_BAD_LENGTH
    _check(spec, store, table, q, lens, 64, 0, *got, only=[b for b in range(70) if b != 3])


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_far_and_negative_scales(fmt):
    rng = np.random.default_rng(23)
    lens = [300]
    spec = (20, 1, 16, 64, fmt)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (1, 2, 64))
    for scale in (0.0, -0.3, 40.0):
        got = _attend(spec, store.dev(), q, table, lens, 90, 3, scale=scale)
        _check(spec, store, table, q, lens, 90, 3, *got, scale=scale)
