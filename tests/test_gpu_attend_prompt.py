"""GPU parity of attention of many new tokens (kvpage_attend_prompt) against
the formula in 64 bits."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import Store, bits, host_f64, place, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from serving_util import (ALL_FORMATS, check_rows, default_scale, i32, largest_steps, put_all, rows_see, status, store_of)

pytestmark = pytest.mark.gpu
NONE = 0x7FC0


def _attend(spec, dev, q, starts, table, lens, window=0, sinks=0, st=None, layout="tokens", scale=None):
    n, hq, d = q.shape
    out = place(np.full((n, hq, d), 0x4242, np.uint16), layout)
    lse = torch.full((n, hq), 7.0, device=DEV)
    need = ka.kvpage_attend_prompt_workspace_bytes(spec, len(lens), n, hq, table.shape[1] * spec[2], window, sinks)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ka.kvpage_attend_prompt(spec, dev, place(q, layout), i32(starts), i32(table), i32(lens), out, ws, window=window,
                            sinks=sinks, lse=lse, scale=scale, dev_status=st)
    torch.cuda.synchronize()
    return out, lse


def _check(spec, store, table, q, starts, lens, window, sinks, out, lse, scale=None, only=None):
    heads, d = spec[1], spec[3]
    o, l = host_f64(out), host_f64(lse)
    for b, n in enumerate(lens):
        if only is not None and b not in only:
            continue
        at = slice(starts[b], starts[b + 1])
        k, v = sequence(store, table, b, n) if n else (np.zeros((heads, 0, d)),) * 2
        check_rows(o[at], l[at], oa.f64(q)[at], k, v, default_scale(d) if scale is None else scale, spec[4],
                   largest_steps(store), rows_see(starts[b + 1] - starts[b], n, window, sinks), (spec, b, n, window, sinks))
    inside = np.zeros(len(o), bool)
    inside[starts[0]:starts[-1]] = True
    assert np.all(l[~inside] == 7.0) and np.all(out.view(torch.int16).cpu().numpy()[~inside] == 0x4242)


def _case(fmt, d, heads, group, page, new, lens, window, sinks, before=0, behind=0, layout="tokens", scale=None):
    rng = np.random.default_rng(sum(lens) + 31 * sum(new) + window + d)
    spec = (sum(-(-n // page) for n in lens) + 3, heads, page, d, fmt)
    say("prompt", spec, new, lens, window, sinks, layout)
    store, table = store_of(rng, spec, lens)
    starts = (before + np.concatenate([[0], np.cumsum(new)])).tolist()
    q = bits(rng, (starts[-1] + behind, heads * group, d), 1.5)
    q[:before], q[starts[-1]:] = NONE, NONE
    st = status()
    out, lse = _attend(spec, store.dev(), q, starts, table, lens, window, sinks, st, layout, scale)
    assert int(st) == 0
    _check(spec, store, table, q, starts, lens, window, sinks, out, lse, scale)


CASES = [
    # heads, group, page, new tokens, lengths with them
    (1, 1, 16, [1], [1]),
    (2, 4, 16, [3, 0, 33, 1], [3, 40, 100, 700]),
    (1, 4, 32, [130], [130]),
    (3, 7, 64, [70, 5], [200, 64]),
    (2, 1, 16, [129, 63, 64, 65], [129, 63, 128, 66]),
    (1, 16, 256, [40], [513]),
    (1, 40, 16, [7, 9], [9, 300]),
    (1, 130, 16, [3], [20]),
    (8, 4, 16, [300], [900]),
]


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, group, page, new, lens", CASES)
def test_prompts(fmt, d, heads, group, page, new, lens):
    _case(fmt, d, heads, group, page, new, lens, 0, 0, layout="heads" if group == 4 else "fused" if group == 7 else "tokens")


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window, sinks", [(1, 0), (16, 1), (64, 4), (65, 63), (100, 64), (200, 65), (33, 500)])
@pytest.mark.parametrize("heads, group, page, new, lens", [(2, 4, 16, [40, 0, 100], [700, 5, 100]), (1, 1, 64, [500], [1000]),
                                                           (1, 7, 32, [90, 1], [90, 400])])
def test_windows(fmt, d, window, sinks, heads, group, page, new, lens):
    _case(fmt, d, heads, group, page, new, lens, window, sinks)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("new, lens", [([4], [6000]), ([1, 6, 5], [3000, 40, 2500]), ([130], [4000])])
def test_few_rows_over_long_contexts(fmt, new, lens):
    """The tokens are shared out and the shares joined."""
    for heads, group, d, window in ((2, 4, 128, 0), (1, 1, 64, 0), (1, 8, 64, 2000)):
        _case(fmt, d, heads, group, 64, new, lens, window, 3, before=2, behind=3)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_more_rows_than_tokens_and_rows_of_no_sequence(fmt):
    """Rows that stand before the first token see nothing: zeros and -inf; rows outside all sequences stay as they were."""
    _case(fmt, 64, 2, 2, 16, [10, 5, 200], [4, 0, 150], 0, 0, before=3, behind=7)
    _case(fmt, 128, 1, 4, 16, [10, 5, 70], [4, 0, 40], 9, 2, before=1)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_scales(fmt):
    for scale in (0.0, -0.2, 30.0):
        _case(fmt, 64, 1, 4, 16, [50], [90], 0, 0, scale=scale)


def test_more_sequences_than_lanes():
    rng = np.random.default_rng(40)
    new = [int(x) for x in rng.integers(0, 9, 150)]
    lens = [m + int(x) for m, x in zip(new, rng.integers(0, 200, 150))]
    _case(ka.KVC_PAGE_INT8, 64, 1, 4, 16, new, lens, 0, 0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("what", ["key", "value", "value inf"])
def test_non_finite_tokens_reach_the_rows_that_see_them(fmt, d, what):
    """A row is not finite exactly where it sees a token that is not: the others are as if that token were any other."""
    rng = np.random.default_rng(41)
    heads, group, page, m, n, window = 2, 4, 16, 150, 200, 60
    bad = [77, 139]
    spec = (20, heads, page, d, fmt)
    store, table = store_of(rng, spec, [n])
    dev = store.dev()
    x = np.full((1, heads, d), 0x3F80, np.uint16)
    y = x.copy()
    y[0, 1, d - 1] = 0x7F80 if what == "value inf" else NONE
    for t in bad:
        slot = torch.tensor([int(table[0, t // page]) * page + t % page], device=DEV)
        ka.kvpage_write(spec, dev, to_dev(y if what == "key" else x), to_dev(x if what == "key" else y), slot)
    torch.cuda.synchronize()
    store.host[:] = dev.cpu().numpy()
    q = bits(rng, (m, heads * group, d))
    for win, sinks in ((0, 0), (window, 2), (window, 80)):
        out, lse = _attend(spec, dev, q, [0, m], table, [n], win, sinks)
        o, l = host_f64(out), host_f64(lse)
        see = rows_see(m, n, win, sinks)
        hit = see[:, bad].any(-1)
        k, v = sequence(store, table, 0, n)
        v = np.where(np.isfinite(v), v, 0)
        k = np.where(np.isfinite(k), k, 0)
        wrong = ~np.isfinite(o)
        assert not wrong[:, :group].any() and not wrong[~hit].any()
        # a key takes the whole row, a value its channel (a block, or the whole vector, with a step)
        first = 0 if what == "key" or fmt in (ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8) else d - 32 if fmt == ka.KVC_PAGE_FP4 else d - 1
        assert wrong[hit][:, group:, first:].all() and not wrong[:, :, :first].any()
        steps = largest_steps(store)
        for rows, hs in ((slice(None), slice(0, group)), (~hit, slice(group, None))):
            h = 0 if hs.start == 0 else 1
            check_rows(o[rows][:, hs], l[rows][:, hs], oa.f64(q)[rows][:, hs], k[h:h + 1], v[h:h + 1], default_scale(d), fmt,
                       steps, see[rows], (fmt, what, win, sinks))


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_a_query_that_is_nan_stays_in_its_row(fmt):
    rng = np.random.default_rng(42)
    spec = (9, 1, 16, 64, fmt)
    store, table = store_of(rng, spec, [100])
    q = bits(rng, (40, 2, 64))
    clean = _attend(spec, store.dev(), q, [0, 40], table, [100])
    q[7, 1, 3] = NONE
    out, lse = _attend(spec, store.dev(), q, [0, 40], table, [100])
    assert torch.isnan(out[7, 1]).all() and torch.isnan(lse[7, 1])
    keep = torch.ones(40, 2, dtype=torch.bool, device=DEV)
    keep[7, 1] = False
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("fmt", [ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8])
def test_values_of_very_different_sizes(fmt):
    """Steps that grow and fall by 2^60 along the tokens: what the exponent taken out of the weights has to follow."""
    rng = np.random.default_rng(43)
    d, n, m = 64, 320, 200
    spec = (20, 1, 16, d, fmt)
    for order in (np.linspace(-30, 30, n), np.linspace(30, -30, n)):
        store = Store(spec)
        k, v = bits(rng, (n, 1, d)), bits(rng, (n, 1, d))
        e = (v >> 7 & 255).astype(int) + np.round(order).astype(int)[:, None, None]
        v = ((v & 0x807F) | (e << 7)).astype(np.uint16)
        put_all(store.host, spec, k, v, np.arange(n))
        table = np.arange(20, dtype=np.int32)[None]
        q = bits(rng, (m, 2, d))
        out, lse = _attend(spec, store.dev(), q, [0, m], table, [n])
        kk, vv = sequence(store, table, 0, n)
        check_rows(host_f64(out), host_f64(lse), oa.f64(q), kk, vv, default_scale(d), fmt, largest_steps(store),
                   rows_see(m, n), fmt)


def test_bad_pages_lengths_and_starts_are_reported():
    rng = np.random.default_rng(44)
    spec = (30, 1, 16, 64, ka.KVC_PAGE_INT8)
    new, lens = [20, 10, 30, 4], [100, 50, 30, 80]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    store, table = store_of(rng, spec, lens)
    dev, q = store.dev(), bits(rng, (64, 2, 64))
    ref, ref_lse = _attend(spec, dev, q, starts, table, lens)
    wrong = table.copy()
    wrong[0, 6], wrong[3, 0] = 30, -1
    st = status()
    out, lse = _attend(spec, dev, q, starts, wrong, lens, st=st)
    assert int(st) == ka.KVC_DEV_BAD_PAGE and torch.equal(out[20:60], ref[20:60]) and torch.equal(lse[20:60], ref_lse[20:60])
    full = np.where(table < 0, 0, table)
    for length in (-1, 113, -(1 << 31), (1 << 31) - 1):
        st = status()
        out, lse = _attend(spec, dev, q, starts, full, [100, length, 30, 80], st=st)
        assert int(st) == ka.KVC_DEV_BAD_LENGTH
        keep = list(range(20)) + list(range(30, 64))
        assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])
    for bad in ([0, 20, 30, 60, 65], [-1, 20, 30, 60, 64], [0, 20, 10, 60, 64], [0, 1 << 30, 30, 60, 64], [0, 20, 30, -9, 64]):
        st = status()
        _attend(spec, dev, q, bad, table, lens, st=st)
        assert int(st) == ka.KVC_DEV_BAD_START, bad


def test_calls_repeat_and_neighbours_stay():
    """Strided outputs leave what lies between them; shared pages, tables that are columns of a wider one; the same bits."""
    rng = np.random.default_rng(45)
    spec = (60, 2, 16, 64, ka.KVC_PAGE_FP8)
    store, table = store_of(rng, spec, [900])
    wide = np.full((3, 70), 99, np.int32)
    wide[:, :57] = table[0]
    new, lens = [30, 2, 50], [900, 600, 50]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    q = bits(rng, (82, 6, 64))
    dev, tab = store.dev(), i32(wide)[:, :57]
    big = torch.full((84, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    out, lse = big[1:83, 1:7], torch.full((83, 6), 9.0, device=DEV)
    need = ka.kvpage_attend_prompt_workspace_bytes(spec, 3, 82, 6, 57 * 16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    runs = []
    for _ in range(2):
        ka.kvpage_attend_prompt(spec, dev, to_dev(q), i32(starts), tab, i32(lens), out, ws, lse=lse[:82])
        torch.cuda.synchronize()
        runs.append((out.clone(), lse.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[1:83, 1:7] = False
    assert bool((big[mask] == 3.0).all()) and bool((lse[82] == 9.0).all())
    for b, n in enumerate(lens):
        at = slice(starts[b], starts[b + 1])
        k, v = sequence(store, np.repeat(table, 3, 0), b, n)
        check_rows(host_f64(out)[at], host_f64(lse)[at], oa.f64(q)[at], k, v, default_scale(64), spec[4],
                   largest_steps(store), rows_see(new[b], n), b)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_one_new_token_is_single_token_attention(fmt):
    rng = np.random.default_rng(46)
    lens = [70, 1, 2000, 300]
    spec = (160, 2, 16, 128, fmt)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (4, 8, 128))
    starts = [0, 1, 2, 3, 4]
    for window, sinks in ((0, 0), (100, 4)):
        out, lse = _attend(spec, store.dev(), q, starts, table, lens, window, sinks)
        _check(spec, store, table, q, starts, lens, window, sinks, out, lse)


def test_offsets_past_32_bits():
    rng = np.random.default_rng(47)
    heads, page, d, n, m = 8, 256, 128, 700, 100
    for fmt in ALL_FORMATS:
        each = oa.page_layout((1, heads, page, d, fmt))[2]
        num = (1 << 32) // each + 4
        spec, small = (num, heads, page, d, fmt), (3, heads, page, d, fmt)
        big = torch.empty(ka.kvpage_bytes(spec), dtype=torch.uint8, device=DEV)
        store, table = store_of(rng, small, [n])
        few = store.dev()
        big[-3 * each:] = few
        q = bits(rng, (m, 16, d))
        a = _attend(spec, big, q, [0, m], table + (num - 3), [n])
        b = _attend(small, few, q, [0, m], table, [n])
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        del big
