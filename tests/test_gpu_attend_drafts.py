"""GPU parity of attention of few new tokens of each sequence (drafts to be verified, the last tokens of a prompt), which
kvpage_attend_prompt takes another way than long prompts (where tables hold more than 256 tokens a sequence): against
the formula in 64 bits."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import Store, bits, host_f64, sequence
from gpu_util import DEV, to_dev
from oracle import attend as oa
from serving_util import ALL_FORMATS, check_rows, default_scale, largest_steps, put_all, rows_see, status, store_of
from test_gpu_attend_prompt import _attend, _case, _check

pytestmark = pytest.mark.gpu
NONE = 0x7FC0


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, group, page, new, lens", [
    (1, 1, 16, [1], [1]),
    (2, 4, 16, [5, 0, 8, 1], [500, 40, 8, 700]),
    (3, 7, 64, [4, 2], [2000, 64]),                   # a token's rows in two units
    (1, 1, 32, [31, 33], [31, 1500]),
    (2, 4, 16, [4, 2, 3], [500, 40, 800]),            # one row tile (the others: two)
    (1, 4, 16, [60, 1, 1, 1, 1, 1, 1, 1, 1], [90, 1, 200, 17, 300, 16, 33, 40, 1000]),  # several row blocks of one
    (1, 16, 256, [2], [513]),
    (4, 2, 16, [3] * 20, list(range(3, 22)) + [300]),
])
def test_drafts(fmt, d, heads, group, page, new, lens):
    _case(fmt, d, heads, group, page, new, lens, 0, 0, layout="heads" if group == 4 else "fused" if group == 7 else "tokens")


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window, sinks", [(1, 0), (2, 1), (16, 16), (33, 4), (100, 65), (64, 500), (3000, 4)])
def test_windows_over_drafts(fmt, d, window, sinks):
    _case(fmt, d, 2, 4, 16, [6, 0, 8, 3], [700, 5, 8, 100], window, sinks)
    _case(fmt, d, 1, 1, 64, [20, 9], [1000, 2100], window, sinks, before=1, behind=2)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_more_drafts_than_tokens(fmt):
    _case(fmt, 64, 2, 2, 16, [10, 5, 7], [4, 0, 350], 0, 0, before=3, behind=7)
    _case(fmt, 128, 1, 4, 16, [6, 5, 7], [4, 0, 400], 9, 2, before=1)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_scales_of_drafts(fmt):
    for scale in (0.0, -0.2, 30.0):
        _case(fmt, 64, 1, 4, 16, [5], [300], 0, 0, scale=scale)


@pytest.mark.parametrize("n", [64, 65, 300])
def test_drafts_of_many_sequences(n):
    rng = np.random.default_rng(n)
    new = [int(x) for x in rng.integers(0, 7, n)]
    lens = [m + int(x) for m, x in zip(new, rng.integers(0, 400, n))]
    _case(ka.KVC_PAGE_INT8, 64, 1, 4, 16, new, lens, 0, 0, before=2, behind=1)
    _case(ka.KVC_PAGE_BF16, 64, 1, 4, 16, new, lens, 30, 2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("what", ["key", "value", "value inf"])
def test_non_finite_tokens_reach_the_drafts_that_see_them(fmt, d, what):
    """A row is not finite exactly where it sees a token that is not: the others are as if that token were any other."""
    rng = np.random.default_rng(61)
    heads, group, page, m, n, window = 2, 2, 16, 12, 400, 60
    spec = (40, heads, page, d, fmt)
    store, table = store_of(rng, spec, [n])
    dev = store.dev()
    x = np.full((1, heads, d), 0x3F80, np.uint16)
    y = x.copy()
    y[0, 1, d - 1] = 0x7F80 if what == "value inf" else NONE
    bad = [334, 394]  # at the windows' first tokens, and among the drafts
    for t in bad:
        slot = torch.tensor([int(table[0, t // page]) * page + t % page], device=DEV)
        ka.kvpage_write(spec, dev, to_dev(y if what == "key" else x), to_dev(x if what == "key" else y), slot)
    torch.cuda.synchronize()
    store.host[:] = dev.cpu().numpy()
    q = bits(rng, (m, heads * group, d))
    for win, sinks in ((0, 0), (window, 2), (window, 350)):
        out, lse = _attend(spec, dev, q, [0, m], table, [n], win, sinks)
        o, l = host_f64(out), host_f64(lse)
        see = rows_see(m, n, win, sinks)
        hit = see[:, bad].any(-1)
        k, v = sequence(store, table, 0, n)
        v = np.where(np.isfinite(v), v, 0)
        k = np.where(np.isfinite(k), k, 0)
        wrong = ~np.isfinite(o)
        assert not wrong[:, :group].any() and not wrong[~hit].any()
        first = 0 if what == "key" or fmt in (ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8) else d - 32 if fmt == ka.KVC_PAGE_FP4 else d - 1
        assert wrong[hit][:, group:, first:].all() and not wrong[:, :, :first].any()
        steps = largest_steps(store)
        for rows, hs in ((slice(None), slice(0, group)), (~hit, slice(group, None))):
            h = 0 if hs.start == 0 else 1
            check_rows(o[rows][:, hs], l[rows][:, hs], oa.f64(q)[rows][:, hs], k[h:h + 1], v[h:h + 1], default_scale(d), fmt,
                       steps, see[rows], (fmt, what, win, sinks))


@pytest.mark.parametrize("fmt", [ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8])
def test_drafted_values_of_very_different_sizes(fmt):
    """Steps that grow by 2^60 along the drafts: a row that does not see the large ones keeps its own bits."""
    rng = np.random.default_rng(62)
    d, n, m = 64, 60, 30
    spec = (20, 1, 16, d, fmt)
    store = Store(spec)
    k, v = bits(rng, (n, 1, d)), bits(rng, (n, 1, d))
    e = (v >> 7 & 255).astype(int) + np.round(np.linspace(-30, 30, n)).astype(int)[:, None, None]
    v = ((v & 0x807F) | (e << 7)).astype(np.uint16)
    put_all(store.host, spec, k, v, np.arange(n))
    table = np.arange(20, dtype=np.int32)[None]
    q = bits(rng, (m, 1, d))
    out, lse = _attend(spec, store.dev(), q, [0, m], table, [n])
    kk, vv = sequence(store, table, 0, n)
    # a row's own values alone bound its error
    for i in range(m):
        seen = n - m + 1 + i
        check_rows(host_f64(out)[i:i + 1], host_f64(lse)[i:i + 1], oa.f64(q)[i:i + 1], kk[:, :seen], vv[:, :seen],
                   default_scale(d), fmt, largest_steps(store), rows_see(1, seen), (fmt, i))


def test_bad_pages_lengths_and_starts_of_drafts_are_reported():
    rng = np.random.default_rng(63)
    spec = (40, 1, 16, 64, ka.KVC_PAGE_INT8)
    new, lens = [5, 3, 7, 1], [300, 50, 30, 80]
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    store, table = store_of(rng, spec, lens)
    dev, q = store.dev(), bits(rng, (16, 2, 64))
    ref, ref_lse = _attend(spec, dev, q, starts, table, lens)
    wrong = table.copy()
    wrong[0, 6], wrong[3, 0] = 30, -1
    st = status()
    out, lse = _attend(spec, dev, q, starts, wrong, lens, st=st)
    assert int(st) == ka.KVC_DEV_BAD_PAGE and torch.equal(out[5:15], ref[5:15]) and torch.equal(lse[5:15], ref_lse[5:15])
    full = np.where(table < 0, 0, table)
    for length in (-1, 305, -(1 << 31), (1 << 31) - 1):
        st = status()
        out, lse = _attend(spec, dev, q, starts, full, [300, length, 30, 80], st=st)
        assert int(st) == ka.KVC_DEV_BAD_LENGTH
        keep = list(range(5)) + list(range(8, 16))
        assert torch.equal(out[keep], ref[keep]) and torch.equal(lse[keep], ref_lse[keep])
    for bad in ([0, 5, 8, 15, 17], [-1, 5, 8, 15, 16], [0, 5, 3, 15, 16], [0, 1 << 30, 8, 15, 16], [0, 5, 8, -9, 16],
                [0, 16, 0, 16, 16]):
        st = status()
        _attend(spec, dev, q, bad, table, lens, st=st)
        assert int(st) == ka.KVC_DEV_BAD_START, bad


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_drafts_agree_with_a_long_prompt(fmt):
    """The same tokens at the end of a long batch and alone: two kernels, one formula."""
    rng = np.random.default_rng(64)
    lens = [900, 400]
    spec = (90, 2, 16, 128, fmt)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (304, 8, 128))
    for window, sinks in ((0, 0), (50, 4)):
        for starts, rows in (([0, 300, 304], slice(0, 304)), ([0, 4, 8], slice(296, 304))):
            out, lse = _attend(spec, store.dev(), q[rows], starts, table, lens, window, sinks)
            _check(spec, store, table, q[rows], starts, lens, window, sinks, out, lse)
