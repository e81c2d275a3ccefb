"""Attention through every plan: two row tiles a wave, units that stay whole
however long, parts by the hundred joined by one wave or by four, pools and
tails together. Each test asks the library which plan its call takes, so that
a changed threshold cannot move it off its kernel unseen."""

import math

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv
from attend_util import FORMATS, Store, bits, check_attend, host_f64, random_sequences, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from plan_util import one_wave_joins, page_plan, pool_plan, put_all
from test_gpu_attend import _pool_check

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _steps(fmt, most):
    """The largest step of values up to `most`, or None."""
    return None if fmt == ka.KVC_PAGE_BF16 else np.array([most / (127 if fmt == ka.KVC_PAGE_INT8 else 448)])


def _sequences(rng, spec, lens, cols):
    """random_sequences for many tokens: values of N(0, 1/4), all below 4."""
    num, heads, page, d, fmt = spec
    order, at = rng.permutation(num), 0
    table = np.full((len(lens), cols), -7, np.int32)
    slots = []
    for b, n in enumerate(lens):
        need = -(-n // page)
        table[b, :need] = order[at:at + need]
        at += need
        t = np.arange(n)
        slots.append(table[b, t // page].astype(np.int64) * page + t % page)
    assert at <= num
    slots = np.concatenate(slots)
    store = Store(spec)
    put_all(store.host, spec, bits(rng, (len(slots), heads, d)), bits(rng, (len(slots), heads, d), 0.5), slots)
    return store, table


def _call(spec, dev, q, table, lens, ws=None):
    n, hq, d = q.shape
    out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if ws is None:
        ws = torch.full((ka.kvpage_attend_workspace_bytes(spec, n, hq, table.shape[1] * spec[2]),), 0xFF, dtype=torch.uint8,
                        device=DEV)
    ka.kvpage_attend(spec, dev, to_dev(q), table, _i32(lens), out, ws, lse=lse, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    return out, lse


def _check(spec, store, table, lens, q, out, lse, which):
    o, l = host_f64(out), host_f64(lse)
    for b in which:
        k, v = sequence(store, table, b, lens[b])
        check_attend(o[b], l[b], oa.f64(q)[b], k, v, 1 / math.sqrt(spec[3]), spec[4] != 0, _steps(spec[4], 4.0), (b, lens[b]))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d, heads, group, page, lens, cols", [
    (128, 1, 48, 16, [5000, 333], 1024), (128, 2, 33, 64, [4200, 0], 128), (128, 1, 70, 256, [4097, 31, 129], 64),
    (64, 1, 17, 16, [700, 5000, 1, 0], 1024), (64, 2, 40, 32, [129, 3000], 256),
])
def test_two_row_tiles_over_pages(fmt, d, heads, group, page, lens, cols):
    rng = np.random.default_rng(d + group)
    spec = (sum(-(-n // page) for n in lens) + 2, heads, page, d, fmt)
    p = page_plan(spec, len(lens), heads * group, cols)
    say("two row tiles", spec, group, lens, p.W)
    assert p.rt == 2 and not p.whole
    store, table = _sequences(rng, spec, lens, cols)
    q = bits(rng, (len(lens), heads * group, d))
    out, lse = _call(spec, store.dev(), q, _i32(table), lens)
    _check(spec, store, table, lens, q, out, lse, range(len(lens)))


@pytest.mark.parametrize("fmt", FORMATS)
def test_units_that_stay_whole_however_long(fmt):
    """So many sequences that each unit is one workgroup's, with tables above 512 tokens: sequences of several rounds
    of page numbers (4096 tokens each) among short and empty ones."""
    rng = np.random.default_rng(21)
    d, page, n, group, cols = 128, 16, 4100, 2, 563
    lens = rng.choice([0, 1, 5, 17, 40], n)
    far = {3: 9001, 2000: 4097, 2001: 4096, 4099: 513, 4098: 600}
    for b, x in far.items():
        lens[b] = x
    spec = (int(np.sum(-(-lens // page))) + 1, 1, page, d, fmt)
    p = page_plan(spec, n, group, cols)
    assert p.whole and cols * page > 512 and p.units == n
    store, table = _sequences(rng, spec, lens, cols)
    q = bits(rng, (n, group, d))
    out, lse = _call(spec, store.dev(), q, _i32(table), lens)
    _check(spec, store, table, lens, q, out, lse, [*far, *rng.permutation(n)[:200]])
    assert bool((out[torch.from_numpy(lens == 0).to(DEV)] == 0).all()) and bool(torch.isfinite(out).all())


def test_hundreds_of_parts_joined_by_one_wave():
    """One long sequence among many short ones: 313 parts of one row, more than one for each lane of the wave."""
    rng = np.random.default_rng(22)
    n, page, d, group, cols = 100, 64, 128, 3, 640
    lens = rng.choice([0, 1, 64, 100], n)
    lens[41] = 40000
    spec = (int(np.sum(-(-lens // page))) + 1, 1, page, d, ka.KVC_PAGE_INT8)
    p = page_plan(spec, n, group, cols)
    blocks = int(np.sum(np.maximum(1, -(-lens // 128))))
    assert not p.whole and one_wave_joins(p) and blocks <= p.W   # a block a workgroup
    store, table = _sequences(rng, spec, lens, cols)
    q = bits(rng, (n, group, d))
    out, lse = _call(spec, store.dev(), q, _i32(table), lens)
    _check(spec, store, table, lens, q, out, lse, range(n))


def _encode(rng, shape):
    k, v = (torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).bfloat16() for _ in range(2))
    pool = kv.SharedKVPool.encode(k, v)
    torch.cuda.synchronize()
    return pool.pool, pool.pool.cpu().numpy()


def _pool_call(shape, pool, q, tail=None):
    n, hq, d = q.shape
    out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, hq), 7.0, device=DEV)
    need = ka.kvpool_attend_workspace_bytes(shape, n, hq, *((tail[0], tail[2].shape[1] * tail[0][2]) if tail else ()))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ka.kvpool_attend(shape, pool, 0, to_dev(q), out, ws, tail=tail, lse=lse)
    torch.cuda.synchronize()
    return out, lse


def _tails(store, table, lens, which, fmt):
    return [(*sequence(store, table, a, lens[a]), _steps(fmt, 4.0)) for a in which]


@pytest.mark.parametrize("d", [64, 128])
def test_hundreds_of_parts_joined_by_four_waves(d):
    """A pool of one kv head whose row has more than 256 parts, more than one for each lane of four waves, alone and
    with tails behind it."""
    rng = np.random.default_rng(d + 23)
    shape, agents, group = (1, 1, 70001, d), 2, 4
    pool, host = _encode(rng, shape)
    q = bits(rng, (agents, group, d))
    p = pool_plan(shape, agents, group)
    assert p.rt == 1 and p.units == 1 and p.W > 256 and not one_wave_joins(p)
    scale = 1 / math.sqrt(d)
    out, lse = _pool_call(shape, pool, q)
    _pool_check(host_f64(out), host_f64(lse), oa.f64(q), host, shape, 0, scale, None, d)
    spec, lens = (400, 1, 16, d, ka.KVC_PAGE_FP8), [5000, 3]
    assert pool_plan(shape, agents, group, True).W > 256 and not page_plan(spec, agents, group, 320, True).whole
    store, table = _sequences(rng, spec, lens, 320)
    out, lse = _pool_call(shape, pool, q, (spec, store.dev(), _i32(table), _i32(lens)))
    _pool_check(host_f64(out), host_f64(lse), oa.f64(q), host, shape, 0, scale, _tails(store, table, lens, range(2), spec[4]), d)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d", [64, 128])
def test_two_row_tiles_over_a_pool_with_tails(fmt, d):
    rng = np.random.default_rng(d + 24)
    shape, agents, group = (1, 2, 16500, d), 15, 4
    pool, host = _encode(rng, shape)
    lens = [300 - 21 * a if a % 4 else a for a in range(agents)]
    spec = (sum(-(-n // 16) for n in lens) + 1, 2, 16, d, fmt)
    q = bits(rng, (agents, 2 * group, d))
    assert pool_plan(shape, agents, 2 * group).rt == 2 and pool_plan(shape, agents, 2 * group, True).rt == 2
    pick = [0, 3, 7, 14]
    out, lse = _pool_call(shape, pool, q)
    _pool_check(host_f64(out)[pick], host_f64(lse)[pick], oa.f64(q)[pick], host, shape, 0, 1 / math.sqrt(d), None, d)
    store, table = _sequences(rng, spec, lens, 20)
    out, lse = _pool_call(shape, pool, q, (spec, store.dev(), _i32(table), _i32(lens)))
    _pool_check(host_f64(out)[pick], host_f64(lse)[pick], oa.f64(q)[pick], host, shape, 0, 1 / math.sqrt(d),
                _tails(store, table, lens, pick, fmt), (d, fmt))


def test_thousands_of_agents_whose_tails_stay_whole():
    rng = np.random.default_rng(25)
    d, n, cols = 128, 4100, 320
    shape = (1, 1, 40, d)
    pool, host = _encode(rng, shape)
    lens = rng.choice([0, 1, 5, 17], n)
    lens[7], lens[4099] = 5000, 4097
    spec = (int(np.sum(-(-lens // 16))) + 1, 1, 16, d, ka.KVC_PAGE_INT8)
    p = page_plan(spec, n, 1, cols, True)
    assert p.whole and cols * 16 > 512
    store, table = _sequences(rng, spec, lens, cols)
    q = bits(rng, (n, 1, d))
    out, lse = _pool_call(shape, pool, q, (spec, store.dev(), _i32(table), _i32(lens)))
    pick = [7, 4099, 0, *rng.permutation(n)[:100]]
    _pool_check(host_f64(out)[pick], host_f64(lse)[pick], oa.f64(q)[pick], host, shape, 0, 1 / math.sqrt(d),
                _tails(store, table, lens, pick, spec[4]), "whole tails")
    assert bool(torch.isfinite(out).all())


def test_one_row_of_a_table_for_all():
    """table_stride 0: sequences (and tails) that read one row of pages to different lengths."""
    rng = np.random.default_rng(26)
    d, page, lens = 64, 16, [700, 0, 33, 700, 16]
    spec = (50, 2, page, d, ka.KVC_PAGE_INT8)
    store, row = random_sequences(rng, spec, [700])
    tab = _i32(row).expand(len(lens), row.shape[1])
    assert tab.stride(0) == 0
    table = np.repeat(row, len(lens), 0)
    q = bits(rng, (len(lens), 6, d))
    out, lse = _call(spec, store.dev(), q, tab, lens)
    _check(spec, store, table, lens, q, out, lse, range(len(lens)))
    shape = (1, 2, 90, d)
    pool, host = _encode(rng, shape)
    out, lse = _pool_call(shape, pool, q, (spec, store.dev(), tab, _i32(lens)))
    _pool_check(host_f64(out), host_f64(lse), oa.f64(q), host, shape, 0, 1 / math.sqrt(d),
                _tails(store, table, lens, range(len(lens)), spec[4]), "one row")


def test_one_workspace_for_every_batch():
    """A workspace of the largest call (whose units stay whole, so it uses hardly any of it) for each smaller one,
    one after another without clearing: the bits of calls with workspaces of their own."""
    rng = np.random.default_rng(27)
    d, page, heads, group, cols = 128, 16, 8, 4, 64
    lens = rng.choice([0, 1, 40, 300, 900], 520, p=[0.2, 0.3, 0.4, 0.08, 0.02])
    lens[0] = 1000
    spec = (int(np.sum(-(-lens // page))) + 1, heads, page, d, ka.KVC_PAGE_FP8)
    assert page_plan(spec, 520, 32, cols).whole and not page_plan(spec, 511, 32, cols).whole
    store, table = _sequences(rng, spec, lens, cols)
    q, dev, tab = bits(rng, (520, heads * group, d)), store.dev(), _i32(table)
    shared = torch.full((ka.kvpage_attend_workspace_bytes(spec, 520, 32, cols * page),), 0xFF, dtype=torch.uint8, device=DEV)
    for n in (520, 511, 300, 64, 15, 1, 512):
        got = _call(spec, dev, q[:n], tab[:n], lens[:n], shared)
        want = _call(spec, dev, q[:n], tab[:n], lens[:n])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), n
        _check(spec, store, table, lens, q, *got, [0, n // 2, n - 1])
