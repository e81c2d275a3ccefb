"""GPU parity of single-token attention over pages (kvpage_attend) and over
the shared pool with tails (kvpool_attend) against the binary64 oracle, with
the bounds of attend_util."""

import math

import numpy as np
import pytest
import torch

import oracle
from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv
from agent_handoff_amd import synth
from attend_util import (FORMATS, U_BF16, bits, check_attend, host_f64, logit_bound, lse_bound, out_bound, place,
                         random_sequences, sequence)
from gpu_util import DEV, say, to_dev, to_host
from oracle import attend as oa

pytestmark = pytest.mark.gpu


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)


def _steps(store):
    """Largest finite step of a store (what weights are scaled by)."""
    spec = store.spec
    if spec[4] == 0:
        return None
    _, at, each = oa.page_layout(spec)
    s = store.host.reshape(spec[0], each)[:, at:at + 8 * spec[1] * spec[2]].copy().view(np.float32)
    return s[np.isfinite(s)] if np.isfinite(s).any() else np.zeros(1)


def _pages_attend(spec, dev, q, table, lens, scale=None, layout="tokens", with_lse=True, status=None):
    n, hq, d = q.shape
    out = place(np.full((n, hq, d), 0x7FC0, np.uint16), layout)
    lse = torch.full((n, hq), 7.0, dtype=torch.float32, device=DEV) if with_lse else None
    cols = table.shape[1] * spec[2]
    ws = torch.full((ka.kvpage_attend_workspace_bytes(spec, n, hq, cols),), 0xFF, dtype=torch.uint8, device=DEV)
    ka.kvpage_attend(spec, dev, place(q, layout), _i32(table), _i32(lens), out, ws, lse=lse, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d, heads, group, page, lens", [
    (128, 1, 1, 16, [1]),
    (64, 2, 4, 16, [0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129]),
    (128, 2, 4, 32, [257, 0, 1, 511, 512, 513]),
    (128, 1, 7, 64, [1000, 63, 64, 65]),
    (64, 1, 16, 128, [100, 300]),
    (128, 1, 17, 16, [40, 290]),
    (64, 3, 33, 16, [77, 0]),
    (128, 1, 70, 256, [600]),
    (64, 1, 2, 16, [4500, 3]),
])
def test_pages(fmt, d, heads, group, page, lens):
    rng = np.random.default_rng(len(lens) + d + group)
    need = sum(-(-n // page) for n in lens)
    spec = (need + 3, heads, page, d, fmt)
    say("attend pages", spec, group, lens)
    store, table = random_sequences(rng, spec, lens)
    q = bits(rng, (len(lens), heads * group, d), 1.5)
    for layout, scale in (("tokens", None), ("fused", 0.31), ("heads", -0.05)):
        status = _status()
        out, lse = _pages_attend(spec, store.dev(), q, table, lens, scale, layout, status=status)
        assert int(status) == 0
        o, l = host_f64(out), host_f64(lse)
        for b, n in enumerate(lens):
            k, v = sequence(store, table, b, n)
            check_attend(o[b], l[b], oa.f64(q)[b], k, v, 1 / math.sqrt(d) if scale is None else scale, fmt != 0,
                         _steps(store), (layout, b, n))


@pytest.mark.parametrize("fmt", FORMATS)
def test_one_token_is_its_value(fmt):
    """A single token has weight 1: the output is its value, rounded once (binary16 holds a code's bits)."""
    rng = np.random.default_rng(3)
    spec = (2, 3, 16, 128, fmt)
    store, table = random_sequences(rng, spec, [1, 1])
    q = bits(rng, (2, 6, 128), 100.0)
    out, lse = _pages_attend(spec, store.dev(), q, table, [1, 1])
    for b in range(2):
        k, v = sequence(store, table, b, 1)
        want = np.repeat(v[:, 0], 2, axis=0)
        tol = U_BF16 if fmt == 0 else U_BF16 + 1.01 * 2.0 ** -11
        assert np.all(np.abs(host_f64(out)[b] - want) <= np.abs(want) * tol + 1e-30)


@pytest.mark.parametrize("fmt", FORMATS)
def test_peaked_flat_and_far_logits(fmt):
    """Weights that are one-hot, all equal (scale 0), or hundreds of powers of two apart; rising and falling
    logits, so that the running maximum moves in every tile or in the first alone."""
    rng = np.random.default_rng(4)
    d, n, page = 64, 700, 16
    spec = (2 * 44 + 1, 1, page, d, fmt)
    for order in (1, -1):
        store, table = random_sequences(rng, spec, [n, n])
        ramp = np.linspace(-3, 3, n)[::order]
        k = np.zeros((n, 1, d), np.float32)
        k[:, 0, 0] = ramp
        k[:, 0, 1:] = 0.01 * rng.standard_normal((n, d - 1))
        t = np.arange(n)
        for b in range(2):
            store.put(synth.f32_to_bf16_bits(k), bits(rng, (n, 1, d), 10.0 ** (3 * b)), table[b, t // page] * page + t % page)
        q = bits(rng, (2, 3, d))
        q[:, 0, 0] = synth.f32_to_bf16_bits(np.float32([50.0]))[0]
        q[:, 1, 0] = synth.f32_to_bf16_bits(np.float32([-300.0]))[0]
        for scale in (0.0, 0.125, 3.0):
            out, lse = _pages_attend(spec, store.dev(), q, table, [n, n], scale)
            for b in range(2):
                kk, vv = sequence(store, table, b, n)
                check_attend(host_f64(out)[b], host_f64(lse)[b], oa.f64(q)[b], kk, vv, scale, fmt != 0, _steps(store),
                             (order, scale, b))


@pytest.mark.parametrize("fmt", [ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8])
def test_values_of_very_different_sizes(fmt):
    """Steps that rise by 2^60 along the sequence, or fall, and zero vectors between them."""
    rng = np.random.default_rng(5)
    d, n, page = 128, 300, 32
    spec = (11, 1, page, d, fmt)
    for order in (1, -1):
        store, table = random_sequences(rng, spec, [n])
        size = (2.0 ** np.linspace(-30, 30, n)[::order]).astype(np.float32)
        v = rng.standard_normal((n, 1, d)).astype(np.float32) * size[:, None, None]
        v[5::7] = 0
        t = np.arange(n)
        slots = table[0, t // page] * page + t % page
        store.put(bits(rng, (n, 1, d)), synth.f32_to_bf16_bits(v), slots)
        q = bits(rng, (1, 4, d))
        out, lse = _pages_attend(spec, store.dev(), q, table, [n])
        kk, vv = sequence(store, table, 0, n)
        check_attend(host_f64(out)[0], host_f64(lse)[0], oa.f64(q)[0], kk, vv, 1 / math.sqrt(d), True, _steps(store), order)


@pytest.mark.parametrize("fmt", FORMATS)
def test_non_finite_values_stay_where_they_belong(fmt):
    """A NaN query row is NaN alone; a NaN key or value that counts makes its heads NaN; unused slots hold NaN
    throughout (the store's filling) and change nothing."""
    rng = np.random.default_rng(6)
    d, page, lens = 64, 16, [40, 40, 21]
    spec = (9, 2, page, d, fmt)
    store, table = random_sequences(rng, spec, lens)
    k, v = bits(rng, (1, 2, d)), bits(rng, (1, 2, d))
    k[0, 0, 3] = 0x7FC0
    store.put(k, v, [table[1, 1] * page + 2])       # head 0 of sequence 1
    q = bits(rng, (3, 4, d))
    q[0, 1, 7] = 0x7FC0
    out, lse = _pages_attend(spec, store.dev(), q, table, lens)
    o, l = host_f64(out), host_f64(lse)
    assert np.all(np.isnan(o[0, 1])) and np.isnan(l[0, 1])
    assert np.all(np.isnan(o[1, :2])) and np.all(np.isnan(l[1, :2]))
    for b, hs in ((0, [0]), (0, [2, 3]), (1, [2, 3]), (2, [0, 1]), (2, [2, 3])):
        kk, vv = sequence(store, table, b, lens[b])
        g = hs[0] // 2
        check_attend(o[b][hs], l[b][hs], oa.f64(q)[b][hs], kk[g:g + 1], vv[g:g + 1], 1 / math.sqrt(d), fmt != 0,
                     _steps(store), (b, hs))


def test_bad_pages_and_lengths_are_reported():
    """Sequences with a page that is none or a length that does not fit say so; the others are right."""
    rng = np.random.default_rng(7)
    spec = (8, 1, 16, 64, ka.KVC_PAGE_INT8)
    lens = [33, 20, 16, 30]
    store, table = random_sequences(rng, spec, lens, cols=3)
    q = bits(rng, (4, 2, 64))
    ref, ref_lse = _pages_attend(spec, store.dev(), q, table, lens)
    bad = table.copy()
    bad[0, 1] = 8
    bad[2, 0] = -1
    status = _status()
    out, lse = _pages_attend(spec, store.dev(), q, bad, lens, status=status)
    assert int(status) == ka.KVC_DEV_BAD_PAGE
    assert torch.equal(out[[1, 3]], ref[[1, 3]]) and torch.equal(lse[[1, 3]], ref_lse[[1, 3]])
    full = table.copy()
    full[full < 0] = 0
    for wrong in (-1, 49, -(1 << 31), (1 << 31) - 1):
        status = _status()
        out, lse = _pages_attend(spec, store.dev(), q, full, [33, wrong, 16, 30], status=status)
        assert int(status) == ka.KVC_DEV_BAD_LENGTH
        assert torch.equal(out[[0, 2, 3]], ref[[0, 2, 3]]) and torch.equal(lse[[0, 2, 3]], ref_lse[[0, 2, 3]])


def test_shared_pages_strided_tables_and_no_lse():
    """Two sequences over the same pages (a fork), tables that are columns of a wider one; lse left out."""
    rng = np.random.default_rng(8)
    spec = (6, 2, 16, 128, ka.KVC_PAGE_BF16)
    store, table = random_sequences(rng, spec, [70])
    wide = np.full((3, 9), 99, np.int32)
    wide[:, :5] = table[0]
    lens = [70, 69, 3]
    q = bits(rng, (3, 4, 128))
    dev, tab = store.dev(), _i32(wide)[:, :5]
    out = torch.empty(3, 4, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(ka.kvpage_attend_workspace_bytes(spec, 3, 4, 80), dtype=torch.uint8, device=DEV)
    ka.kvpage_attend(spec, dev, to_dev(q), tab, _i32(lens), out, ws)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        k, v = sequence(store, np.repeat(table, 3, 0), b, n)
        check_attend(host_f64(out)[b], None, oa.f64(q)[b], k, v, 1 / math.sqrt(128), False, None, b)


def test_neighbours_stay_and_calls_repeat_bit_for_bit():
    """Rows behind the last sequence and between strided rows are left as they were; a second call gives the same bits."""
    rng = np.random.default_rng(9)
    spec = (80, 2, 16, 64, ka.KVC_PAGE_FP8)
    lens = [600, 5, 300]
    store, table = random_sequences(rng, spec, lens)
    q = bits(rng, (3, 6, 64))
    dev = store.dev()
    big = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    out = big[1:4, 1:7]
    lse = torch.full((4, 6), 9.0, device=DEV)
    ws = torch.empty(ka.kvpage_attend_workspace_bytes(spec, 3, 6, table.shape[1] * 16), dtype=torch.uint8, device=DEV)
    runs = []
    for _ in range(2):
        ka.kvpage_attend(spec, dev, to_dev(q), _i32(table), _i32(lens), out, ws, lse=lse[:3])
        torch.cuda.synchronize()
        runs.append((out.clone(), lse.clone()))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    mask = torch.ones_like(big, dtype=torch.bool)
    mask[1:4, 1:7] = False
    assert bool((big[mask] == 3.0).all()) and bool((lse[3] == 9.0).all())


# ------------------------------------------------------------------ pool

def _pool_check(got, lse, q, pool, shape, layer, scale, tails, what):
    """tails: (keys, values, steps) of each agent's own tokens or None."""
    d = shape[3]
    keys, rot = oa.pool_rotated(pool, shape, layer)
    vals = rot @ oa.hadamard(d) / math.sqrt(d)
    sizes = np.max(np.abs(rot), -1)
    for a in range(q.shape[0]):
        k, v = keys, vals
        if tails is not None:
            k, v = np.concatenate([keys, tails[a][0]], 1), np.concatenate([vals, tails[a][1]], 1)
        want, wl, p = oa.attend(q[a], k, v, scale)
        dl = logit_bound(q[a], k, scale)
        T = shape[2]
        # the pool's part in rotated space: the transform spreads each bound over all channels
        inner = out_bound(want, p[:, :T], rot, dl, k.shape[1], True, sizes, levels=True)
        b = np.repeat(np.sum(inner, -1, keepdims=True) / math.sqrt(d), d, -1) + np.abs(want) * 2.0 ** -20
        if tails is not None and tails[a][0].shape[1]:
            b = b + out_bound(want, p[:, T:], tails[a][1], dl, k.shape[1], tails[a][2] is not None, tails[a][2])
        b = b + U_BF16 * (np.abs(want) + b)
        err = np.abs(got[a] - want)
        assert np.all(err <= b), f"{what} agent {a}: off by {np.max(err / np.maximum(b, 1e-300))} bounds"
        assert np.all(np.abs(lse[a] - wl) <= lse_bound(wl, dl, k.shape[1])), what


def _pool_attend(shape, pool, layer, q, tail=None, scale=None, layout="tokens", status=None):
    n, hq, d = q.shape
    out = place(np.full((n, hq, d), 0x7FC0, np.uint16), layout)
    lse = torch.full((n, hq), 7.0, device=DEV)
    need = ka.kvpool_attend_workspace_bytes(shape, n, hq, tail[0] if tail else None,
                                            tail[2].shape[1] * tail[0][2] if tail else 0)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ka.kvpool_attend(shape, pool, layer, place(q, layout), out, ws, tail=tail, lse=lse, scale=scale, dev_status=status)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("shape, agents, group", [
    ((1, 1, 1, 64), 1, 1), ((2, 2, 31, 128), 1, 4), ((1, 2, 33, 64), 3, 2), ((3, 1, 100, 128), 15, 4),
    ((1, 1, 257, 64), 64, 3), ((1, 2, 700, 128), 5, 7), ((2, 1, 2051, 128), 2, 1), ((1, 1, 300, 128), 64, 16),
])
def test_pool(shape, agents, group):
    rng = np.random.default_rng(shape[2])
    say("attend pool", shape, agents, group)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 2, shape=shape)
    pool = oracle.pool_encode(k, v)
    dev = torch.from_numpy(pool).to(DEV)
    q = bits(rng, (agents, shape[1] * group, shape[3]), 1.0)
    for layer, layout, scale in ((shape[0] - 1, "tokens", None), (0, "fused", 0.2)):
        status = _status()
        out, lse = _pool_attend(shape, dev, layer, q, None, scale, layout, status)
        assert int(status) == 0
        _pool_check(host_f64(out), host_f64(lse), oa.f64(q), pool, shape, layer,
                    1 / math.sqrt(shape[3]) if scale is None else scale, None, (shape, layer))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape, lens", [((2, 2, 90, 64), [0, 1, 40]), ((1, 1, 600, 128), [300, 0, 17, 16]),
                                        ((1, 2, 5, 128), [0, 0])])
def test_pool_with_tails(fmt, shape, lens):
    rng = np.random.default_rng(11)
    L, H, T, d = shape
    k, v = synth.kv_bits(synth.WORKLOADS[3], 3, shape=shape)
    pool = oracle.pool_encode(k, v)
    page = 16
    spec = (sum(-(-n // page) for n in lens) + 2, H, page, d, fmt)
    store, table = random_sequences(rng, spec, lens, size_v=2.0)
    q = bits(rng, (len(lens), 4 * H, d))
    status = _status()
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), L - 1, q, (spec, store.dev(), _i32(table), _i32(lens)),
                            status=status)
    assert int(status) == 0
    tails = [(*sequence(store, table, a, n), _steps(store)) for a, n in enumerate(lens)]
    _pool_check(host_f64(out), host_f64(lse), oa.f64(q), pool, shape, L - 1, 1 / math.sqrt(d), tails, (fmt, shape))


def test_pool_sizes_far_apart_and_a_heavy_sink():
    """Value vectors from 2^-12 to 2^12 in size, zero vectors, and one token that takes nearly all weight."""
    shape = (1, 1, 400, 128)
    rng = np.random.default_rng(12)
    k = rng.standard_normal(shape).astype(np.float32)
    k[0, 0, 0] = 0
    k[0, 0, 0, 5] = 30
    v = rng.standard_normal(shape).astype(np.float32) * 2.0 ** rng.integers(-12, 13, (1, 1, 400, 1))
    v[0, 0, 0] *= 1e-3
    v[0, 0, 7::9] = 0
    pool = oracle.pool_encode(synth.f32_to_bf16_bits(k), synth.f32_to_bf16_bits(v.astype(np.float32)))
    q = rng.standard_normal((2, 4, 128)).astype(np.float32)
    q[0, :, 5] = 4
    qb = synth.f32_to_bf16_bits(q)
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), 0, qb)
    _pool_check(host_f64(out), host_f64(lse), oa.f64(qb), pool, shape, 0, 1 / math.sqrt(128), None, "sizes")


def test_pool_header_is_checked():
    shape = (1, 1, 40, 64)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 1, shape=shape)
    pool = oracle.pool_encode(k, v)
    pool[8] ^= 1
    spec = (2, 1, 16, 64, 1)
    rng = np.random.default_rng(1)
    store, table = random_sequences(rng, spec, [3, 4])
    q = bits(rng, (2, 2, 64))
    for tail in (None, (spec, store.dev(), _i32(table), _i32([3, 4]))):
        status = _status()
        out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), 0, q, tail, status=status)
        assert int(status) == kv.KVC_DEV_BAD_HEADER
        assert np.all(to_host(out) == 0x7FC0) and bool((lse == 7.0).all())


def test_pool_attention_agrees_with_decode_and_attention():
    """The operator against the path it replaces: kvpool_decode, then plain attention over the decoded cache."""
    shape, agents, group = (2, 2, 500, 128), 3, 4
    rng = np.random.default_rng(13)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 5, shape=shape)
    pool = kv.SharedKVPool.encode(to_dev(k), to_dev(v))
    q = bits(rng, (agents, 2 * group, 128))
    out = pool.attend(1, to_dev(q))
    ko, vo = pool.decode_layers(1, 2)
    torch.cuda.synchronize()
    for a in range(agents):
        want, _, p = oa.attend(oa.f64(q)[a], host_f64(ko[0])[0], host_f64(vo[0])[0], 1 / math.sqrt(128))
        kk, rot = oa.pool_rotated(pool.pool.cpu().numpy(), shape, 1)
        # the decode rounds keys and values to bf16: values 2^-8 of each, logits 2^-8 of sum |q k|
        dl = np.max(np.abs(np.repeat(kk, group, 0)) @ np.abs(oa.f64(q)[a])[..., None], axis=(1, 2)) / math.sqrt(128) * 2.0 ** -8
        vals = np.abs(host_f64(vo[0])[0])
        for h in range(2 * group):
            b = (p[h] @ vals[h // group]) * (2 * dl[h] + 2.0 ** -8) * 1.1 + np.abs(want[h]) * 2.0 ** -8
            inner = np.sum(p[h] @ np.abs(rot[h // group])) / math.sqrt(128) * 2.0 ** -9
            assert np.all(np.abs(host_f64(out)[a, h] - want[h]) <= b + inner)


# ------------------------------------------------------------------ streams, graphs, runs together

def test_two_streams_at_once_and_graph_replays():
    """Two calls of different sequences on two streams with workspaces of their own; then one captured and replayed
    over changed queries, pages, tables and lengths, with eager calls of the same kind in between."""
    rng = np.random.default_rng(14)
    spec = (400, 2, 16, 128, ka.KVC_PAGE_INT8)
    q, ws, out, ref, tabs, lens, devs = [], [], [], [], [], [], []
    for i in range(2):
        n = [700 + i, 900, 64]
        store, table = random_sequences(rng, spec, n, cols=64)
        devs.append(store.dev())
        tabs.append(_i32(table))
        lens.append(_i32(n))
        q.append(to_dev(bits(rng, (3, 8, 128))))
        ws.append(torch.empty(ka.kvpage_attend_workspace_bytes(spec, 3, 8, 1024), dtype=torch.uint8, device=DEV))
        out.append(torch.zeros(3, 8, 128, dtype=torch.bfloat16, device=DEV))
        ref.append(torch.zeros_like(out[-1]))
        ka.kvpage_attend(spec, devs[i], q[i], tabs[i], lens[i], ref[i], ws[i])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for i in range(2):
            ka.kvpage_attend(spec, devs[i], q[i], tabs[i], lens[i], out[i], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(out[i], ref[i])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ka.kvpage_attend(spec, devs[0], q[0], tabs[0], lens[0], out[0], ws[0])
    for step in range(4):
        n = [900 - step, step, 1024]
        store, table = random_sequences(rng, spec, n, cols=64)
        devs[0].copy_(store.dev())
        tabs[0].copy_(_i32(table))
        lens[0].copy_(_i32(n))
        q[0].copy_(to_dev(bits(rng, (3, 8, 128))))
        g.replay()
        ka.kvpage_attend(spec, devs[1], q[1], tabs[1], lens[1], out[1], ws[1])
        torch.cuda.synchronize()
        ka.kvpage_attend(spec, devs[0], q[0], tabs[0], lens[0], ref[0], ws[1])
        torch.cuda.synchronize()
        assert torch.equal(out[0], ref[0]) and torch.equal(out[1], ref[1]), step


@pytest.mark.parametrize("fmt", FORMATS)
def test_agents_generate_behind_a_shared_document(fmt):
    """The operators as they are used: each step turns the projection's rows in place, writes the new keys and values
    to the agents' pages and attends to the document and the pages, all in one captured graph replayed per step.
    Every step's output is checked against the oracle over the stored bytes, and the stored bytes against the rows."""
    rng = np.random.default_rng(15)
    L, H, T, d, agents, group, page, steps = 2, 2, 130, 64, 3, 2, 16, 20
    shape = (L, H, T, d)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 6, shape=shape)
    pool = kv.SharedKVPool.encode(to_dev(k), to_dev(v))
    cache = ka.PagedKV(agents * 2, H, page, d, fmt)
    order = rng.permutation(agents * 2).astype(np.int32).reshape(agents, 2)
    table = _i32(order)
    hq = H * group
    rows = torch.zeros(agents, (hq + 2 * H) * d, dtype=torch.bfloat16, device=DEV)
    q = rows[:, :hq * d].view(agents, hq, d)
    kn, vn = (rows[:, (hq + i * H) * d:(hq + (i + 1) * H) * d].view(agents, H, d) for i in (0, 1))
    pos = torch.zeros(agents, dtype=torch.int64, device=DEV)
    slots = torch.zeros(agents, dtype=torch.int64, device=DEV)
    lens = torch.zeros(agents, dtype=torch.int32, device=DEV)
    w = [bits(rng, d, 1.0) for _ in range(2)]
    wd = [to_dev(x) for x in w]
    f = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    out = torch.empty(agents, hq, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(agents, hq, device=DEV)
    need = ka.kvpool_attend_workspace_bytes(shape, agents, hq, cache.spec, 2 * page)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ka.kvc_norm_rotate(q, kn, pos, f, q, kn, q_weight=wd[0], k_weight=wd[1])
        cache.write(kn, vn, slots)
        ka.kvpool_attend(shape, pool.pool, 1, q, out, ws, tail=(cache.spec, cache.pages, table, lens), lse=lse)
    spec = (agents * 2, H, page, d, fmt)
    seen = oa.pool_rotated(pool.pool.cpu().numpy(), shape, 1)
    host = np.zeros(oa.page_bytes(spec), np.uint8)
    for step in range(steps):
        raw = bits(rng, (agents, (hq + 2 * H) * d))
        rows.copy_(to_dev(raw))
        at = T + step
        pos.fill_(at)
        s = order[:, step // page].astype(np.int64) * page + step % page
        slots.copy_(torch.from_numpy(s))
        lens.fill_(step + 1)
        g.replay()
        torch.cuda.synchronize()
        turned = to_host(rows)
        want = oa.norm_rotate(oa.f64(raw[:, :hq * d]).reshape(agents, hq, d), oa.f64(w[0]), 1e-6, [at] * agents, f, 0)
        assert np.all(np.abs(oa.f64(turned[:, :hq * d]).reshape(want.shape) - want)
                      <= np.abs(want) * 2.0 ** -8 + np.max(np.abs(want)) * 2.0 ** -17)
        oa.page_write(host, spec, turned[:, hq * d:(hq + H) * d].reshape(agents, H, d),
                      turned[:, (hq + H) * d:].reshape(agents, H, d), s)
        assert np.array_equal(cache.pages.cpu().numpy(), host), step
        t = np.arange(step + 1)
        tails = []
        for a in range(agents):
            kk, vv = oa.page_values(host, spec, order[a, t // page].astype(np.int64) * page + t % page)
            tails.append((kk.transpose(1, 0, 2), vv.transpose(1, 0, 2), None if fmt == 0 else np.array([1.0])))
        _pool_check(host_f64(out), host_f64(lse), oa.f64(turned[:, :hq * d]).reshape(agents, hq, d),
                    pool.pool.cpu().numpy(), shape, 1, 1 / math.sqrt(d), tails, step)
    assert seen[0].shape == (H, T, d)


def test_holders_attend():
    """PagedKV.attend and SharedKVPool.attend (with a PagedKV as tail) give the calls' results."""
    rng = np.random.default_rng(16)
    spec = (9, 2, 16, 64, ka.KVC_PAGE_INT8)
    lens = [40, 9, 0]
    store, table = random_sequences(rng, spec, lens)
    cache = ka.PagedKV(*spec)
    cache.pages.copy_(store.dev())
    q = bits(rng, (3, 4, 64))
    want, _ = _pages_attend(spec, store.dev(), q, table, lens)
    assert torch.equal(cache.attend(to_dev(q), _i32(table), _i32(lens)), want)
    shape = (1, 2, 50, 64)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 7, shape=shape)
    pool = kv.SharedKVPool.encode(to_dev(k), to_dev(v))
    want, _ = _pool_attend(shape, pool.pool, 0, q, (spec, store.dev(), _i32(table), _i32(lens)))
    assert torch.equal(pool.attend(0, to_dev(q), tail=(cache, _i32(table), _i32(lens))), want)
    e = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert cache.attend(e, _i32(np.zeros((0, 2))), _i32([])).shape == e.shape
    assert pool.attend(0, e).shape == e.shape


@pytest.mark.parametrize("seqs, heads", [(64, 2), (65, 1), (257, 1), (700, 1)])
def test_many_ragged_sequences(seqs, heads):
    """Work shared out over many sequences, empty ones among them, with tables wide enough that it is shared
    (not one workgroup each)."""
    rng = np.random.default_rng(seqs)
    d, page = 64, 16
    lens = rng.choice([0, 1, 127, 128, 129, 200, 640], seqs, p=[0.3, 0.2, 0.1, 0.1, 0.1, 0.15, 0.05])
    lens[0], lens[-1] = 0, 641
    spec = (int(np.sum(-(-lens // page))) + 1, heads, page, d, ka.KVC_PAGE_INT8)
    store, table = random_sequences(rng, spec, lens, cols=1024 // page)
    q = bits(rng, (seqs, 2 * heads, d))
    out, lse = _pages_attend(spec, store.dev(), q, table, lens)
    o, l = host_f64(out), host_f64(lse)
    for b, n in enumerate(lens):
        k, v = sequence(store, table, b, n)
        check_attend(o[b], l[b], oa.f64(q)[b], k, v, 1 / math.sqrt(d), True, _steps(store), (b, n))


@pytest.mark.parametrize("shape, agents, group", [((1, 2, 8200, 64), 15, 4), ((1, 1, 16500, 128), 40, 2), ((1, 1, 8321, 128), 33, 4),
                                                  ((1, 1, 9001, 64), 64, 4)])
def test_pool_many_rows(shape, agents, group):
    """Pools long enough that several row groups of a workgroup share the widened tokens; ends inside a step."""
    rng = np.random.default_rng(agents)
    k, v = synth.kv_bits(synth.WORKLOADS[3], 8, shape=shape)
    pool = oracle.pool_encode(k, v)
    q = bits(rng, (agents, shape[1] * group, shape[3]), 1.0)
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), 0, q)
    pick = [0, agents // 2, agents - 1]
    _pool_check(host_f64(out)[pick], host_f64(lse)[pick], oa.f64(q)[pick], pool, shape, 0, 1 / math.sqrt(shape[3]), None,
                (shape, agents))
    spec = (agents + 2, shape[1], 16, shape[3], ka.KVC_PAGE_FP8)
    lens = [i % 17 for i in range(agents)]
    store, table = random_sequences(rng, spec, lens)
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), 0, q, (spec, store.dev(), _i32(table), _i32(lens)))
    tails = [(*sequence(store, table, a, lens[a]), _steps(store)) for a in pick]
    _pool_check(host_f64(out)[pick], host_f64(lse)[pick], oa.f64(q)[pick], pool, shape, 0, 1 / math.sqrt(shape[3]), tails,
                (shape, agents, "tails"))


def _hot(rng, n, heads, group, seqs, d, at):
    """Queries of 2^11..2^12 a channel and keys [n, heads, d] of about 2^10, one of which (token at) has the
    queries' signs at 2^14: logits up to 10^9, that token's far above the rest."""
    sign = np.where(rng.random(d) < 0.5, -1.0, 1.0)
    k = rng.standard_normal((n, heads, d)) * 2.0 ** 10
    if at is not None:
        k[at] = sign * 2.0 ** 14 * (1 + rng.random((heads, d)) / 8)
    q = sign * 2.0 ** 11 * (1 + rng.random((seqs, heads * group, d)))
    return synth.f32_to_bf16_bits(q.astype(np.float32)), synth.f32_to_bf16_bits(k.astype(np.float32))


def _far(q, keys, scale, at):
    """Every row's logit at `at` passes all others by far more than what logits may be off."""
    group = q.shape[0] // keys.shape[0]
    for h in range(q.shape[0]):
        x = keys[h // group] @ q[h] * scale
        rest = np.delete(x, at)
        assert x[at] - np.max(rest, initial=-np.inf) > 100 + 2 * np.max(logit_bound(q, keys, scale))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n, at", [(1, 0), (200, 3), (700, 699), (5000, 2500)])
def test_logits_of_a_thousand_million(fmt, n, at):
    """One token takes all the weight (its difference to the maximum is 0 whatever the maximum's rounding):
    the output is its value, each rounding as for a single token."""
    rng = np.random.default_rng(n)
    d, heads, group, page = 128, 2, 4, 16
    spec = (-(-n // page) + 1, heads, page, d, fmt)
    store, table = random_sequences(rng, spec, [n])
    q, k = _hot(rng, n, heads, group, 1, d, at)
    t = np.arange(n)
    store.put(k, bits(rng, (n, heads, d)), table[0, t // page] * page + t % page)
    out, lse = _pages_attend(spec, store.dev(), q, table, [n])
    keys, values = sequence(store, table, 0, n)
    q64, scale = oa.f64(q)[0], 1 / math.sqrt(d)
    _far(q64, keys, scale, at)
    want = np.repeat(values[:, at], group, axis=0)
    tol = U_BF16 if fmt == 0 else U_BF16 + 1.01 * 2.0 ** -11
    assert np.all(np.abs(host_f64(out)[0] - want) <= np.abs(want) * tol + 1e-30)
    wl = oa.attend(q64, keys, values, scale)[1]
    assert np.all(np.abs(host_f64(lse)[0] - wl) <= lse_bound(wl, logit_bound(q64, keys, scale), n))


@pytest.mark.parametrize("d, T, group", [(128, 300, 4), (64, 9000, 2)])
def test_pool_logits_of_a_thousand_million(d, T, group):
    """The same with a pool, where the first agent's token lies in the pool and the second one's in its tail."""
    rng = np.random.default_rng(d)
    heads, page, lens = 2, 16, [5, 40]
    shape, spec = (1, heads, T, d), (6, heads, page, d, 1)
    q, k = _hot(rng, T, heads, group, 2, d, T // 2)
    v = bits(rng, (heads, T, d))
    pool = oracle.pool_encode(k.transpose(1, 0, 2)[None].copy(), v[None])
    store, table = random_sequences(rng, spec, lens)
    q[1] ^= 0x8000  # the second agent turns away from the pool's token ...
    tk = rng.standard_normal((lens[1], heads, d)).astype(np.float32)
    tk[7] = -oa.f64(k[T // 2])  # ... towards one of its own
    t = np.arange(lens[1])
    store.put(synth.f32_to_bf16_bits(tk), bits(rng, (lens[1], heads, d)), table[1, t // page] * page + t % page)
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), 0, q, (spec, store.dev(), _i32(table), _i32(lens)))
    keys, rot = oa.pool_rotated(pool, shape, 0)
    vals, scale = rot @ oa.hadamard(d) / math.sqrt(d), 1 / math.sqrt(d)
    for a, at in ((0, T // 2), (1, T + 7)):
        k2, v2 = sequence(store, table, a, lens[a])
        kk, vv, q64 = np.concatenate([keys, k2], 1), np.concatenate([vals, v2], 1), oa.f64(q)[a]
        _far(q64, kk, scale, at)
        want = np.repeat(vv[:, at], group, axis=0)
        if a == 0:  # weight and level rounded to binary16 in rotated space, binary32 sums of d
            b = np.repeat(np.sum(np.abs(rot[:, at]), -1), group)[:, None] / math.sqrt(d) * (2.01 * 2.0 ** -11 + 2.0 ** -20)
        else:
            b = np.abs(want) * 1.01 * 2.0 ** -11
        b = b + U_BF16 * (np.abs(want) + b) + 1e-30
        assert np.all(np.abs(host_f64(out)[a] - want) <= b)
        wl = oa.attend(q64, kk, vv, scale)[1]
        assert np.all(np.abs(host_f64(lse)[a] - wl) <= lse_bound(wl, logit_bound(q64, kk, scale), T + lens[a]))


def test_pool_offsets_past_32_bits():
    """The second layer of a pool of 6 GB gives the bits of the same layer in a pool of its own."""
    H, T, d, n = 4, (1 << 22) - 3, 128, 2
    gen = torch.Generator(device=DEV).manual_seed(5)
    k, v = (torch.empty(2, H, T, d, dtype=torch.bfloat16, device=DEV).normal_(generator=gen) for _ in range(2))
    q = torch.empty(n, 2 * H, d, dtype=torch.bfloat16, device=DEV).normal_(0, 2, generator=gen)
    got = []
    for shape, kk, vv, layer in (((2, H, T, d), k, v, 1), ((1, H, T, d), k[1:], v[1:], 0)):
        pool = torch.empty(kv.kvpool_bytes(shape), dtype=torch.uint8, device=DEV)
        ws = torch.empty(kv.kvpool_workspace_bytes(shape), dtype=torch.uint8, device=DEV)
        kv.kvpool_encode(shape, kk, vv, pool, ws, _status())
        out, lse = _pool_attend(shape, pool, layer, to_host(q))
        got.append((out, lse))
    assert pool.numel() * 2 > 1 << 32
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])
    assert bool(torch.isfinite(got[0][0]).all())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("e", [-90, 110])
def test_keys_far_from_their_queries_in_size(fmt, e):
    """Keys of about 2^e and queries of about 2^-e: ordinary logits."""
    rng = np.random.default_rng(e + 100)
    d, n, page, heads = 128, 150, 32, 2
    spec = (6, heads, page, d, fmt)
    store, table = random_sequences(rng, spec, [n])
    t = np.arange(n)
    store.put(bits(rng, (n, heads, d), 2.0 ** e), bits(rng, (n, heads, d)), table[0, t // page] * page + t % page)
    q = bits(rng, (1, 3 * heads, d), 2.0 ** -e)
    out, lse = _pages_attend(spec, store.dev(), q, table, [n])
    k, v = sequence(store, table, 0, n)
    check_attend(host_f64(out)[0], host_f64(lse)[0], oa.f64(q)[0], k, v, 1 / math.sqrt(d), fmt != 0, _steps(store), e)
