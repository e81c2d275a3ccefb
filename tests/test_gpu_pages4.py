"""GPU parity of 4-bit pages (KVC_PAGE_FP4): codes and powers bit for bit,
values read back exactly, and single-token attention over them, alone and as
tails behind a pool, against the oracle."""

import math

import numpy as np
import pytest
import torch

import oracle
from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import synth
from attend_util import Store, bits, check_attend, host_f64, place, sequence
from gpu_util import DEV, say, to_dev, to_host
from oracle import attend as oa
from serving_util import i32, status, store_of
from test_gpu_attend import _pages_attend, _pool_attend, _pool_check

pytestmark = pytest.mark.gpu
FP4 = ka.KVC_PAGE_FP4


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, page, num, n, layout", [(1, 16, 1, 1, "tokens"), (3, 16, 9, 100, "heads"),
                                                        (8, 64, 5, 15, "fused"), (2, 256, 2, 301, "tokens"),
                                                        (5, 32, 140, 4200, "heads")])
def test_write_and_read(d, heads, page, num, n, layout):
    rng = np.random.default_rng(n + d)
    spec = (num, heads, page, d, FP4)
    say("pages", spec, n, layout)
    k, v = bits(rng, (n, heads, d), 3.0), bits(rng, (n, heads, d), 1e-3)
    slots = rng.permutation(num * page)[:n].astype(np.int64)
    if n > 2:
        slots[1], slots[2] = -1, num * page   # padding, and one outside
    store = Store(spec)
    dev, st = store.dev(), status()
    sl = torch.from_numpy(slots).to(DEV)
    ka.kvpage_write(spec, dev, place(k, layout), place(v, layout), sl, st)
    torch.cuda.synchronize()
    assert int(st) == (ka.KVC_DEV_BAD_SLOT if n > 2 else 0)
    store.put(k, v, slots)
    got = dev.cpu().numpy()
    bad = np.nonzero(got != store.host)[0]
    assert bad.size == 0, f"{bad.size} bytes differ, first at {bad[0]}"
    mark = np.full((n, heads, d), 0x4242, np.uint16)
    ko, vo = place(mark, layout), place(mark, layout)
    ka.kvpage_read(spec, dev, sl, ko, vo, st)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < num * page)
    for t, w in zip((ko, vo), oa.page_values(store.host, spec, slots[live])):
        assert np.all(to_host(t)[~live] == 0x4242)
        assert np.array_equal(host_f64(t)[live], w)


def test_every_exponent_ties_and_non_finite():
    """Every bf16 exponent as a block's maximum, with values all over the range below; ties; zeros, Inf and NaN."""
    d, n = 64, 300
    rng = np.random.default_rng(7)
    k = bits(rng, (n, 1, d))
    for i in range(254):
        b = rng.integers(0, 1 << 16, d).astype(np.uint16)
        e = np.minimum(b >> 7 & 255, i + 1)
        k[i, 0] = (b & 0x807F) | (e << 7).astype(np.uint16)
        k[i, 0, 0] = (k[i, 0, 0] & 0x807F) | (i + 1) << 7
    ties = np.concatenate([np.arange(-32, 32) * 0.25 * 0.875])
    k[254, 0] = synth.f32_to_bf16_bits(np.clip(np.round(ties * 4) / 4, -7, 7).astype(np.float32))
    k[254, 0, 0], k[254, 0, 32] = synth.f32_to_bf16_bits(np.float32([7, -7]))
    k[255] = 0
    k[256, 0] = rng.integers(1, 128, d)               # denormals alone
    k[257, 0, 3], k[258, 0, 35], k[259, 0, 9] = 0x7F80, 0xFF80, 0x7FC1
    k[260, 0] = 0x8000                                # -0
    k[261, 0], k[261, 0, 63] = 0, 0x0001
    k[262, 0], k[262, 0, 1] = 0x7F7F, 0xFF7F          # the largest
    spec = (10, 1, 32, d, FP4)
    slots = np.arange(n, dtype=np.int64)
    store = Store(spec)
    dev = store.dev()
    v = k[::-1].copy()
    ka.kvpage_write(spec, dev, to_dev(k), to_dev(v), torch.from_numpy(slots).to(DEV))
    torch.cuda.synchronize()
    store.put(k, v, slots)
    assert np.array_equal(dev.cpu().numpy(), store.host)
    ko, vo = (torch.empty(n, 1, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    ka.kvpage_read(spec, dev, torch.from_numpy(slots).to(DEV), ko, vo)
    torch.cuda.synchronize()
    want = oa.page_values(store.host, spec, slots)[0]
    r = host_f64(ko)
    assert np.array_equal(np.isnan(r), np.isnan(want)) and np.array_equal(r[~np.isnan(r)], want[~np.isnan(r)])
    assert np.isnan(r[257, 0, :32]).all() and np.isfinite(r[257, 0, 32:]).all() and np.isnan(r[258, 0, 32:]).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, group, page, lens", [(1, 1, 16, [1]), (2, 4, 16, [0, 31, 32, 33, 100]),
                                                      (8, 4, 64, [700, 1, 129, 2000]), (3, 7, 32, [513, 127, 128, 64]),
                                                      (1, 40, 16, [5000, 17]), (2, 1, 256, [300, 0, 4097])])
def test_attention(d, heads, group, page, lens):
    rng = np.random.default_rng(sum(lens) + d)
    spec = (sum(-(-n // page) for n in lens) + 3, heads, page, d, FP4)
    say("pages", spec, lens)
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (len(lens), heads * group, d), 1.5)
    out, lse = _pages_attend(spec, store.dev(), q, table, lens)
    o, l = host_f64(out), host_f64(lse)
    for b, n in enumerate(lens):
        kk, vv = sequence(store, table, b, n)
        check_attend(o[b], l[b], oa.f64(q)[b], kk, vv, 1 / math.sqrt(d), False, None, (spec, b))


def test_non_finite_blocks_stay_where_they_belong():
    """A NaN block of one kv head's value makes 32 channels of its query heads NaN; one of a key all of them; blocks
    behind the length, and other sequences', none."""
    rng = np.random.default_rng(12)
    d, lens = 128, [40, 200, 37]
    spec = (30, 2, 16, d, FP4)
    store, table = store_of(rng, spec, lens)
    steps, each = oa.page_layout(spec)[1:]

    def power(b, j, h, t, block):
        return int(table[b, t // 16]) * each + steps + ((j * 2 + h) * 16 + t % 16) * 4 + block

    store.host[power(0, 1, 1, 39, 2)] = 255    # a value
    store.host[power(1, 0, 0, 130, 1)] = 255   # a key
    q = bits(rng, (3, 4, d))
    out, lse = _pages_attend(spec, store.dev(), q, table, lens)
    o, l = host_f64(out), host_f64(lse)
    assert np.isnan(o[0, 2:, 64:96]).all() and np.isfinite(o[0, 2:, :64]).all() and np.isfinite(o[0, 2:, 96:]).all()
    assert np.isnan(o[1, :2]).all() and np.isnan(l[1, :2]).all()
    for b, hs in ((0, [0, 1]), (1, [2, 3]), (2, [0, 1]), (2, [2, 3])):
        kk, vv = sequence(store, table, b, lens[b])
        g = hs[0] // 2
        check_attend(o[b][hs], l[b][hs], oa.f64(q)[b][hs], kk[g:g + 1], vv[g:g + 1], 1 / math.sqrt(d), False, None, (b, hs))


@pytest.mark.parametrize("shape, lens", [((2, 2, 100, 64), [0, 5, 33]), ((1, 4, 4096, 128), [250, 0, 17, 300]),
                                         ((3, 1, 700, 128), [1, 64])])
def test_tails_behind_a_pool(shape, lens):
    rng = np.random.default_rng(shape[2])
    L, H, T, d = shape
    spec = (sum(-(-n // 16) for n in lens) + 2, H, 16, d, FP4)
    pool = oracle.pool_encode(bits(rng, (L, H, T, d)), bits(rng, (L, H, T, d)))
    store, table = store_of(rng, spec, lens)
    q = bits(rng, (len(lens), H * 4, d), 1.5)
    st = status()
    out, lse = _pool_attend(shape, torch.from_numpy(pool).to(DEV), L - 1, q, (spec, store.dev(), i32(table), i32(lens)),
                            status=st)
    assert int(st) == 0
    tails = [(*sequence(store, table, b, m), None) for b, m in enumerate(lens)]
    _pool_check(host_f64(out), host_f64(lse), oa.f64(q), pool, shape, L - 1, 1 / math.sqrt(d), tails, shape)


def test_offsets_past_32_bits():
    """A store above 4 GiB: its last pages are written, read and attended to as those of a small one."""
    rng = np.random.default_rng(14)
    heads, page, d, n = 8, 256, 128, 600
    each = oa.page_layout((1, heads, page, d, FP4))[2]
    num = (1 << 32) // each + 4
    spec = (num, heads, page, d, FP4)
    pages = torch.empty(ka.kvpage_bytes(spec), dtype=torch.uint8, device=DEV)
    k, v = bits(rng, (n, heads, d)), bits(rng, (n, heads, d), 0.5)
    last = np.array([num - 1, num - 3, num - 2])
    t = np.arange(n)
    slots = torch.from_numpy(last[t // page].astype(np.int64) * page + t % page).to(DEV)
    ka.kvpage_write(spec, pages, to_dev(k), to_dev(v), slots)
    small = (3, heads, page, d, FP4)
    few = torch.zeros(ka.kvpage_bytes(small), dtype=torch.uint8, device=DEV)
    ka.kvpage_write(small, few, to_dev(k), to_dev(v), torch.arange(n, device=DEV))
    q = to_dev(bits(rng, (1, 32, d)))
    outs = []
    for sp, store, row in ((spec, pages, last), (small, few, [0, 1, 2])):
        out = torch.empty(1, 32, d, dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(ka.kvpage_attend_workspace_bytes(sp, 1, 32, 3 * page), dtype=torch.uint8, device=DEV)
        ka.kvpage_attend(sp, store, q, i32([row]), i32([n]), out, ws)
        ko, vo = (torch.empty(n, heads, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        sl = slots if sp is spec else torch.arange(n, device=DEV)
        ka.kvpage_read(sp, store, sl, ko, vo)
        outs.append((out, ko, vo))
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)
