"""GPU parity of attention of many new tokens where each block is a workgroup's, over long contexts, and of NaN and Inf in the
first tiles of blocks, shared out or not; the plans are as the library names them."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import bits, host_f64, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from prompt_util import plan_name, prompt_plan
from serving_util import ALL_FORMATS, check_rows, default_scale, largest_steps, rows_see, status, store_of
from test_gpu_attend_prompt import _attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads, group, new, lens, window, sinks", [
    (80, 1, [700, 0, 601], [1000, 40, 601], 0, 0),
    (26, 4, [650, 651], [651, 1900], 0, 0),
    (80, 1, [701, 600], [1500, 700], 600, 5),
    (14, 13, [333, 340], [1100, 340], 700, 33),
    (90, 1, [1300], [900], 0, 0),                 # 400 rows that see nothing
])
def test_blocks_over_long_contexts(fmt, d, heads, group, new, lens, window, sinks):
    rng = np.random.default_rng(91)
    spec = (sum(-(-n // 32) for n in lens) + 2, heads, 32, d, fmt)
    store, table = store_of(rng, spec, lens)
    starts = np.concatenate([[0], np.cumsum(new)]).tolist()
    plan = prompt_plan(spec, len(lens), starts[-1], heads * group, table.shape[1], window, sinks)
    say("prompt in blocks", spec, group, new, lens, window, sinks, plan.blocks)
    assert plan_name(plan) == "blocks" and table.shape[1] * 32 > 512
    q = bits(rng, (starts[-1], heads * group, d), 1.5)
    st = status()
    out, lse = _attend(spec, store.dev(), q, starts, table, lens, window, sinks, st)
    assert int(st) == 0
    o, l = host_f64(out), host_f64(lse)
    assert np.isfinite(o).all()
    steps = largest_steps(store)
    for b, n in enumerate(lens):
        at = slice(starts[b], starts[b + 1])
        k, v = sequence(store, table, b, n)
        for h in (0, 1, heads // 2, heads - 1):
            hs = slice(h * group, (h + 1) * group)
            check_rows(o[at, hs], l[at, hs], oa.f64(q)[at, hs], k[h:h + 1], v[h:h + 1], default_scale(d), fmt, steps,
                       rows_see(new[b], n, window, sinks), (spec, b, h))


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name, heads", [("blocks", 162), ("shared", 6)])
def test_non_finite_values_in_the_first_tiles_of_blocks(fmt, d, name, heads):
    """With a window, the first tile of a block holds tokens that its first rows see and the others do not: those stay as if
    the token were any other, whichever wave brings the tile. Each head has one such token."""
    rng = np.random.default_rng(93)
    m, n, window, page = 640, 1400, 700, 64
    # rows stand at 760 to 1399; what blocks of 128 of them see begins with 61, 189, 317, 445
    bad = np.array([62, 75, 190, 319, 446, 470])[np.arange(heads) % 6]
    spec = (n // page + 2, heads, page, d, fmt)
    store, table = store_of(rng, spec, [n])
    assert plan_name(prompt_plan(spec, 1, m, heads, table.shape[1], window)) == name
    dev = store.dev()
    tokens = np.unique(bad)
    slots = np.array([int(table[0, t // page]) * page + t % page for t in tokens])
    k, v = (bits(rng, (len(tokens), heads, d)) for _ in range(2))
    for h, t in enumerate(bad):
        v[tokens == t, h, d - 1] = 0x7FC0 if h % 2 else 0x7F80
    ka.kvpage_write(spec, dev, to_dev(k), to_dev(v), torch.tensor(slots, device=DEV))
    torch.cuda.synchronize()
    store.host[:] = dev.cpu().numpy()
    q = bits(rng, (m, heads, d))
    out, lse = _attend(spec, dev, q, [0, m], table, [n], window)
    again = _attend(spec, dev, q, [0, m], table, [n], window)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse, again[1])
    o, l, see = host_f64(out), host_f64(lse), rows_see(m, n, window)
    first = 0 if fmt in (ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8) else d - 32 if fmt == ka.KVC_PAGE_FP4 else d - 1
    k, v = sequence(store, table, 0, n)
    for h in range(heads):
        hit = see[:, bad[h]]
        assert 0 < hit.sum() < m
        wrong = ~np.isfinite(o[:, h])
        assert wrong[hit][:, first:].all() and not wrong[~hit].any() and not wrong[:, :first].any(), h
        if h < 6 or h == heads - 1:
            hs = slice(h, h + 1)
            check_rows(o[~hit][:, hs], l[~hit][:, hs], oa.f64(q)[~hit][:, hs], k[hs], np.where(np.isfinite(v[hs]), v[hs], 0),
                       default_scale(d), fmt, largest_steps(store), see[~hit], (fmt, h))
