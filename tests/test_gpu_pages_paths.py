"""The paged cache through both forms of its kernels (one vector of each group
of lanes at a time, or four), in every pair of row layouts, at the largest
number of heads."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import FORMATS, Store, bits, host_f64, place
from gpu_util import DEV, say, to_dev, to_host
from oracle import attend as oa
from plan_util import put_all

pytestmark = pytest.mark.gpu


def _four_at_a_time(n, heads, d):
    """launch_page's rule: the GPU stays full with four vectors for each group of d / 8 lanes."""
    return 2 * n * heads >= 4 * (256 // (d // 8)) * 1024


def _write_and_read(rng, spec, n, slots, layouts):
    num, heads, page, d, fmt = spec
    k, v = bits(rng, (n, heads, d), 3.0), bits(rng, (n, heads, d), 1e-3)
    store = Store(spec)
    dev, status = store.dev(), torch.zeros(1, dtype=torch.int32, device=DEV)
    sl = torch.from_numpy(slots).to(DEV)
    ka.kvpage_write(spec, dev, place(k, layouts[0]), place(v, layouts[1]), sl, status)
    torch.cuda.synchronize()
    put_all(store.host, spec, k, v, slots)
    bad = np.nonzero(dev.cpu().numpy() != store.host)[0]
    assert bad.size == 0, f"{bad.size} bytes differ, first at {bad[0]}"
    outside = slots >= num * page
    assert int(status) == (ka.KVC_DEV_BAD_SLOT if outside.any() else 0)
    mark = np.full((n, heads, d), 0x4242, np.uint16)
    ko, vo = place(mark, layouts[0]), place(mark, layouts[1])
    ka.kvpage_read(spec, dev, sl, ko, vo)
    torch.cuda.synchronize()
    live = (slots >= 0) & ~outside
    for t, w in zip((ko, vo), oa.page_values(store.host, spec, slots[live])):
        assert np.all(to_host(t)[~live] == 0x4242)
        # the product in binary32 (2^-24), then bf16 (half a step); bf16 stores are copies
        assert np.all(np.abs(host_f64(t)[live] - w) <= (0 if fmt == 0 else 2.0 ** -8 + 2.0 ** -23) * np.abs(w))


LAYOUTS = [("tokens", "heads"), ("heads", "tokens"), ("fused", "fused"), ("heads", "heads")]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("layouts", LAYOUTS)
@pytest.mark.parametrize("d, n, heads", [(128, 4133, 8), (64, 8219, 8), (128, 11003, 3), (64, 61, 5), (128, 75, 3)])
def test_layouts(fmt, layouts, d, n, heads):
    rng = np.random.default_rng(n)
    say("pages", fmt, layouts, d, n, heads)
    assert _four_at_a_time(n, heads, d) == (n > 1000)
    page = 32
    spec = (-(-n // page) + 2, heads, page, d, fmt)
    slots = rng.permutation(spec[0] * page)[:n].astype(np.int64)
    slots[5], slots[n // 2], slots[n - 2] = -1, spec[0] * page, -(1 << 40)   # padding, and one outside
    _write_and_read(rng, spec, n, slots, layouts)


@pytest.mark.parametrize("layout", ["tokens", "heads"])
def test_the_most_heads(layout):
    """65536 heads: with heads first, as many rows of the launch's grid."""
    rng = np.random.default_rng(5)
    spec = (1, 1 << 16, 16, 64, ka.KVC_PAGE_INT8)
    _write_and_read(rng, spec, 3, np.array([7, -1, 2], np.int64), (layout, layout))
