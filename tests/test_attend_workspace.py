"""A program allocates a workspace once, for its largest call: the sizes that the
queries give never fall with more sequences (agents), tokens or rows, across every
change of plan, and a call takes the workspace of any larger one. No GPU."""

import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv

COUNTS = sorted({n for c in (1, 2, 3, 8, 32, 39, 64, 100, 128, 191, 192, 256, 384, 511, 512, 513, 767, 768, 1000, 1023, 1024,
                             2047, 2048, 4095, 4096, 6143, 6144, 8191) for n in (c - 1, c, c + 1) if n > 0})
TOKENS = sorted({t for c in (16, 128, 256, 512, 1024, 1280, 2048, 4096, 8192, 16384, 32768, 131072, 1 << 20)
                 for t in (c - 16, c, c + 16) if t > 0})


def _rises(sizes, what):
    assert all(s > 0 for s in sizes), what
    for i in range(1, len(sizes)):
        assert sizes[i] >= sizes[i - 1], (what, i, sizes[i - 1], sizes[i])


@pytest.mark.parametrize("heads, d, group", [(8, 128, 4), (32, 64, 1), (2, 128, 33), (1, 64, 17), (1, 128, 48), (2, 64, 40),
                                             (4, 128, 16), (1, 128, 1)])
def test_page_workspaces_never_fall(heads, d, group):
    spec = (4, heads, 16, d, 1)
    most = {(n, t): ka.kvpage_attend_workspace_bytes(spec, n, heads * group, t) for n in COUNTS for t in TOKENS
            if n * heads * group < 1 << 23 and n * (t // 128 + 1) < 1 << 31}
    for t in TOKENS:
        _rises([most[n, t] for n in COUNTS if (n, t) in most], ("sequences", t))
    for n in COUNTS:
        _rises([most[n, t] for t in TOKENS if (n, t) in most], ("tokens", n))


@pytest.mark.parametrize("heads, d, group", [(8, 128, 4), (32, 64, 1), (1, 64, 4), (2, 128, 7)])
@pytest.mark.parametrize("pool_tokens", [100, 512, 513, 4096, 131071])
def test_pool_workspaces_never_fall(heads, d, group, pool_tokens):
    spec, shape = (4, heads, 16, d, 1), (1, heads, pool_tokens, d)
    counts = [n for n in COUNTS if n * heads * group < 1 << 23]

    def size(n, t=None, s=shape):
        return ka.kvpool_attend_workspace_bytes(s, n, heads * group, *(() if t is None else (spec, t)))

    _rises([size(n) for n in counts], "agents")
    for t in (16, 512, 4096, 32768):
        _rises([size(n, t) for n in counts], ("agents", t))
    for n in (1, 15, 64, 511, 512, 1000):
        _rises([size(n)] + [size(n, t) for t in TOKENS], ("tails", n))
        _rises([size(n, 64, (1, heads, t, d)) for t in TOKENS], ("pool", n))


def test_the_sizes_that_fell():
    """The pairs at which the sizes used to fall."""
    for spec, hq, few, many, tokens in (((4, 8, 16, 128, 1), 32, 511, 512, 4096), ((4, 32, 16, 64, 1), 32, 191, 192, 4096)):
        a, b = (ka.kvpage_attend_workspace_bytes(spec, n, hq, tokens) for n in (few, many))
        assert 0 < a <= b
    a, b = (ka.kvpage_attend_workspace_bytes((4, 2, 16, 128, 1), 39, 66, t) for t in (1280, 2048))
    assert 0 < a <= b
    shape, spec = (1, 8, 100, 128), (4, 8, 16, 128, 1)
    a, b = (ka.kvpool_attend_workspace_bytes(shape, n, 32, spec, 4096) for n in (511, 512))
    assert 0 < a <= b


fake_addresses = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only host")
A = 1 << 40


@fake_addresses
@pytest.mark.parametrize("n", [1, 32, 511, 512, 700])
def test_a_call_takes_the_workspace_of_a_larger_one(n):
    """The size is looked at before the alignment of q, which is wrong in each of these calls: nothing is launched."""
    spec = ka.kvc_pages(600, 8, 16, 128, 1)
    ws = ka.kvpage_attend_workspace_bytes(spec, 700, 32, 4096)
    rows = [ka.kvc_rows(i * A + 8, 32 * 128, 128) for i in (1, 2)]
    L = kv.library()

    def call(size, cols):
        return L.kvpage_attend(spec, 3 * A, ka.kvpage_bytes(spec), n, 32, rows[0], 4 * A, cols, cols, 5 * A, 0.1, rows[1], None,
                               6 * A, size, None, None)

    for cols in (1, 32, 33, 100, 256):
        assert call(ws, cols) == kv.KVC_E_ALIGN
        assert call(0, cols) == kv.KVC_E_SIZE
