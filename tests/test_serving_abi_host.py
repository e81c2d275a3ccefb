"""Host-side checks of kvpage_append, kvpage_attend_window,
kvpage_attend_prompt and 4-bit pages: sizes against the oracle, workspaces that
never fall, and every refusal, all before any device work."""

import ctypes

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from agent_handoff_amd import kvcodec as kv
from oracle import attend as oa

fake_addresses = pytest.mark.skipif(torch.cuda.device_count() != 0, reason="fake device addresses: CPU-only host")
L = kv.library()
A = 1 << 40
N, HQ, HK, D = 5, 8, 2, 64


@pytest.mark.parametrize("spec", [(1, 1, 16, 64, 4), (7, 3, 16, 64, 4), (960, 8, 16, 128, 4), (5, 8, 256, 128, 4)])
def test_four_bit_pages_agree_with_oracle(spec):
    assert ka.kvpage_bytes(spec) == oa.page_bytes(spec) > 0
    assert 2 * ka.kvpage_bytes(spec) < 1.1 * ka.kvpage_bytes((*spec[:4], 1)) + 512 * spec[0]


def test_invalid_formats():
    for fmt in (3, 5, 8, 0xFFFFFFFF):
        spec = (4, 2, 16, 64, fmt)
        assert ka.kvpage_bytes(spec) == 0
        assert ka.kvpage_attend_window_workspace_bytes(spec, 1, 4, 64, 16, 0) == 0
        assert ka.kvpage_attend_prompt_workspace_bytes(spec, 1, 4, 4, 64) == 0


# ---------------------------------------------------------------- workspaces

COUNTS = sorted({n for c in (1, 2, 8, 15, 32, 64, 100, 256, 511, 767, 1023, 2047, 4095) for n in (c, c + 1)})
TOKENS = sorted({t for c in (16, 128, 256, 512, 1024, 2048, 8192, 32768, 1 << 20) for t in (c - 16, c, c + 16) if t > 0})
WINDOWS = [1, 15, 16, 17, 100, 112, 113, 496, 497, 512, 1024, 5000, 1 << 20, 1 << 31, 0xFFFFFFFF]
SINKS = [0, 1, 4, 16, 17, 100, 4096, 0xFFFFFFFF]


def _rises(sizes, what):
    assert all(s > 0 for s in sizes), what
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), (what, sizes)


@pytest.mark.parametrize("heads, d, group", [(8, 128, 4), (32, 64, 1), (1, 64, 17), (2, 128, 33)])
def test_window_workspaces_never_fall(heads, d, group):
    spec = (4, heads, 16, d, 4)

    def size(n, t, w, s):
        return ka.kvpage_attend_window_workspace_bytes(spec, n, heads * group, t, w, s)

    for w in WINDOWS:
        for t in TOKENS[::3]:
            _rises([size(n, t, w, 4) for n in COUNTS], ("sequences", w, t))
            _rises([size(7, t, w, s) for s in SINKS], ("sinks", w, t))
        for n in COUNTS[::5]:
            _rises([size(n, t, w, 4) for t in TOKENS], ("tokens", w, n))
    for n in COUNTS[::5]:
        for t in TOKENS[::3]:
            most = ka.kvpage_attend_workspace_bytes(spec, n, heads * group, t)
            _rises([size(n, t, w, 4) for w in WINDOWS] + [most], ("window", n, t))
            assert size(n, t, 0, 9) == most


@pytest.mark.parametrize("heads, d, group", [(8, 128, 4), (32, 64, 1), (1, 64, 17), (2, 128, 33), (1, 128, 200)])
def test_prompt_workspaces_never_fall(heads, d, group):
    spec = (4, heads, 16, d, 0)

    def size(b, n, t, w=0, s=0):
        return ka.kvpage_attend_prompt_workspace_bytes(spec, b, n, heads * group, t, w, s)

    for t in TOKENS:
        for b in (1, 7, 100):
            _rises([size(b, n, t) for n in COUNTS], ("rows", t, b))
        for n in (1, 40, 5000):
            _rises([size(b, n, t) for b in COUNTS], ("sequences", t, n))
            _rises([size(3, n, t, w, 4) for w in WINDOWS] + [size(3, n, t)], ("window", t, n))
            _rises([size(3, n, t, 100, s) for s in SINKS], ("sinks", t, n))
    for b in (1, 7, 100):
        for n in COUNTS:
            _rises([size(b, n, t) for t in TOKENS], ("tokens", b, n))
            assert size(0, n, 4096) > 0 and size(b, 0, 4096) > 0


def test_prompt_sizes_out_of_range():
    spec = (4, 2, 16, 64, 1)
    f = ka.kvpage_attend_prompt_workspace_bytes
    assert f(spec, 1, 10, 5, 64) == 0 and f(spec, 1, 10, 0, 64) == 0          # heads that do not divide
    assert f(spec, 1, 1 << 28, 4, 64) == 0 and f(spec, 1 << 20, 10, 4, 64) == 0
    assert f(spec, 1, 10, 4, 1 << 31) == 0 and f(spec, 1, 10, 4, (1 << 31) - 16) > 0


# ---------------------------------------------------------------- refusals
# Raw C calls with made-up device addresses, on hosts without a GPU only.

def rows(base, ts=None, hs=D, heads=HK):
    return ka.kvc_rows(base, heads * D if ts is None else ts, hs)


SPEC = ka.kvc_pages(6, HK, 16, D, ka.KVC_PAGE_FP4)
PB = ka.kvpage_bytes(SPEC)


def _append(spec=SPEC, pages=A, size=PB, n=N, hq=HQ, q=None, k=None, v=None, qw=5 * A, kw=6 * A, eps=1e-6, pos=7 * A, pairs=32,
            pairing=0, f=True, slots=8 * A, qo=None, status=9 * A):
    q = rows(2 * A, heads=HQ) if q is None else q
    k = rows(3 * A) if k is None else k
    v = rows(4 * A) if v is None else v
    qo = rows(10 * A, heads=HQ) if qo is None else qo
    fr = np.ones(64, np.float32)
    return L.kvpage_append(spec, pages, size, n, hq, q or None, k or None, v or None, qw, kw, eps, pos,
                           fr.ctypes.data if f else None, pairs, pairing, slots, qo or None, status, None)


@fake_addresses
def test_append_refusals():
    assert _append(n=0) == kv.KVC_OK
    for bad in ({"spec": ka.kvc_pages(6, HK, 24, D, 1)}, {"spec": ka.kvc_pages(6, HK, 16, D, 3)}, {"hq": (1 << 16) + 1},
                {"n": (1 << 26) - 3}, {"q": rows(2 * A, ts=1 << 62)}, {"v": rows(4 * A, hs=1 << 61)}):
        assert _append(**bad) == kv.KVC_E_SHAPE, bad
    for bad in ({"pairs": 4}, {"pairs": 40}, {"pairing": 2}, {"eps": -1e-6}, {"eps": float("nan")}, {"eps": float("inf")}):
        assert _append(**bad) == kv.KVC_E_RANGE, bad
    for bad in ({"spec": None}, {"pages": None}, {"q": False}, {"k": False}, {"v": rows(0)}, {"qo": False}, {"slots": None},
                {"pos": None}, {"f": False}):
        assert _append(**bad) == kv.KVC_E_NULL, bad
    assert _append(size=PB - 1) == kv.KVC_E_SIZE
    for bad in ({"pages": A + 128}, {"q": rows(2 * A + 2)}, {"qo": rows(10 * A, ts=HQ * D + 4)}, {"k": rows(3 * A, hs=D + 1)},
                {"v": rows(4 * A + 8)}, {"qw": 5 * A + 8}, {"kw": 6 * A + 2}, {"pos": 7 * A + 4}, {"slots": 8 * A + 4},
                {"status": 9 * A + 2}):
        assert _append(**bad) == kv.KVC_E_ALIGN, bad
    for bad in ({"qo": rows(3 * A, heads=HQ)}, {"qo": rows(4 * A + 2 * D, heads=HQ)},  # over the keys, the values
                {"qo": rows(2 * A + 2 * D, heads=HQ)},                               # shifted over its own input
                {"qo": rows(10 * A, ts=0, heads=HQ)}, {"qo": rows(10 * A, hs=D // 2)},
                {"qo": rows(A, heads=HQ)}, {"qo": rows(8 * A)}, {"qo": rows(7 * A)}, {"qo": rows(5 * A)}, {"qo": rows(6 * A)},
                {"k": rows(A + 256)}, {"v": rows(A + PB - 256)}, {"q": rows(A, heads=HQ)}, {"slots": A + 64}, {"pos": A + 64},
                {"kw": A + 64}, {"status": A + 64}, {"status": 8 * A + 8}, {"status": 10 * A}, {"status": 3 * A},
                {"status": 7 * A}):
        assert _append(**bad) == kv.KVC_E_ALIAS, bad


@fake_addresses
def test_append_without_queries_looks_at_none():
    """Past every check, the launch fails for want of a GPU."""
    assert _append() == kv.KVC_E_HIP
    assert _append(hq=0, q=False, qo=False, qw=3) == kv.KVC_E_HIP
    assert _append(pairs=0, pos=None, f=False) == kv.KVC_E_HIP
    assert _append(qo=rows(2 * A, heads=HQ)) == kv.KVC_E_HIP   # in place


WS = ka.kvpage_attend_window_workspace_bytes(SPEC, N, HQ, 64, 40, 4)


def _window(spec=SPEC, pages=A, size=PB, n=N, hq=HQ, q=None, table=3 * A, cols=4, stride=4, lens=4 * A, window=40, sinks=4,
            scale=0.125, out=None, lse=6 * A, ws=7 * A, ws_bytes=WS, status=8 * A):
    q = rows(2 * A, heads=HQ) if q is None else q
    out = rows(5 * A, heads=HQ) if out is None else out
    return L.kvpage_attend_window(spec, pages, size, n, hq, q or None, table, cols, stride, lens, window, sinks, scale,
                                  out or None, lse, ws, ws_bytes, status, None)


PWS = ka.kvpage_attend_prompt_workspace_bytes(SPEC, 2, N, HQ, 64)


def _prompt(spec=SPEC, pages=A, size=PB, seqs=2, n=N, hq=HQ, q=None, starts=9 * A, table=3 * A, cols=4, stride=4, lens=4 * A,
            window=0, sinks=0, scale=0.125, out=None, lse=6 * A, ws=7 * A, ws_bytes=PWS, status=8 * A):
    q = rows(2 * A, heads=HQ) if q is None else q
    out = rows(5 * A, heads=HQ) if out is None else out
    return L.kvpage_attend_prompt(spec, pages, size, seqs, n, hq, q or None, starts, table, cols, stride, lens, window, sinks,
                                  scale, out or None, lse, ws, ws_bytes, status, None)


@fake_addresses
@pytest.mark.parametrize("f", [_window, _prompt])
def test_attention_refusals(f):
    assert f(n=0) == kv.KVC_OK
    for bad in ({"spec": None}, {"pages": None}, {"q": False}, {"table": None}, {"lens": None}, {"out": rows(0)},
                {"ws": None}):
        assert f(**bad) == kv.KVC_E_NULL, bad
    for bad in ({"spec": ka.kvc_pages(6, HK, 16, 96, 4)}, {"spec": ka.kvc_pages(6, HK, 16, D, 3)}, {"hq": 7}, {"hq": 0},
                {"cols": 0}, {"cols": 1 << 27}, {"n": 1 << 27}, {"q": rows(2 * A, ts=1 << 62)}):
        assert f(**bad) == kv.KVC_E_SHAPE, bad
    for bad in ({"scale": float("inf")}, {"scale": float("nan")}, {"scale": 3e38}, {"stride": 3}, {"stride": 1 << 31}):
        assert f(**bad) == kv.KVC_E_RANGE, bad
    assert f(size=PB - 1) == kv.KVC_E_SIZE and f(ws_bytes=0) == kv.KVC_E_SIZE
    for bad in ({"pages": A + 16}, {"q": rows(2 * A + 8)}, {"out": rows(5 * A, hs=D + 4)}, {"table": 3 * A + 2},
                {"lens": 4 * A + 1}, {"lse": 6 * A + 2}, {"ws": 7 * A + 64}, {"status": 8 * A + 1}):
        assert f(**bad) == kv.KVC_E_ALIGN, bad
    for bad in ({"out": rows(2 * A, heads=HQ)}, {"out": rows(A, heads=HQ)}, {"out": rows(3 * A, heads=HQ)},
                {"out": rows(5 * A, ts=0)}, {"lse": 5 * A}, {"ws": A}, {"ws": 2 * A}, {"status": 7 * A + 16},
                {"lse": 4 * A}, {"status": 3 * A}, {"lse": 2 * A}):
        assert f(**bad) == kv.KVC_E_ALIAS, bad
    assert f() == kv.KVC_E_HIP and f(lse=None, status=None) == kv.KVC_E_HIP
    assert f(window=0xFFFFFFFF, sinks=0xFFFFFFFF, ws_bytes=1 << 30) == kv.KVC_E_HIP


@fake_addresses
def test_prompt_refusals():
    assert _prompt(seqs=0) == kv.KVC_OK
    assert _prompt(starts=None) == kv.KVC_E_NULL and _prompt(starts=9 * A + 2) == kv.KVC_E_ALIGN
    assert _prompt(seqs=1 << 20) == kv.KVC_E_SHAPE
    for bad in ({"out": rows(9 * A, heads=HQ)}, {"lse": 9 * A + 8}, {"ws": 9 * A}, {"status": 9 * A}):
        assert _prompt(**bad) == kv.KVC_E_ALIAS, bad
    few = ka.kvpage_attend_prompt_workspace_bytes(SPEC, 1, 1, 8, 1 << 15)   # shared out
    assert few > 256
    assert _prompt(seqs=1, n=1, cols=1 << 11, stride=1 << 11, ws_bytes=few) == kv.KVC_E_HIP
    assert _prompt(seqs=1, n=1, cols=1 << 11, stride=1 << 11, ws_bytes=256) == kv.KVC_E_SIZE


@fake_addresses
def test_calls_take_the_workspace_of_larger_ones():
    """The size is looked at before the alignment of q, which is wrong in each of these calls: nothing is launched."""
    spec = ka.kvc_pages(600, 8, 16, 128, 4)
    bad = ka.kvc_rows(2 * A + 8, 32 * 128, 128)
    most = ka.kvpage_attend_prompt_workspace_bytes(spec, 40, 9000, 32, 1 << 20, 0, 0)
    wide = ka.kvpage_attend_window_workspace_bytes(spec, 700, 32, 1 << 20, 4096, 100)
    for n in (1, 3, 32, 33, 200, 700, 5000, 9000):
        for cols in (1, 17, 100, 5000, 1 << 16):
            for window, sinks in ((0, 0), (1, 0), (100, 4), (4096, 100)):
                for b in (1, 15, 40):
                    assert _prompt(spec=spec, size=1 << 40, n=n, seqs=b, hq=32, cols=cols, stride=cols, q=bad, window=window,
                                   sinks=sinks, ws_bytes=most) == kv.KVC_E_ALIGN
                if window and n <= 700:
                    assert _window(spec=spec, size=1 << 40, n=n, hq=32, cols=cols, stride=cols, q=bad, window=window,
                                   sinks=sinks, ws_bytes=wide) == kv.KVC_E_ALIGN


# ---------------------------------------------------------------- the binding's own checks

def test_binding_refuses_wrong_tensors():
    spec = (4, 2, 16, 64, 4)
    pages = torch.zeros(ka.kvpage_bytes(spec), dtype=torch.uint8)
    b = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    i64, f = torch.zeros(3, dtype=torch.int64), np.ones(32, np.float32)
    good = dict(spec=spec, pages=pages, q=q, k=b, v=b, positions=i64, inv_freq=f, slots=i64, q_out=q.clone())
    for bad in (dict(k=b[:2]), dict(v=b.half()), dict(slots=i64.int()), dict(q_out=None), dict(q_out=q[:, :2]), dict(positions=None),
                dict(positions=i64[:2]), dict(q=q[..., :32]), dict(k_weight=b[0, 0, :32]), dict(pages=pages.view(torch.int32)),
                dict(inv_freq=None), dict(dev_status=torch.zeros(2, dtype=torch.int32)), dict(pairing=-1), dict(spec=spec[:4])):
        with pytest.raises(ValueError):
            ka.kvpage_append(**{**good, **bad})
    with pytest.raises(ValueError, match="GPU"):
        ka.kvpage_append(**good)
    with pytest.raises(TypeError):
        ka.kvpage_append(spec, pages, q, b, b, i64, f, i64)
    table, lens, ws = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(4096, dtype=torch.uint8)
    good = dict(spec=spec, pages=pages, q=q, table=table, lens=lens, window=4, sinks=1, out=q.clone(), ws=ws)
    for bad in (dict(window=-1), dict(window=1 << 32), dict(sinks=None), dict(lens=lens[:2]), dict(table=table.long()),
                dict(out=q[:, :2]), dict(lse=torch.zeros(3, 2))):
        with pytest.raises(ValueError):
            ka.kvpage_attend_window(**{**good, **bad})
    with pytest.raises(ValueError, match="GPU"):
        ka.kvpage_attend_window(**good)
    starts = torch.zeros(4, dtype=torch.int32)
    good = dict(spec=spec, pages=pages, q=q, starts=starts, table=table, lens=lens, out=q.clone(), ws=ws)
    for bad in (dict(starts=starts.long()), dict(starts=starts[:0]), dict(starts=starts[:3]), dict(starts=starts[None]),
                dict(lens=lens[:1]), dict(table=table[:1]), dict(out=q[:2]), dict(window=-1), dict(q=q[0])):
        with pytest.raises(ValueError):
            ka.kvpage_attend_prompt(**{**good, **bad})
    with pytest.raises(ValueError, match="GPU"):
        ka.kvpage_attend_prompt(**good)


def test_structures():
    assert ctypes.sizeof(ka.kvc_pages) == 20 and ka.KVC_PAGE_FP4 == 4 and ka.KVC_DEV_BAD_START == 128
