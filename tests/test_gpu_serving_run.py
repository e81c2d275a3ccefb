"""The serving operators as a program uses them together: prompts in chunks,
then single tokens with a window, over one paged cache; on two streams; and in
replayed graphs."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import Store, bits, check_attend, host_f64, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from serving_util import ALL_FORMATS, check_rows, default_scale, half, i32, largest_steps, rows_see, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("d, window, sinks", [(128, 0, 0), (64, 50, 4)])
def test_conversations(fmt, d, window, sinks):
    """Three conversations: a chunk of each prompt, a second one (one conversation's only token), then single tokens.
    Attention is checked over what the pages hold, the pages against rotation and write one after the other."""
    rng = np.random.default_rng(d)
    heads, group, page, seqs = 2, 4, 16, 3
    hq, cols = heads * group, 16
    cache = ka.PagedKV(seqs * cols, heads, page, d, fmt)
    spec = tuple(getattr(cache.spec, f) for f, _ in cache.spec._fields_)
    say("conversations", spec, window, sinks)
    twin = torch.zeros_like(cache.pages)
    table = rng.permutation(seqs * cols).astype(np.int32).reshape(seqs, cols)
    freq = (10000.0 ** (-np.arange(d // 2) / (d // 2))).astype(np.float32)
    qw, kw = to_dev(bits(rng, (d,))), to_dev(bits(rng, (d,)))
    lens = np.zeros(seqs, np.int64)
    st = status()
    for new in ([70, 33, 5], [30, 1, 64], [1, 1, 1], [1, 1, 1]):
        at = np.concatenate([np.arange(a, a + m) for a, m in zip(lens, new)])
        seq = np.repeat(np.arange(seqs), new)
        lens = lens + new
        n = len(at)
        fused = to_dev(bits(rng, (n, hq + 2 * heads, d)))
        q, k, v = fused[:, :hq], fused[:, hq:hq + heads], fused[:, hq + heads:]
        slots = torch.from_numpy(table[seq, at // page].astype(np.int64) * page + at % page).to(DEV)
        pos = torch.from_numpy(at).to(DEV)
        turned = cache.append(q, k, v, pos, freq, slots, q_weight=qw, k_weight=kw, dev_status=st)
        qo, ko = torch.empty_like(turned), torch.empty(n, heads, d, dtype=torch.bfloat16, device=DEV)
        ka.kvc_norm_rotate(q, k, pos, freq, qo, ko, q_weight=qw, k_weight=kw)
        ka.kvpage_write(spec, twin, ko, v, slots)
        torch.cuda.synchronize()
        assert torch.equal(turned, qo) and torch.equal(cache.pages, twin)
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        lse = torch.empty(n, hq, device=DEV)
        if max(new) > 1:
            out = cache.attend_prompt(turned, i32(starts), i32(table), i32(lens), lse=lse, dev_status=st, window=window, sinks=sinks)
        else:
            out = cache.attend(turned, i32(table), i32(lens), lse=lse, dev_status=st, window=window, sinks=sinks)
        torch.cuda.synchronize()
        store = Store(spec)
        store.host[:] = cache.pages.cpu().numpy()
        o, l, qq = host_f64(out), host_f64(lse), host_f64(turned)
        for b in range(seqs):
            s = slice(starts[b], starts[b + 1])
            kk, vv = sequence(store, table, b, int(lens[b]))
            see = rows_see(new[b], int(lens[b]), window, sinks)
            if max(new) > 1:
                check_rows(o[s], l[s], qq[s], kk, vv, default_scale(d), fmt, largest_steps(store), see, (spec, b))
            else:
                check_attend(o[s][0], l[s][0], qq[s][0], kk[:, see[0]], vv[:, see[0]], default_scale(d), half(fmt),
                             largest_steps(store), (spec, b))
    assert int(st) == 0


class _Step:
    """One call of each operator on buffers of its own: tokens of two sequences appended, attended to as a prompt (shared
    out and joined) and as single tokens with a window."""

    def __init__(self, rng, fmt, n=6, length=3000):
        self.spec = (2 * 48, 2, 64, 128, fmt)
        self.length, self.n = length, n
        self.pages = torch.zeros(ka.kvpage_bytes(self.spec), dtype=torch.uint8, device=DEV)
        self.table = i32(rng.permutation(96).reshape(2, 48))
        full = torch.arange(length, device=DEV)
        slots = (self.table[:, full // 64].long() * 64 + full % 64).flatten()
        ka.kvpage_write(self.spec, self.pages, to_dev(bits(rng, (2 * length, 2, 128))), to_dev(bits(rng, (2 * length, 2, 128))), slots)
        self.rows = to_dev(bits(rng, (2 * n, 12, 128)))
        at = torch.arange(length - n, length, device=DEV)
        self.slots = (self.table[:, at // 64].long() * 64 + at % 64).flatten()
        self.pos = at.repeat(2)
        self.freq = (10000.0 ** (-np.arange(64) / 64)).astype(np.float32)
        self.starts, self.lens = i32([0, n, 2 * n]), i32([length, length])
        self.q = torch.zeros(2 * n, 8, 128, dtype=torch.bfloat16, device=DEV)
        self.outs = [torch.zeros_like(self.q), torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)]
        self.lses = [torch.zeros(2 * n, 8, device=DEV), torch.zeros(2, 8, device=DEV)]
        a = ka.kvpage_attend_prompt_workspace_bytes(self.spec, 2, 2 * n, 8, 48 * 64)
        b = ka.kvpage_attend_window_workspace_bytes(self.spec, 2, 8, 48 * 64, 1500, 4)
        assert a > 256 and b > 256
        self.ws = [torch.empty(x, dtype=torch.uint8, device=DEV) for x in (a, b)]

    def run(self):
        r = self.rows
        ka.kvpage_append(self.spec, self.pages, r[:, :8], r[:, 8:10], r[:, 10:], self.pos, self.freq, self.slots, self.q)
        ka.kvpage_attend_prompt(self.spec, self.pages, self.q, self.starts, self.table, self.lens, self.outs[0], self.ws[0],
                                lse=self.lses[0])
        ka.kvpage_attend_window(self.spec, self.pages, self.q[self.n - 1::self.n], self.table, self.lens, 1500, 4, self.outs[1],
                                self.ws[1], lse=self.lses[1])

    def result(self):
        return [t.clone() for t in (self.pages, self.q, *self.outs, *self.lses)]

    def clear(self):
        for t in (self.q, *self.outs, *self.lses):
            t.zero_()


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_two_streams_at_once(fmt):
    rng = np.random.default_rng(60)
    steps = [_Step(rng, fmt), _Step(rng, fmt)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.result())
        s.clear()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, stream in zip(steps, streams):
            with torch.cuda.stream(stream):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert _same(s.result(), w)


@pytest.mark.parametrize("fmt", ALL_FORMATS)
def test_replayed_graphs(fmt):
    """Two graphs with workspaces of their own, replayed with new rows, eager work in between."""
    rng = np.random.default_rng(61)
    steps = [_Step(rng, fmt), _Step(rng, fmt)]
    graphs = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run()
        graphs.append(g)
    for turn in range(4):
        fresh = [to_dev(bits(rng, s.rows.shape)) for s in steps]
        want = []
        for s, r in zip(steps, fresh):
            s.rows.copy_(r)
            s.run()
            torch.cuda.synchronize()
            want.append(s.result())
            s.clear()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert _same(s.result(), w), turn


def test_the_stream_given_is_the_one_used():
    """Work given a stream by its handle waits for what that stream holds, and not for the current one."""
    rng = np.random.default_rng(62)
    s = _Step(rng, ka.KVC_PAGE_FP4)
    s.run()
    torch.cuda.synchronize()
    want = s.result()
    s.clear()
    stream = torch.cuda.Stream()
    fresh = s.rows.clone()
    s.rows.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        s.rows.copy_(fresh)
    r = s.rows
    ka.kvpage_append(s.spec, s.pages, r[:, :8], r[:, 8:10], r[:, 10:], s.pos, s.freq, s.slots, s.q, stream=stream)
    ka.kvpage_attend_prompt(s.spec, s.pages, s.q, s.starts, s.table, s.lens, s.outs[0], s.ws[0], lse=s.lses[0],
                            stream=stream.cuda_stream)
    ka.kvpage_attend_window(s.spec, s.pages, s.q[s.n - 1::s.n], s.table, s.lens, 1500, 4, s.outs[1], s.ws[1], lse=s.lses[1],
                            stream=stream)
    torch.cuda.synchronize()
    assert _same(s.result(), want)


def test_empty_calls():
    spec = (2, 2, 16, 64, ka.KVC_PAGE_FP4)
    pages = torch.zeros(ka.kvpage_bytes(spec), dtype=torch.uint8, device=DEV)
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    i64 = torch.zeros(0, dtype=torch.int64, device=DEV)
    ws = torch.zeros(512, dtype=torch.uint8, device=DEV)
    ka.kvpage_append(spec, pages, none, kv, kv, i64, np.ones(32, np.float32), i64, none.clone())
    ka.kvpage_attend_window(spec, pages, none, i32(np.zeros((0, 2))), i32([]), 5, 1, none.clone(), ws)
    ka.kvpage_attend_prompt(spec, pages, none, i32([0, 0]), i32([[0, 1]]), i32([7]), none.clone(), ws)
    some = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    ka.kvpage_attend_prompt(spec, pages, torch.zeros_like(some), i32([2, 2]), i32([[0, 1]]), i32([7]), some, ws)
    ka.kvpage_attend_prompt(spec, pages, torch.zeros_like(some), i32([0]), i32(np.zeros((0, 2))), i32([]), some, ws)
    torch.cuda.synchronize()
    assert bool((some == 5.0).all()) and not pages.any()


def test_formula_of_a_small_prompt():
    """Written out token by token, without the other tests' helpers."""
    rng = np.random.default_rng(63)
    spec = (3, 1, 16, 64, ka.KVC_PAGE_BF16)
    cache = ka.PagedKV(*spec)
    k, v, q = bits(rng, (20, 1, 64)), bits(rng, (20, 1, 64)), bits(rng, (7, 2, 64))
    cache.write(to_dev(k), to_dev(v), torch.arange(20, device=DEV))
    out = cache.attend_prompt(to_dev(q), i32([0, 7]), i32([[0, 1, 2]]), i32([20]), window=6, sinks=2)
    torch.cuda.synchronize()
    o = host_f64(out)
    for i in range(7):
        p = 13 + i
        tokens = [t for t in range(p + 1) if t < 2 or t > p - 6]
        for h in range(2):
            w = np.array([np.exp(oa.f64(q)[i, h] @ oa.f64(k)[t, 0] / 8) for t in tokens])
            want = sum(a * oa.f64(v)[t, 0] for a, t in zip(w / w.sum(), tokens))
            assert np.all(np.abs(o[i, h] - want) <= 2.0 ** -8 * (np.abs(want) + np.abs(oa.f64(v)[:, 0]).max(0)) * 1.01)
