"""GPU parity of attention of new tokens of very many sequences, a workgroup a block: the time grows with the sequences, not with
their square, and what is wrong with any of them is reported."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import bits, host_f64, sequence
from gpu_util import DEV, say, to_dev
from oracle import attend as oa
from prompt_util import plan_name, prompt_plan
from serving_util import ALL_FORMATS, check_rows, default_scale, i32, largest_steps, rows_see, status, store_of

pytestmark = pytest.mark.gpu


def many(rng, n, spec, most_new, cols):
    """A store of pages that all sequences share, and sequences of up to most_new tokens over up to cols pages."""
    store, table = store_of(rng, spec, [spec[0] * spec[2]])
    new = rng.integers(0, most_new + 1, n)
    lens = np.minimum(new + rng.integers(0, cols * spec[2], n), cols * spec[2])
    lens[rng.integers(0, n, n // 50)] = 0                  # rows that see nothing
    return store, rng.choice(table[0], (n, cols)).astype(np.int32), new, lens


def check(store, table, q, starts, new, lens, out, lse, only):
    spec = store.spec
    for b in only:
        at = slice(starts[b], starts[b] + new[b])
        n = int(lens[b])
        k, v = sequence(store, table, b, n) if n else (np.zeros((spec[1], 0, spec[3])),) * 2
        check_rows(host_f64(out[at]), host_f64(lse[at]), oa.f64(q[at]), k, v, default_scale(spec[3]), spec[4],
                   largest_steps(store), rows_see(int(new[b]), n), (spec, int(b), n))


@pytest.mark.parametrize("fmt", ALL_FORMATS)
@pytest.mark.parametrize("n, most_new, heads, group, d", [(65, 40, 2, 4, 64), (300, 5, 3, 2, 128), (1000, 70, 1, 4, 64)])
def test_more_sequences_than_a_wave_holds(fmt, n, most_new, heads, group, d):
    rng = np.random.default_rng(n)
    spec = (16, heads, 16, d, fmt)
    store, table, new, lens = many(rng, n, spec, most_new, 8)
    starts = 3 + np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1]) + 2
    say("many sequences", spec, n, rows)
    plan = prompt_plan(spec, n, rows, heads * group, 8)
    assert plan_name(plan) == "blocks"
    q = bits(rng, (rows, heads * group, d))
    out = torch.full((rows, heads * group, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows, heads * group), 7.0, device=DEV)
    ws = torch.empty(plan.bytes, dtype=torch.uint8, device=DEV)
    st = status()
    ka.kvpage_attend_prompt(spec, store.dev(), to_dev(q), i32(starts), i32(table), i32(lens), out, ws, lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    for edge in (slice(0, 3), slice(rows - 2, rows)):
        assert bool((out[edge] == 3.0).all()) and bool((lse[edge] == 7.0).all())
    assert bool(torch.isfinite(out).all())
    check(store, table, q, starts, new, lens, out, lse, range(n) if n < 400 else rng.choice(n, 200, replace=False))


def test_time_grows_with_the_sequences():
    """16384 sequences of up to two new tokens: some 2 ms; 30 where each workgroup counts them all."""
    rng = np.random.default_rng(3)
    n, heads, group, d = 16384, 8, 4, 128
    spec = (16, heads, 16, d, ka.KVC_PAGE_BF16)
    store, table, new, lens = many(rng, n, spec, 2, 3)
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1])
    plan = prompt_plan(spec, n, rows, heads * group, 3)
    assert plan_name(plan) == "blocks"
    q = bits(rng, (rows, heads * group, d))
    dev, qd, s, t, ln = store.dev(), to_dev(q), i32(starts), i32(table), i32(lens)
    out = torch.zeros_like(qd)
    lse = torch.zeros(rows, heads * group, device=DEV)
    ws = torch.empty(plan.bytes, dtype=torch.uint8, device=DEV)
    times = []
    for _ in range(4):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        ka.kvpage_attend_prompt(spec, dev, qd, s, t, ln, out, ws, lse=lse)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    say("many sequences", n, times)
    assert min(times) < 10
    check(store, table, q, starts, new, lens, out, lse, rng.choice(n, 60, replace=False))


def test_what_is_wrong_is_reported_wherever_it_is():
    """Lengths of sequences without new tokens too, and wrong starts of the first, the last and one in the middle."""
    rng = np.random.default_rng(4)
    n, spec = 333, (16, 1, 16, 64, ka.KVC_PAGE_INT8)
    store, table, new, lens = many(rng, n, spec, 4, 8)
    new[[0, 100, n - 1]] = 0, 0, 3
    starts = np.concatenate([[0], np.cumsum(new)])
    rows = int(starts[-1])
    q, dev = to_dev(bits(rng, (rows, 2, 64))), store.dev()
    ws = torch.empty(prompt_plan(spec, n, rows, 2, 8).bytes, dtype=torch.uint8, device=DEV)

    def call(starts, lens):
        out, st = torch.full((rows, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV), status()
        ka.kvpage_attend_prompt(spec, dev, q, i32(starts), i32(table), i32(lens), out, ws, dev_status=st)
        torch.cuda.synchronize()
        return out, int(st)

    ref, st = call(starts, lens)
    assert st == 0
    for b in (0, 100, 200, n - 1):
        for length in (-1, 129):
            wrong = lens.copy()
            wrong[b] = length
            out, st = call(starts, wrong)
            assert st == ka.KVC_DEV_BAD_LENGTH, b
            keep = torch.ones(rows, dtype=torch.bool, device=DEV)
            keep[starts[b]:starts[b + 1]] = False
            assert torch.equal(out[keep], ref[keep])
    for at, value in ((0, -1), (1, rows + 1), (100, -(1 << 31)), (150, 1 << 30), (200, 0), (n, rows + 1), (n, 0)):
        wrong = starts.copy()
        wrong[at] = value
        assert call(wrong, lens)[1] == ka.KVC_DEV_BAD_START, (at, value)
