"""GPU parity of attention of many new tokens over values whose sizes only some rows see, through each of its plans: every row
against the bound of what it sees alone."""

import numpy as np
import pytest

from agent_handoff_amd import kvattend as ka
from attend_util import Store, bits, host_f64, sequence
from oracle import attend as oa
from prompt_util import check_each_row, growing_values, plan_name, prompt_plan, value_steps
from serving_util import default_scale, put_all, rows_see
from test_gpu_attend_prompt import _attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [ka.KVC_PAGE_INT8, ka.KVC_PAGE_FP8])
@pytest.mark.parametrize("name, n, m, group, cols", [("few", 60, 30, 1, 20), ("blocks", 320, 200, 2, 20), ("shared", 600, 400, 2, 40)])
@pytest.mark.parametrize("low, high", [(-30, 30), (30, -30), (-8, 8)])
def test_sizes_of_values_that_only_some_rows_see(fmt, name, n, m, group, cols, low, high):
    """Each row is bound by the values that it sees alone: small ones seen first keep their bits beside large ones that
    later rows see."""
    rng = np.random.default_rng(92)
    d = 64
    spec = (cols, 1, 16, d, fmt)
    assert plan_name(prompt_plan(spec, 1, m, group, cols)) == name
    store = Store(spec)
    put_all(store.host, spec, bits(rng, (n, 1, d)), growing_values(rng, n, d, low, high), np.arange(n))
    table = np.arange(cols, dtype=np.int32)[None]
    q = bits(rng, (m, group, d))
    out, lse = _attend(spec, store.dev(), q, [0, m], table, [n])
    k, v = sequence(store, table, 0, n)
    check_each_row(host_f64(out), host_f64(lse), oa.f64(q), k, v, value_steps(store.host, spec, np.arange(n)),
                   default_scale(d), fmt, rows_see(m, n), (fmt, name))
