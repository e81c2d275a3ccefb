"""Wrong starts in attention of many new tokens, through each of its plans: reported, and everything around outputs and
workspace stays as it was."""

import numpy as np
import pytest
import torch

from agent_handoff_amd import kvattend as ka
from attend_util import bits
from gpu_util import DEV, say, to_dev
from prompt_util import plan_name, prompt_plan
from serving_util import i32, status, store_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name, rows, lens", [("shared", 400, [900, 700, 500, 800]), ("few", 64, [900, 700, 500, 800]),
                                              ("blocks", 200, [300, 200, 100, 250])])
def test_wrong_starts_write_nowhere_else(d, name, rows, lens):
    """Outputs and workspace lie inside larger buffers, whose margins stay as they are, whatever lists of parts an earlier
    call has left in the workspace: numbers that could be a list's, and such as could not."""
    rng = np.random.default_rng(94)
    heads, group, page = 2, 2, 16
    spec = (200, heads, page, d, ka.KVC_PAGE_INT8)
    store, table = store_of(rng, spec, lens)
    cols = table.shape[1]
    plan = prompt_plan(spec, len(lens), rows, heads * group, cols)
    assert plan_name(plan) == name
    dev, tab, n = store.dev(), i32(table), i32(lens)
    q = to_dev(bits(rng, (rows, heads * group, d)))
    edge = 64
    out = torch.full((rows + 2 * edge, heads * group, d), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((rows + 2 * edge, heads * group), 7.0, device=DEV)
    room = 1 << 20
    ws = torch.empty(plan.bytes + 2 * room, dtype=torch.uint8, device=DEV)
    need = plan.bytes
    words = ws[room:room + need].view(torch.int32)
    inside = slice(edge, edge + rows)
    fills = [-1, 0, 1, 2, 0x7FFFFFFF, 511, None]
    for starts in ([0, rows, 0, rows, rows], [0, 20, 10, 30, rows + 1], [-5, 10, 20, 30, rows], [rows, 30, 20, 0, rows],
                   [0, 1 << 30, 30, 60, rows], [0, 10, 20, 30, -(1 << 31)]):
        for fill in fills:
            ws.fill_(0xA5)
            if fill is None:   # lists of small numbers
                words.copy_(torch.from_numpy(rng.integers(0, 40, words.numel()).astype(np.int32)))
            else:
                words.fill_(fill)
            st = status()
            say("wrong starts", name, d, starts, fill)
            ka.kvpage_attend_prompt(spec, dev, q, i32(starts), tab, n, out[inside], ws[room:room + need], lse=lse[inside],
                                    dev_status=st)
            torch.cuda.synchronize()
            assert int(st) == ka.KVC_DEV_BAD_START
            assert bool((ws[:room] == 0xA5).all()) and bool((ws[room + need:] == 0xA5).all())
            assert bool((out[:edge] == 3.0).all()) and bool((out[edge + rows:] == 3.0).all())
            assert bool((lse[:edge] == 7.0).all()) and bool((lse[edge + rows:] == 7.0).all())
