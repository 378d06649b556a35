"""Lengths and pages that break the contract of the draft trees' attention, over the page sizes,
row counts and context lengths that take different paths through it."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu

POOLS = [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"), ("q4", "f32")]
# drafts: one query tile and a word of drafts, two tiles, eight tiles and eight words; tables of a
# few key tiles (segments stay whole) and of many (cut and merged)
SHAPES = [(8, [200, 90, 130]), (64, [200, 90, 130]), (255, [300, 260, 400]),
          (8, [2000, 90, 900]), (64, [2000, 90, 900]), (255, [1500, 260, 700])]


def run(inp, d):
    ws = B.new_tree_workspace(d["q"], d["pool"] if inp.c.pool == "q4" else d["pool"][0], d["table"])
    ws[256:] = 0xff  # whatever was there
    got = tr.call(inp, d, workspace=ws).double().cpu().numpy()
    return got, B.pa_check_device_flag(ws)[1]


@pytest.mark.parametrize("pool,dtype", POOLS)
@pytest.mark.parametrize("ps", [12, 16])
@pytest.mark.parametrize("L,ctx", SHAPES, ids=lambda x: str(x).replace(" ", ""))
def test_lengths(pool, dtype, ps, L, ctx):
    """Sequences in every place whose length is below L, negative or above the capacity get zero
    rows; the others are not disturbed."""
    inp = tr.Inputs(tr.Case(4, 2, L, ps, ctx, pool, dtype, seed=L + ps))
    want, tol = tr.attend(inp)
    cap = inp.table.shape[1] * ps
    for b, bad_len in enumerate((L - 1, -1, cap + 1)):
        d = inp.device()
        d["ctx"][b] = bad_len
        got, flag = run(inp, d)
        assert (got[b] == 0).all() and flag == B.PA_FLAG_BAD_CONTEXT
        others = [x for x in range(3) if x != b]
        assert ref.worst(got[others], want[others], tol[others]) <= 1.0
    d = inp.device()
    d["ctx"][:] = 0
    got, flag = run(inp, d)
    assert (got == 0).all() and flag == B.PA_FLAG_BAD_CONTEXT


@pytest.mark.parametrize("pool,dtype", POOLS)
@pytest.mark.parametrize("ps", [12, 16])
@pytest.mark.parametrize("L,ctx", SHAPES, ids=lambda x: str(x).replace(" ", ""))
def test_pages(pool, dtype, ps, L, ctx):
    """Keys behind bad page ids read as zeros: before the drafts, among them, a sequence's first
    page and its last."""
    inp = tr.Inputs(tr.Case(4, 2, L, ps, ctx, pool, dtype, seed=L + ps + 1))
    d = inp.device()
    last = (ctx[2] - 1) // ps
    for at, page in (((0, 3), inp.P), ((1, 0), -1), ((2, last), 1 << 30), ((2, last - 1), -(1 << 31))):
        for t in inp.dense:
            t[inp.table[at]] = 0
        d["table"][at] = page
    want, tol = tr.attend(inp)
    got, flag = run(inp, d)
    assert ref.worst(got, want, tol) <= 1.0 and flag == B.PA_FLAG_BAD_PAGE
