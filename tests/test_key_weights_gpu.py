"""Key weights on the GPU (bf16 and 4-bit pages) against 64 bits."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


CASES = [
    Case(1, 1, 1, 1, 1, [1]),
    Case(3, 4, 2, 1, 128, [33, 257, 1000], spare=1),
    Case(2, 7, 1, 1, 12, [129, 700]),
    Case(2, 8, 2, 2, 64, [600, 65]),
    Case(2, 3, 2, 3, 3, [3, 250]),
    Case(2, 4, 2, 32, 16, [32, 400]),
    Case(1, 2, 2, 130, 24, [333]),
    Case(2, 4, 1, 9, 16, [900, 5], causal=False),
    Case(1, 4, 1, 1, 16, [4000]),
]
CASES = [Case(**{**c.__dict__, "pool": p, "dtype": t}) for c in CASES
         for p, t in (("bf16", "bf16"), ("q4", "bf16"), ("q4", "f32"))]


def run(inp, d, w_in, w_out, ws=None, ctx=None):
    c = inp.c
    args = (d["table"], d["ctx"] if ctx is None else ctx, c.ps, inp.scale, c.causal)
    kw = dict(key_weights=w_in, key_weights_out=w_out, workspace=ws)
    if c.pool == "q4":
        return B.paged_attention_q4(d["q"], d["pool"], *args, **kw)
    return B.paged_attention_weights(d["q"], *d["pool"], *args, **kw)


def workspace(inp, d):
    if inp.c.pool == "q4":
        return B.new_q4_workspace(d["q"], d["pool"], d["table"])
    return B.new_weights_workspace(d["q"], d["pool"][0], d["table"])


@pytest.mark.parametrize("c", CASES, ids=str)
def test_weights(c):
    import torch
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(inp, d)
    want, added, tol, w_tol = ref.attend(inp)
    live = np.arange(inp.cap)[None, None] < inp.ctx[:, None, None]
    # out of place onto a wider array of junk
    out_w = torch.full((c.B, c.H_kv, inp.cap + 5), float("nan"), device="cuda")
    in_w = torch.nn.functional.pad(d["w"], (0, 5), value=float("nan"))
    in_w[:, :, :inp.cap][torch.from_numpy(~live).cuda().expand(c.B, c.H_kv, -1)] = float("nan")
    out = run(inp, d, in_w, out_w, ws)
    assert B.pa_check_device_flag(ws)[1] == 0
    assert ref.worst(_np(out), want, tol) <= 1
    got = _np(out_w)
    assert not got[:, :, inp.cap:].any()
    w = np.where(live, added + inp.w, 0.0)
    assert ref.worst(got[:, :, :inp.cap], w, w_tol + 2.0 ** -24 * w) <= 1
    # without what was there: each (sequence, kv head) hands out its rows' weight
    none_w = torch.empty_like(d["w"])
    run(inp, d, None, none_w, ws)
    assert ref.worst(_np(none_w), added, w_tol) <= 1
    assert np.allclose(_np(none_w).sum(-1), c.G * c.L, rtol=1e-4)
    # in place, twice
    acc = d["w"].clone()
    run(inp, d, acc, acc, ws)
    assert torch.equal(acc, out_w[:, :, :inp.cap])
    run(inp, d, acc, acc, ws)
    w2 = np.where(live, 2 * added + inp.w, 0.0)
    assert ref.worst(_np(acc), w2, 2 * w_tol + 2.0 ** -23 * w2) <= 1


@pytest.mark.parametrize("pool", ["bf16", "q4"])
@pytest.mark.parametrize("L", [1, 20])
def test_bad_lengths_and_pages(pool, L):
    import torch
    c = Case(4, 2, 2, L, 16, [40, 100, 64, 50], pool=pool)
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(inp, d)
    ctx = torch.tensor([L - 1, 100, 113, 50], dtype=torch.int32, device="cuda")
    w = torch.full_like(d["w"], float("nan"))
    out = run(inp, d, d["w"], w, ws, ctx)
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_CONTEXT
    want, added, tol, w_tol = ref.attend(inp, skip=(0, 2))
    assert ref.worst(_np(out), want, tol) <= 1
    assert not w[0].any() and not w[2].any()
    full = (added + inp.w)[[1, 3]]
    live = np.arange(inp.cap)[None, None] < inp.ctx[[1, 3]][:, None, None]
    assert ref.worst(_np(w)[[1, 3]], full * live, w_tol[[1, 3]] + 2.0 ** -24 * full) <= 1
    ws.zero_()
    d["table"][1, 2] = inp.P + 3  # keys 32 .. 47 of sequence 1
    run(inp, d, None, w, ws)
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_PAGE
    for x in inp.dense:
        x[inp.table[1, 2]] = 0  # they read as zeros
    _, added, _, w_tol = ref.attend(inp)
    assert ref.worst(_np(w), added, w_tol) <= 1


def test_peaked_rows():
    """Scores hundreds apart: all weight on one key, the rest exactly as small
    as 64 bits says."""
    c = Case(1, 4, 1, 1, 16, [500])
    for pool in ("bf16", "q4"):
        inp = ref.Inputs(Case(**{**c.__dict__, "pool": pool}))
        inp.scale = 8.0
        d = inp.device()
        w = d["w"].clone()
        out = run(inp, d, None, w)
        want, added, tol, w_tol = ref.attend(inp)
        assert ref.worst(_np(out), want, tol) <= 1
        # probabilities below fp32's normal range flush to zero
        assert ref.worst(_np(w), added, w_tol + 2.0 ** -125) <= 1
