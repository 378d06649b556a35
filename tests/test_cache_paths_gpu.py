"""The cache operators where their kernels share work: more sequences than a
block counts at once, pools beyond 32-bit offsets, workspaces full of junk,
shared by graphs and by calls of other shapes, two streams at once."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def workspace(c, d):
    if c.pool == "q4":
        return B.new_q4_workspace(d["q"], d["pool"], d["table"])
    return B.new_weights_workspace(d["q"], d["pool"][0], d["table"])


def attend(inp, d, ws, weights=True, **kw):
    """(out, key weights or None)"""
    import torch
    c = inp.c
    w = torch.empty_like(d["w"]) if weights else None
    args = (d["table"], d["ctx"], c.ps, inp.scale, c.causal)
    kw = dict(kw, workspace=ws, key_weights_out=w, key_weights=d["w"] if weights else None)
    if c.pool == "q4":
        return B.paged_attention_q4(d["q"], d["pool"], *args, **kw), w
    return B.paged_attention_weights(d["q"], *d["pool"], *args, **kw), w


def check(inp, out, w, skip=()):
    want, added, tol, w_tol = ref.attend(inp, skip)
    assert ref.worst(_np(out), want, tol) <= 1
    if w is not None:
        live = np.arange(inp.cap)[None, None] < inp.ctx[:, None, None]
        live[list(skip)] = False
        full = np.where(live, added + inp.w, 0.0)
        assert ref.worst(_np(w), full, w_tol + 2.0 ** -24 * full) <= 1


def spread(n, lo, hi):
    return [lo + (37 * i) % (hi - lo) for i in range(n)]


# one case per kernel; spare table entries keep the capacity above what the
# short-table and whole-prompt forms take
PATHS = [
    Case(2, 4, 2, 1, 16, [300, 900]),                              # short table
    Case(2, 4, 2, 1, 16, [300, 1900]),                             # shares of all keys
    Case(2, 4, 2, 2, 16, [300, 1900], dtype="f32"),
    Case(2, 4, 2, 13, 16, [400, 90], dtype="f32", spare=70),       # 64-row blocks
    Case(2, 4, 2, 13, 16, [400, 1300], pool="bf16"),
    Case(2, 4, 2, 40, 16, [700, 41]),                              # tiles
    Case(2, 4, 2, 40, 16, [700, 41], pool="bf16"),
    Case(2, 4, 2, 65, 12, [900, 66], pool="bf16"),                 # tiles, a short last one
    Case(2, 4, 2, 100, 16, [700, 141]),                            # whole prompts
]


@pytest.mark.parametrize("c", [
    Case(300, 1, 1, 1, 16, spread(300, 1, 60), spare=70),
    Case(300, 2, 1, 1, 16, spread(300, 1, 60), pool="bf16", spare=70),
    Case(300, 4, 1, 12, 16, spread(300, 12, 60), dtype="f32", spare=70),
    Case(600, 8, 1, 8, 16, spread(600, 8, 90), spare=6),
    Case(600, 8, 1, 8, 16, spread(600, 8, 90), pool="bf16", spare=6),
    Case(520, 4, 1, 33, 16, spread(520, 33, 80), spare=15),
    # few rows, tables wide enough to count as many keys
    Case(2, 4, 2, 10, 16, [900, 90], spare=2100),
    Case(2, 4, 2, 5, 16, [900, 90], pool="bf16", spare=4200),
    # one query tile: a sequence's pieces of one, two and more key tiles
    Case(90, 8, 2, 16, 16, spread(90, 16, 700)),
    Case(90, 4, 2, 25, 16, spread(90, 25, 700), pool="bf16"),
], ids=str)
def test_many_sequences_and_wide_tables(c):
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    out, w = attend(inp, d, ws)
    assert B.pa_check_device_flag(ws)[1] == 0
    check(inp, out, w)


@pytest.mark.parametrize("pool", ["q4", "bf16"])
@pytest.mark.parametrize("L", [40, 65])
def test_bad_lengths_and_pages_on_tiles(pool, L):
    import torch
    c = Case(4, 4, 2, L, 16, [400, 100, 264, 150], pool=pool, spare=30)
    inp = ref.Inputs(c)
    d = inp.device()
    good = d["ctx"]
    ws = workspace(c, d)
    d["ctx"] = torch.tensor([L - 1, 100, inp.cap + 1, 150], dtype=torch.int32, device="cuda")
    out, w = attend(inp, d, ws)
    assert B.pa_check_device_flag(ws, clear=True)[1] == B.PA_FLAG_BAD_CONTEXT
    check(inp, out, w, skip=(0, 2))
    d["ctx"] = good
    d["table"][0, 3] = inp.P
    d["table"][3, 0] = -1
    out, w = attend(inp, d, ws)
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_PAGE
    for x in inp.dense:  # their keys read as zeros
        x[inp.table[0, 3]] = 0
        x[inp.table[3, 0]] = 0
    check(inp, out, w)


@pytest.mark.parametrize("c,weights", [(c, True) for c in PATHS] +
                         [(c, False) for c in PATHS if c.pool == "q4"], ids=str)
def test_captured_on_junk(c, weights):
    """A workspace of junk behind its first bytes serves a call, and two graphs
    of calls of different shapes in turn."""
    import torch
    inp = ref.Inputs(c)
    other = ref.Inputs(Case(**{**c.__dict__, "B": 1, "ctx": c.ctx[1:], "seed": 9}))
    d, e = inp.device(), other.device()
    ws = max((workspace(x.c, y) for x, y in ((inp, d), (other, e))), key=lambda t: t.numel())
    flat = ws.view(-1).view(torch.uint8)
    flat[256:] = 0xff  # (the first 256 bytes are the flag and counters, zero between calls)
    first = attend(inp, d, ws, weights)
    flat[256:] = 0x7f
    second = attend(other, e, ws, weights)
    check(inp, *first)
    check(other, *second)
    graphs = []
    for i, dd in ((inp, d), (other, e)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = attend(i, dd, ws, weights)
        graphs.append((g, got))
    for k in (0, 1, 1, 0):
        graphs[k][0].replay()
    torch.cuda.synchronize()
    for (_, got), want in zip(graphs, (first, second)):
        assert torch.equal(got[0], want[0])
        assert not weights or torch.equal(got[1], want[1])
    assert B.pa_check_device_flag(ws)[1] == 0


def test_two_streams_at_once():
    import torch
    sets = []
    for c in PATHS:
        inp = ref.Inputs(c)
        d = inp.device()
        sets.append((inp, d, workspace(c, d)))
    want = [attend(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(3):
        for i, s in enumerate(sets):
            got.append((i, attend(*s, stream=streams[(i + turn) % 2])))
        torch.cuda.synchronize()
    for i, (out, w) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(w, want[i][1])


@pytest.mark.parametrize("mult", [2.0 ** -100, 2.0 ** -30, 2.0 ** 60])
@pytest.mark.parametrize("pool,L", [("q4", 1), ("q4", 5), ("q4", 40), ("bf16", 5), ("bf16", 40)])
def test_queries_far_from_one(pool, L, mult):
    c = Case(1, 4, 1, L, 16, [300], pool=pool, spare=4)
    inp = ref.Inputs(c)
    inp.q = ref.bf16((inp.q * np.float32(mult)).astype(np.float32))
    inp.scale = float(np.float32(0.1 / mult))
    d = inp.device()
    check(inp, *attend(inp, d, workspace(c, d)))


def far(inp, pages):
    """The inputs with their pool at the end of one of `pages` pages."""
    import torch
    d = inp.device()
    old = d["pool"]
    grown = []
    for t in old:
        x = torch.empty(pages, *t.shape[1:], dtype=t.dtype, device="cuda")
        x[pages - inp.P:] = t
        grown.append(x)
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (pages - inp.P), d["table"])
    d["pool"] = B.Q4Pool(*grown) if inp.c.pool == "q4" else grown
    return d, old


@pytest.mark.parametrize("pool,L", [("q4", 1), ("q4", 20), ("q4", 40), ("q4", 200),
                                    ("bf16", 1), ("bf16", 12), ("bf16", 40)])
def test_beyond_32_bit_offsets(pool, L):
    """Rows whose byte offsets pass 32 bits give what the same rows at the
    start of a pool give."""
    import torch
    c = Case(2, 4, 2, L, 128, [300, 201], pool=pool, spare=1)
    inp = ref.Inputs(c, extra_pages=4)
    near = inp.device()
    ws = workspace(c, near)
    want = attend(inp, near, ws)
    pages = (2 ** 32 // (64 if pool == "q4" else 256)) // (2 * 128) + 64
    d, old = far(inp, pages)
    got = attend(inp, d, ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    if L > 1:
        return
    # eviction to the far pages, and (4-bit) an append there
    base = pages - inp.P
    dst = torch.from_numpy(inp.free[:4].reshape(2, 2).astype(np.int32)).cuda()
    args = (d["ctx"], d["w"], 150, 20)
    if pool == "q4":
        B.evict_kv_q4(old, near["table"], *args, dst)
        B.evict_kv_q4(d["pool"], d["table"], *args, dst + base)
        x = torch.randn(2, 2, 1, 128, device="cuda").bfloat16()
        B.append_kv_q4(x, -x, old, near["table"], d["ctx"])
        B.append_kv_q4(x, -x, d["pool"], d["table"], d["ctx"])
        near_rows = B.gather_kv_q4(old, near["table"], d["ctx"], 300)
        far_rows = B.gather_kv_q4(d["pool"], d["table"], d["ctx"], 300)
        assert all(torch.equal(a, b) for a, b in zip(near_rows, far_rows))
    else:
        B.evict_kv(*old, near["table"], *args, dst)
        B.evict_kv(*d["pool"], d["table"], *args, dst + base)
    for a, b in zip(old, d["pool"]):
        assert torch.equal(a.view(torch.uint8), b[base:].view(torch.uint8))


@pytest.mark.parametrize("Bn,H,ps,ctx,keep,recent", [
    (80, 4, 16, spread(80, 1, 200), 60, 7),   # more heads than are resident at 1024 threads
    (1, 1, 128, [52000], 20000, 11),          # more keys than shared memory holds
], ids=["heads", "keys"])
def test_evict_forms(Bn, H, ps, ctx, keep, recent):
    import test_evict_gpu as e
    inp = ref.Inputs(Case(Bn, 1, H, 1, ps, ctx, pool="q4"), extra_pages=Bn * -(-keep // ps))
    w = np.random.default_rng(2).random(inp.w.shape).astype(np.float32)
    e.check(inp, "q4", np.round(w, 2), keep, recent)
