"""Eviction on the GPU: kept positions, weights, lengths and rows, bit for bit."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def device_pool(inp, dtype):
    import torch
    d = inp.device()
    if dtype == "f32":
        d["pool"] = [t.float() + 1e-3 for t in d["pool"]]
    return d


def check(inp, dtype, w, keep, recent, ctx=None):
    import torch
    c = inp.c
    d = device_pool(inp, dtype)
    ctx = np.array(c.ctx if ctx is None else ctx, np.int32)
    npg = -(-keep // c.ps)
    dst = inp.free[:c.B * npg].reshape(c.B, npg).astype(np.int32)
    before = [t.clone() for t in d["pool"]]
    ws = B.new_cache_workspace()
    args = (d["table"], torch.from_numpy(ctx).cuda(), torch.from_numpy(w).cuda(), keep, recent,
            torch.from_numpy(dst).cuda())
    if dtype == "q4":
        new = B.evict_kv_q4(d["pool"], *args, workspace=ws)
    else:
        new = B.evict_kv(*d["pool"], *args, workspace=ws)
    assert B.pa_check_device_flag(ws)[1] == 0
    kept, lens = ref.evict(w, ctx, keep, recent)
    assert np.array_equal(new.kept.cpu().numpy(), kept)
    assert np.array_equal(new.context_lens.cpu().numpy(), lens)
    want_w = np.where(kept >= 0, np.take_along_axis(w, np.maximum(kept, 0), 2), 0)
    assert np.array_equal(new.key_weights.cpu().numpy().view(np.int32),
                          want_w.astype(np.float32).view(np.int32))
    b, h, j = np.nonzero(kept >= 0)
    s = kept[b, h, j]
    for got, old in zip(d["pool"], before):
        exp = old.clone()
        exp[dst[b, j // c.ps], h, j % c.ps] = old[inp.table[b, s // c.ps], h, s % c.ps]
        assert torch.equal(got.view(torch.uint8), exp.view(torch.uint8))


CASES = [
    # B, H_kv, ps, ctx, keep, recent
    (1, 1, 1, [1], 1, 0),
    (2, 2, 16, [17, 40], 16, 3),
    (3, 1, 3, [10, 50, 29], 29, 29),
    (2, 2, 12, [600, 513], 100, 0),
    (2, 1, 64, [512, 1025], 511, 64),
    (4, 2, 16, [0, 5, 100, 64], 64, 10),
    (1, 1, 128, [5000], 1, 1),
    (1, 2, 128, [9000], 4097, 1000),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("Bn,H,ps,ctx,keep,recent", CASES, ids=lambda v: str(v).replace(" ", ""))
def test_evict(dtype, Bn, H, ps, ctx, keep, recent):
    c = Case(Bn, 1, H, 1, ps, ctx, pool="q4" if dtype == "q4" else "bf16", spare=1)
    inp = ref.Inputs(c, extra_pages=Bn * -(-keep // ps))
    rng = np.random.default_rng(keep)
    w = np.exp(rng.standard_normal(inp.w.shape) * 3).astype(np.float32)
    check(inp, dtype, w, keep, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "nan", "tiny", "unused"])
def test_order_of_weights(kind):
    c = Case(2, 1, 2, 1, 16, [700, 1100], pool="q4")
    inp = ref.Inputs(c, extra_pages=40)
    rng = np.random.default_rng(3)
    w = rng.standard_normal(inp.w.shape).astype(np.float32)
    if kind == "equal":
        w[:] = 0.25
    elif kind == "few":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    elif kind == "signs":
        w = rng.choice(np.array([0.0, -0.0, 1.0, -1.0, np.inf, -np.inf], np.float32), w.shape)
    elif kind == "nan":
        w[rng.random(w.shape) < 0.02] = np.nan
    elif kind == "tiny":
        w = (rng.integers(0, 5, w.shape) * 1e-45).astype(np.float32)
    else:
        w[0, :, 700:], w[1, :, 1100:] = 1e30, np.nan  # past the contexts
    check(inp, "q4", w, 300, 50)


def test_long_contexts():
    c = Case(1, 1, 2, 1, 128, [40000], pool="q4")
    inp = ref.Inputs(c, extra_pages=160)
    w = np.random.default_rng(1).random(inp.w.shape).astype(np.float32)
    check(inp, "q4", np.round(w, 3), 20001, 77)


def test_errors_are_recorded():
    import torch
    c = Case(3, 1, 2, 1, 16, [100, 50, 64], pool="q4")
    inp = ref.Inputs(c, extra_pages=9)
    d = inp.device()
    dst = torch.from_numpy(inp.free[:9].reshape(3, 3).astype(np.int32)).cuda()
    ctx = torch.tensor([-1, 50, 10 ** 6], dtype=torch.int32, device="cuda")
    ws = B.new_cache_workspace()
    new = B.evict_kv_q4(d["pool"], d["table"], ctx, d["w"], 40, 5, dst, workspace=ws)
    assert B.pa_check_device_flag(ws, clear=True)[1] == B.PA_FLAG_BAD_CONTEXT
    assert new.context_lens.tolist() == [0, 40, 0]
    assert (new.kept[0] == -1).all() and not new.key_weights[2].any()
    before = [t.clone() for t in d["pool"]]
    d["table"][0, 0], dst[1, 1] = inp.P, -5
    B.evict_kv_q4(d["pool"], d["table"], d["ctx"], d["w"], 40, 5, dst, workspace=ws)
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_PAGE
    used = set(dst[dst >= 0].tolist())
    for pg in set(range(inp.P)) - used:
        assert all(torch.equal(a[pg], b[pg]) for a, b in zip(before, d["pool"]))


def test_captured():
    import torch
    c = Case(2, 1, 2, 1, 16, [300, 200], pool="bf16")
    inp = ref.Inputs(c, extra_pages=20)
    d = inp.device()
    dst = torch.from_numpy(inp.free[:20].reshape(2, 10).astype(np.int32)).cuda()
    ws = B.new_cache_workspace()
    B.evict_kv(*d["pool"], d["table"], d["ctx"], d["w"], 150, 20, dst, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        new = B.evict_kv(*d["pool"], d["table"], d["ctx"], d["w"], 150, 20, dst, workspace=ws)
    for seed in range(2):
        w = np.random.default_rng(seed).random(inp.w.shape).astype(np.float32)
        d["w"].copy_(torch.from_numpy(w))
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(new.kept.cpu().numpy(), ref.evict(w, c.ctx, 150, 20)[0])
