"""4-bit pages on the GPU: what the append stores (bit for bit), the dense
read-back, and attention over such pages against 64 bits."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _flag(ws):
    return B.pa_check_device_flag(ws)[1]


def _hard_rows(rng, n, dtype):
    """Rows of every magnitude, with exact ties between codes and scales,
    zeros, subnormals, infinities and values past the range."""
    x = rng.standard_normal((n, 128)).astype(np.float32)
    x *= np.exp2(rng.integers(-20, 14, (n, 8))).astype(np.float32).repeat(16, 1)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0], np.float32)
    for i in range(0, n, 3):  # x = a border * a scale, the group's largest 6 * scale
        s = ref.E4M3[rng.integers(1, 127, 8)].astype(np.float32).repeat(16)
        x[i] = rng.choice(mids, 128) * s * rng.choice([-1, 1], 128)
        x[i, ::16] = 6 * s[::16]
    for i in range(1, n, 7):  # the largest value on a border between two scales
        m = (ref.E4M3[1:] + ref.E4M3[:-1])[rng.integers(0, 125, 8)].astype(np.float32) / 2
        x[i] = rng.standard_normal(128).astype(np.float32) * 0.1 * m.repeat(16)
        x[i, ::16] = 6 * m
    x[2, :16], x[2, 16:32], x[2, 32] = 0, 1e-40, np.inf
    x[5, 40], x[5, 70], x[5, 90] = -3e38, -0.0, 2690
    return ref.bf16(x) if dtype == "bf16" else x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Bn,H,L,ps,ctx", [
    (1, 1, 1, 1, [1]), (3, 2, 5, 3, [5, 17, 40]), (2, 4, 129, 16, [129, 300]),
    (5, 1, 33, 128, [33, 64, 65, 200, 1000])])
def test_append_and_read_back(dtype, Bn, H, L, ps, ctx):
    import torch
    c = Case(Bn, 1, H, L, ps, ctx, spare=1)
    inp, d = ref.Inputs(c), None
    d = inp.device()
    rng = np.random.default_rng(Bn * 100 + L)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    new = [_hard_rows(rng, max(6, Bn * H * L), dtype)[:Bn * H * L].reshape(Bn, H, L, 128)
           for _ in range(2)]
    want = [t.copy() for t in inp.raw]
    for i, x in enumerate(new):
        codes, scales = ref.quantise(x)
        for b in range(Bn):
            for t in range(L):
                s = ctx[b] - L + t
                pg, slot = inp.table[b, s // ps], s % ps
                want[2 * i][pg, :, slot] = codes[b, :, t]
                want[2 * i + 1][pg, :, slot] = scales[b, :, t]
    kn, vn = (torch.from_numpy(x).to(dt).cuda() for x in new)
    ws = B.append_kv_q4(kn, vn, d["pool"], d["table"], d["ctx"])
    for got, w in zip(d["pool"], want):
        assert np.array_equal(got.cpu().numpy(), w)
    # the last L + 2 positions, and the first 40, dense
    for n, tail in ((L + 2, True), (40, False)):
        k, v = B.gather_kv_q4(d["pool"], d["table"], d["ctx"], n, tail=tail, dtype=dt, workspace=ws)
        for got, codes, scales in ((k, want[0], want[1]), (v, want[2], want[3])):
            dense = ref.dequantise(codes, scales)
            for b, S in enumerate(ctx):
                rows = ref.rows_of(dense, inp.table, b, S, ps)
                w = np.zeros((H, n, 128))
                if tail:
                    m = min(n, S)
                    w[:, n - m:] = rows[:, S - m:]
                else:
                    m = min(n, S)
                    w[:, :m] = rows[:, :m]
                assert np.array_equal(_np(got[b]), w)
    assert _flag(ws) == 0


def test_append_nan_poisons_its_group_only():
    import torch
    c = Case(1, 1, 1, 1, 16, [7])
    d = ref.Inputs(c).device()
    x = torch.ones(1, 1, 1, 128, device="cuda")
    x[..., 20] = float("nan")
    B.append_kv_q4(x, x, d["pool"], d["table"], d["ctx"])
    k, _ = B.gather_kv_q4(d["pool"], d["table"], d["ctx"], 1, tail=True, dtype=torch.float32)
    bad = torch.isnan(k[0, 0, 0]).cpu()
    assert bad[16:32].all() and bad.sum() == 16


def test_append_errors_are_recorded_and_skipped():
    import torch
    c = Case(3, 1, 2, 4, 16, [40, 20, 33])
    inp = ref.Inputs(c)
    d = inp.device()
    before = [t.clone() for t in d["pool"]]
    ctx = torch.tensor([3, 20, 1000], dtype=torch.int32, device="cuda")
    table = d["table"].clone()
    table[1, 1] = inp.P  # positions 16 .. 19 of sequence 1
    x = torch.ones(3, 2, 4, 128, device="cuda")
    ws = B.append_kv_q4(x, x, d["pool"], table, ctx)
    assert _flag(ws) == B.PA_FLAG_BAD_CONTEXT | B.PA_FLAG_BAD_PAGE
    assert all(torch.equal(a, b) for a, b in zip(before, d["pool"]))
    k, v = B.gather_kv_q4(d["pool"], table, ctx, 5)
    assert not k[0, :, 3:].any() and not k[2].any() and not v[2].any()


CASES = [
    Case(1, 1, 1, 1, 1, [1]),
    Case(2, 1, 2, 1, 16, [31, 32]),
    Case(3, 4, 2, 1, 128, [33, 257, 1000]),
    Case(2, 7, 1, 1, 12, [129, 700], spare=3),
    Case(2, 8, 2, 1, 64, [600, 65]),
    Case(2, 3, 2, 3, 3, [3, 250]),
    Case(2, 4, 1, 5, 24, [5, 511]),
    Case(1, 16, 1, 2, 16, [300]),
    Case(2, 4, 2, 17, 16, [17, 400]),
    Case(2, 2, 2, 65, 128, [65, 513]),
    Case(1, 4, 2, 200, 64, [333]),
    Case(3, 4, 2, 65, 16, [65, 129, 700], spare=9),
    Case(2, 5, 2, 70, 12, [71, 300]),
    Case(2, 4, 2, 1, 16, [2500, 7], causal=False),
    Case(2, 2, 2, 40, 8, [20, 300], causal=False),
    Case(1, 2, 1, 1, 16, [4000], spare=200),
]
CASES += [Case(**{**c.__dict__, "dtype": "f32"}) for c in CASES]
# many rows per kv head: whole and short last tiles, group sizes that do not
# divide a tile, contexts that cross every SM's share, many short sequences
CASES += [
    Case(1, 1, 1, 300, 16, [300]),
    Case(2, 7, 1, 130, 16, [130, 513]),
    Case(1, 48, 1, 3, 64, [260]),
    Case(1, 128, 1, 1, 16, [390]),
    Case(1, 100, 1, 5, 16, [129]),
    Case(1, 130, 1, 1, 16, [100]),
    Case(1, 4, 2, 16, 128, [3900], spare=4),
    Case(2, 4, 1, 97, 16, [2000, 97]),
    Case(1, 8, 1, 33, 8, [3000]),
    Case(40, 4, 2, 65, 16, [65 + 7 * i for i in range(40)]),
    Case(2, 4, 1, 66, 16, [66, 200]),
    Case(2, 4, 2, 129, 24, [100, 40], causal=False),
    Case(2, 3, 1, 43, 1, [43, 140]),
]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_attention(c):
    inp = ref.Inputs(c)
    d = inp.device()
    ws = B.new_q4_workspace(d["q"], d["pool"], d["table"])
    out = B.paged_attention_q4(d["q"], d["pool"], d["table"], d["ctx"], c.ps, inp.scale, c.causal,
                               workspace=ws)
    want, _, tol, _ = ref.attend(inp)
    assert _flag(ws) == 0
    assert ref.worst(_np(out), want, tol) <= 1
    assert out.dtype == d["q"].dtype
    again = B.paged_attention_q4(d["q"], d["pool"], d["table"], d["ctx"], c.ps, inp.scale,
                                 c.causal, workspace=ws)
    assert (again == out).all()


@pytest.mark.parametrize("mult", [2.0 ** -130, 2.0 ** -30, 2.0 ** 60])
def test_queries_far_from_one(mult):
    """Queries outside f16's range, with a scale that brings the scores back."""
    import torch
    c = Case(1, 4, 1, 1, 16, [200])
    inp = ref.Inputs(c)
    q = (inp.q * np.float32(mult)).astype(np.float32)
    inp.q = ref.bf16(q)
    inp.scale = float(np.float32(min(0.1 / mult, 1e30)))
    d = inp.device()
    out = B.paged_attention_q4(d["q"], d["pool"], d["table"], d["ctx"], c.ps, inp.scale)
    want, _, tol, _ = ref.attend(inp)
    assert ref.worst(_np(out), want, tol) <= 1
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 33])
def test_bad_sequences_and_pages(dtype, L):
    """A sequence whose length breaks the contract gets zero rows, a key
    behind a bad page reads as zeros; the others are as alone."""
    import torch
    c = Case(4, 2, 2, L, 16, [40, 100, 64, 50], dtype=dtype)
    inp = ref.Inputs(c)
    d = inp.device()
    ws = B.new_q4_workspace(d["q"], d["pool"], d["table"])
    for bad in (10 ** 6, inp.cap + 1, -3):
        ws.zero_()
        ctx = torch.tensor([0, 100, bad, 50], dtype=torch.int32, device="cuda")
        out = B.paged_attention_q4(d["q"], d["pool"], d["table"], ctx, c.ps, inp.scale,
                                   workspace=ws)
        want, _, tol, _ = ref.attend(inp, skip=(0, 2))
        assert _flag(ws) == B.PA_FLAG_BAD_CONTEXT
        assert ref.worst(_np(out), want, tol) <= 1
    ws.zero_()
    table = d["table"].clone()
    table[1, 0] = -1
    out = B.paged_attention_q4(d["q"], d["pool"], table, d["ctx"], c.ps, inp.scale, workspace=ws)
    assert _flag(ws) == B.PA_FLAG_BAD_PAGE
    for x in inp.dense:  # a page of zeros for the first 16 keys of sequence 1
        x[inp.table[1, 0]] = 0
    want, _, tol, _ = ref.attend(inp)
    assert ref.worst(_np(out), want, tol) <= 1


def test_table_of_unread_junk_and_shared_pages():
    """Two sequences on the same pages get the same rows as private copies."""
    c = Case(2, 4, 2, 1, 16, [100, 100])
    inp = ref.Inputs(c)
    inp.table[1, :7] = inp.table[0, :7]
    inp.q[1] = inp.q[0]
    d = inp.device()
    out = B.paged_attention_q4(d["q"], d["pool"], d["table"], d["ctx"], c.ps)
    assert (out[0] == out[1]).all()


def test_captured_and_on_another_stream():
    import torch
    c = Case(3, 4, 2, 1, 16, [300, 17, 900])
    inp = ref.Inputs(c)
    d = inp.device()
    ws = B.new_q4_workspace(d["q"], d["pool"], d["table"])
    out = torch.zeros_like(d["q"])
    w = torch.zeros_like(d["w"])

    def call(**kw):
        B.paged_attention_q4(d["q"], d["pool"], d["table"], d["ctx"], c.ps, inp.scale,
                             key_weights=d["w"], key_weights_out=w, out=out, workspace=ws, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    torch.cuda.synchronize()
    first, first_w = out.clone(), w.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]  # two graphs, one workspace
    for g in graphs:
        with torch.cuda.graph(g):
            call()
    for g in graphs + graphs:
        out.zero_()
        w.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(w, first_w)
    assert _flag(ws) == 0


def test_whole_flow():
    """Prompt appended in 4 bits and attended with key weights, the cache
    trimmed, then decode steps on the trimmed cache: every output against 64
    bits over what is stored."""
    import torch
    Bn, H, G, ps, keep, recent = 2, 2, 4, 16, 48, 9
    rng = np.random.default_rng(5)

    def normal(*shape):
        return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).bfloat16().cuda()
    pool = B.new_q4_pool(40, H, ps)
    lens = [70, 100]
    table = torch.arange(14, dtype=torch.int32, device="cuda").view(2, 7)
    ctx = torch.tensor([100, 100], dtype=torch.int32, device="cuda")
    ws = B.append_kv_q4(normal(Bn, H, 100, 128), normal(Bn, H, 100, 128), pool, table, ctx)
    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def check(q, out, table, ctx, w_out, w_in):
        inp = ref.Inputs(Case(Bn, G, H, q.shape[2], ps, ctx.tolist()))
        inp.table, inp.ctx, inp.q = table.cpu().numpy(), ctx.cpu().numpy(), q.float().cpu().numpy()
        raw = [t.cpu().numpy() for t in pool]
        inp.dense = [ref.dequantise(*raw[:2]), ref.dequantise(*raw[2:])]
        inp.w = np.zeros(tuple(w_out.shape))
        want, w, tol, w_tol = ref.attend(inp)
        assert ref.worst(_np(out), want, tol) <= 1
        w += _np(w_in) * (np.arange(w.shape[2]) < inp.ctx[:, None, None])
        assert ref.worst(_np(w_out), w, w_tol + 2.0 ** -23 * w) <= 1

    q = normal(Bn, H * G, 8, 128)
    w = torch.zeros(Bn, H, 112, device="cuda")
    out = B.paged_attention_q4(q, pool, table, ctx, ps, key_weights_out=w)
    check(q, out, table, ctx, w, torch.zeros_like(w))
    dst = torch.arange(20, 28, dtype=torch.int32, device="cuda").view(2, 4)
    new = B.evict_kv_q4(pool, table, ctx, w, keep, recent, dst, workspace=ws)
    assert new.context_lens.tolist() == [48, 48]
    kept, _ = ref.evict(w.cpu().numpy(), lens, keep, recent)
    assert np.array_equal(new.kept.cpu().numpy(), kept)
    table, ctx = dst, new.context_lens
    w = torch.zeros(Bn, H, 64, device="cuda")
    w[:, :, :keep] = new.key_weights
    for step in range(3):
        ctx = ctx + 1
        B.append_kv_q4(normal(Bn, H, 1, 128), normal(Bn, H, 1, 128), pool, table, ctx,
                       workspace=ws)
        q = normal(Bn, H * G, 1, 128)
        before = w.clone()
        out = B.paged_attention_q4(q, pool, table, ctx, ps, key_weights=w, key_weights_out=w)
        check(q, out, table, ctx, w, before)
    assert _flag(ws) == 0
