"""Draft trees on the GPU against their 64-bit forms: visibility, attention over
bf16, fp32 and 4-bit pages, compaction."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


# ---- visibility ------------------------------------------------------------------
@pytest.mark.parametrize("L", [1, 2, 31, 32, 33, 64, 100, 255, 1001, 1024])
def test_mask_and_depths(L):
    import torch
    rng = np.random.default_rng(L)
    parents = np.concatenate([tr.random_parents(rng, 3, L), tr.random_parents(rng, 2, L, 0.02),
                              np.arange(-1, L - 1, dtype=np.int32)[None],   # one chain
                              np.full((1, L), -1, np.int32),                # roots alone
                              np.full((1, L), -2, np.int32)])               # no draft
    if L > 40:
        parents[0, L // 3] = -2  # what follows it is no draft either
    see = tr.visible(parents)
    ws = B.new_cache_workspace()
    mask, depths = B.tree_mask(torch.from_numpy(parents).cuda(), workspace=ws)
    assert np.array_equal(mask.cpu().numpy(), tr.words(see))
    assert np.array_equal(depths.cpu().numpy(), see.sum(-1) - 1)
    assert B.pa_check_device_flag(ws)[1] == 0


def test_mask_of_parents_that_break_the_contract():
    import torch
    parents = np.array([[-1, 1, 0, 2, -5, 4, 99, -2, 7]], np.int32)
    ws = B.new_cache_workspace()
    mask, depths = B.tree_mask(torch.from_numpy(parents).cuda(), workspace=ws)
    assert mask[0, :, 0].tolist() == [1, 0, 5, 13, 0, 0, 0, 0, 0]
    assert depths[0].tolist() == [0, -1, 1, 2, -1, -1, -1, -1, -1]
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_TREE


# ---- attention -------------------------------------------------------------------
CASES = [
    tr.Case(1, 1, 1, 16, [1]),                                 # one key, itself
    tr.Case(4, 2, 1, 16, [1, 2, 300]),                         # single tokens
    tr.Case(4, 2, 8, 16, [8, 9, 300]),                         # no position before the drafts
    tr.Case(4, 2, 16, 128, [16, 127, 128, 129, 900]),
    tr.Case(3, 2, 13, 12, [13, 200, 900]),                     # odd sizes
    tr.Case(7, 1, 5, 1, [5, 130, 257]),                        # pages of one slot
    tr.Case(8, 1, 16, 64, [40, 700]),                          # 128 rows
    tr.Case(3, 1, 43, 24, [43, 500]),                          # 129 rows
    tr.Case(4, 2, 64, 8, [64, 65, 2000]),                      # 256 rows
    tr.Case(4, 1, 65, 16, [65, 300, 1111]),                    # 260 rows
    tr.Case(2, 2, 255, 64, [255, 256, 700]),                   # 510 rows, trees over several tiles
    tr.Case(1, 3, 300, 128, [300, 431, 1000]),                 # a tree wider than two tiles
    tr.Case(1, 1, 1024, 16, [1024, 1500]),
    tr.Case(1, 2, 129, 16, [129, 4000, 300], spare=40),        # wide tables, long contexts
    tr.Case(4, 8, 16, 16, [100 + 61 * i for i in range(20)]),  # many sequences
    tr.Case(2, 4, 3, 16, [20000]),
    tr.Case(32, 1, 9, 16, [77, 1000]),                         # a large group
    tr.Case(4, 2, 33, 16, [33, 150, 700], kind="any"),
    tr.Case(2, 1, 140, 64, [140, 141, 600], kind="any"),
]


def variants():
    for c in CASES:
        for pool, dtype in (("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"), ("q4", "f32")):
            yield tr.Case(**{**c.__dict__, "pool": pool, "dtype": dtype})


@pytest.mark.parametrize("c", list(variants()), ids=str)
def test_attention(c):
    inp = tr.Inputs(c)
    want, tol = tr.attend(inp)
    d = inp.device()
    ws = B.new_tree_workspace(d["q"], d["pool"] if c.pool == "q4" else d["pool"][0], d["table"])
    out = tr.call(inp, d, workspace=ws)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert ref.worst(got, want, tol) <= 1.0
    assert (got[~inp.drafted[:, None].repeat(c.G * c.H_kv, 1)] == 0).all()
    assert B.pa_check_device_flag(ws)[1] == 0
    again = tr.call(inp, d, workspace=ws)  # what the first call left in the workspace
    assert out.equal(again)


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"),
                                        ("q4", "f32")])
def test_sequences_that_break_the_contract(pool, dtype):
    c = tr.Case(4, 2, 8, 16, [200, 90, 333, 40], pool, dtype)
    inp = tr.Inputs(c)
    cap = inp.table.shape[1] * c.ps
    for bad_len in (7, -1, cap + 1):
        want, tol = tr.attend(inp, skip=(1,))
        d = inp.device()
        d["ctx"][1] = bad_len
        ws = B.new_tree_workspace(d["q"], d["pool"] if pool == "q4" else d["pool"][0], d["table"])
        got = tr.call(inp, d, workspace=ws).double().cpu().numpy()
        assert (got[1] == 0).all()
        assert ref.worst(got, want, tol) <= 1.0
        assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_CONTEXT


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"),
                                        ("q4", "f32")])
def test_keys_behind_bad_pages_read_as_zeros(pool, dtype):
    c = tr.Case(4, 2, 8, 16, [200, 90], pool, dtype)
    inp = tr.Inputs(c)
    d = inp.device()
    for t in inp.dense:  # the pages behind the entries that break
        t[inp.table[0, 3]] = 0
        t[inp.table[1, 0]] = 0
    want, tol = tr.attend(inp)
    d["table"][0, 3] = inp.P
    d["table"][1, 0] = -1
    ws = B.new_tree_workspace(d["q"], d["pool"] if pool == "q4" else d["pool"][0], d["table"])
    got = tr.call(inp, d, workspace=ws).double().cpu().numpy()
    assert ref.worst(got, want, tol) <= 1.0
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_PAGE


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"),
                                        ("q4", "f32")])
def test_nan_rows(pool, dtype):
    """A NaN in a query row or in a key that a row sees makes that row NaN, and
    no other; a draft's NaN key reaches its descendants alone."""
    c = tr.Case(2, 2, 40, 16, [40, 400, 1300], pool, dtype, seed=3)
    inp = tr.Inputs(c)
    d = inp.device()
    want, tol = tr.attend(inp)
    live = np.flatnonzero(inp.drafted[1])
    d["q"][0, 1, 0, 5] = float("nan")
    node = int(live[len(live) // 3])
    s = 400 - c.L + node
    page, slot = int(inp.table[1, s // c.ps]), s % c.ps
    if pool == "q4":
        d["pool"].key_scales[page, 0, slot, 2] = 0x7f
    else:
        d["pool"][0][page, 0, slot, 33] = float("nan")
    got = tr.call(inp, d).double().cpu().numpy()
    nan = np.zeros(got.shape[:3], bool)
    nan[0, 1, 0] = True
    nan[1, :c.G] = inp.see[1][:, node]  # kv head 0
    assert (np.isnan(got).all(-1) == nan).all()
    assert ref.worst(got[~nan], want[~nan], tol[~nan]) <= 1.0


def test_workspace_of_the_largest_call_serves_smaller_ones():
    import torch
    big = tr.Inputs(tr.Case(4, 2, 64, 16, [2000, 1999, 1000, 64]))
    d = big.device()
    ws = B.new_tree_workspace(d["q"], d["pool"][0], d["table"])
    ws[256:] = 0xff  # whatever was there
    for c in (big.c, tr.Case(4, 2, 1, 16, [1500]), tr.Case(4, 2, 8, 16, [30, 200]),
              tr.Case(4, 2, 33, 16, [1999])):
        inp = tr.Inputs(c)
        d = inp.device()
        want, tol = tr.attend(inp)
        got = tr.call(inp, d, workspace=ws).double().cpu().numpy()
        assert ref.worst(got, want, tol) <= 1.0
    torch.cuda.synchronize()
    assert B.pa_check_device_flag(ws)[1] == 0


def test_large_scores_and_scales():
    """Scores far apart: the softmax picks its key; scale 0: the plain mean."""
    for pool, dtype in (("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16")):
        inp = tr.Inputs(tr.Case(2, 1, 6, 16, [500], pool, dtype, seed=9))
        for scale in (0.0, 30.0):
            inp.scale = scale
            want, tol = tr.attend(inp)
            got = tr.call(inp, inp.device()).double().cpu().numpy()
            assert ref.worst(got, want, tol) <= 1.0


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"),
                                        ("q4", "f32")])
def test_light_keys(pool, dtype):
    """Where the heaviest key's values are 0 the output is the light keys', to the
    precision of their own weights."""
    inp = tr.Inputs(tr.Case(4, 2, 24, 16, [300, 24], pool, dtype, seed=2))
    inp.scale *= 8  # other keys weigh 2^-10 and less
    for b, S in enumerate(inp.ctx):
        K = ref.rows_of(inp.dense[0], inp.table, b, S, 16)
        for h in range(2):
            q = inp.q[b, 4 * h:4 * h + 4][:, inp.drafted[b]].astype(np.float64)
            see = inp.see[b][inp.drafted[b]]
            x = np.einsum("gld,sd->gls", q, np.nan_to_num(K[h]))
            hide = np.concatenate([np.zeros((len(see), S - 24), bool), ~see], 1)
            heavy = np.unique(np.where(hide, -np.inf, x).argmax(-1))
            page, slot = inp.table[b, heavy // 16], heavy % 16
            inp.raw[-1 if pool != "q4" else 2][page, h, slot] = 0
            inp.dense[1][page, h, slot] = 0
    want, tol = tr.attend(inp)
    got = tr.call(inp, inp.device()).double().cpu().numpy()
    assert ref.worst(got, want, tol) <= 1.0


# ---- compaction ------------------------------------------------------------------
def paths_of(rng, drafted, L):
    out = []
    for b in range(len(drafted)):
        n = [0, L, 1, L // 2][b % 4]
        out.append(np.sort(rng.choice(L, n, replace=False)).astype(np.int32))
    return out


@pytest.mark.parametrize("pool", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("L,ps,H", [(1, 16, 2), (5, 1, 3), (16, 128, 8), (63, 12, 2), (300, 16, 1),
                                    (1000, 64, 2)])
def test_compaction(pool, L, ps, H):
    import torch
    ctx = [L, L + 1, L + 37, 2 * L + 500, L + 129]
    inp = tr.Inputs(tr.Case(1, H, L, ps, ctx, pool, "f32" if pool == "f32" else "bf16", seed=L))
    rng = np.random.default_rng(L + ps)
    paths = paths_of(rng, inp.drafted, L)
    path = np.full((len(ctx), max(len(p) for p in paths) + 3), 12345, np.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = p
    d = inp.device()
    bufs = list(d["pool"])
    want = [t.cpu().clone() for t in bufs]
    for b, (S, p) in enumerate(zip(ctx, paths)):
        src, dst = S - L + p, S - L + np.arange(len(p))
        for t in want:
            rows = t[inp.table[b, src // ps], :, src % ps].clone()
            t[inp.table[b, dst // ps], :, dst % ps] = rows
    ws = B.new_cache_workspace()
    args = (d["table"], d["ctx"], torch.from_numpy(path).cuda(),
            torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"), L)
    lens = B.compact_kv_q4(d["pool"], *args, workspace=ws) if pool == "q4" else \
        B.compact_kv(*bufs, *args, workspace=ws)
    assert lens.tolist() == [S - L + len(p) for S, p in zip(ctx, paths)]
    assert B.pa_check_device_flag(ws)[1] == 0
    for got, w in zip(bufs, want):
        assert got.cpu().contiguous().view(torch.uint8).equal(w.contiguous().view(torch.uint8))


def test_compaction_of_bad_paths_moves_nothing():
    import torch
    L = 6
    inp = tr.Inputs(tr.Case(1, 2, L, 16, [50] * 7))
    d = inp.device()
    path = np.array([[0, 2, 1], [0, 6, 6], [-1, 0, 1], [1, 1, 2], [0, 1, 2], [0, 1, 2], [3, 4, 5]],
                    np.int32)
    lens = np.array([3, 2, 1, 2, 4, -1, 3], np.int32)
    before = [t.clone() for t in d["pool"]]
    ws = B.new_cache_workspace()
    got = B.compact_kv(*d["pool"], d["table"][:6], d["ctx"][:6], torch.from_numpy(path[:6]).cuda(),
                       torch.from_numpy(lens[:6]).cuda(), L, workspace=ws)
    assert got.tolist() == [44] * 6
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_TREE
    for a, t in zip(before, d["pool"]):
        assert a.view(torch.int16).equal(t.view(torch.int16))
    ctx = torch.tensor([5, 0, 17 * 16], dtype=torch.int32, device="cuda")  # too short, too long
    ws = B.new_cache_workspace()
    got = B.compact_kv(*d["pool"], d["table"][:3], ctx, torch.from_numpy(path[4:]).cuda(),
                       torch.from_numpy(lens[[0, 0, 0]]).cuda(), L, workspace=ws)
    assert got.tolist() == ctx.tolist()
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_CONTEXT
    for a, t in zip(before, d["pool"]):
        assert a.view(torch.int16).equal(t.view(torch.int16))
    d["table"][0, 3] = 1 << 20  # the page of positions 48 and 49: rows from and to it stay
    ws = B.new_cache_workspace()
    got = B.compact_kv(*d["pool"], d["table"][:1], d["ctx"][:1],
                       torch.from_numpy(path[6:]).cuda(), torch.from_numpy(lens[6:]).cuda(), L,
                       workspace=ws)
    assert got.tolist() == [47] and B.pa_check_device_flag(ws)[1] == B.PA_FLAG_BAD_PAGE
    want = before[0].clone()
    page = int(inp.table[0, 2])
    want[page, :, 12] = before[0][page, :, 15]  # draft 3, position 47; drafts 4 and 5 are behind it
    assert want.view(torch.int16).equal(d["pool"][0].view(torch.int16))
