"""Draft trees and page sharing as a server runs them: captured steps, other
streams, shared workspaces, pools past 32-bit offsets."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def capture(fn):
    import torch
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


@pytest.mark.parametrize("pool,dtype", [("bf16", "bf16"), ("f32", "f32"), ("q4", "bf16"),
                                        ("q4", "f32")])
def test_two_captured_calls_share_a_workspace(pool, dtype):
    """One of a few long sequences (cut and merged), one of many short ones; both
    are replayed in turn with the lengths and trees of the moment."""
    import torch
    runs = []
    for c, other in ((tr.Case(4, 2, 64, 16, [3000, 900, 64, 1500], pool, dtype), [700, 3000, 99, 64]),
                     (tr.Case(4, 2, 8, 16, [100 + 30 * i for i in range(8)], pool, dtype),
                      [310 - 30 * i for i in range(8)])):
        a = tr.Inputs(c)
        b = tr.Inputs(tr.Case(**{**c.__dict__, "ctx": other, "seed": 5}))
        runs.append((a, b))
    P = max(i.P for r in runs for i in r)
    width = max(i.table.shape[1] for r in runs for i in r)

    def padded(inp):
        """Its tensors with P pages and tables of the common width."""
        d = inp.device()
        d["table"] = torch.nn.functional.pad(d["table"], (0, width - inp.table.shape[1]), value=-7)
        bufs = [torch.cat([t, t.new_zeros((P - t.shape[0], *t.shape[1:]))]) for t in d["pool"]]
        d["pool"] = B.Q4Pool(*bufs) if pool == "q4" else bufs
        return d
    sets = [[padded(i) for i in r] for r in runs]
    big = max((s[0] for s in sets),
              key=lambda d: B.new_tree_workspace(d["q"], d["pool"] if pool == "q4" else d["pool"][0],
                                                 d["table"]).numel())
    ws = B.new_tree_workspace(big["q"], big["pool"] if pool == "q4" else big["pool"][0],
                              big["table"])
    graphs, outs = [], []
    for r, s in zip(runs, sets):
        out = torch.empty_like(s[0]["q"])
        tr.call(r[0], s[0], out=out, workspace=ws)  # kernels are set up outside the capture
        torch.cuda.synchronize()
        graphs.append(capture(lambda: tr.call(r[0], s[0], out=out, workspace=ws)))
        outs.append(out)
    for turn in range(4):
        for r, s, g, out in zip(runs, sets, graphs, outs):
            inp = r[turn % 2]
            if turn < 2:
                want, tol = tr.attend(inp)
                r[turn].want = want, tol
            src = padded(inp)
            for k in ("q", "table", "ctx", "mask"):
                s[0][k].copy_(src[k])
            for x, y in zip(s[0]["pool"], src["pool"]):
                x.copy_(y)
            out.fill_(7)
            g.replay()
            want, tol = inp.want
            assert ref.worst(out.double().cpu().numpy(), want, tol) <= 1.0
    assert B.pa_check_device_flag(ws)[1] == 0


def test_a_captured_step():
    """Grow, copy, append, mask, attend, keep a path, shrink: one graph, replayed
    step after step, does what the calls do one by one."""
    import torch
    rng = np.random.default_rng(8)
    rows, H, G, L, ps, width, P = 5, 2, 4, 20, 16, 20, 160
    i32 = dict(dtype=torch.int32, device="cuda")

    def state():
        s = dict(table=torch.full((rows, width), -1, **i32), ctx=torch.zeros(rows, **i32),
                 refs=torch.zeros(P, **i32),
                 k=torch.zeros(P, H, ps, 128, dtype=torch.bfloat16, device="cuda"))
        s["v"] = s["k"].clone()
        s["ws"] = B.new_pages_workspace(s["table"], s["refs"])
        B.resize_pages(s["table"], s["ctx"], s["refs"], torch.tensor([37, 5, 80, 0, 0], **i32), ps,
                       workspace=s["ws"])
        B.fork_pages(s["table"], s["ctx"], s["refs"], torch.tensor([0, 2], **i32),
                     torch.tensor([3, 4], **i32), ps, workspace=s["ws"])
        return s
    x = {n: torch.zeros(rows, h, L, 128, dtype=torch.bfloat16, device="cuda")
         for n, h in (("q", H * G), ("k", H), ("v", H))}
    parents, path = torch.zeros(rows, L, **i32), torch.zeros(rows, L, **i32)
    path_lens = torch.zeros(rows, **i32)

    def step(s):
        copies = B.resize_pages(s["table"], s["ctx"], s["refs"], s["ctx"] + L, ps, workspace=s["ws"])
        B.copy_pages(s["k"], s["v"], copies, workspace=s["cache_ws"])
        B.append_kv(x["k"], x["v"], s["k"], s["v"], s["table"], s["ctx"])
        mask, _ = B.tree_mask(parents, workspace=s["cache_ws"])
        out = B.paged_attention_tree(x["q"], s["k"], s["v"], s["table"], s["ctx"], mask, ps,
                                     workspace=s["tree_ws"])
        lens = B.compact_kv(s["k"], s["v"], s["table"], s["ctx"], path, path_lens, L,
                            workspace=s["cache_ws"])
        B.resize_pages(s["table"], s["ctx"], s["refs"], lens, ps, workspace=s["ws"])
        return out
    one, two = state(), state()
    for s in (one, two):
        s["cache_ws"] = B.new_cache_workspace()
        s["tree_ws"] = B.new_tree_workspace(x["q"], s["k"], s["table"])
    parents.fill_(-1)
    step(one)
    step(two)
    torch.cuda.synchronize()
    got = [None]

    def captured():
        got[0] = step(two)
    g = capture(captured)
    for _ in range(6):
        p = tr.random_parents(rng, rows, L)
        parents.copy_(torch.from_numpy(p))
        for n in x.values():
            n.copy_(torch.randn(n.shape, device="cuda"))
        keep = rng.integers(0, 4, rows)
        rowsof = np.full((rows, L), -1, np.int32)
        for b in range(rows):
            rowsof[b, :keep[b]] = np.sort(rng.choice(L // 2, keep[b], replace=False))
        path.copy_(torch.from_numpy(rowsof))
        path_lens.copy_(torch.from_numpy(keep.astype(np.int32)))
        want = step(one)
        g.replay()
        assert want.equal(got[0])
        for k in ("table", "ctx", "refs", "k", "v"):
            assert one[k].equal(two[k])
    for s in (one, two):
        for w in ("ws", "cache_ws", "tree_ws"):
            assert B.pa_check_device_flag(s[w])[1] == 0


def test_calls_follow_the_current_stream():
    """Inputs become ready late on a stream of their own."""
    import torch
    inp = tr.Inputs(tr.Case(4, 2, 40, 16, [700, 1500, 40]))
    want, tol = tr.attend(inp)
    d = inp.device()
    late = {k: d[k].clone() for k in ("q", "ctx", "mask")}
    parents = torch.full((3, 40), -2, dtype=torch.int32, device="cuda")
    chain = torch.arange(-1, 39, dtype=torch.int32, device="cuda").expand(3, 40).contiguous()
    for k in late:
        d[k].zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        for k, t in late.items():
            d[k].copy_(t)
        parents.copy_(chain)
        out = tr.call(inp, d)
        mask, depths = B.tree_mask(parents)
    s.synchronize()
    assert ref.worst(out.double().cpu().numpy(), want, tol) <= 1.0
    assert depths[1].tolist() == list(range(40))


@pytest.mark.parametrize("pool", ["bf16", "f32", "q4"])
def test_pages_past_32_bit_offsets(pool):
    import torch
    inp = tr.Inputs(tr.Case(2, 2, 12, 16, [300, 77], pool, "f32" if pool == "f32" else "bf16"))
    d = inp.device()
    size = next(iter(d["pool"])).itemsize
    row = 64 if pool == "q4" else 128  # of the widest buffer, in elements
    P = 2 ** 32 // (2 * 16 * row) + 2 * inp.P
    if torch.cuda.mem_get_info()[0] < 2 * P * 32 * row * size + (4 << 30):
        pytest.skip("not enough free memory")
    base = P - inp.P
    bufs = []
    for t in d["pool"]:
        far = torch.empty((P, *t.shape[1:]), dtype=t.dtype, device="cuda")
        far[base:] = t
        bufs.append(far)
    d["pool"] = B.Q4Pool(*bufs) if pool == "q4" else bufs
    used = torch.arange(d["table"].shape[1], device="cuda") * 16 < d["ctx"][:, None]
    d["table"] = torch.where(used, d["table"] + base, d["table"]).int()
    want, tol = tr.attend(inp)
    assert ref.worst(tr.call(inp, d).double().cpu().numpy(), want, tol) <= 1.0
    # the last page copied to the first, a draft moved ahead
    copies = torch.tensor([[P - 1, 0, 16]], dtype=torch.int32, device="cuda")
    B.copy_pages_q4(d["pool"], copies) if pool == "q4" else B.copy_pages(*bufs, copies)
    args = (d["table"], d["ctx"], torch.tensor([[3], [11]], dtype=torch.int32, device="cuda"),
            torch.ones(2, dtype=torch.int32, device="cuda"), 12)
    before = [t[base:].clone() for t in bufs]
    lens = B.compact_kv_q4(d["pool"], *args) if pool == "q4" else B.compact_kv(*bufs, *args)
    assert lens.tolist() == [289, 66]
    for t, b in zip(bufs, before):
        assert t[0].view(torch.uint8).equal(t[P - 1].view(torch.uint8))
        for seq, (S, i) in enumerate(((300, 3), (77, 11))):
            src, dst = S - 12 + i, S - 12
            b[int(inp.table[seq, dst // 16]), :, dst % 16] = \
                b[int(inp.table[seq, src // 16]), :, src % 16]
        assert t[base:].view(torch.uint8).equal(b.view(torch.uint8))


def test_calls_at_once():
    """Two streams and two host threads, a workspace each: neither disturbs the other."""
    import threading
    import torch
    jobs = []
    for c in (tr.Case(4, 2, 64, 16, [1500, 700, 64]), tr.Case(4, 2, 24, 16, [900, 400], "q4"),
              tr.Case(2, 2, 12, 16, [800, 31], "f32", "f32")):
        inp = tr.Inputs(c)
        d = inp.device()
        ws = B.new_tree_workspace(d["q"], d["pool"] if c.pool == "q4" else d["pool"][0], d["table"])
        jobs.append((inp, d, ws, torch.cuda.Stream(), []))
    torch.cuda.synchronize()

    def work(inp, d, ws, stream, outs):
        with torch.cuda.stream(stream):
            for _ in range(20):
                outs.append(tr.call(inp, d, workspace=ws))
    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for inp, d, ws, _, outs in jobs:
        want, tol = tr.attend(inp)
        assert len(outs) == 20 and all(o.equal(outs[0]) for o in outs)
        assert ref.worst(outs[0].double().cpu().numpy(), want, tol) <= 1.0
        assert B.pa_check_device_flag(ws)[1] == 0


def test_captured_first_calls():
    """A call may be captured before any other of its kind was made (in a process of its own)."""
    import os
    import subprocess
    import sys
    program = """
import torch, tree_ref as tr, cache_ref as ref
from paged_kv_cache_03_gb300 import binding as B
for pool, dtype in (("bf16", "bf16"), ("q4", "bf16"), ("f32", "f32"), ("q4", "f32")):
    for L in (8, 64):
        inp = tr.Inputs(tr.Case(4, 1, L, 16, [2000, 64], pool, dtype))
        d = inp.device()
        ws = B.new_tree_workspace(d["q"], d["pool"] if pool == "q4" else d["pool"][0], d["table"])
        out = torch.empty_like(d["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            tr.call(inp, d, out=out, workspace=ws)
        g.replay()
        want, tol = tr.attend(inp)
        assert ref.worst(out.double().cpu().numpy(), want, tol) <= 1.0
parents = torch.tensor([[-1, 0, 0]], dtype=torch.int32, device="cuda")
ws = B.new_cache_workspace()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    mask, depths = B.tree_mask(parents, workspace=ws)
g.replay()
assert mask[0, :, 0].tolist() == [1, 3, 5] and depths[0].tolist() == [0, 1, 1]
"""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([here, os.path.dirname(here)]))
    r = subprocess.run([sys.executable, "-c", program], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
