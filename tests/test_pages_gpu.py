"""Pages shared between sequences on the GPU: forks, growth, release and copies
against a simulation, and a speculative decoding loop over all of it."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


class Device:
    """A simulation and the same state on the GPU."""

    def __init__(self, rows, width, P, ps):
        import torch
        self.sim = tr.Pages(rows, width, P, ps)
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.ctx = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(P, dtype=torch.int32, device="cuda")
        self.ws = B.new_pages_workspace(self.table, self.refs)

    def dev(self, x):
        import torch
        return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")

    def fork(self, sources, targets, lens=None):
        self.sim.fork(list(sources), list(targets), lens)
        B.fork_pages(self.table, self.ctx, self.refs, self.dev(sources), self.dev(targets),
                     self.sim.ps, None if lens is None else self.dev(lens), workspace=self.ws)

    def resize(self, new):
        want, short = self.sim.resize(new)
        copies = B.resize_pages(self.table, self.ctx, self.refs, self.dev(new), self.sim.ps,
                                workspace=self.ws)
        assert np.array_equal(copies.cpu().numpy(), want)
        return copies, short

    def check(self, flag=0):
        assert np.array_equal(self.table.cpu().numpy(), self.sim.table)
        assert np.array_equal(self.ctx.cpu().numpy(), self.sim.ctx)
        assert np.array_equal(self.refs.cpu().numpy(), self.sim.refs)
        assert self.sim.consistent()
        assert B.pa_check_device_flag(self.ws, clear=True)[1] == flag


@pytest.mark.parametrize("rows,width,P,ps", [(1, 1, 1, 16), (6, 5, 40, 4), (40, 9, 200, 16),
                                             (1500, 3, 9000, 8), (5, 2500, 20000, 1),
                                             (64, 40, 70000, 128)])
def test_random_events(rows, width, P, ps):
    rng = np.random.default_rng(rows + width)
    d = Device(rows, width, P, ps)
    cap = width * ps
    for step in range(12):
        new = rng.integers(0, cap + 1, rows)
        new[rng.random(rows) < 0.3] = -1
        new[rng.random(rows) < 0.2] = 0
        near = rng.random(rows) < 0.3
        new[near] = np.minimum(d.sim.ctx[near] + rng.integers(1, ps + 2, near.sum()), cap)
        _, short = d.resize(new)
        d.check(B.PA_FLAG_NO_PAGES if short else 0)
        empty, full = np.flatnonzero(d.sim.ctx == 0), np.flatnonzero(d.sim.ctx)
        if len(empty) and len(full):
            t = rng.permutation(empty)[:max(1, len(empty) // 2)]
            s = rng.choice(full[:max(1, len(full) // 3)], len(t))  # several of one source
            lens = None if step % 2 else rng.integers(0, d.sim.ctx[s] + 1)
            d.fork(s, t, lens)
            d.check()


def test_the_last_holder_that_grows_keeps_the_page():
    d = Device(5, 4, 12, 8)
    d.resize([13, 0, 0, 0, 0])
    d.fork([0, 0, 0], [1, 3, 4], [13, 11, 13])
    d.check()
    c, _ = d.resize([15, 14, -1, 12, 14])  # all four holders: three copies
    assert c[:, 2].tolist() == [5, 5, 0, 3, 0] and int(d.table[4, 1]) == 1
    d.check()
    d.resize([8, 8, -1, 9, 9])
    d.fork([4], [2])
    c, _ = d.resize([9, 9, 10, 9, 9])  # row 4 holds it and does not grow: a copy
    assert c[:, 2].tolist() == [0, 0, 1, 0, 0]
    d.check()


def test_too_few_pages():
    d = Device(4, 8, 6, 4)
    _, short = d.resize([8, 9, 12, 4])  # 2 + 3 pages, then none for 3 and (after it) none for 1
    assert short and d.ctx.tolist() == [8, 9, 0, 0]
    d.check(B.PA_FLAG_NO_PAGES)
    _, short = d.resize([4, 12, 8, 0])  # one given up in the same call
    assert not short
    d.check()
    d.resize([4, 11, 8, 0])
    d.fork([1], [3], [10])
    # row 1 finds no page for its copy: row 3, which would keep the shared one, stays too
    _, short = d.resize([16, 12, -1, 11])
    assert short and d.ctx.tolist() == [4, 11, 8, 10]
    d.check(B.PA_FLAG_NO_PAGES)


def test_forks_that_break_the_contract():
    d = Device(6, 4, 12, 8)
    d.resize([20, 9, 0, 0, 0, 3])
    state = [t.clone() for t in (d.table, d.ctx, d.refs)]
    # not empty; itself; out of range; a target that another fork has as its source; a length
    for s, t, n in (([0], [1], None), ([2], [2], None), ([6], [2], None), ([0], [-1], None),
                    ([0, 2], [2, 3], None), ([0], [2], [21]), ([0], [2], [-1])):
        B.fork_pages(d.table, d.ctx, d.refs, d.dev(s), d.dev(t), 8,
                     None if n is None else d.dev(n), workspace=d.ws)
        assert B.pa_check_device_flag(d.ws, clear=True)[1] == B.PA_FLAG_BAD_CONTEXT
        if len(s) == 1:
            assert all(a.equal(b) for a, b in zip(state, (d.table, d.ctx, d.refs)))
        else:  # the fork of 2 is refused, and so is the one whose target it reads
            assert d.ctx.tolist() == [20, 9, 20, 0, 0, 3]
            d.ctx[2] = 0
            d.table[2] = -1
            d.refs.copy_(state[2])
    d.fork([0, 1], [3, 3])  # a target twice: the first has it
    d.check(B.PA_FLAG_BAD_CONTEXT)
    assert d.ctx.tolist() == [20, 9, 0, 20, 0, 3]


def test_lengths_and_pages_that_break_the_contract():
    d = Device(3, 2, 12, 8)
    d.resize([9, 9, 9])
    d.check()
    d.resize([17, 10, -5])  # above the capacity; left alone
    d.check(B.PA_FLAG_BAD_CONTEXT)
    d.table[0, 1] = 12      # freed: the entry out of range is not given back
    d.refs[int(d.table[1, 0])] = 0  # held by nobody
    B.resize_pages(d.table, d.ctx, d.refs, d.dev([0, 0, 16]), 8, workspace=d.ws)
    assert B.pa_check_device_flag(d.ws)[1] == B.PA_FLAG_BAD_PAGE
    assert (d.refs >= 0).all() and d.ctx.tolist() == [0, 0, 16]
    assert (d.table[:2] == -1).all()


@pytest.mark.parametrize("pool", ["bf16", "f32", "q4"])
@pytest.mark.parametrize("ps,H", [(1, 1), (3, 2), (12, 3), (16, 8), (128, 2)])
def test_copies(pool, ps, H):
    import torch
    P = 20
    g = torch.Generator(device="cuda").manual_seed(ps)

    def bytes_(*shape):
        return torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    if pool == "q4":
        bufs = [bytes_(P, H, ps, n) for n in (64, 8, 64, 8)]
        p = B.Q4Pool(*bufs)
    else:
        dt = torch.bfloat16 if pool == "bf16" else torch.float32
        bufs = [bytes_(P, H, ps, 128 * dt.itemsize).view(dt) for _ in range(2)]
    copies = [(0, 5, ps), (0, 6, max(1, ps // 2)), (-1, -1, 0), (7, 8, 0), (9, 9, ps),
              (1, 19, ps), (20, 3, 1), (2, 20, 1), (2, -3, 1), (2, 4, ps + 1), (2, 4, -1)]
    want = [t.clone() for t in bufs]
    for t in want:
        for a, b, n in ((0, 5, ps), (0, 6, max(1, ps // 2)), (1, 19, ps)):
            t[b, :, :n] = t[a, :, :n]
    ws = B.new_cache_workspace()
    c = torch.tensor(copies, dtype=torch.int32, device="cuda")
    for part, flag in ((c[:6], 0), (c, B.PA_FLAG_BAD_PAGE), (c[:0], 0)):
        B.copy_pages_q4(p, part, workspace=ws) if pool == "q4" else \
            B.copy_pages(*bufs, part, workspace=ws)
        assert B.pa_check_device_flag(ws, clear=True)[1] == flag
        for a, b in zip(bufs, want):
            assert a.view(torch.uint8).equal(b.view(torch.uint8))


@pytest.mark.parametrize("pool", ["bf16", "q4"])
def test_speculative_steps_with_forks(pool):
    """Sequences decode with drafted trees: grow, append, attend, keep a path,
    shrink; one is forked on the way.  What the cache holds in the end is what
    the kept tokens appended one after the other would have left, and every
    attention is that of its drafts over it."""
    import torch
    rng = np.random.default_rng(4)
    H, G, L, ps, rows, width, P = 2, 4, 12, 16, 4, 12, 40
    d = Device(rows, width, P, ps)
    dt = torch.bfloat16
    kv = B.new_q4_pool(P, H, ps) if pool == "q4" else \
        [torch.zeros(P, H, ps, 128, dtype=dt, device="cuda") for _ in range(2)]
    append = (lambda k, v, t, c: B.append_kv_q4(k, v, kv, t, c)) if pool == "q4" else \
        (lambda k, v, t, c: B.append_kv(k, v, *kv, t, c))
    copy = (lambda c: B.copy_pages_q4(kv, c)) if pool == "q4" else (lambda c: B.copy_pages(*kv, c))

    def new(*shape):
        return ref.bf16(rng.standard_normal(shape).astype(np.float32))

    def cuda(x):
        return torch.from_numpy(x).to(dt).cuda()
    held = {b: [np.zeros((H, 0, 128))] * 2 for b in range(rows)}  # what every row should hold

    def stored(x):
        return ref.dequantise(*ref.quantise(x)) if pool == "q4" else x
    # prompts in rows 0 and 1
    copies, _ = d.resize([21, 40, 0, 0])
    for b, n in ((0, 21), (1, 40)):
        x = [new(1, H, n, 128) for _ in range(2)]
        append(cuda(x[0]), cuda(x[1]), d.table[b:b + 1], d.ctx[b:b + 1])
        held[b] = [stored(t[0]) for t in x]
    live = [0, 1]
    for step in range(5):
        if step == 1:
            d.fork([0, 1], [2, 3], [d.sim.ctx[0], 25])
            held[2], held[3] = held[0], [t[:, :25] for t in held[1]]
            live = [0, 1, 2, 3]
        n = len(live)
        want = d.sim.ctx.copy()
        want[live] += L
        copies, short = d.resize(want)
        assert not short
        copy(copies)
        parents = tr.random_parents(rng, n, L)
        see = tr.visible(parents)
        mask, depths = B.tree_mask(torch.from_numpy(parents).cuda())
        x = [new(n, H, L, 128) for _ in range(2)]
        q = new(n, H * G, L, 128)
        table, ctx = d.table[:n], d.ctx[:n]
        append(cuda(x[0]), cuda(x[1]), table, ctx)
        out = B.paged_attention_tree_q4(cuda(q), kv, table, ctx, mask, ps) if pool == "q4" else \
            B.paged_attention_tree(cuda(q), *kv, table, ctx, mask, ps)
        out = out.double().cpu().numpy()
        paths = []
        for b in live:
            there = see[b].any(-1)
            K, V = (np.concatenate([h, stored(t[b])], 1) for h, t in zip(held[b], x))
            show = np.concatenate([np.ones((L, K.shape[1] - L), bool), see[b]], 1)
            for h in range(H * G):
                s = q[b, h].astype(np.float64) @ K[h // G].T / np.sqrt(128)
                s[~show] = -np.inf
                p = np.exp(s[there] - s[there].max(-1, keepdims=True))
                o = p @ V[h // G] / p.sum(-1, keepdims=True)
                # p and the output in bf16, scores as in tree_ref
                tol = 4 * 2.0 ** -8 * (p @ np.abs(V[h // G]) / p.sum(-1, keepdims=True))
                assert (np.abs(out[b, h][there] - o) <= tol).all()
                assert (out[b, h][~there] == 0).all()
            node, path = int(rng.choice(np.flatnonzero(there))), []
            while node >= 0:
                path.insert(0, node)
                node = int(parents[b, node])
            paths.append(path)
            held[b] = [np.concatenate([h, stored(t[b])[:, path]], 1) for h, t in zip(held[b], x)]
        path = np.full((n, L), -1, np.int32)
        for b, p in enumerate(paths):
            path[b, :len(p)] = p
        args = (table, ctx, torch.from_numpy(path).cuda(), d.dev([len(p) for p in paths]), L)
        lens = B.compact_kv_q4(kv, *args) if pool == "q4" else B.compact_kv(*kv, *args)
        assert lens.tolist() == [held[b][0].shape[1] for b in live]
        want = np.full(rows, -1)
        want[live] = lens.cpu().numpy()
        d.resize(want)
        d.check()
        for b in live:
            S = held[b][0].shape[1]
            if pool == "q4":
                got = B.gather_kv_q4(kv, d.table[b:b + 1], d.ctx[b:b + 1], S, dtype=torch.float32)
            else:
                at = torch.arange(S, device="cuda")
                got = [t[d.table[b].long()[at // ps], :, at % ps].transpose(0, 1)[None] for t in kv]
            for g, h in zip(got, held[b]):
                assert np.array_equal(g[0].double().cpu().numpy(), h)
    d.resize([0] * rows)
    assert (d.refs == 0).all() and (d.table == -1).all()
    d.check()
