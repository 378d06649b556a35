"""Plain 64-bit forms of draft trees (visibility, attention, compaction) and of
page sharing, and the seeded inputs of their tests, in numpy."""
from __future__ import annotations

import dataclasses
import math

import numpy as np

import cache_ref as ref
from paged_kv_cache_03_gb300 import binding as B


def visible(parents):
    """[B, L, L]: draft i sees draft n, by walking up from every draft."""
    Bn, L = parents.shape
    see = np.zeros((Bn, L, L), bool)
    for b in range(Bn):
        for i in range(L):
            p = int(parents[b, i])
            if p == -1:
                see[b, i, i] = True
            elif 0 <= p < i and see[b, p, p]:
                see[b, i] = see[b, p]
                see[b, i, i] = True
    return see


def words(see):
    """int32 words [B, L, W] of truth values [B, L, L]."""
    L = see.shape[-1]
    W = (L + 31) // 32
    x = np.zeros((*see.shape[:-1], 32 * W), np.uint64)
    x[..., :L] = see
    w = (x.reshape(*see.shape[:-1], W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def random_parents(rng, Bn, L, spread=1.0):
    """Trees with slots without a draft at the end of some."""
    parents = np.full((Bn, L), -2, np.int32)
    for b in range(Bn):
        n = L if b % 2 == 0 else int(rng.integers(max(1, L // 2), L + 1))
        for i in range(n):
            lo = max(0, int(i - 1 - spread * i))
            parents[b, i] = -1 if i == 0 or rng.random() < 0.05 else rng.integers(lo, i)
    return parents


@dataclasses.dataclass
class Case:
    G: int
    H_kv: int
    L: int
    ps: int
    ctx: list
    pool: str = "bf16"   # or "f32", "q4"
    dtype: str = "bf16"  # of the query
    seed: int = 0
    spare: int = 0       # table entries past the longest sequence's pages
    kind: str = "tree"   # or "any": any set of drafts, some rows empty

    def __str__(self):
        return (f"{self.pool}-{self.dtype}-G{self.G}H{self.H_kv}L{self.L}ps{self.ps}-"
                f"{self.kind}-{len(self.ctx)}x{max(self.ctx)}")


class Inputs:
    """Pools, table, query and visibility of a case.  Unused slots, unused
    pages and slots without a draft hold NaN, unused table entries junk."""

    def __init__(self, c: Case):
        rng = np.random.default_rng(c.seed + 11)
        self.c, Bn = c, len(c.ctx)
        npg = [-(-s // c.ps) for s in c.ctx]
        self.P = sum(npg) + 2
        perm = rng.permutation(self.P)
        self.table = np.full((Bn, max(npg) + c.spare), -7, np.int32)
        at = 0
        for b in range(Bn):
            self.table[b, :npg[b]] = perm[at:at + npg[b]]
            at += npg[b]
        self.ctx = np.array(c.ctx, np.int32)
        self.scale = float(np.float32(1 / math.sqrt(128)))
        if c.kind == "tree":
            self.see = visible(random_parents(rng, Bn, c.L, 0.5))
        else:
            self.see = rng.random((Bn, c.L, c.L)) < 0.4
            self.see[rng.random((Bn, c.L)) < 0.2] = False  # no drafts, though others' bits say so
        self.drafted = self.see.any(-1)
        self.mask = words(self.see)
        self.see &= self.drafted[:, None, :]
        used = np.zeros((self.P, c.ps), bool)
        for b, s in enumerate(c.ctx):
            i = np.concatenate([np.arange(s - c.L), s - c.L + np.flatnonzero(self.drafted[b])])
            used[self.table[b, i // c.ps], i % c.ps] = True
        q = rng.standard_normal((Bn, c.H_kv * c.G, c.L, 128)).astype(np.float32) * 1.5
        q[~self.drafted[:, None].repeat(c.H_kv * c.G, 1)] = np.nan
        self.q = ref.bf16(q) if c.dtype == "bf16" else q
        off = ~used[:, None].repeat(c.H_kv, 1)
        self.raw, self.dense = [], []  # raw: what goes to the device
        for mult in (1.5, 1.0):
            x = rng.standard_normal((self.P, c.H_kv, c.ps, 128)).astype(np.float32) * mult
            if c.pool == "q4":
                codes, scales = ref.quantise(x)
                scales[off] = 0x7f
                self.raw += [codes, scales]
                self.dense.append(ref.dequantise(codes, scales))
            else:
                x = ref.bf16(x) if c.pool == "bf16" else x
                x[off] = np.nan
                self.raw.append(x)
                self.dense.append(x.astype(np.float64))

    def device(self):
        import torch
        d = {}
        dt = torch.bfloat16 if self.c.dtype == "bf16" else torch.float32
        d["q"] = torch.from_numpy(self.q).to(dt).cuda()
        d["table"] = torch.from_numpy(self.table).cuda()
        d["ctx"] = torch.from_numpy(self.ctx).cuda()
        d["mask"] = torch.from_numpy(self.mask).cuda()
        if self.c.pool == "q4":
            d["pool"] = B.Q4Pool(*[torch.from_numpy(t).cuda() for t in self.raw])
        else:
            d["pool"] = [torch.from_numpy(t).to(dt).cuda() for t in self.raw]
        return d


def call(inp, d, **kw):
    """The attention through the framework."""
    args = (d["table"], d["ctx"], d["mask"], inp.c.ps, inp.scale)
    if inp.c.pool == "q4":
        return B.paged_attention_tree_q4(d["q"], d["pool"], *args, **kw)
    return B.paged_attention_tree(d["q"], *d["pool"], *args, **kw)


def attend(inp: Inputs, skip=()):
    """64-bit output and its tolerance; sequences in `skip` are zeros.  The
    tolerance counts roundings; p are probabilities:

    * the output's type: half a step, eps / 2 of the result;
    * scores: 128 products, exact (bf16, 4 bits) or rounded by 2^-24 (fp32), are
      added in fp32; a partial sum is at most T = scale * sum |q k|, and 128
      additions each off by at most 2^-23 T (the tensor cores cut) make 2^-16 T;
      with the scaling and the exponential's own 2^-21 at most 2^-15 T + 2^-20
      relative in every p (T of the row's largest score, both in p and the sum);
    * fp32 operands enter the products as two f16 parts, which hold all but 2^-22 of
      a value (and 2^-40 of the largest of its 8 rows): q and k 2^-21 T together,
      inside the 2^-16 T that the line above leaves; p and v 2^-21 relative, inside
      the S 2^-24 below, whose worst case no sum of rounded terms comes near;
    * p of bf16 queries is rounded to bf16 over bf16 pages: 2^-8; over 4-bit pages to
      f16: 2^-11; the sums add them unrounded.  Weights in f16, one part or two, are 2^7
      times p / (the row's largest p, or one up to 2^8 times smaller that the maximum so
      far stands for): from 2^-14 on they are rounded relatively (two parts: 2^-22, the
      low one being cut at 2^-25), below that to steps of 2^-24, so at most 2^-25 2^-7 of
      the row's largest p is lost of each;
    * sums of S terms in fp32: 2^-24 S at worst;
    * a p below 2^-126 of the row's largest is 0 in fp32 (the smallest normal
      number): at most 2^-126 of every value is lost (times the row's largest p).
    """
    c = inp.c
    out = np.zeros(inp.q.shape)
    tol = np.full(inp.q.shape, 1e-300)
    eps = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -24
    pop = 0.0 if c.dtype == "f32" else 2.0 ** -11 if c.pool == "q4" else 2.0 ** -8
    lost = 2.0 ** -126 if c.pool == c.dtype == "bf16" else 2.0 ** -32
    for b, S in enumerate(inp.ctx):
        if b in skip:
            continue
        there = inp.drafted[b]
        if not there.any():
            continue
        show = np.concatenate([np.ones((c.L, S - c.L), bool), inp.see[b]], 1)[there]
        keys = np.concatenate([np.ones(S - c.L, bool), there])  # the others are NaN
        show = show[:, keys]
        K = ref.rows_of(inp.dense[0], inp.table, b, S, c.ps)[:, keys]
        V = ref.rows_of(inp.dense[1], inp.table, b, S, c.ps)[:, keys]
        for h in range(c.G * c.H_kv):
            k, v, q = K[h // c.G], V[h // c.G], inp.q[b, h][there].astype(np.float64)
            x = q @ k.T * inp.scale
            T = (np.abs(q) @ np.abs(k).T * inp.scale).max(-1, keepdims=True)
            x[~show] = -np.inf
            top = x.max(-1, keepdims=True)
            p = np.exp(x - np.where(np.isinf(top), 0, top))
            p /= np.maximum(p.sum(-1, keepdims=True), 1e-300)  # (an empty row: zeros)
            rel = T * 2.0 ** -15 + 2.0 ** -20 + S * 2.0 ** -24
            o = p @ v
            out[b, h, there] = o
            tol[b, h, there] = (rel + pop) * (p @ np.abs(v)) + eps * np.abs(o) + \
                lost * p.max(-1, keepdims=True) * np.abs(v).sum(0)
    return out, tol


# ---- pages ---------------------------------------------------------------------
class Pages:
    """Table, lengths and page counts, one event after the other."""

    def __init__(self, rows, width, P, ps):
        self.ps, self.P = ps, P
        self.table = np.full((rows, width), -1, np.int32)
        self.ctx = np.zeros(rows, np.int32)
        self.refs = np.zeros(P, np.int32)

    def n(self, length):
        return -(-int(length) // self.ps)

    def fork(self, sources, targets, lens=None):
        before = self.ctx.copy()
        for i, (s, t) in enumerate(zip(sources, targets)):
            S = int(before[s]) if lens is None else int(lens[i])
            if s in targets or t in targets[:i] or before[t] != 0 or not 0 <= S <= before[s]:
                continue
            self.table[t] = -1
            self.table[t, :self.n(S)] = self.table[s, :self.n(S)]
            for e in self.table[t, :self.n(S)]:
                self.refs[e] += 1
            self.ctx[t] = S

    def resize(self, new):
        rows, ps = range(len(self.ctx)), self.ps
        cap = self.table.shape[1] * ps
        copies = np.full((len(self.ctx), 3), (-1, -1, 0), np.int32)
        for b in rows:
            if 0 <= new[b] < self.ctx[b]:
                for e in range(self.n(new[b]), self.n(self.ctx[b])):
                    self.refs[self.table[b, e]] -= 1
                    self.table[b, e] = -1
                self.ctx[b] = new[b]
        grow = [b for b in rows if self.ctx[b] < new[b] <= cap]
        last = {b: int(self.table[b, self.ctx[b] // ps]) for b in grow if self.ctx[b] % ps}
        free, full, short = list(np.flatnonzero(self.refs == 0)), self.refs.copy(), False
        for b in grow:
            S, N = int(self.ctx[b]), int(new[b])
            same = [x for x in last if last[x] == last.get(b)]
            held = b in last and full[last[b]] > 1
            keep = held and len(same) == full[last[b]] and same[-1] == b
            copy = held and not keep
            take = self.n(N) - self.n(S) + copy
            short |= take > len(free)
            if short and (take > 0 or keep):
                continue
            if copy:
                copies[b] = last[b], free[0], S % ps
                self.refs[last[b]] -= 1
            at = S // ps if copy else self.n(S)
            for e in range(take):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[b, at + e] = p
            self.ctx[b] = N
        return copies, short

    def consistent(self):
        held = np.zeros(self.P, np.int64)
        for b, S in enumerate(self.ctx):
            for e in self.table[b, :self.n(S)]:
                held[e] += 1
        return (held == self.refs).all()
