"""Plain 64-bit forms of the cache operators (4-bit rows, key weights,
eviction) and the seeded inputs of their tests, in numpy."""
from __future__ import annotations

import dataclasses
import math

import numpy as np

from paged_kv_cache_03_gb300 import binding as B
from paged_kv_cache_03_gb300 import synth

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_values():
    """The finite non-negative e4m3 values; the index is the byte."""
    v = [m * 2.0 ** -9 for m in range(8)]
    for e in range(1, 16):
        v += [(8 + m) * 2.0 ** (e - 10) for m in range(8)]
    return np.array(v[:127])


E4M3 = e4m3_values()


def nearest(x, values):
    """Index of the nearest of ascending values, ties to the even index."""
    mid = (values[1:] + values[:-1]) / 2
    lo, hi = np.searchsorted(mid, x, "left"), np.searchsorted(mid, x, "right")
    return np.where(lo % 2 == 0, lo, hi)


def quantise(x):
    """(codes [..., 64], scales [..., 8]) of rows [..., 128] (no NaN)."""
    g = np.asarray(x, np.float64).reshape(*x.shape[:-1], 8, 16)
    s = np.clip(nearest(np.abs(g).max(-1) / 6, E4M3), 1, 126)
    mag = nearest(np.minimum(np.abs(g) / E4M3[s][..., None], 6.0), E2M1)
    code = (mag + 8 * np.signbit(g)).reshape(x.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8), s.astype(np.uint8)


def dequantise(codes, scales):
    both = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 128)
    val = np.where(both >= 8, -E2M1[both & 7], E2M1[both & 7])
    s = np.append(E4M3, np.nan)[np.minimum(scales, 127)]
    return (val.reshape(*val.shape[:-1], 8, 16) * s[..., None]).reshape(val.shape)


def rows_of(dense, table, b, S, ps):
    """[H_kv, S, 128] of sequence b from a pool [P, H_kv, ps, 128]."""
    s = np.arange(S)
    return dense[table[b, s // ps], :, s % ps].transpose(1, 0, 2)


@dataclasses.dataclass
class Case:
    B: int
    G: int
    H_kv: int
    L: int
    ps: int
    ctx: list
    pool: str = "q4"     # or "bf16"
    dtype: str = "bf16"  # of the query
    causal: bool = True
    seed: int = 0
    spare: int = 0       # table entries past the longest sequence's pages

    def __str__(self):
        return (f"{self.pool}-{self.dtype}-B{self.B}G{self.G}H{self.H_kv}L{self.L}ps{self.ps}"
                f"{'' if self.causal else '-full'}-{max(self.ctx)}")


def bf16(x):
    return synth.bf16_to_f32(synth.bf16_bits(np.asarray(x, np.float32)))


class Inputs:
    """Pools, table and query of a case.  Unused slots and pages hold NaN,
    unused table entries junk."""

    def __init__(self, c: Case, extra_pages=0):
        rng = np.random.default_rng(c.seed + 1)
        npg = [-(-s // c.ps) for s in c.ctx]
        self.c, self.P = c, sum(npg) + 2 + extra_pages
        perm = rng.permutation(self.P)
        self.free = perm[sum(npg):]
        self.table = np.full((c.B, max(npg) + c.spare), -7, np.int32)
        at = 0
        used = np.zeros((self.P, c.ps), bool)
        for b, s in enumerate(c.ctx):
            self.table[b, :npg[b]] = perm[at:at + npg[b]]
            at += npg[b]
            i = np.arange(s)
            used[self.table[b, i // c.ps], i % c.ps] = True
        self.ctx = np.array(c.ctx, np.int32)
        self.cap = self.table.shape[1] * c.ps
        self.scale = float(np.float32(1 / math.sqrt(128)))
        q = rng.standard_normal((c.B, c.H_kv * c.G, c.L, 128)).astype(np.float32) * 1.5
        self.q = bf16(q) if c.dtype == "bf16" else q
        self.raw, self.dense = [], []  # raw: what goes to the device
        for mult in (1.5, 1.0):
            x = rng.standard_normal((self.P, c.H_kv, c.ps, 128)).astype(np.float32) * mult
            if c.pool == "q4":
                codes, scales = quantise(x)
                scales[~used[:, None].repeat(c.H_kv, 1)] = 0x7f
                self.raw += [codes, scales]
                self.dense.append(dequantise(codes, scales))
            else:
                x = bf16(x)
                x[~used[:, None].repeat(c.H_kv, 1)] = np.nan
                self.raw.append(x)
                self.dense.append(x.astype(np.float64))
        self.w = rng.random((c.B, c.H_kv, self.cap)).astype(np.float32)

    def device(self):
        import torch
        d = {}
        dt = torch.bfloat16 if self.c.dtype == "bf16" else torch.float32
        d["q"] = torch.from_numpy(self.q).to(dt).cuda()
        d["table"] = torch.from_numpy(self.table).cuda()
        d["ctx"] = torch.from_numpy(self.ctx).cuda()
        d["w"] = torch.from_numpy(self.w).cuda()
        if self.c.pool == "q4":
            d["pool"] = B.Q4Pool(*[torch.from_numpy(t).cuda() for t in self.raw])
        else:
            d["pool"] = [torch.from_numpy(t).bfloat16().cuda() for t in self.raw]
        return d


def attend(inp: Inputs, skip=()):
    """64-bit (out, added weights, tolerance of out, of the weights); sequences
    in `skip` are zeros.  The tolerances count roundings; p are probabilities:

    * the output's type: half a step, eps / 2 of the result;
    * scores: 128 products are exact and are added in fp32 by 8 (16 for fp32
      queries) instructions; a partial sum is at most T = scale * sum |q k|,
      an instruction adds 17 terms, each cut by at most 2^-23 T: with the
      scaling and the exponential's own 2^-21 at most 2^-15 T + 2^-20
      relative in every p;
    * p as an operand: 2^-11 for f16 (4-bit pages, few rows), 2^-22 for its two
      parts (fp32), 2^-8 for bf16 (bf16 pages; 4-bit pages and more than 8 rows
      per kv head, which may go through bf16 copies of the pages), and as much
      again where the row sum adds the rounded weights; parts below f16's range
      lose up to 2^-25 of the row's largest p each;
    * sums of S terms in fp32: 2^-24 S at worst, S below 2^12 here.
    """
    c = inp.c
    out = np.zeros(inp.q.shape)
    tol = np.zeros(inp.q.shape)
    w = np.zeros(inp.w.shape)
    w_tol = np.zeros(inp.w.shape)
    eps = 2.0 ** -8 if c.dtype == "bf16" else 2.0 ** -24
    many = c.pool == "bf16" or c.G * c.L > 8
    pop = 2.0 ** -22 if c.dtype == "f32" else 2 * 2.0 ** -8 if many else 2.0 ** -11
    for b, S in enumerate(inp.ctx):
        if b in skip:
            continue
        K = rows_of(inp.dense[0], inp.table, b, S, c.ps)
        V = rows_of(inp.dense[1], inp.table, b, S, c.ps)
        for h in range(c.G * c.H_kv):
            k, v, q = K[h // c.G], V[h // c.G], inp.q[b, h].astype(np.float64)
            x = q @ k.T * inp.scale
            T = (np.abs(q) @ np.abs(k).T * inp.scale).max(-1, keepdims=True)
            if c.causal:
                x[np.arange(S)[None] > np.arange(c.L)[:, None] + S - c.L] = -np.inf
            p = np.exp(x - x.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            rel = T * 2.0 ** -15 + 2.0 ** -20 + S * 2.0 ** -24
            out[b, h] = p @ v
            tol[b, h] = (rel + pop) * (p @ np.abs(v)) + eps * np.abs(out[b, h]) + \
                2.0 ** -25 * p.max(-1, keepdims=True) * np.abs(v).sum(0)
            w[b, h // c.G, :S] += p.sum(0)
            w_tol[b, h // c.G, :S] += (2 * rel * p).sum(0)
    return out, w, tol, w_tol


def evict(w, ctx, keep, recent):
    """(kept [B, H, keep], lengths) of weights [B, H, S]."""
    kept = np.full((*w.shape[:2], keep), -1, np.int32)
    for b, S in enumerate(ctx):
        for h in range(w.shape[1]):
            n = min(S, keep)
            last = S if S <= keep else recent
            x = w[b, h, :S - last].astype(np.float64)
            x = np.where(np.isnan(x), np.inf, x) + 0.0
            nan = np.isnan(w[b, h, :S - last])
            order = np.lexsort((np.arange(S - last), -x, ~nan))
            kept[b, h, :n] = np.sort(np.append(order[:n - last], np.arange(S - last, S)))
    return kept, np.minimum(ctx, keep).astype(np.int32)


def worst(got, want, tol):
    """The largest error in units of its tolerance."""
    return float(np.max(np.abs(got - want) / np.maximum(tol, 1e-300)))
