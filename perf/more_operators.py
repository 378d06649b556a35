"""Timed cases of the operators that speculative decoding and branching need
over a page pool: the visibility of a tree of drafted tokens, attention of such
a tree over the cache, compaction of the accepted drafts, and pages that are
shared, taken, copied and given back when sequences fork, grow and end.

``run`` computes a case in plain torch (``own`` false) or through the
framework's entry points (``own`` true); ``exact`` computes it in 64 bits.

The drafted tokens of a sequence are the last L of its context_lens[b] keys.
parents[b, i] < i is the draft that draft i follows, -1 for the last token
before the drafts, -2 for a slot without a draft; such slots are seen by nobody
and their outputs are 0.  Bit n of word n // 32 of mask[b, i] says that draft i
sees draft n (its ancestors and itself); every draft sees the keys before them.

A 4-bit row is 128 values: 64 bytes of e2m1 codes (dim 2i in the low half of
byte i) and 8 e4m3 scales, one per 16 dims; a value is code * scale.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
GROUP = 16
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
ROW = {"bf16": 4 * D, "f32": 8 * D, "q4": 144}  # bytes of a key and its value


# ---------------------------------------------------------------- the cases --
def _case(op, B, G, H_kv, L, page_size, ctx, pool="bf16", dtype="bf16", n=0, name=None):
    """B sequences of ctx keys, L of them drafted; n: rows forked from them."""
    c = dict(op=op, pool=pool, dtype=dtype, B=B, G=G, H_kv=H_kv, L=L, page_size=page_size,
             ctx_lo=ctx[0], ctx_hi=ctx[1], n=n)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one sequence with a few drafts, where latency counts
        _case("tree", 1, 4, 2, 8, 16, (300, 300), name="tree one short"),
        # a serving batch, a small tree each
        _case("tree", 64, 4, 8, 16, 128, (128, 4096), name="tree batch"),
        # wide trees over ragged contexts
        _case("tree", 16, 4, 8, 63, 64, (1000, 8000), name="tree wide"),
        # long contexts in small pages
        _case("tree", 16, 4, 8, 32, 16, (32768, 32768), name="tree long"),
        # a cache held in 4 bits
        _case("tree", 32, 4, 8, 24, 64, (500, 8000), pool="q4", name="tree 4-bit"),
        # fp32, a group of 3, page size and lengths that are no powers of two
        _case("tree", 3, 3, 5, 13, 12, (200, 900), pool="f32", dtype="f32", name="tree fp32"),
        # the visibility of a batch's trees, once per step for all layers
        _case("mask", 64, 1, 1, 64, 16, (64, 64), name="mask batch"),
        # large trees, odd size
        _case("mask", 8, 1, 1, 1001, 16, (1001, 1001), name="mask large"),
        # the drafts' rows stored, then the accepted ones moved together
        _case("compact", 64, 4, 8, 16, 128, (128, 1024), name="compact batch"),
        _case("compact", 16, 4, 8, 63, 64, (1000, 4000), pool="q4", name="compact 4-bit"),
        # a step of a beam search: 64 beams end, 64 are forked from 16 and grow
        _case("pages", 16, 4, 8, 1, 128, (128, 4096), n=64, name="pages beams"),
        # samples of long prompts in small pages, room for 32 drafts each
        _case("pages", 8, 4, 4, 32, 16, (4000, 32000), pool="q4", n=48, name="pages samples"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["tree", "tree", "tree", "mask", "compact", "pages"])
        pool = rng.choice(["bf16", "bf16", "q4", "f32"])
        dtype = "bf16" if pool == "bf16" else "f32" if pool == "f32" else \
            rng.choice(["bf16", "bf16", "f32"])
        G, H_kv = rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([1, 2, 4, 5, 8])
        B, ps = _log(rng, 1, 64), rng.choice([8, 12, 16, 24, 64, 128])
        L = _log(rng, 8, 1024) if op == "mask" else _log(rng, 1, 255)
        hi = max(L, _log(rng, 32, 32768))
        lo = max(L, int(hi * rng.uniform(0.2, 1.0)))
        if op == "mask":
            c = _case(op, B, 1, 1, L, 16, (L, L))
            if B * L >= 64 and B * L ** 3 <= 8 * 1001 ** 3:
                return c
            continue
        c = _case(op, B, G, H_kv, L, ps, (lo, hi), pool, dtype,
                  _log(rng, 1, 128) if op == "pages" else 0)
        rows = (B + c["n"] // 8) * H_kv * hi  # (forks share what they do not copy)
        scores = B * H_kv * G * L * hi if op == "tree" else 0
        if rows * ROW[pool] <= 16 * 8 * 32768 * ROW["bf16"] / (1 if op == "tree" else 2) and \
                scores <= 16 * 8 * 4 * 32 * 32768 / (1 if pool != "f32" else 4):
            return c


def _lens(case, seed):
    r = random.Random(seed * 7919 + 17)
    return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]


def _words(L):
    return (L + 31) // 32


def _accepted(case):
    """Mean number of accepted drafts."""
    return min(case["L"], 1 + 0.5 * math.log(case["L"]) * 1.5)


def work(case):
    B, H, G, L, ps, n = (case[k] for k in ("B", "H_kv", "G", "L", "page_size", "n"))
    # expected context: the cases draw lengths evenly between their bounds
    mean = (case["ctx_lo"] + case["ctx_hi"]) / 2
    row = ROW[case["pool"]]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "mask":
        return {"bytes": B * L * (4 + 4 + 4 * _words(L)), "flops": B * L * L}
    if case["op"] == "compact":
        acc = _accepted(case)
        b = B * H * (L * (2 * D * es + row) + acc * 2 * row) + B * (4 * acc + 12)
        if case["pool"] == "q4":  # the read-back of the last L rows
            b += B * H * L * (row + 4 * D)
        return {"bytes": b, "flops": B * H * L * D * (8 if case["pool"] == "q4" else 1)}
    if case["op"] == "pages":
        entries = n * (mean / ps)
        part = (ps - 1) / 2  # rows of a last page that is not full
        b = entries * (4 + 4 + 8 + 8) + n * (L / ps + 1) * 8 + n * H * part * 2 * row
        if case["pool"] == "q4":
            b += n * H * (ps + L) * (row + 4 * D)
        return {"bytes": b, "flops": entries * 4}
    pairs = B * H * G * L * (mean - L + 1 + math.log(L))
    b = B * H * mean * row + 2 * B * H * G * L * D * es + B * L * _words(L) * 4
    return {"bytes": b, "flops": 4 * D * pairs}


# --------------------------------------------------------------- the inputs --
def _quant(x):
    """Codes [..., 64] and scales [..., 8] (bytes) of fp32 rows [..., 128]."""
    g = x.float().unflatten(-1, (D // GROUP, GROUP))
    s = (g.abs().amax(-1) / 6.0).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    y = g / s.float().unsqueeze(-1)
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for i, m in enumerate(MID):  # a tie goes to the even code
        code += (a > m) if i % 2 == 0 else (a >= m)
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def _dequant(codes, scales, lut):
    """fp32 rows [..., 128]; lut: the 16 values of a code."""
    both = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    s = scales.view(torch.float8_e4m3fn).float()
    return (both.unflatten(-1, (D // GROUP, GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _pages(n, page_size):
    return (n + page_size - 1) // page_size


def _trees(case, seed):
    """parents [B, L] and, of each tree, a path from its root (ascending)."""
    r = random.Random(seed * 104729 + 5)
    B, L = case["B"], case["L"]
    parents = np.full((B, L), -2, np.int32)
    paths = []
    for b in range(B):
        n = r.randint((3 * L + 3) // 4, L)  # the other slots hold no draft
        for i in range(n):
            parents[b, i] = -1 if i == 0 or r.random() < 0.02 else r.randrange(i)
        node, path = r.randrange(n), []
        while node >= 0:
            path.append(node)
            node = int(parents[b, node])
        path = path[::-1]
        paths.append(path[:r.randint(min(1, len(path)), len(path))] if r.random() < 0.95 else [])
    return parents, paths


def _words_of(see):
    """int32 words [..., W] of truth values [..., L]."""
    L = see.shape[-1]
    x = torch.nn.functional.pad(see.long(), (0, 32 * _words(L) - L)).unflatten(-1, (-1, 32))
    return (x << torch.arange(32, device=see.device)).sum(-1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, G, L, ps, n = (case[k] for k in ("B", "H_kv", "G", "L", "page_size", "n"))
    st = dict(case=case, ps=ps)
    if case["op"] == "mask":
        st["parents"] = torch.from_numpy(_trees(case, seed)[0]).cuda()
        return st
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, mult=1.0):
        return torch.randn(shape, generator=g, device="cuda") * mult

    def cuda(x):
        return torch.from_numpy(np.asarray(x, np.int32)).cuda()

    lens = _lens(case, seed)
    npg = [_pages(s, ps) for s in lens]
    grow = L if case["op"] == "pages" else 0
    width = _pages(case["ctx_hi"] + grow, ps)
    # the longest sequences' pages, those that forks take, and a few that stay free
    total = B * width + n * (1 + _pages(L, ps)) + 3
    perm = torch.randperm(total, generator=g, device="cuda").int().cpu().numpy()
    table = np.full((B + n, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :npg[b]] = perm[at:at + npg[b]]
        at += npg[b]
    st.update(lens=lens, cap=width * ps, table=cuda(table), ctx=cuda(lens + [0] * n),
              lut=torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda"),
              scale=float(np.float32(1.0 / math.sqrt(D))))
    if case["pool"] == "q4":
        # page by page, so that the unrounded pool never stands in memory
        parts = []
        for mult in (1.5, 1.0):
            codes = torch.empty(total, H, ps, D // 2, dtype=torch.uint8, device="cuda")
            scales = torch.empty(total, H, ps, D // GROUP, dtype=torch.uint8, device="cuda")
            step = max(1, (1 << 25) // (H * ps * D))
            for p in range(0, total, step):
                k = min(step, total - p)
                codes[p:p + k], scales[p:p + k] = _quant(normal(k, H, ps, D, mult=mult))
            parts += [codes, scales]
        st["pool"] = parts
    else:
        pdt = torch.bfloat16 if case["pool"] == "bf16" else torch.float32
        st["pool"] = [normal(total, H, ps, D, mult=m).to(pdt) for m in (1.5, 1.0)]
    if case["op"] == "pages":
        r = random.Random(seed * 31 + 3)
        src = [r.randrange(B) for _ in range(n)]
        refs = np.zeros(total, np.int32)
        refs[perm[:at]] = 1
        st.update(refs=cuda(refs), src=cuda(src), tgt=cuda(range(B, B + n)), sources=src,
                  ended=cuda([-1] * B + [0] * n),
                  grown=cuda([-1] * B + [lens[s] + L for s in src]))
        _plain_pages(st)  # the rows to be forked into hold what a step before left
        return st
    parents, paths = _trees(case, seed)
    if case["op"] == "compact":
        new_dt = dt if case["pool"] == "q4" else st["pool"][0].dtype
        st["k_new"] = normal(B, H, L, D, mult=1.5).to(new_dt)
        st["v_new"] = normal(B, H, L, D).to(new_dt)
        most = max(1, max(len(p) for p in paths))
        st["paths"] = paths
        st["path"] = cuda([p + [-1] * (most - len(p)) for p in paths])
        st["path_lens"] = cuda([len(p) for p in paths])
        return st
    st["query"] = normal(B, H * G, L, D).to(dt)
    st["parents"] = parents
    st["mask"] = _words_of(_visible(torch.from_numpy(parents).cuda()))
    return st


# ---------------------------------------------------------- the plain forms --
def _visible(parents):
    """[B, L, L]: draft i sees draft n."""
    L = parents.shape[1]
    i = torch.arange(L, device="cuda")
    see = (parents[:, :, None] == i) | (i[:, None] == i)
    for _ in range(max(1, (L - 1).bit_length())):  # paths twice as long each time
        see = (see.float() @ see.float()) > 0
    lost = (see & ((parents < -1) | (parents >= i))[:, None, :]).any(-1)  # no draft, or after none
    return see & ~lost[:, :, None]


def _where(table, pos, ps):
    """Page and slot of logical positions pos [B, n] (clamped into the table)."""
    pos = pos.clamp(min=0)
    lp = (pos // ps).clamp(max=table.shape[1] - 1)
    return table.gather(1, lp).clamp(min=0).long(), pos % ps


def _dense(st, parts, table, pos):
    """fp32 rows [B, H_kv, n, 128] at logical positions pos [B, n]."""
    pg, slot = _where(table, pos, st["ps"])
    rows = [t[pg, :, slot] for t in parts]  # [B, n, H_kv, ...]
    x = _dequant(*rows, st["lut"]) if len(rows) == 2 else rows[0].float()
    return x.transpose(1, 2)


def _tail(st, table, ctx, n):
    """Rows at the last n positions of each context, bf16, 0 before its start."""
    pos = ctx.long()[:, None] - n + torch.arange(n, device="cuda")
    ok = (pos >= 0)[:, None, :, None]
    return [(_dense(st, st["pool"][k:k + 2], table, pos) * ok).bfloat16() for k in (0, 2)]


def _plain_mask(st):
    see = _visible(st["parents"])
    return _words_of(see), (see.sum(-1) - 1).to(torch.int32)


def _plain_tree(st):
    c, q = st["case"], st["query"]
    B, H, G, L = c["B"], c["H_kv"], c["G"], c["L"]
    half = len(st["pool"]) // 2
    bits = (st["mask"][..., None] >> torch.arange(32, device="cuda")) & 1
    see = bits.flatten(-2)[..., :L] > 0
    drafted = see.any(-1)
    pos = torch.arange(st["cap"], device="cuda").expand(B, -1)
    rel = pos - (st["ctx"].long()[:, None] - L)  # number of the draft at a position
    among = see.gather(2, rel.clamp(0, L - 1)[:, None].expand(B, L, -1))
    show = ((rel < 0)[:, None] & drafted[:, :, None]) | (among & ((rel >= 0) & (rel < L))[:, None])
    qr = q.float().reshape(B, H, G * L, D)
    s = (qr @ _dense(st, st["pool"][:half], st["table"], pos).transpose(2, 3)) * st["scale"]
    s.view(B, H, G, L, -1).masked_fill_(~show[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-3e38))
    out = p @ _dense(st, st["pool"][half:], st["table"], pos)
    return (out / p.sum(-1, keepdim=True).clamp(min=1e-30)).reshape(q.shape).to(q.dtype)


def _plain_compact(st):
    c, path = st["case"], st["path"].long()
    L, n = c["L"], st["path_lens"].long()[:, None]
    first = st["ctx"].long()[:, None] - L
    new = first + torch.arange(L, device="cuda")
    pg, slot = _where(st["table"], new, st["ps"])
    k, v = st["k_new"].transpose(1, 2), st["v_new"].transpose(1, 2)
    rows = [*_quant(k), *_quant(v)] if c["pool"] == "q4" else [k, v]
    for t, x in zip(st["pool"], rows):
        t[pg, :, slot] = x
    j = torch.arange(path.shape[1], device="cuda")
    fp, fs = _where(st["table"], first + torch.where(j < n, path, j), st["ps"])
    tp, ts = _where(st["table"], first + j, st["ps"])
    for t in st["pool"]:
        t[tp, :, ts] = t[fp, :, fs]
    lens = st["ctx"] - L + st["path_lens"]
    return [lens] + (_tail(st, st["table"], lens, L) if c["pool"] == "q4" else list(st["pool"]))


def _plain_pages(st):
    c, ps, table, ctx, refs = st["case"], st["ps"], st["table"], st["ctx"], st["refs"]
    B, L, n = c["B"], c["L"], c["n"]
    src, tgt = st["src"].long(), st["tgt"].long()
    i = torch.arange(table.shape[1], device="cuda")
    one = torch.ones((), dtype=torch.int32, device="cuda")

    def count(entries, there, by):
        refs.index_add_(0, entries.clamp(min=0).flatten().long(), (there * by).flatten().int())

    # the rows that ended give their pages back
    old = table[tgt]
    count(old, old >= 0, -one)
    # forks share every page of their sources
    new = table[src]
    count(new, new >= 0, one)
    table[tgt] = new
    # room for L more: the pages needed, and a page of its own in a shared one's place
    have = _pages(ctx[src].long(), ps)
    want = _pages(ctx[src].long() + L, ps)
    rows = ctx[src].long() % ps
    last = new.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0]
    own_copy = (rows > 0) & (refs[last.long()] > 1)
    take = want - have + own_copy
    first = have - own_copy.long()
    ids = torch.argsort((refs > 0).int(), stable=True)  # the free pages first, ascending
    k = i - first[:, None] + (take.cumsum(0) - take)[:, None]
    fresh = (i >= first[:, None]) & (i < want[:, None])
    got = torch.where(fresh, ids[k.clamp(0, ids.numel() - 1)].int(), table[tgt])
    count(last, own_copy, -one)
    count(got, fresh, one)
    table[tgt] = got
    ctx[tgt] = (ctx[src] + L).int()
    mine = got.gather(1, first[:, None].clamp(max=i.numel() - 1))[:, 0]
    copies = torch.stack([last.long(), mine.long(), rows], 1)
    copies = torch.where(own_copy[:, None], copies, torch.tensor([-1, -1, 0], device="cuda"))
    # the rows of those pages, all layers alike: here one
    a = torch.where(own_copy, last, mine).long()
    inside = torch.arange(ps, device="cuda") < rows[:, None]
    for t in st["pool"]:
        t[mine.long()] = torch.where(inside[:, None, :, None] & own_copy[:, None, None, None],
                                     t[a], t[mine.long()])
    copies = torch.cat([torch.tensor([[-1, -1, 0]], device="cuda").expand(B, 3), copies])
    tail = _tail(st, table[B:], ctx[B:], ps + L) if c["pool"] == "q4" else list(st["pool"])
    return [table, ctx, refs, copies.int()] + tail


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"mask": _plain_mask, "tree": _plain_tree, "compact": _plain_compact,
            "pages": _plain_pages}[op](state)


# ------------------------------------------------- the framework's operators --
def _own(st, op):
    from paged_kv_cache_03_gb300 import binding as pa
    c, ps = st["case"], st["ps"]
    q4 = c["pool"] == "q4"
    if "ws" not in st:  # a serving loop makes these once
        if q4 and "pool" in st:
            st["q4"] = pa.Q4Pool(*st["pool"])
        if op == "tree":
            st["ws"] = pa.new_tree_workspace(st["query"], st["q4"] if q4 else st["pool"][0],
                                             st["table"])
        elif op == "pages":
            st["ws"] = pa.new_pages_workspace(st["table"], st["refs"])
        else:
            st["ws"] = pa.new_cache_workspace("cuda")
    ws = st["ws"]
    if op == "mask":
        return pa.tree_mask(st["parents"], workspace=ws)
    table, ctx = st["table"], st["ctx"]
    if op == "tree":
        if q4:
            return pa.paged_attention_tree_q4(st["query"], st["q4"], table, ctx, st["mask"], ps,
                                              st["scale"], workspace=ws)
        return pa.paged_attention_tree(st["query"], *st["pool"], table, ctx, st["mask"], ps,
                                       st["scale"], workspace=ws)
    if op == "compact":
        if q4:
            pa.append_kv_q4(st["k_new"], st["v_new"], st["q4"], table, ctx, workspace=ws)
            lens = pa.compact_kv_q4(st["q4"], table, ctx, st["path"], st["path_lens"], c["L"],
                                    workspace=ws)
            return [lens, *pa.gather_kv_q4(st["q4"], table, lens, c["L"], tail=True,
                                           workspace=ws)]
        pa.append_kv(st["k_new"], st["v_new"], *st["pool"], table, ctx, workspace=ws)
        lens = pa.compact_kv(*st["pool"], table, ctx, st["path"], st["path_lens"], c["L"],
                             workspace=ws)
        return [lens, *st["pool"]]
    refs, B = st["refs"], c["B"]
    pa.resize_pages(table, ctx, refs, st["ended"], ps, workspace=ws)
    pa.fork_pages(table, ctx, refs, st["src"], st["tgt"], ps, workspace=ws)
    copies = pa.resize_pages(table, ctx, refs, st["grown"], ps, workspace=ws)
    if q4:
        pa.copy_pages_q4(st["q4"], copies, workspace=ws)
        tail = pa.gather_kv_q4(st["q4"], table[B:], ctx[B:], ps + c["L"], tail=True, workspace=ws)
    else:
        pa.copy_pages(*st["pool"], copies, workspace=ws)
        tail = st["pool"]
    return [table, ctx, refs, copies, *tail]


# ------------------------------------------------------------- in 64 bits --
def _e4m3_values():
    """All finite non-negative e4m3 values, ascending: index = byte."""
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(x, values):
    """Index of the nearest of ascending `values`, ties to the even index."""
    mid = (values[1:] + values[:-1]) / 2
    lo = torch.searchsorted(mid, x.contiguous(), right=False)  # a tie counts as below
    hi = torch.searchsorted(mid, x.contiguous(), right=True)
    return torch.where(lo % 2 == 0, lo, hi)


def _exact_round(x):
    """What 4 bits hold of fp64 rows [..., 128], by nearest values."""
    g = x.reshape(-1, GROUP)
    scales = _e4m3_values()
    s = scales[_nearest(g.abs().amax(1) / 6, scales).clamp(min=1)][:, None]
    levels = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    return (levels[_nearest(g.abs() / s, levels)] * s * torch.sign(g)).reshape(x.shape)


def _exact_values(parts):
    """fp64 rows of bf16 or fp32 rows, or of codes and scales."""
    if len(parts) == 1:
        return parts[0].double()
    byte = parts[0].int()
    code = torch.stack((byte % 16, byte // 16), -1).reshape(*byte.shape[:-1], D)
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[(code % 8).long()]
    val = torch.where(code >= 8, -mag, mag).reshape(*byte.shape[:-1], 8, GROUP)
    return (val * _e4m3_values()[parts[1].long()][..., None]).reshape(*byte.shape[:-1], D)


def _exact_rows(st, parts, table, b, pos):
    """fp64 rows [H_kv, n, 128] of sequence b at positions pos [n]."""
    pg = table[b].long()[pos // st["ps"]]
    return _exact_values([t.transpose(1, 2)[pg, pos % st["ps"]].transpose(0, 1) for t in parts])


def _exact_mask(parents):
    """Visibility [B, L, L] by walking up from every draft."""
    B, L = parents.shape
    see = np.zeros((B, L, L), bool)
    for b in range(B):
        for i in range(L):
            p = int(parents[b, i])
            if p == -1:
                see[b, i, i] = True
            elif 0 <= p < i and see[b, p, p]:
                see[b, i] = see[b, p]
                see[b, i, i] = True
    return see


def _exact_pages(case, st):
    """The pages' state by a simulation, one event after the other."""
    B, L, ps, n = case["B"], case["L"], case["page_size"], case["n"]
    table, ctx, refs = (st[k].cpu().numpy().copy() for k in ("table", "ctx", "refs"))
    copies = np.full((B + n, 3), (-1, -1, 0), np.int32)
    for row in range(B, B + n):
        for e in table[row][table[row] >= 0]:
            refs[e] -= 1
        table[row] = -1
    for row, s in zip(range(B, B + n), st["sources"]):
        table[row], ctx[row] = table[s], ctx[s]
        for e in table[row][table[row] >= 0]:
            refs[e] += 1
    free = iter(np.flatnonzero(refs == 0))
    for row in range(B, B + n):
        have, want = _pages(int(ctx[row]), ps), _pages(int(ctx[row]) + L, ps)
        part = int(ctx[row]) % ps
        if part and refs[table[row, have - 1]] > 1:
            new = next(free)
            copies[row] = (table[row, have - 1], new, part)
            refs[table[row, have - 1]] -= 1
            refs[new] = 1
            table[row, have - 1] = new
        for j in range(have, want):
            table[row, j] = next(free)
            refs[table[row, j]] = 1
        ctx[row] += L
    return table, ctx, refs, copies


def exact(case, seed):
    st = prepare(case, seed)
    B, H, G, L, ps = (case[k] for k in ("B", "H_kv", "G", "L", "page_size"))
    if case["op"] == "mask":
        see = torch.from_numpy(_exact_mask(st["parents"].cpu().numpy()))
        W = _words(L)
        words = np.zeros((B, L, W), np.uint32)
        for i in range(L):
            words[:, :, i // 32] |= see[:, :, i].numpy().astype(np.uint32) << np.uint32(i % 32)
        return words.view(np.int32), (see.sum(-1) - 1).int()
    half = len(st["pool"]) // 2
    pools = [st["pool"][:half], st["pool"][half:]]
    q4 = case["pool"] == "q4"
    if case["op"] == "compact":
        lens = np.array([s - L + len(p) for s, p in zip(st["lens"], st["paths"])], np.int32)
        rows = [torch.zeros(B, H, L, D, dtype=torch.float64, device="cuda") if q4
                else p[0].double() for p in pools]
        for b, (S, path) in enumerate(zip(st["lens"], st["paths"])):
            for i, new in enumerate((st["k_new"], st["v_new"])):
                new = _exact_round(new[b].double()) if q4 else new[b].double()
                moved = new.clone()  # [H, L, 128]
                moved[:, :len(path)] = new[:, path]
                if q4:
                    n = max(0, min(L - len(path), S - L))  # rows before the drafts
                    at = torch.arange(S - L - n, S - L, device="cuda")
                    rows[i][b, :, L - len(path) - n:L - len(path)] = \
                        _exact_rows(st, pools[i], st["table"], b, at)
                    rows[i][b, :, L - len(path):] = moved[:, :len(path)]
                else:
                    at = torch.arange(S - L, S, device="cuda")
                    pg = st["table"][b].long()[at // ps]
                    rows[i].transpose(1, 2)[pg, at % ps] = moved.transpose(0, 1)
        return [lens, *rows]
    if case["op"] == "pages":
        # (prepare's own pass has run: start again from rows that hold nothing)
        table, ctx, refs, copies = _exact_pages(case, _emptied(st))
        tails = []
        for part in pools:
            if q4:
                n, new = ps + L, torch.from_numpy(table).cuda()
                rows = torch.zeros(case["n"], H, n, D, dtype=torch.float64, device="cuda")
                for i in range(case["n"]):
                    m = min(n, int(ctx[B + i]))
                    at = torch.arange(int(ctx[B + i]) - m, int(ctx[B + i]), device="cuda")
                    rows[i, :, n - m:] = _exact_rows(st, part, new, B + i, at)
                    if copies[B + i, 1] >= 0:  # rows before the fork's length: its source's
                        old = at < int(ctx[B + i]) - L
                        rows[i, :, n - m:][:, old] = \
                            _exact_rows(st, part, st["table"], st["sources"][i], at[old])
                tails.append(rows)
            else:
                rows = part[0].double()
                for a, d, m in copies:
                    if d >= 0:
                        rows[int(d), :, :int(m)] = part[0][int(a), :, :int(m)].double()
                tails.append(rows)
        return [table, ctx, refs, copies, *tails]
    see = torch.from_numpy(_exact_mask(st["parents"])).cuda()
    out = torch.zeros(B, H * G, L, D, dtype=torch.float64, device="cuda")
    for b, S in enumerate(st["lens"]):
        at = torch.arange(S, device="cuda")
        K = _exact_rows(st, pools[0], st["table"], b, at)
        V = _exact_rows(st, pools[1], st["table"], b, at)
        there = see[b].diagonal()
        show = torch.cat([torch.ones(L, S - L, dtype=torch.bool, device="cuda"), see[b]], 1)[there]
        for h in range(H * G):
            x = st["query"][b, h][there].double() @ K[h // G].T * st["scale"]
            x[~show] = -math.inf
            out[b, h, there] = torch.softmax(x, -1) @ V[h // G]
    return out


def _emptied(st):
    """The page state without the forked rows."""
    table, ctx, refs = (st[k].clone() for k in ("table", "ctx", "refs"))
    B = st["case"]["B"]
    for e in table[B:].flatten().tolist():
        if e >= 0:
            refs[e] -= 1
    table[B:], ctx[B:] = -1, 0
    return dict(st, table=table, ctx=ctx, refs=refs)
