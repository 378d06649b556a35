"""Timed cases of the operators around a page pool that is held in 4 bits or
trimmed by attention weight: append (quantise), attention over 4-bit pages,
attention that also accumulates each key's weight, and eviction.

``run`` computes a case in plain torch (``own`` false) or through the
framework's entry points (``own`` true); ``exact`` computes it in 64 bits.

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


# ---------------------------------------------------------------- the cases --
def _case(op, B, G, H_kv, L, page_size, ctx, pool="q4", dtype="bf16", causal=True, keep=0,
          recent=0, name=None):
    c = dict(op=op, pool=pool, dtype=dtype, B=B, G=G, H_kv=H_kv, L=L, page_size=page_size,
             ctx_lo=ctx[0], ctx_hi=ctx[1], causal=causal, keep=keep, recent=recent)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of a serving batch: a row per sequence and kv head
        _case("append", 64, 4, 8, 1, 128, (128, 4096), name="append decode"),
        # four prompts written at once
        _case("append", 4, 4, 8, 2048, 128, (2048, 2048), name="append prompt"),
        # a chunk in fp32, odd length, small pages
        _case("append", 2, 2, 4, 65, 16, (300, 1000), dtype="f32", name="append fp32 chunk"),
        # one short decode, where latency counts; a page size that is no power of two
        _case("attend", 1, 4, 2, 1, 12, (300, 300), dtype="f32", name="attend one short"),
        # a decode step of a serving batch
        _case("attend", 64, 4, 8, 1, 128, (128, 4096), name="attend decode"),
        # decodes over long contexts in small pages
        _case("attend", 16, 4, 8, 1, 16, (32768, 32768), name="attend long decode"),
        # continuation chunks over ragged contexts
        _case("attend", 8, 4, 8, 65, 128, (1000, 8000), name="attend chunks"),
        # four whole prompts
        _case("attend", 4, 4, 8, 2048, 128, (2048, 2048), name="attend prompts"),
        # a decode step that keeps the heavy-hitter scores, bf16 pages
        _case("weigh", 64, 4, 8, 1, 128, (128, 4096), pool="bf16", name="weigh decode bf16"),
        # the last 32 positions of prompts score their keys before an eviction
        _case("weigh", 8, 4, 8, 32, 128, (1000, 8000), pool="q4", name="weigh window"),
        # halving long contexts, bf16 pages
        _case("evict", 16, 4, 8, 1, 128, (8192, 8192), pool="bf16", keep=4096, recent=512,
              name="evict bf16"),
        # a ragged batch trimmed to a budget, some sequences already within it
        _case("evict", 32, 4, 8, 1, 64, (500, 4096), pool="q4", keep=1024, recent=65,
              name="evict 4-bit"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["append", "attend", "attend", "weigh", "evict"])
        pool = "q4" if op in ("append", "attend") else rng.choice(["q4", "bf16"])
        dtype = "bf16" if pool == "bf16" or op == "evict" else rng.choice(["bf16", "bf16", "f32"])
        G = rng.choice([1, 2, 3, 4, 7, 8])
        H_kv = rng.choice([1, 2, 4, 8])
        B = _log(rng, 1, 64)
        L = 1 if op == "evict" or (op != "append" and rng.random() < 0.4) else _log(rng, 1, 2048)
        ps = rng.choice([8, 12, 16, 24, 64, 128])
        hi = max(L, _log(rng, 32, 32768))
        lo = max(L, int(hi * rng.uniform(0.2, 1.0)))
        keep = recent = 0
        if op == "evict":
            keep = max(1, int(hi * rng.uniform(0.1, 1.0)))
            recent = int(keep * rng.uniform(0.0, 0.5))
        c = _case(op, B, G, H_kv, L, ps, (lo, hi), pool, dtype, rng.random() < 0.8, keep, recent)
        rows = B * H_kv * hi
        scores = rows * G * L if op in ("attend", "weigh") else 0
        if rows * 144 <= 16 * 8 * 32768 * 144 * (1 if pool == "q4" else 0.5) and \
                scores <= 4 * 32 * 2048 * 2048 // 2:
            return c


def _lens(case, seed):
    r = random.Random(seed * 7919 + 17)
    return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]


def _visible(case, S):
    L = case["L"]
    return L * S - L * (L - 1) // 2 if case["causal"] else L * S


def work(case):
    B, H, G, L = case["B"], case["H_kv"], case["G"], case["L"]
    # expected context: the cases draw lengths evenly between their bounds
    mean = (case["ctx_lo"] + case["ctx_hi"]) / 2
    row = 144 if case["pool"] == "q4" else 4 * D
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "append":
        # rows in, 4-bit rows out, and the read-back of what was stored
        n = B * H * L
        return {"bytes": n * (2 * D * es + 2 * 144 + 2 * D * es), "flops": n * 2 * D * 4}
    if case["op"] == "evict":
        lo, hi, keep = case["ctx_lo"], case["ctx_hi"], case["keep"]
        if hi <= keep:
            kept = mean
        elif lo >= keep:
            kept = keep
        else:
            kept = ((keep - lo) * (lo + keep) / 2 + (hi - keep) * keep) / (hi - lo)
        back = 2 * D * 2 + 144 if case["pool"] == "q4" else 0  # the 4-bit rows' read-back
        return {"bytes": B * H * (4 * mean + kept * (2 * row + 8 + back)), "flops": B * H * mean}
    pairs = B * H * G * _visible(case, mean)
    b = B * H * mean * row + 2 * B * H * G * L * D * es
    if case["op"] == "weigh":
        b += 8 * B * H * mean
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
    return [(s + page_size - 1) // page_size for s in n]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, H, G, L, ps = case["B"], case["H_kv"], case["G"], case["L"], case["page_size"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32

    def normal(*shape, mult=1.0):
        return torch.randn(shape, generator=g, device="cuda") * mult

    lens = _lens(case, seed)
    npg = _pages(lens, ps)
    new = _pages([min(s, case["keep"]) for s in lens], ps)  # pages an eviction writes
    width, new_width = max(_pages([case["ctx_hi"]], ps)[0], 1), max(max(new), 1)
    total = sum(npg) + sum(new)
    perm = torch.randperm(total, generator=g, device="cuda").int().cpu().numpy()
    table = np.full((B, width), -1, np.int32)
    dst = np.full((B, new_width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :npg[b]] = perm[at:at + npg[b]]
        at += npg[b]
        dst[b, :new[b]] = perm[at:at + new[b]]
        at += new[b]
    st = dict(case=case, lens=lens, ps=ps, cap=width * ps,
              table=torch.from_numpy(table).cuda(),
              ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"),
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
                n = min(step, total - p)
                codes[p:p + n], scales[p:p + n] = _quant(normal(n, H, ps, D, mult=mult))
            parts += [codes, scales]
        st["pool"] = parts
    else:
        st["pool"] = [normal(total, H, ps, D, mult=m).to(dt) for m in (1.5, 1.0)]
    if case["op"] == "append":
        st["k_new"], st["v_new"] = normal(B, H, L, D, mult=1.5).to(dt), normal(B, H, L, D).to(dt)
    elif case["op"] == "evict":
        st["dst"], st["dst_cap"] = torch.from_numpy(dst).cuda(), new_width * ps
        # accumulated weights: a few heavy keys, many light ones, some equal
        w = torch.exp(normal(B, H, st["cap"]) * 2.0)
        st["weights"] = torch.where(w < 0.5, torch.full_like(w, 0.125), w)
    else:
        st["query"] = normal(B, H * G, L, D).to(dt)
        if case["op"] == "weigh":
            # what a call like this one adds on average, times a spread
            w = torch.exp(normal(B, H, st["cap"])) * (G * L / case["ctx_hi"])
            live = torch.arange(st["cap"], device="cuda")[None, :] < st["ctx"][:, None]
            st["weights"] = w * live[:, None, :]
    return st


# ---------------------------------------------------------- the plain forms --
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


def _plain_append(st):
    c, dt = st["case"], st["k_new"].dtype
    pos = st["ctx"].long()[:, None] - c["L"] + torch.arange(c["L"], device="cuda")
    pg, slot = _where(st["table"], pos, st["ps"])
    outs = []
    for i, x in ((0, st["k_new"]), (2, st["v_new"])):
        codes, scales = _quant(x.transpose(1, 2))
        st["pool"][i][pg, :, slot] = codes
        st["pool"][i + 1][pg, :, slot] = scales
        outs.append(_dense(st, st["pool"][i:i + 2], st["table"], pos).to(dt))
    return outs


def _plain_attend(st, weigh):
    c, q = st["case"], st["query"]
    B, H, G, L = c["B"], c["H_kv"], c["G"], c["L"]
    half = len(st["pool"]) // 2
    pos = torch.arange(st["cap"], device="cuda").expand(B, -1)
    qr = q.float().reshape(B, H, G * L, D)
    s = (qr @ _dense(st, st["pool"][:half], st["table"], pos).transpose(2, 3)) * st["scale"]
    see = st["ctx"].long()[:, None].expand(B, L)  # keys each query position sees
    if c["causal"]:
        see = see - L + 1 + torch.arange(L, device="cuda")
    hide = pos[:, None, :] >= see[:, :, None]  # [B, L, cap]
    s.view(B, H, G, L, -1).masked_fill_(hide[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = (p @ _dense(st, st["pool"][half:], st["table"], pos)).reshape(q.shape).to(q.dtype)
    if not weigh:
        return out
    live = (pos < st["ctx"][:, None])[:, None, :]
    return out, torch.where(live, st["weights"] + p.sum(2), torch.zeros_like(st["weights"]))


def _plain_evict(st):
    c = st["case"]
    B, H, keep, recent = c["B"], c["H_kv"], c["keep"], c["recent"]
    S = st["ctx"].long()[:, None, None]
    pos = torch.arange(st["cap"], device="cuda").expand(B, H, -1)
    w = torch.where(pos < S, st["weights"], torch.full_like(st["weights"], float("-inf")))
    w = torch.where((pos < S) & ((pos >= S - recent) | (S <= keep)),
                    torch.full_like(w, float("inf")), w)
    rank = w.sort(stable=True, dim=-1, descending=True).indices[..., :keep]
    lens = st["ctx"].clamp(max=keep)
    n = rank.shape[-1]
    i = torch.arange(n, device="cuda")
    live = i < lens.long()[:, None, None]
    kept = rank.masked_fill(~live, st["cap"]).sort(-1).values.masked_fill(~live, -1)
    kept = torch.nn.functional.pad(kept, (0, keep - n), value=-1)
    src = kept.clamp(min=0)
    weights = torch.where(kept >= 0, st["weights"].gather(2, src.clamp(max=st["cap"] - 1)),
                          torch.zeros((), device="cuda"))
    # rows of every (b, kv head), copied to the destination's pages
    # (a place past a sequence's length repeats its first copy)
    b = torch.arange(B, device="cuda")[:, None, None]
    h = torch.arange(H, device="cuda")[None, :, None]
    j = torch.where(kept >= 0, torch.arange(keep, device="cuda"), 0)
    s = torch.where(kept >= 0, kept, kept[..., :1])
    fp = st["table"][b, s // st["ps"]].long()
    tp = st["dst"][b, j // st["ps"]].long()
    for t in st["pool"]:
        t[tp, h, j % st["ps"]] = t[fp, h, s % st["ps"]]
    if c["pool"] == "q4":  # read back dense, 0 past each length
        at = torch.arange(keep, device="cuda").expand(B, -1)
        ok = (at < lens[:, None])[:, None, :, None]
        rows = [(_dense(st, st["pool"][k:k + 2], st["dst"], at) * ok).bfloat16() for k in (0, 2)]
    else:
        rows = list(st["pool"])
    return rows + [lens, weights, kept.int()]


def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    if op == "append":
        return _plain_append(state)
    if op == "evict":
        return _plain_evict(state)
    return _plain_attend(state, op == "weigh")


# ------------------------------------------------- the framework's operators --
def _own(st, op):
    from paged_kv_cache_03_gb300 import binding as pa
    c = st["case"]
    if c["pool"] == "q4" and "q4" not in st:
        st["q4"] = pa.Q4Pool(*st["pool"])
    if "ws" not in st:  # a serving loop allocates it once
        if op in ("append", "evict"):
            st["ws"] = pa.new_cache_workspace("cuda")
        else:
            st["ws"] = pa.new_q4_workspace(st["query"], st["q4"], st["table"]) \
                if c["pool"] == "q4" else \
                pa.new_weights_workspace(st["query"], st["pool"][0], st["table"])
    ws, table, ctx, ps = st["ws"], st["table"], st["ctx"], st["ps"]
    if op == "append":
        pa.append_kv_q4(st["k_new"], st["v_new"], st["q4"], table, ctx, workspace=ws)
        return list(pa.gather_kv_q4(st["q4"], table, ctx, c["L"], tail=True,
                                    dtype=st["k_new"].dtype, workspace=ws))
    if op == "evict":
        if c["pool"] == "q4":
            new = pa.evict_kv_q4(st["q4"], table, ctx, st["weights"], c["keep"], c["recent"],
                                 st["dst"], workspace=ws)
            rows = list(pa.gather_kv_q4(st["q4"], st["dst"], new.context_lens, c["keep"],
                                        workspace=ws))
        else:
            new = pa.evict_kv(*st["pool"], table, ctx, st["weights"], c["keep"], c["recent"],
                              st["dst"], workspace=ws)
            rows = list(st["pool"])
        return rows + [new.context_lens, new.key_weights, new.kept]
    if op == "attend":
        return pa.paged_attention_q4(st["query"], st["q4"], table, ctx, ps, st["scale"],
                                     c["causal"], workspace=ws)
    weights = torch.empty_like(st["weights"])
    if c["pool"] == "q4":
        out = pa.paged_attention_q4(st["query"], st["q4"], table, ctx, ps, st["scale"],
                                    c["causal"], key_weights=st["weights"],
                                    key_weights_out=weights, workspace=ws)
    else:
        out = pa.paged_attention_weights(st["query"], *st["pool"], table, ctx, ps, st["scale"],
                                         c["causal"], key_weights=st["weights"],
                                         key_weights_out=weights, workspace=ws)
    return out, weights


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


def _exact_rows(st, parts, table, b, pos):
    """fp64 rows [H_kv, n, 128] of sequence b at positions pos [n]."""
    pg = table[b].long()[pos // st["ps"]]
    rows = [t.transpose(1, 2)[pg, pos % st["ps"]].transpose(0, 1) for t in parts]
    if len(rows) == 1:
        return rows[0].double()
    byte = rows[0].int()
    code = torch.stack((byte % 16, byte // 16), -1).reshape(*byte.shape[:-1], D)
    mag = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[(code % 8).long()]
    val = torch.where(code >= 8, -mag, mag).reshape(*byte.shape[:-1], 8, GROUP)
    return (val * _e4m3_values()[rows[1].long()][..., None]).reshape(*byte.shape[:-1], D)


def exact(case, seed):
    st = prepare(case, seed)
    B, H, G, L = case["B"], case["H_kv"], case["G"], case["L"]
    half = len(st["pool"]) // 2
    if case["op"] == "append":
        return [_exact_round(x.double()) for x in (st["k_new"], st["v_new"])]
    if case["op"] == "evict":
        keep, recent, w = case["keep"], case["recent"], st["weights"].cpu().numpy()
        kept = np.full((B, H, keep), -1, np.int32)
        weights = np.zeros((B, H, keep))
        for b, S in enumerate(st["lens"]):
            n, last = min(S, keep), min(recent, S)
            for h in range(H):
                order = np.lexsort((np.arange(S - last), -w[b, h, :S - last].astype(np.float64)))
                at = np.sort(np.append(order[:n - last], np.arange(S - last, S)))
                kept[b, h, :n] = at
                weights[b, h, :n] = w[b, h, at]
        if case["pool"] == "q4":
            rows = [torch.zeros(B, H, keep, D, dtype=torch.float64, device="cuda") for _ in "kv"]
        else:
            rows = [t.double() for t in st["pool"]]
        for b, S in enumerate(st["lens"]):
            n = min(S, keep)
            at = torch.arange(n, device="cuda")
            to = st["dst"][b].long()[at // st["ps"]]
            for i in range(2):
                all_rows = _exact_rows(st, st["pool"][i * half:(i + 1) * half], st["table"], b,
                                       torch.arange(S, device="cuda"))
                for h in range(H):
                    src = torch.from_numpy(kept[b, h, :n]).cuda().long()
                    if case["pool"] == "q4":
                        rows[i][b, h, :n] = all_rows[h, src]
                    else:
                        rows[i][to, h, at % st["ps"]] = all_rows[h, src]
        lens = np.minimum(np.array(st["lens"], np.int32), keep)
        return rows + [lens, weights, kept]
    out = torch.empty(B, H * G, L, D, dtype=torch.float64, device="cuda")
    weights = torch.zeros(B, H, st["cap"], dtype=torch.float64, device="cuda")
    for b, S in enumerate(st["lens"]):
        pos = torch.arange(S, device="cuda")
        K = _exact_rows(st, st["pool"][:half], st["table"], b, pos)
        V = _exact_rows(st, st["pool"][half:], st["table"], b, pos)
        last = S - L + torch.arange(L, device="cuda") if case["causal"] else \
            torch.full((L,), S - 1, device="cuda")
        for h in range(H * G):
            x = st["query"][b, h].double() @ K[h // G].T * st["scale"]
            x[pos[None, :] > last[:, None]] = -math.inf
            p = torch.softmax(x, -1)
            out[b, h] = p @ V[h // G]
            weights[b, h // G, :S] += p.sum(0)
        if case["op"] == "weigh":
            weights[b, :, :S] += st["weights"][b, :, :S].double()
    return out if case["op"] == "attend" else (out, weights)
