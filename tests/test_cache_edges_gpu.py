"""The cache operators where their kernels' parts meet: hand-overs between the
roles of a CTA, states that cross shares, values at the ends of the types."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B
from test_cache_paths_gpu import PATHS, attend, check, spread, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("c", [
    # one query tile; pieces of one key tile (no second half to join), of two, of three,
    # several of them a CTA, in changing order
    Case(300, 8, 2, 8, 16, spread(300, 8, 128)),
    Case(300, 8, 2, 8, 16, spread(300, 8, 256)),
    Case(260, 8, 2, 8, 16, [[100, 300, 120, 200, 60][i % 5] for i in range(260)]),
    Case(260, 4, 2, 17, 16, [[100, 300, 300, 90][i % 4] for i in range(260)], pool="bf16"),
], ids=str)
def test_short_pieces_of_one_query_tile(c):
    import torch
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    out, w = attend(inp, d, ws)
    check(inp, out, w)
    for _ in range(40):
        again = attend(inp, d, ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], w)
    assert B.pa_check_device_flag(ws)[1] == 0


def test_evictions_back_to_back():
    """Evictions without a wait between them, their outputs in the same memory:
    each copies the rows that its own selection chose."""
    import torch
    c = Case(8, 1, 4, 1, 16, spread(8, 200, 900), pool="bf16")
    keep, n = 128, 24
    inp = ref.Inputs(c, extra_pages=8 * 8)
    d = inp.device()
    dst = torch.from_numpy(inp.free[:64].reshape(8, 8).astype(np.int32)).cuda()
    ws = B.new_cache_workspace()
    rng = np.random.default_rng(11)
    ws_in = [torch.from_numpy(rng.random(inp.w.shape).astype(np.float32)).cuda() for _ in range(n)]
    torch.cuda.synchronize()
    got = []
    for w in ws_in:
        new = B.evict_kv(*d["pool"], d["table"], d["ctx"], w, keep, 16, dst, workspace=ws)
        got.append((new.kept.clone(), [t[dst.long()].clone() for t in d["pool"]]))
        del new
    b, h = np.arange(8)[:, None, None], np.arange(4)[None, :, None]
    at = np.arange(keep)
    for w, (kept, rows) in zip(ws_in, got):
        want, _ = ref.evict(w.cpu().numpy(), c.ctx, keep, 16)
        assert np.array_equal(kept.cpu().numpy(), want)
        for t, x in zip(d["pool"], rows):
            src = t[inp.table[b, want // 16], h, want % 16]
            assert torch.equal(x[b, at // 16, h, at % 16].view(torch.uint8), src.view(torch.uint8))


def test_fp32_weights_back_to_back():
    """fp32 queries one after the other through one workspace, without a wait:
    the weights are those of each query, not of the one before."""
    import torch
    c = Case(3, 4, 2, 12, 16, [300, 90, 500], dtype="f32")
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    rng = np.random.default_rng(4)
    qs = [rng.standard_normal(inp.q.shape).astype(np.float32) * 1.5 for _ in range(6)]
    dev = [torch.from_numpy(q).cuda() for q in qs]
    torch.cuda.synchronize()
    got = []
    for q in dev + dev:
        d["q"] = q
        got.append(attend(inp, d, ws))
    for q, first, again in zip(qs, got, got[6:]):
        inp.q = q
        check(inp, *first)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def one_heavy_key(Bn, G, L, n, dtype, gap):
    """Bn sequences over the same n keys of one kv head, all values 1: key n // 3
    scores `gap` log2 units, the others 0.  Every output is exactly 1."""
    import torch
    ps = 128
    P = n // ps
    codes = torch.zeros(P, 1, ps, 64, dtype=torch.uint8, device="cuda")
    scales = torch.full((P, 1, ps, 8), 0x38, dtype=torch.uint8, device="cuda")  # 1.0
    codes[(n // 3) // ps, 0, (n // 3) % ps] = 0x22                              # 1.0, twice
    values = torch.full_like(codes, 0x22)
    pool = B.Q4Pool(codes, scales, values, scales.clone())
    table = torch.arange(P, dtype=torch.int32, device="cuda").repeat(Bn, 1)
    ctx = torch.full((Bn,), n, dtype=torch.int32, device="cuda")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    q = torch.ones(Bn, G, L, 128, device="cuda").to(dt)
    scale = float(np.float32(gap * np.log(2) / 128))
    out = B.paged_attention_q4(q, pool, table, ctx, ps, scale, False)
    return float((out.double() - 1).abs().max())


# log2 units below the heaviest key: f16 has steps of 2^-24 at its lower end
@pytest.mark.parametrize("gap", [22.3, 25.5, 30.0])
@pytest.mark.parametrize("Bn,L,n", [(640, 1, 32768), (320, 16, 32768), (2, 1, 4096)],
                         ids=["walk", "block", "short"])
def test_many_light_keys_fp32(Bn, L, n, gap):
    """Counted: the two parts of a weight 2^-22; a row sum and an O that take n / 64 sums of
    a step, each add off by 2^-24; a step's products, 68 terms cut by 2^-23; joining lanes,
    warps and shares, 64 adds.  (Weights below f16's steps, if they were lost, would be a
    quarter of 32768 * 2^-25.5 in the heaviest key's warp: 1.7e-4.)"""
    tol = 2.0 ** -22 + (2 * n / 64 + 64) * 2.0 ** -24 + 68 * 2.0 ** -23
    assert one_heavy_key(Bn, 4, L, n, "f32", gap) <= tol


@pytest.mark.parametrize("L", [1, 16, 65])
def test_many_light_keys_bf16(L):
    """bf16 queries: 2^15 keys that weigh 2^-25.5 are 2^-10.5 of the row; lost or not, the
    output is within half a step of 1."""
    assert one_heavy_key(160, 4, L, 32768, "bf16", 25.5) <= 2.0 ** -8


# every path, its states whole and cut over shares, key chunks and remainder rows
NAN_CASES = [(c, True) for c in PATHS] + [(c, False) for c in PATHS if c.pool == "q4"] + [
    (Case(1, 4, 1, 1, 16, [3900]), True),
    (Case(1, 4, 1, 3, 16, [3900], pool="bf16"), True),
    (Case(1, 4, 1, 13, 16, [3900], dtype="f32"), True),
    (Case(1, 4, 1, 32, 16, [3900]), True),
    (Case(1, 4, 1, 65, 16, [3900], pool="bf16"), True),
    (Case(1, 2, 1, 200, 16, [310]), False),              # whole prompts, keys cut in chunks
    (Case(1, 4, 1, 130, 16, [600]), False),              # ... and a last tile of few rows
    (Case(2, 2, 2, 40, 8, [300, 120], causal=False), True),
]


@pytest.mark.parametrize("c,weights", NAN_CASES, ids=str)
@pytest.mark.parametrize("where", ["query", "key"])
def test_nan_rows(where, c, weights):
    """A row whose query, or a key it sees, holds a NaN is NaN on every path, and so are the
    weights of the keys it sees; nothing else changes."""
    import torch
    if where == "key" and not c.causal:
        return  # every row sees every key
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    out, w = attend(inp, d, ws, weights)
    S, L = c.ctx[0], c.L
    pos = np.arange(L) + (S - L if c.causal else S)  # the last key that a row of sequence 0 sees
    rows = np.zeros((c.B, c.H_kv, c.G, L), bool)
    if where == "query":
        rows[0, c.H_kv - 1, c.G // 2, 0] = rows[0, 0, 0, L // 2] = rows[0, 0, c.G - 1, L - 1] = True
        d["q"] = d["q"].clone()
        d["q"].view(c.B, c.H_kv, c.G, L, 128)[torch.from_numpy(rows).cuda()] = float("nan")
    else:
        k = S - 1 - L // 2
        rows[0, 0] = pos >= k
        page, slot = inp.table[0, k // c.ps], k % c.ps
        if c.pool == "q4":
            d["pool"].key_scales[page, 0, slot] = 0x7f
        else:
            d["pool"][0][page, 0, slot] = float("nan")
    got, got_w = attend(inp, d, ws, weights)
    assert B.pa_check_device_flag(ws)[1] == 0
    bad = torch.from_numpy(rows.reshape(c.B, c.H_kv * c.G, L)).cuda()
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], out[~bad])
    if weights:
        far = np.where(rows, pos, -1).max((2, 3))  # the last key that a NaN row sees
        bad = np.arange(inp.cap) <= far[:, :, None]
        bad &= np.arange(inp.cap) < inp.ctx[:, None, None]
        bad = torch.from_numpy(bad).cuda()
        assert torch.isnan(got_w[bad]).all() and torch.equal(got_w[~bad], w[~bad])


@pytest.mark.parametrize("pool,dtype", [("q4", "bf16"), ("q4", "f32"), ("bf16", "bf16")])
def test_one_workspace_for_every_smaller_call(pool, dtype):
    """Sized for the largest batch, chunk and table, a workspace serves the decode steps,
    short chunks, small batches and narrow tables."""
    def case(Bn, L, spare):
        return Case(Bn, 4, 2, L, 16, spread(Bn, L, 300), pool=pool, dtype=dtype, spare=spare)
    big = case(16, 65, 1000)
    ws = workspace(big, ref.Inputs(big).device())
    for c in (big, case(16, 1, 1000), case(3, 2, 1000), case(16, 8, 60), case(1, 16, 3), case(2, 33, 0),
              case(16, 1, 0)):
        inp = ref.Inputs(c)
        d = inp.device()
        for weights in ((True, False) if pool == "q4" else (True,)):
            out, w = attend(inp, d, ws, weights)
            check(inp, out, w)
    assert B.pa_check_device_flag(ws)[1] == 0


def test_workspace_sizes_are_monotone():
    """pa_*_workspace_bytes of any shape with at most the B, L and table of another."""
    rng = np.random.default_rng(8)
    for _ in range(300):
        G, H = int(rng.choice([1, 2, 4, 7, 8, 16, 48, 130])), int(rng.choice([1, 2, 8]))
        dtype, ps = int(rng.choice([B.PA_BF16, B.PA_F32])), int(rng.choice([1, 12, 16, 128]))
        top = [int(np.exp(rng.uniform(0, np.log(m)))) for m in (500, 5000, 100000 // ps)]

        def sizes(Bn, L, n):
            sh = B.make_shape(Bn, G * H, H, L, 128, 1000, ps, n, dtype)
            got = [B.pa_q4_workspace_bytes(sh, False), B.pa_q4_workspace_bytes(sh, True)]
            return got + ([B.pa_weights_workspace_bytes(sh)] if dtype == B.PA_BF16 else [])
        most = sizes(*top)
        assert min(most) > 0
        for _ in range(20):
            less = [int(rng.integers(1, m + 1)) if rng.random() < 0.7 else m for m in top]
            assert all(a <= b for a, b in zip(sizes(*less), most))


@pytest.mark.parametrize("pool,dtype", [("q4", "bf16"), ("q4", "f32"), ("bf16", "bf16")])
def test_weights_of_few_rows_over_very_wide_tables(pool, dtype):
    """A table of 2 million slots a sequence: the scores are not stored (4 bytes a row and
    slot would pass 512 MiB), the weights are the same."""
    c = Case(4, 8, 2, 1, 128, [300, 1, 129, 1000], pool=pool, dtype=dtype, spare=16400)
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    assert 4 * 2 * 8 * inp.cap * 4 > 2 ** 29 >= ws.numel() - 2 ** 26
    out, w = attend(inp, d, ws)
    check(inp, out, w)
    again = attend(inp, d, ws)
    assert (again[0] == out).all() and (again[1] == w).all()
    assert B.pa_check_device_flag(ws)[1] == 0


def test_whole_prompts_in_groups():
    """Whole prompts whose bf16 copies do not fit together (tables of 65536 slots and 8 kv
    heads: 268 MB a sequence, 1 GiB in all): six sequences go as four and two.  Every
    sequence is as in a call of its group alone, and against 64 bits; a bad length and a bad
    page in the second group stay where they are."""
    import torch
    H, G, L, ps, n = 8, 16, 2048, 128, 512
    ctx = [2048, 2500, 4100, 3001, 2222, 2600]
    gen = torch.Generator(device="cuda").manual_seed(1)
    npg = [-(-s // ps) for s in ctx]
    P = sum(npg) + 3
    perm = torch.randperm(P, generator=gen, device="cuda").int()
    table = torch.full((6, n), -9, dtype=torch.int32, device="cuda")
    at = 0
    for b, k in enumerate(npg):
        table[b, :k] = perm[at:at + k]
        at += k
    pool = B.new_q4_pool(P, H, ps)
    for t in (pool.key_codes, pool.value_codes):
        t.copy_(torch.randint(0, 256, t.shape, generator=gen, device="cuda"))
    for t in (pool.key_scales, pool.value_scales):  # 0.25 .. 0.94
        t.copy_(torch.randint(0x28, 0x38, t.shape, generator=gen, device="cuda"))
    q = torch.randn(6, H * G, L, 128, generator=gen, device="cuda").bfloat16()
    lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ws = B.new_q4_workspace(q, pool, table, False)
    assert ws.numel() > 4 * n * ps * H * 512

    def call(b0, b1, table=table, lens=lens):
        return B.paged_attention_q4(q[b0:b1], pool, table[b0:b1], lens[b0:b1], ps, workspace=ws)
    out = call(0, 6)
    assert torch.equal(call(0, 4), out[:4]) and torch.equal(call(4, 6), out[4:])
    assert B.pa_check_device_flag(ws)[1] == 0

    def against_64_bits(out, table, seqs):
        K, V = B.gather_kv_q4(pool, table, lens, max(ctx), dtype=torch.float32)
        for b in seqs:
            for h, l in ((0, 0), (G + 3, 1000), (H * G - 1, L - 1)):
                S = ctx[b] - L + l + 1
                k, v = K[b, h // G, :S].double(), V[b, h // G, :S].double()
                x = q[b, h, l].double()
                p = torch.softmax(k @ x * float(np.float32(128 ** -0.5)), 0)
                T = float((k.abs() @ x.abs()).max()) * 128 ** -0.5
                want = p @ v
                # roundings as in cache_ref.attend: scores, P in bf16 and in its sum, the output
                tol = (T * 2.0 ** -15 + 2.0 ** -12 + 2.0 ** -7) * (p @ v.abs()) + 2.0 ** -8 * want.abs() + \
                    2.0 ** -25 * p.max() * v.abs().sum(0)
                assert ((out[b, h, l].double() - want).abs() <= tol).all(), (b, h, l)
    against_64_bits(out, table, range(6))
    bad = lens.clone()
    bad[5] = n * ps + 1
    got = call(0, 6, lens=bad)
    assert B.pa_check_device_flag(ws, clear=True)[1] == B.PA_FLAG_BAD_CONTEXT
    assert torch.equal(got[:5], out[:5]) and not got[5].any()
    hole = table.clone()
    hole[4, 3] = P + 7
    got = call(0, 6, table=hole)
    assert B.pa_check_device_flag(ws, clear=True)[1] == B.PA_FLAG_BAD_PAGE
    assert torch.equal(got[:4], out[:4]) and torch.equal(got[5], out[5])
    against_64_bits(got, hole, [4])


@pytest.mark.parametrize("pool", ["q4", "bf16"])
def test_evicted_weights_go_on_without_a_copy(pool):
    """key_weights_out of an eviction is the key_weights of the next attention call."""
    import torch
    c = Case(3, 4, 2, 1, 16, [300, 40, 500], pool=pool)
    inp = ref.Inputs(c, extra_pages=3 * 5)
    d = inp.device()
    dst = torch.from_numpy(inp.free[:15].reshape(3, 5).astype(np.int32)).cuda()
    evict = B.evict_kv_q4 if pool == "q4" else B.evict_kv
    pages = (d["pool"],) if pool == "q4" else d["pool"]
    args = (*pages, d["table"], d["ctx"], d["w"], 60, 7, dst)
    plain = evict(*args)
    w2 = torch.full((3, 2, 80), float("nan"), device="cuda")
    new = evict(*args, key_weights_out=w2)
    assert new.key_weights is w2 and torch.equal(w2[:, :, :60], plain.key_weights)
    assert not w2[:, :, 60:].any() and torch.equal(new.kept, plain.kept)
    assert plain.key_weights.shape == (3, 2, 60)
    # the attention that follows, with w2 in place and with a copy
    copy = torch.nn.functional.pad(plain.key_weights, (0, 20))
    d["table"], d["ctx"] = dst, new.context_lens
    call = B.paged_attention_q4 if pool == "q4" else B.paged_attention_weights
    outs = [call(d["q"], *pages, dst, new.context_lens, 16, key_weights=w, key_weights_out=w)
            for w in (w2, copy)]
    assert torch.equal(*outs) and torch.equal(w2, copy)
    for bad in (w2[:, :, :59].contiguous(), w2.double(), w2[:2].contiguous(), w2.cpu(),
                w2.transpose(0, 1).contiguous().transpose(0, 1)):
        with pytest.raises(ValueError):
            evict(*args, key_weights_out=bad)
    with pytest.raises(B.PagedAttentionError):  # not in place
        evict(*args, key_weights_out=d["w"])


def test_streams_as_raw_handles():
    """A raw handle, 0 (the default stream) and a stream object, from another current stream."""
    import torch
    c = Case(2, 4, 2, 1, 16, [300, 1900])
    inp = ref.Inputs(c)
    d = inp.device()
    ws = workspace(c, d)
    want = attend(inp, d, ws)
    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(other):
        for stream in (side, side.cuda_stream, 0):
            got = attend(inp, d, ws, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_small_rows_scaled_by_a_power_of_two():
    """Values of a few thousandths are below the scales' range; stored times 2^10, with the key's
    factor taken out of `scale` and the value's out of the output, the attention is that of
    rows 0.18 of a group's largest value off at most."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    k, v = normal(1, 2, 200, 128) * 2.0 ** -9, normal(1, 2, 200, 128) * 2.0 ** -9
    q = (normal(1, 8, 1, 128) * 2.0 ** 9).bfloat16()
    table = torch.arange(13, dtype=torch.int32, device="cuda").view(1, 13)
    ctx = torch.tensor([200], dtype=torch.int32, device="cuda")
    scale = 128 ** -0.5
    pool = B.new_q4_pool(13, 2, 16)
    B.append_kv_q4(k * 1024, v * 1024, pool, table, ctx)
    K, V = (t.double() / 1024 for t in B.gather_kv_q4(pool, table, ctx, 200, dtype=torch.float32))
    for stored, x in ((K, k), (V, v)):
        a = x.view(1, 2, 200, 8, 16).abs().amax(-1, keepdim=True)
        assert ((stored - x).view(1, 2, 200, 8, 16).abs() <= 0.18 * a).all()
    out = B.paged_attention_q4(q, pool, table, ctx, 16, scale / 1024).double() / 1024
    s = q.double().view(1, 2, 4, 128) @ K.transpose(2, 3) * scale
    p = torch.softmax(s, -1)
    T = (q.double().abs().view(1, 2, 4, 128) @ K.abs().transpose(2, 3) * scale).amax(-1, keepdim=True)
    tol = (T * 2.0 ** -15 + 2.0 ** -11 + 2.0 ** -12) * (p @ V.abs()) + 2.0 ** -8 * (p @ V).abs() + \
        2.0 ** -25 * p.amax(-1, keepdim=True) * V.abs().sum(2, keepdim=True)
    assert ((out.view(1, 2, 4, 128) - p @ V).abs() <= tol).all()


@pytest.mark.parametrize("G,L,status", [(1, 2 ** 27, B.PA_ERR_UNSUPPORTED), (8, 2 ** 24, B.PA_ERR_UNSUPPORTED),
                                        (1, 2 ** 27 - 1, B.PA_ERR_WORKSPACE)])
def test_too_many_rows_for_the_weights(G, L, status):
    """Refused on the host.  (No workspace: nothing could be launched in any case.)"""
    fake = 1 << 20
    sh = B.make_shape(1, G, 1, L, 128, 16, 16, 8, B.PA_F32)
    st = B.pa_paged_attention_q4(sh, fake, (fake,) * 4, fake, fake, 0.1, 0, None, fake, 128, fake,
                                 fake, 0, 0)
    assert st == status
