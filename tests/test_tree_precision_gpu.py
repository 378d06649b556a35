"""The attention of draft trees over fp32 operands against its 64-bit form, by the root mean
square of the error: a worst case counts every rounding at its largest and leaves room for a lost
half of an operand, the mean square does not (tests/test_tree_precision_cpu.py)."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from tree_precision import LIMIT, rms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool", ["f32", "q4"])
@pytest.mark.parametrize("G,H,L,ps,ctx", [
    (4, 2, 1, 16, [2, 300]), (4, 2, 16, 128, [16, 129, 900]), (3, 2, 13, 12, [13, 200, 900]),
    (4, 2, 64, 8, [64, 65, 2000]), (1, 3, 300, 128, [300, 431, 1000]), (2, 4, 3, 16, [8000]),
    (4, 8, 16, 16, [100 + 61 * i for i in range(20)])], ids=str)
def test_two_parts(pool, G, H, L, ps, ctx):
    inp = tr.Inputs(tr.Case(G, H, L, ps, ctx, pool, "f32", seed=L))
    want, _ = tr.attend(inp)
    got = tr.call(inp, inp.device()).double().cpu().numpy()
    assert rms(got, want) <= LIMIT


def long_pieces(pool):
    """20 sequences of 8 kv heads and the same 8000 keys: a CTA has thousands of keys of a row."""
    inp = tr.Inputs(tr.Case(1, 8, 2, 128, [8000], pool, "f32", seed=1))
    rng = np.random.default_rng(2)
    inp.q = rng.standard_normal((20, 8, 2, 128)).astype(np.float32) * 1.5
    inp.ctx = np.full(20, 8000, np.int32)
    for name in ("table", "see", "mask", "drafted"):
        setattr(inp, name, getattr(inp, name).repeat(20, 0))
    return inp


@pytest.mark.parametrize("pool", ["f32", "q4"])
def test_long_contexts(pool):
    """Sums over thousands of keys are not cut: what the tensor cores cut grows with their number."""
    inp = long_pieces(pool)
    want, _ = tr.attend(inp)
    got = tr.call(inp, inp.device()).double().cpu().numpy()
    assert rms(got, want) <= LIMIT


@pytest.mark.parametrize("pool", ["f32", "q4"])
def test_long_contexts_of_climbing_scores(pool):
    """The same where the maximum moves on the way: scores climb by 28 powers of two in all."""
    inp = long_pieces(pool)
    inp.q[..., 0] = 8
    at = np.arange(8000)
    page, slot = inp.table[0, at // 128], at % 128
    x = np.zeros((8000, 8, 128), np.float32)  # of which the first 16 dims are taken
    x[..., 0] = (at // 400 * 1.4)[:, None]  # 8 * 26.6 / sqrt(128) = 18.8
    if pool == "q4":
        codes, scales = ref.quantise(x)
        inp.raw[0][page, :, slot, :8], inp.raw[1][page, :, slot, 0] = codes[..., :8], scales[..., 0]
        x = ref.dequantise(codes, scales)
    else:
        inp.raw[0][page, :, slot, :16] = x[..., :16]
    inp.dense[0][page, :, slot, :16] = x[..., :16]
    want, tol = tr.attend(inp)
    got = tr.call(inp, inp.device()).double().cpu().numpy()
    assert ref.worst(got, want, tol) <= 1.0
    # scores of 20 cut at 24 additions: 20 * 24 * 2^-25 beside what LIMIT counts
    assert rms(got, want) <= LIMIT + 20 * 24 * 2.0 ** -25
