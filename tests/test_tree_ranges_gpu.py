"""The attention of draft trees where numbers are large."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B
from tree_precision import LIMIT, rms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pool,L,ps,ctx", [
    ("bf16", 8, 16, [300, 200]),     # whole segments
    ("bf16", 8, 16, [3000, 900]),    # cut and merged
    ("bf16", 64, 16, [1500, 700]),   # two query tiles side by side
    ("bf16", 8, 12, [900, 300]),     # pages that are not a multiple of 8
    ("f32", 8, 16, [900, 300]),
])
def test_large_values_behind_climbing_scores(pool, L, ps, ctx):
    """Values near 2^100, and scores that rise by 60 powers of two behind the first 128 keys:
    sums of weights times values stay numbers all the same."""
    inp = tr.Inputs(tr.Case(4, 2, L, ps, ctx, pool, pool, seed=21))
    inp.q[..., 0] = 16
    for b, S in enumerate(ctx):
        at = np.arange(S)
        page, slot = inp.table[b, at // ps], at % ps
        for t in (inp.raw[0], inp.dense[0]):  # 16 * 29.5 / sqrt(128) = 41.7 = 60.2 ln 2
            t[page, :, slot, 0] = np.where(at < 128, 0, 29.5)[:, None]
    inp.raw[1] *= np.float32(2.0 ** 100)
    inp.dense[1] *= 2.0 ** 100
    want, tol = tr.attend(inp)
    d = inp.device()
    ws = B.new_tree_workspace(d["q"], d["pool"][0], d["table"])
    got = tr.call(inp, d, workspace=ws).double().cpu().numpy()
    assert np.isfinite(got).all()
    assert ref.worst(got, want, tol) <= 1.0
    assert B.pa_check_device_flag(ws)[1] == 0


def test_rows_of_mixed_magnitude():
    """What an fp32 key or value row holds of its numbers does not hang on its neighbours', seen or
    not: in every eight rows of the context a value row 2^45 times as large whose key weighs 0,
    and among the drafts large ones on branches of their own."""
    L, S, ps = 24, 700, 16
    inp = tr.Inputs(tr.Case(4, 2, L, ps, [S], "f32", "f32", seed=5))
    inp.see[0] = np.eye(L, dtype=bool)  # every draft a root
    inp.mask = tr.words(inp.see)
    rng = np.random.default_rng(6)
    inp.q[:] = rng.standard_normal(inp.q.shape) * 1.5
    inp.q[..., 0] = 4
    at = np.arange(S)
    page, slot = inp.table[0, at // ps], at % ps
    K, V = (rng.standard_normal((S, 2, 128)).astype(np.float32) * m for m in (1.5, 1.0))
    heavy = at[(at % 8 == 3) & (at < S - L)]
    K[heavy] = 0
    K[heavy, :, 0] = -2.0 ** 20  # a score of -2^22 / sqrt(128)
    V[heavy] *= np.float32(2.0 ** 45)
    large = [1, 9, 17]
    K[S - L + np.array(large)] *= np.float32(2.0 ** 40)
    V[S - L + np.array(large)] *= np.float32(2.0 ** 45)
    inp.raw[0][page, :, slot], inp.raw[1][page, :, slot] = K, V
    rows = [i for i in range(L) if i not in large]
    want = np.zeros(inp.q.shape)
    for h in range(8):
        k, v = (t[:, h // 4].astype(np.float64) for t in (K, V))
        for i in rows:
            keys = np.append(np.arange(S - L), S - L + i)
            x = k[keys] @ inp.q[0, h, i].astype(np.float64) * inp.scale
            p = np.exp(x - x.max())
            want[0, h, i] = p @ v[keys] / p.sum()
    got = tr.call(inp, inp.device()).double().cpu().numpy()
    assert rms(got[:, :, rows], want[:, :, rows]) <= LIMIT
