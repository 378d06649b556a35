"""The attention of draft trees where numbers are large."""
import numpy as np
import pytest

import cache_ref as ref
import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

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
