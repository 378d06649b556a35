"""The limit of tests/test_tree_precision_gpu.py: two parts of every operand keep it with room to
spare, and an operand that has lost its low part breaks it (CPU only)."""
import numpy as np
import pytest

import tree_precision as tp


def inputs(S, rows=16):
    rng = np.random.default_rng(S)
    q, k, v = (rng.standard_normal((n, 128)).astype(np.float32).astype(np.float64) * m
               for n, m in ((rows, 1.5), (S, 1.5), (S, 1.0)))
    x = q @ k.T / np.sqrt(128)
    p = np.exp(x - x.max(-1, keepdims=True))
    return q, k, v, 1 / np.sqrt(128), p @ v / p.sum(-1, keepdims=True)


@pytest.mark.parametrize("S", [40, 300, 2000, 8000])
def test_a_lost_part_breaks_the_limit(S):
    q, k, v, scale, want = inputs(S)
    assert tp.rms(tp.attend(q, k, v, scale), want) <= tp.LIMIT / 4
    for lost in "qkvp":
        assert tp.rms(tp.attend(q, k, v, scale, lost), want) >= 8 * tp.LIMIT, lost
