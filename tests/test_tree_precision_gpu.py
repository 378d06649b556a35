"""The attention of draft trees over fp32 operands against its 64-bit form, by the root mean
square of the error: a worst case counts every rounding at its largest and leaves room for a lost
half of an operand, the mean square does not (tests/test_tree_precision_cpu.py)."""
import pytest

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
