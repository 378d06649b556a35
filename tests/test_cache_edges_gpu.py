"""The cache operators where their kernels' parts meet: hand-overs between the
roles of a CTA, states that cross shares, values at the ends of the types."""
import numpy as np
import pytest

import cache_ref as ref
from cache_ref import Case
from paged_kv_cache_03_gb300 import binding as B
from test_cache_paths_gpu import attend, check, spread, workspace

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
