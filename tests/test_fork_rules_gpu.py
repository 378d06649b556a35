"""Which forks of a call are made: every rule of the header by itself."""
import pytest

import tree_ref as tr
from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu

# rows of these lengths in pages of 8 slots; sources, targets, lens, and the rows that change
ROWS = [20, 9, 0, 0, 5, 0]
CALLS = {
    "a source that a made fork names": ([0, 2], [2, 3], None, {2: 20}),
    "... and the other way round": ([2, 0], [3, 2], None, {2: 20}),
    "a source that a refused fork names, its target not empty": ([0, 1], [1, 3], None, {}),
    "a source that a refused fork names, its own source out of range": ([6, 1], [1, 3], None, {}),
    "its own target": ([2, 0], [2, 3], None, {3: 20}),
    "a target named twice: the first has it": ([0, 1], [3, 3], None, {3: 20}),
    "... though it is not made": ([7, 1], [3, 3], None, {}),
    "... for its length": ([0, 1], [3, 3], [21, 9], {}),
    "a length above the source's": ([1, 0], [2, 3], [10, 20], {3: 20}),
    "a negative length": ([1, 0], [2, 3], [9, -1], {2: 9}),
    "no length": ([1, 0], [2, 3], [0, 17], {3: 17}),
    "rows out of range": ([0, -1, 0, 1], [-1, 2, 6, 3], None, {3: 9}),
    "a target that is not empty": ([0, 1], [4, 5], None, {5: 9}),
}


@pytest.mark.parametrize("name", CALLS)
def test_forks(name):
    import torch
    sources, targets, lens, made = CALLS[name]

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    sim = tr.Pages(6, 4, 16, 8)
    sim.resize(ROWS)
    table, ctx, refs = (ints(x) for x in (sim.table, sim.ctx, sim.refs))
    ws = B.new_cache_workspace()
    B.fork_pages(table, ctx, refs, ints(sources), ints(targets), 8, None if lens is None else ints(lens),
                 workspace=ws)
    assert ctx.tolist() == [made.get(b, S) for b, S in enumerate(ROWS)]
    for b, S in made.items():
        s = sources[targets.index(b)]
        n = -(-S // 8)
        sim.table[b, :n] = sim.table[s, :n]
        sim.refs[sim.table[s, :n]] += 1
    assert table.tolist() == sim.table.tolist() and refs.tolist() == sim.refs.tolist()
    refused = len(made) < len(sources) and name != "no length"
    assert B.pa_check_device_flag(ws)[1] == (B.PA_FLAG_BAD_CONTEXT if refused else 0)
