"""As many pages as a shape can have."""
import pytest

from paged_kv_cache_03_gb300 import binding as B

pytestmark = pytest.mark.gpu


def test_no_free_page_among_the_most():
    """2^31 - 1 pages of one slot, all held but for the last: the search for free ones ends there."""
    import torch
    P = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 16 * P + (4 << 30):
        pytest.skip("not enough free memory")
    i32 = dict(dtype=torch.int32, device="cuda")
    refs = torch.ones(P, **i32)
    refs[-1] = 0
    table, ctx = torch.full((3, 2), -1, **i32), torch.zeros(3, **i32)
    ws = B.new_pages_workspace(table, refs)
    copies = B.resize_pages(table, ctx, refs, torch.tensor([1, 1, 2], **i32), 1, workspace=ws)
    assert B.pa_check_device_flag(ws)[1] == B.PA_FLAG_NO_PAGES
    assert table.tolist() == [[P - 1, -1], [-1, -1], [-1, -1]] and ctx.tolist() == [1, 0, 0]
    assert copies.tolist() == [[-1, -1, 0]] * 3 and int(refs[-1]) == 1
