"""Sizes of draft trees and of shared pages that a C int does not hold (CPU only)."""
import pytest

from paged_kv_cache_03_gb300 import binding as B


@pytest.mark.parametrize("n", [0, -1, 1 << 31, (1 << 32) + 16])
def test_sizes(n):
    import torch

    def z(*s, dtype=torch.int32):
        return torch.zeros(s, dtype=dtype)
    with pytest.raises(ValueError, match="page_size"):
        B.fork_pages(z(4, 2), z(4), z(9), z(2), z(2), n)
    with pytest.raises(ValueError, match="page_size"):
        B.resize_pages(z(4, 2), z(4), z(9), z(4), n)
    with pytest.raises(ValueError, match="L must"):
        B._compact("", None, (), (4, 2, 16), B.PA_BF16, torch.device("cpu"), z(2, 2), z(2), z(2, 3), z(2), n, None)
