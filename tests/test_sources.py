"""What the library's sources may not hold (CPU only)."""
import glob
import os

HERE = os.path.dirname(os.path.abspath(__file__))


def test_no_multicast_loads():
    """One library serves every process, whatever memory its pool pointers name, so no
    copy and no arrival goes to several CTAs at once."""
    files = glob.glob(os.path.join(HERE, "..", "paged_kv_cache_03_gb300", "csrc", "*.cu*"))
    assert len(files) > 10
    for f in files:
        with open(f) as src:
            assert ".multicast" not in src.read(), os.path.basename(f)
