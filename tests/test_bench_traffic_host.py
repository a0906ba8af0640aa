"""The captured DRAM traffic that the bench line quotes belongs to the GEMM source that is there."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("workload", ["kimi_T8192", "dsv4", "kimi_T16", "small_T32", "small_T1", "tiny"])
def test_the_captures_are_of_the_gemm_that_is_built(workload):
    """An edit of the GEMM's source, of its kernels or not, leaves the roofline without its traffic until the captures
    are taken again: what other operators need of it goes into their own sources."""
    sys.path.insert(0, ROOT)
    import bench

    assert bench.fc1_traffic(workload) is not None
