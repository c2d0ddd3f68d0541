"""Rules on the kernels' sources that no run shows."""
import os

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_03_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.listdir(CSRC)))
def test_no_tma_load_is_a_multicast(name):
    # the kernels run as replicas on several GPUs too, where a load into several CTAs may not be used
    # (a commit that signals both CTAs of a pair is no load)
    with open(os.path.join(CSRC, name)) as f:
        for line in f:
            assert not ("cp.async.bulk" in line and "multicast::cluster" in line), line
