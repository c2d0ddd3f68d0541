"""Sizes at the ends of what the kernels index (no GPU: the calls are refused
on the host)."""
import ctypes

import pytest

NULL = None


@pytest.fixture(scope="module")
def bsq():
    from block_scaled_precision_03_gb300 import _build
    import block_scaled_precision_03_gb300 as b
    _build.build()
    b.lib()
    return b


@pytest.mark.parametrize("cols", [(1 << 30) + 1, (1 << 31) - 300, (1 << 31) - 256, 1 << 31, 1 << 40])
def test_expert_rows_wider_than_the_kernels_count(bsq, cols):
    # the kernels count a row's elements in 32 bits and look up to 622592 elements past the last one
    # they move (4 steps of 128 threads in 1216 pieces), which has to stay below 2^31
    L = bsq.lib()
    from block_scaled_precision_03_gb300.ops import BsqMoePlanC as Plan
    plan, n = ctypes.byref(Plan(1, 1, 1, 256, 256, 256)), cols
    assert L.bsq_moe_gather(256, n, 1, n, plan, 256, n, NULL) == 2
    assert L.bsq_moe_dispatch(256, n, 1, n, 256, 1, plan, 256, n, NULL, 0, NULL) == 2
    assert L.bsq_moe_combine(256, n, 1, n, 256, plan, 256, n, NULL) == 2
    assert L.bsq_moe_combine_backward(256, n, 256, n, 1, n, 256, plan, 256, n, 256, NULL) == 2
