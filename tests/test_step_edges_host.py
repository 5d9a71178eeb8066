"""Sizes at the edge of what the training step's operators take, checked on the host."""
import ctypes

import pytest
import torch

# the addresses are made up, so a check that let one through must not find a device
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks, run without a GPU")


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_grouped_gemm_gb300 as m
    return m


@pytest.mark.parametrize("T,k,code", [(2 ** 26 - 64, 32, 0), (2 ** 26 - 63, 32, 2), (2 ** 26 - 1, 32, 2),
                                      (2 ** 27 - 1, 16, 2), (2 ** 27 - 128, 16, 0)])
def test_route_grad_of_nearly_2_31_choices(moe, T, k, code):
    """Places in the lists have 32 bits and run up to a segment of 1024 choices past the last one."""
    c, n = moe.Cfg(T, 128, 64, k, 1, 1, 128, 0, 1, 2.5, moe.MOE_BF16, moe.MOE_BF16), ctypes.c_size_t(0)
    assert moe.validate(c) == 0
    L, at = moe._lib, [(i + 1) << 40 for i in range(9)]
    assert L.moe_route_grad_query(ctypes.byref(c), ctypes.byref(n)) == code
    if code:
        assert L.moe_route_grad(ctypes.byref(c), *at[:8], 0, at[8], None) == code
