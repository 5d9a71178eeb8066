"""Sizes and arguments at the end of what the training calls take, checked on the host: nothing here
launches GPU work."""
import ctypes

import pytest

OK = 1 << 20   # an aligned address that the checks never dereference


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_grouped_gemm_gb300 as m
    return m


@pytest.mark.parametrize("size,code", [(2 ** 31 - 1, 2), (2 ** 31 - 512, 2), (2 ** 31 - 520, 0)])
@pytest.mark.parametrize("dim", ["rows", "n", "k"])
def test_sizes_that_leave_no_room_for_a_tile(moe, dim, size, code):
    """Tiles of up to 256 rows or columns and k-steps of 64 are counted in 32 bits: sizes that
    rounding up to them would carry past 2^31 are refused."""
    if dim != "rows":
        size = size // 8 * 8
    shape = {**dict(rows=16, E=4, n=8, k=8), dim: size}
    g, n = ctypes.byref(moe.GroupCfg(**shape)), ctypes.c_size_t(0)
    L = moe._lib
    assert L.moe_grouped_query(g, ctypes.byref(n)) == code
    if code:
        assert L.moe_grouped_mm(g, OK, OK, OK, OK, OK, None) == code
        assert L.moe_grouped_mm_dx(g, OK, OK, OK, OK, OK, None) == code
        assert L.moe_grouped_mm_dw(g, OK, OK, OK, OK, 0, 0, OK, None) == code
