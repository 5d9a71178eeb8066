"""Refusals of the training calls, checked on the host: nothing here launches GPU work."""
import ctypes
import os
import sys

import pytest
import torch

OK = 1 << 20   # an aligned address that the checks never dereference


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_grouped_gemm_gb300 as m
    return m


def cfg(moe, **change):
    return ctypes.byref(moe.GroupCfg(**{**dict(rows=16, E=4, n=64, k=128), **change}))


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), 1), (dict(E=0), 1), (dict(n=0), 1), (dict(k=-8), 1),
    (dict(E=1025), 2), (dict(n=60), 2), (dict(k=100), 2),
    (dict(), 0), (dict(rows=0), 0), (dict(n=8, k=8, E=1024), 0)])
def test_group_shapes(moe, change, code):
    L, n = moe._lib, ctypes.c_size_t(0)
    g = cfg(moe, **change)
    assert L.moe_grouped_query(g, ctypes.byref(n)) == code
    if code:
        assert n.value == 0
        assert L.moe_grouped_mm(g, OK, OK, OK, OK, OK, None) == code
        assert L.moe_grouped_mm_dx(g, OK, OK, OK, OK, OK, None) == code
        assert L.moe_grouped_mm_dw(g, OK, OK, OK, OK, 0, 0, OK, None) == code
    else:
        assert n.value >= 16


def test_grouped_pointers(moe):
    L, g = moe._lib, cfg(moe)
    assert L.moe_grouped_query(None, None) == 1
    assert L.moe_grouped_query(g, None) == 1
    for fn, args in ((L.moe_grouped_mm, [OK] * 5), (L.moe_grouped_mm_dx, [OK] * 5)):
        for i in range(5):
            assert fn(g, *[None if j == i else a for j, a in enumerate(args)], None) == 1
            assert fn(g, *[OK + 8 if j == i else a for j, a in enumerate(args)], None) == 3
        assert fn(None, *args, None) == 1
    for i in range(4):
        a = [OK] * 4
        a[i] = None
        assert L.moe_grouped_mm_dw(g, *a, 0, 0, OK, None) == 1
        a[i] = OK + 2
        assert L.moe_grouped_mm_dw(g, *a, 0, 0, OK, None) == 3
    assert L.moe_grouped_mm_dw(g, OK, OK, OK, OK, 0, 0, None, None) == 1
    for dtype in (-1, 1, 2, 4):
        assert L.moe_grouped_mm_dw(g, OK, OK, OK, OK, dtype, 0, OK, None) == 1
    assert L.moe_grouped_mm_dw(g, OK, OK, OK, OK, moe.MOE_BF16, 1, OK, None) == 1  # bf16 sums


def test_no_rows_is_no_work(moe):
    L, g = moe._lib, cfg(moe, rows=0)
    assert L.moe_grouped_mm(g, None, OK, OK, None, OK, None) == 0
    assert L.moe_grouped_mm_dx(g, None, OK, OK, None, OK, None) == 0
    assert L.moe_grouped_mm(g, None, None, OK, None, OK, None) == 1   # counts still needed
    assert L.moe_act_save(0, 128, None, None, None, None) == 0
    assert L.moe_act_load(0, 0, 128, None, None, None, None, None, None) == 0
    assert L.moe_swiglu_save(0, 128, None, None, None, None, None) == 0
    assert L.moe_swiglu_grad(0, 128, None, None, None, None, None, None) == 0
    assert L.moe_combine_grad(0, 2, 128, 0, None, None, None, None, None, None, None, None) == 0


@pytest.mark.parametrize("rows,cols,code", [(-1, 128, 1), (4, 0, 1), (4, 64, 2), (4, 200, 2),
                                            (2 ** 30, 128, 2)])
def test_row_shapes(moe, rows, cols, code):
    L = moe._lib
    assert L.moe_act_save(rows, cols, OK, OK, OK, None) == code
    assert L.moe_act_load(rows, 4, cols, OK, OK, OK, OK, None, None) == code
    assert L.moe_swiglu_save(rows, cols, OK, OK, OK, OK, None) == code
    assert L.moe_swiglu_grad(rows, cols, OK, OK, OK, OK, OK, None) == code
    assert L.moe_combine_grad(rows, 2, cols, 8, OK, OK, OK, OK, OK + 16, OK, None, None) == code
    assert L.moe_combine_grad(4, 2, 128, -1, OK, OK, OK, OK, OK + 16, OK, None, None) == 1


def test_row_pointers(moe):
    L = moe._lib
    for fn, head, n in ((L.moe_act_save, (4, 128), 3), (L.moe_swiglu_save, (4, 128), 4),
                        (L.moe_swiglu_grad, (4, 128), 4)):
        tail = [OK] if fn is L.moe_swiglu_grad else []   # a: may be NULL, not misaligned
        for i in range(n):
            a = [OK] * n
            a[i] = None
            assert fn(*head, *a, *tail, None) == 1
            a[i] = OK + 4
            assert fn(*head, *a, *tail, None) == 3
    assert L.moe_swiglu_grad(4, 128, OK, OK, OK, OK, OK + 8, None) == 3
    assert L.moe_act_load(4, 3, 128, OK, OK, None, OK, None, None) == 1    # no index, too few rows
    assert L.moe_act_load(4, -1, 128, OK, OK, OK, OK, None, None) == 1
    assert L.moe_act_load(4, 4, 128, OK, OK, OK + 4, OK, None, None) == 3
    assert L.moe_act_load(4, 4, 128, OK, OK, OK, None, None, None) == 1
    assert L.moe_act_load(4, 4, 128, OK, OK, OK, OK, OK + 2, None) == 3    # status
    args = [OK, OK, OK, OK, 2 * OK, OK]
    for i in range(6):
        a = list(args)
        a[i] = None
        assert L.moe_combine_grad(4, 2, 128, 8, *a, None, None) == 1
        a[i] = OK + 4
        assert L.moe_combine_grad(4, 2, 128, 8, *a, None, None) == 3
    assert L.moe_combine_grad(4, 2, 128, 8, OK, OK, OK, OK, OK, OK, None, None) == 1  # in place
    assert L.moe_combine_grad(4, 2, 128, 8, *args, OK + 1, None) == 3
    assert L.moe_combine_grad(4, 0, 128, 8, *args, None, None) == 1
    assert L.moe_combine_grad(4, 33, 128, 8, *args, None, None) == 2
    assert L.moe_combine_grad(2 ** 27, 32, 128, 8, *args, None, None) == 2   # T * k


def test_binding_refuses_other_tensors(moe):
    """Types, shapes and places are checked before a pointer reaches the library."""
    g = moe.GroupCfg(rows=16, E=4, n=64, k=128)
    x, w = torch.zeros(16, 128, dtype=torch.bfloat16), torch.zeros(4, 64, 128, dtype=torch.bfloat16)
    y, c = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        moe.grouped_mm(g, x, c, w, y, ws)
    with pytest.raises(ValueError, match="x must be"):
        moe.grouped_mm(g, x.float(), c, w, y, ws)
    with pytest.raises(ValueError, match="shape"):
        moe.grouped_mm(g, x[:8], c, w, y, ws)
    with pytest.raises(ValueError, match="2-D"):
        moe.act_save(x[0], x, x)
    with pytest.raises(ValueError):
        moe.combine_grad(x, c, x, x, x, x)
    with pytest.raises(moe.MoEError):
        moe.grouped_ws_bytes(moe.GroupCfg(rows=16, E=4, n=63, k=128))


def test_train_layer_takes_one_rank_bf16(moe):
    import synth
    from combine_grouped_gemm_gb300.train import MoETrainLayer
    for name in ("dsv3_decode", "dsv3_fp8_prefill"):
        with pytest.raises(ValueError, match="R == 1"):
            MoETrainLayer(synth.CONFIGS[name], None, None, {}, "cpu")


@pytest.mark.gpu
def test_example_lowers_its_loss():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples"))
    import train_experts
    losses = train_experts.main(steps=12)
    assert losses[-1] < 0.7 * losses[0]
