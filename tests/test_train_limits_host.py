"""Sizes and arguments at the end of what the training calls take, checked on the host: nothing here
launches GPU work."""
import ctypes

import pytest
import torch

# the addresses are made up, so a check that let one through must not find a device
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks, run without a GPU")

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


def refuses_overlap(call, sizes, out, allowed=()):
    """Each way in which array `out` can meet another one is an invalid argument. sizes: name ->
    bytes, of arrays at fake addresses 1 TB apart."""
    base = {n: (i + 1) << 40 for i, n in enumerate(sizes)}
    for other in sizes:
        if other == out:
            continue
        meets = [base[other] + sizes[other] - 16, base[other] - sizes[out] + 16]
        if other not in allowed:
            meets.append(base[other])
        for at in meets:
            assert call(**{**base, out: at}) == 1, (out, other, at)


def test_outputs_that_meet_an_input_are_refused(moe):
    """Every call's blocks run in any order: a result over an input would change what other blocks
    read. (sizes: whole multiples of 16 bytes, at least 32)"""
    L = moe._lib
    rows, E, n, k = 16, 8, 64, 128
    g = ctypes.byref(moe.GroupCfg(rows=rows, E=E, n=n, k=k))
    x, w, y = 2 * rows * k, 2 * E * n * k, 2 * rows * n
    ws = moe.grouped_ws_bytes(moe.GroupCfg(rows=rows, E=E, n=n, k=k)) // 16 * 16

    def mm(a, counts, w, out, ws):
        return L.moe_grouped_mm(g, a, counts, w, out, ws, None)

    def dx(a, counts, w, out, ws):
        return L.moe_grouped_mm_dx(g, a, counts, w, out, ws, None)

    def dw(a, counts, w, out, ws, dtype=moe.MOE_F32):
        return L.moe_grouped_mm_dw(g, a, w, counts, out, dtype, 0, ws, None)
    refuses_overlap(mm, dict(a=x, counts=4 * E, w=w, out=y, ws=ws), "out")
    refuses_overlap(dx, dict(a=y, counts=4 * E, w=w, out=x, ws=ws), "out")
    refuses_overlap(dw, dict(a=y, counts=4 * E, w=x, out=2 * w, ws=ws), "out")
    refuses_overlap(lambda **p: dw(dtype=moe.MOE_BF16, **p),
                    dict(a=y, counts=4 * E, w=x, out=w, ws=ws), "out")
    for f, s in ((mm, dict(a=x, counts=4 * E, w=w, out=y, ws=ws)),
                 (dx, dict(a=y, counts=4 * E, w=w, out=x, ws=ws)),
                 (dw, dict(a=y, counts=4 * E, w=x, out=2 * w, ws=ws))):
        refuses_overlap(f, s, "ws")

    rows, d = 16, 256
    save = dict(x=2 * rows * d, q=rows * d, scales=rows * d // 32)
    for out in ("q", "scales"):
        refuses_overlap(lambda x, q, scales: L.moe_act_save(rows, d, x, q, scales, None), save, out)
    load = dict(q=8 * d, scales=8 * d // 32, index=4 * rows, out=2 * rows * d)
    refuses_overlap(lambda q, scales, index, out: L.moe_act_load(
        rows, 8, d, q, scales, index, out, None, None), load, "out")
    swi = dict(gu=4 * rows * d, a=2 * rows * d, q=2 * rows * d, scales=rows * d // 16)
    for out in ("a", "q", "scales"):
        refuses_overlap(lambda gu, a, q, scales: L.moe_swiglu_save(rows, d, gu, a, q, scales, None),
                        swi, out)
    grad = dict(q=2 * rows * d, scales=rows * d // 16, da=2 * rows * d, dgu=4 * rows * d,
                a=2 * rows * d)
    for out in ("dgu", "a"):   # a may be da itself: one thread reads and writes an element
        refuses_overlap(lambda q, scales, da, dgu, a: L.moe_swiglu_grad(
            rows, d, q, scales, da, dgu, a, None), grad, out, ("da",) if out == "a" else ())
    T, k = 8, 4
    comb = dict(ebuf=2 * rows * d, row_of=4 * T * k, topk_w=4 * T * k, dy=2 * T * d,
                debuf=2 * rows * d, dtopk_w=4 * T * k)
    for out in ("debuf", "dtopk_w"):   # dtopk_w may be topk_w itself, likewise
        refuses_overlap(lambda ebuf, row_of, topk_w, dy, debuf, dtopk_w: L.moe_combine_grad(
            T, k, d, rows, ebuf, row_of, topk_w, dy, debuf, dtopk_w, None, None),
            comb, out, ("topk_w",) if out == "dtopk_w" else ())


class OnDevice(torch.Tensor):
    """A tensor that says it lies on CUDA device `place`."""
    place = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.place


def test_tensors_of_another_device_are_refused(moe, monkeypatch):
    """The kernels run on the current device: its streams, its memory."""
    monkeypatch.setattr(moe, "_device", lambda: 0)
    bf, i32, f32, u8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8

    def make(*shapes):
        return [torch.zeros(s, dtype=t).as_subclass(OnDevice) for t, *s in shapes]
    g = moe.GroupCfg(rows=16, E=4, n=64, k=128)
    x, c, w, y, ws = make((bf, 16, 128), (i32, 4), (bf, 4, 64, 128), (bf, 16, 64), (u8, 1 << 20))
    dw, = make((f32, 4, 64, 128))
    r, q, s, i, o = make((bf, 16, 128), (u8, 16, 128), (f32, 1, 16), (i32, 8), (bf, 8, 128))
    gu, q2, s2, a, dgu = make((bf, 16, 256), (u8, 16, 256), (f32, 2, 16), (bf, 16, 128),
                              (bf, 16, 256))
    ro, tw, dy, de, dt = make((i32, 8, 2), (f32, 8, 2), (bf, 8, 128), (bf, 16, 128), (f32, 8, 2))
    st, = make((i32, 4))
    calls = [(moe.grouped_mm, (g, x, c, w, y, ws)), (moe.grouped_mm_dx, (g, y, c, w, x, ws)),
             (moe.grouped_mm_dw, (g, y, x, c, dw, ws)), (moe.act_save, (r, q, s)),
             (lambda *t: moe.act_load(*t[:4], status=t[4]), (q, s, i, o, st)),
             (moe.swiglu_save, (gu, a, q2, s2)), (moe.swiglu_grad, (q2, s2, a, dgu, r)),
             (lambda *t: moe.combine_grad(*t[:6], status=t[6]), (r, ro, tw, dy, de, dt, st))]
    for fn, args in calls:
        for t in args:
            if isinstance(t, torch.Tensor):
                t.place = 1
                with pytest.raises(ValueError, match="device"):
                    fn(*args)
                t.place = 0
