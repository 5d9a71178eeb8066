"""The training calls on the GPU: arrays that lie next to each other or in place of one another."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def normal(seed, *shape, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(BF)


def test_arrays_next_to_each_other(moe):
    """x and y in one allocation, one right after the other, either way round."""
    g = moe.GroupCfg(rows=100, E=2, n=64, k=136)
    c = torch.tensor([60, 40], dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")
    x, w = normal(1, 100, 136), normal(2, 2, 64, 136)
    ref = torch.empty((100, 64), dtype=BF, device="cuda")
    moe.grouped_mm(g, x, c, w, ref, ws)
    for first in (True, False):
        both = torch.zeros(100 * (64 + 136), dtype=BF, device="cuda")
        xs = both[:13600] if first else both[6400:]
        ys = both[13600:] if first else both[:6400]
        xs.copy_(x.view(-1))
        moe.grouped_mm(g, xs.view(100, 136), c, w, ys.view(100, 64), ws)
        assert torch.equal(ys.view(100, 64), ref) and torch.equal(xs.view(100, 136), x)
    with pytest.raises(moe.MoEError):   # y's first row over x's last
        moe.grouped_mm(g, both[:13600].view(100, 136), c, w,
                       both[13600 - 64:13600 - 64 + 6400].view(100, 64), ws)


def test_outputs_in_place_of_an_input(moe):
    rows, f = 77, 256
    gu, da = normal(1, rows, 2 * f), normal(2, rows, f)
    a, q = torch.empty_like(da), torch.empty((rows, 2 * f), dtype=torch.uint8, device="cuda")
    s = torch.empty((2 * f // 128, rows), device="cuda")
    moe.swiglu_save(gu, a, q, s)
    dgu, dgu2, a = torch.empty_like(gu), torch.empty_like(gu), torch.empty_like(da)
    moe.swiglu_grad(q, s, da, dgu, a)
    here = da.clone()
    moe.swiglu_grad(q, s, here, dgu2, here)
    assert torch.equal(dgu, dgu2) and torch.equal(here, a)

    for T in (5, 12000):   # a CTA a choice, a warp a choice
        k, d = 2, 1152
        row_of = torch.randperm(T * k, device="cuda").to(torch.int32).view(T, k)
        w = torch.rand((T, k), device="cuda")
        ebuf, dy = normal(3, T * k, d), normal(4, T, d)
        de, dw = torch.empty_like(ebuf), torch.empty_like(w)
        moe.combine_grad(ebuf, row_of, w, dy, de, dw)
        de2, here = torch.empty_like(ebuf), w.clone()
        moe.combine_grad(ebuf, row_of, here, dy, de2, here)
        assert torch.equal(de, de2) and torch.equal(here, dw)
