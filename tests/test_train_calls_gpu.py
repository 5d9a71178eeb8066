"""The training calls on the GPU: arrays that lie next to each other or in place of one another, the
element-wise calls' large and ragged sizes, the codes against the dispatch's, the precision of long
weight gradients."""
import dataclasses

import pytest
import torch

import synth
from test_train_gpu import awkward, check, quantise

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


@pytest.mark.parametrize("rows,f", [(3648 + 1, 2048), (3648 + 16, 2048), (3648 + 17, 2048),
                                    (3648 + 63, 2048), (58368 + 3, 128), (58368 + 61, 128)])
def test_swiglu_save_of_many_rows(moe, rows, f):
    """From 3648 tiles of 16 rows x 128 columns on, a CTA takes 64 rows, 16 at a time with the next
    ones' loads ahead; the last CTA has 1 to 63 of them."""
    gu = awkward(6, rows, 2 * f)
    a = torch.empty((rows, f), dtype=BF, device="cuda")
    q = torch.empty((rows, 2 * f), dtype=torch.uint8, device="cuda")
    s = torch.empty((2 * f // 128, rows), device="cuda")
    moe.swiglu_save(gu, a, q, s)
    rq, rs = quantise(gu)
    assert torch.equal(q.cpu(), rq) and torch.equal(s.cpu(), rs)
    g, u = gu.double().chunk(2, 1)
    ref = g * torch.sigmoid(g) * u
    # as for small sizes: the exponential is off by 2^-21 + 2^-24 |g| of its size
    check(a, ref, 2.0 ** -16 * ref.abs() + 1e-36 * u.abs(), "bf16")


@pytest.mark.parametrize("T,d", [(1, 256), (48, 256), (1000, 7168)])
def test_codes_and_scales_are_the_dispatch_s(moe, T, d):
    """act_save of x and the e4m3 dispatch of x: the same bytes for every row sent."""
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=T, d=d, R=1, act="fp8", w="fp8")
    x = awkward(3, T, d)
    if T > 1:
        x[1, ::128] = 3e38          # a block scale near the end of the range
    idx = torch.stack([torch.randperm(cfg.E, device="cuda")[:cfg.k] for _ in range(T)])
    b = moe.Buffers(cfg)
    b["topk_idx"].copy_(idx)
    moe.dispatch(cfg, x, b["topk_idx"], b["recv"], b["recv_scales"], b["counts"], b["row_of"])
    q = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    s = torch.empty((d // 128, T), device="cuda")
    moe.act_save(x, q, s)
    for i in range(cfg.k):
        rows = b["row_of"][:, i].long()
        assert torch.equal(b["recv"].view(torch.uint8)[rows], q)
        assert torch.equal(b["recv_scales"][:, rows], s)


def test_fp32_weight_gradients_are_summed_in_short_runs(moe):
    """A group of 8300 rows whose reduction is not split (81 units). The tensor core truncates: each
    addition of 16 products loses up to 2^-23 of the running sum, 2^-24 in the mean, which for sums
    that grow like the root of their length is 2/3 of 2^-24 of the result an addition. Sums of 512
    rows, 32 additions, are off by 1.3e-6 that way, joined by rounded additions that add little;
    one sum of 8300 rows would be off by up to 2e-5 (measured: 2.1e-6 after 2048 rows, 4.4e-6
    after 4096)."""
    g = moe.GroupCfg(rows=8300, E=1, n=2304, k=2304)
    c = torch.tensor([8300], dtype=torch.int32, device="cuda")
    x, dy = normal(1, g.rows, g.k), normal(2, g.rows, g.n)
    dw = torch.empty((1, g.n, g.k), device="cuda")
    ws = torch.zeros(moe.grouped_ws_bytes(g), dtype=torch.uint8, device="cuda")
    moe.grouped_mm_dw(g, dy, x, c, dw, ws)
    ref = dy.double().t() @ x.double()
    assert float((dw[0].double() - ref).norm() / ref.norm()) < 1.5e-6
