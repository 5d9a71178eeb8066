"""The training step of an MoE block put together: forward, backward and update against the formulas
in 64 bits, captured and replayed, and the serving block against its stages."""
import dataclasses

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def setup(T=192, shared=128, d=256, seed=0, **kw):
    from combine_grouped_gemm_gb300.train import MoETrainBlock
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=T, d=d, R=1, d_ff_shared=shared)
    inp = synth.make_router_inputs(cfg, "cuda")
    W = synth.make_expert_weights(cfg, "cuda")
    W = {k: v for k, v in W.items() if v is not None and not k.endswith("_s")}
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def vec(lo, hi):
        return torch.rand(d, generator=g, device="cuda") * (hi - lo) + lo
    block = MoETrainBlock(cfg, inp["w_gate"], inp["bias"], W, vec(0.8, 1.2), vec(0.8, 1.2),
                          vec(0.1, 0.9), eps=1e-5, res_scale=0.9, out_scale=0.7, **kw)
    x = (torch.randn((T, d), generator=g, device="cuda") * 2).to(block.stream_dtype)
    dh = (torch.randn((T, d), generator=g, device="cuda") * 0.1).to(block.stream_dtype)
    return cfg, inp, W, block, x, dh


def reference(cfg, inp, W, block, x, dh, idx):
    """The block in 64 bits by autograd, with the kernel's choice of experts."""
    d = lambda t: t.detach().double().requires_grad_(True)   # noqa: E731
    P = {n: d(w) for n, (w, _) in block.parameters().items()}
    X = d(x)

    def norm(t):
        return t * (t.square().mean(1, keepdim=True) + 1e-5) ** -0.5
    n = norm(X) * P["w_in"]
    s = torch.sigmoid(n @ P["w_gate"].t()).gather(1, idx.long())
    w = s / s.sum(1, keepdim=True) * cfg.route_scale
    y = 0

    def expert(t, w13, w2):
        gate, up = (t @ w13.t()).chunk(2, 1)
        return (torch.nn.functional.silu(gate) * up) @ w2.t()
    for e in range(cfg.E):
        hit = (idx == e).double()
        y = y + expert(n, P["w13"][e], P["w2"][e]) * (w * hit).sum(1, keepdim=True)
    if cfg.d_ff_shared:
        y = y + expert(n, P["ws13"], P["ws2"])
    h = 0.9 * X + 0.7 * P["gate"] * norm(y) * P["w_out"]
    h.backward(dh.double())
    return h, dict({"d" + n: p.grad for n, p in P.items()}, dx=X.grad)


def rel(a, b):
    return float((a.double() - b.reshape(a.shape)).norm() / b.norm())


@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("T,shared", [(1, 128), (37, 0), (192, 128), (700, 128)])
def test_block_gradients(moe, T, shared, st):
    """Every gradient of the block. The chain rounds to bf16 at n, the products and their gradients
    (2^-9 of their size in the mean, six of them one after another), and to 8 bits at the kept
    activations (e4m3: a mean relative error of 2^-5.5, on x and the gate/up product): the norm of a
    gradient's error stays below 2^-9 * 6 + 2^-5.5 * 2 < 0.06 of its norm."""
    cfg, inp, W, block, x, dh = setup(T, shared, stream_dtype=st)
    h = block.forward(x)
    grads = block.backward(dh)
    ref_h, ref = reference(cfg, inp, W, block, x, dh, block.layer.bufs["topk_idx"])
    assert rel(h, ref_h.detach()) < 0.01
    for name, r in ref.items():
        assert rel(grads[name], r) < 0.06, name
    assert moe.read_status(block.layer.bufs["ws"]) == 0
    assert moe.read_status(block.layer.router_ws) == 0
    assert moe.read_status(block.layer.routed.ws) == 0
    # summed over a second micro-batch: twice the weights' gradients, bit by bit
    first = {k: v.clone() for k, v in grads.items()}
    block.forward(x)
    block.backward(dh, accumulate=True)
    for name, v in block.grads.items():
        same = name in ("dx", "dtopk_w")
        assert torch.equal(v, first[name] if same else first[name] + first[name]), name


@pytest.mark.parametrize("bits", [32, 8])
def test_step_updates_every_weight(moe, bits):
    """A step after a backward moves the masters as AdamW's first step does: by lr times the sign of
    the gradient where that is far above eps, and the weights are their masters rounded."""
    from combine_grouped_gemm_gb300.train import AdamW
    cfg, inp, W, block, x, dh = setup(64)
    opt = AdamW(block.parameters(), lr=1e-3, weight_decay=0.0, max_norm=1e9, state_bits=bits)
    block.forward(x)
    block.backward(dh)
    before = {n: t["p"].clone() for n, t in zip(opt.names, opt.tensors)}
    opt.step()
    total = 0.0
    for n, t in zip(opt.names, opt.tensors):
        weight, grad = block.parameters()[n]
        total += float(grad.double().square().sum())
        big = grad.abs() > 1e-4
        moved = (t["p"] - before[n])[big]
        # 1 / (1 + eps/|g|) with eps/|g| <= 1e-4; the difference of two fp32 values of size <= 2
        assert bool(((moved + 1e-3 * grad[big].sign()).abs() <= 1e-3 * 2e-4 + 2.0 ** -22).all()), n
        assert weight.dtype is F32 or torch.equal(weight, t["p"].to(BF)), n
        assert weight.dtype is not F32 or t["p"] is weight
    assert abs(float(opt.norm) - total ** 0.5) <= 1e-5 * total ** 0.5
    assert opt.steps == 1 and moe.read_status(opt.state) == 0
    # saved, gone on, loaded and gone on again: the same
    saved = opt.state_dict()
    opt.step(lr=5e-4)
    after = {n: t["p"].clone() for n, t in zip(opt.names, opt.tensors)}
    opt.load_state_dict(saved)
    opt.step()
    for n, t in zip(opt.names, opt.tensors):
        assert torch.equal(after[n], t["p"]), n
    with pytest.raises(ValueError, match="other weights"):
        opt.load_state_dict(dict(saved, tensors={}))


def test_captured_training_steps(moe):
    """Forward, backward and update captured once and replayed on new tokens give what eager steps
    give, while an eager block of its own lives beside."""
    from combine_grouped_gemm_gb300.train import AdamW

    def make():
        cfg, inp, W, block, x, dh = setup(96)
        return block, AdamW(block.parameters(), lr=1e-3, max_norm=0.5, state_bits=8), x, dh
    a, oa, xa, da = make()
    b, ob, xb, db = make()
    ha = torch.empty_like(xa)
    a.forward(xa, ha)     # one eager run: the one-time shared-memory limits
    a.backward(da)
    saved = oa.state_dict()
    oa.step()
    oa.load_state_dict(saved)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.forward(xa, ha)
        a.backward(da)
        oa.step()
    for i in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        xa.copy_(torch.randn(xa.shape, generator=g, device="cuda"))
        xb.copy_(xa)
        graph.replay()
        hb = b.forward(xb)
        b.backward(db)
        ob.step()
        torch.cuda.synchronize()
        assert torch.equal(ha, hb)
        for (n, (wa, ga)), (wb, gb) in zip(a.parameters().items(), b.parameters().values()):
            assert torch.equal(ga, gb) and torch.equal(wa, wb), (i, n)
    assert oa.steps == ob.steps == 3


def test_block_keeps_its_contract(moe):
    cfg, inp, W, block, x, dh = setup(32)
    with pytest.raises(RuntimeError, match="forward"):
        block.backward(dh)
    with pytest.raises(ValueError, match="another"):
        block.forward(x, x)
    with pytest.raises(ValueError, match="x must be"):
        block.forward(x.float())
    block.forward(x)
    block.backward(dh)
    with pytest.raises(RuntimeError, match="forward"):
        block.backward(dh)


def test_train_layer_without_router_is_as_before(moe):
    """train_router adds to dx; everything else of the layer stays bit by bit."""
    from combine_grouped_gemm_gb300.train import MoETrainLayer
    cfg, inp, W, block, x, dh = setup(64)
    a = MoETrainLayer(cfg, inp["w_gate"], inp["bias"], W)
    b = MoETrainLayer(cfg, inp["w_gate"], inp["bias"], W, train_router=True)
    assert torch.equal(a.forward(x), b.forward(x))
    ga, gb = a.backward(dh), b.backward(dh)
    assert "dw_gate" not in ga
    for n in ga:
        assert n == "dx" or torch.equal(ga[n], gb[n]), n
    assert not torch.equal(ga["dx"], gb["dx"])


@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("T", [8, 64])
def test_serving_block_is_its_stages(moe, T, st):
    """MoEBlock's chain (norm, layer, norm with gate and residual and the next block's norm) against
    the calls one by one, two blocks in a row, and captured."""
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=T, d_ff_shared=128)
    inp = synth.make_router_inputs(cfg, "cuda")
    W = synth.make_expert_weights(cfg, "cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = [torch.rand(cfg.d, generator=g, device="cuda") + 0.5 for _ in range(5)]
    x = torch.randn((T, cfg.d), generator=g, device="cuda").to(st)
    layers = [moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W) for _ in range(2)]
    first = moe.MoEBlock(layers[0], w[0], w_out=w[1], gate=w[4], w_next=w[2], out_scale=0.5)
    second = moe.MoEBlock(layers[1], w[2], w_out=w[3])
    h1, n1 = first(x)
    n1 = n1.clone()
    h2 = second(h1, n1)
    n, y = torch.empty_like(x, dtype=BF), torch.empty_like(x, dtype=BF)
    moe.norm_in(x, w[0], n)
    layers[0](n, y)
    h, nn = torch.empty_like(x), torch.empty_like(n)
    moe.norm_out(y, x, w[1], w[4], w[2], h, nn, out_scale=0.5)
    assert torch.equal(h, h1) and torch.equal(nn, n1)
    layers[1](n1, y)
    hh = torch.empty_like(x)
    moe.norm_out(y, h, w[3], None, None, hh, None)
    assert torch.equal(hh, h2)
    # called again with its own n (layers that share weights): as from a copy of it
    a, m = first(x)
    keep = m.clone()
    b1, m1 = first(a, m)
    b1, m1 = b1.clone(), m1.clone()
    b2, m2 = first(a, keep)
    assert torch.equal(b1, b2) and torch.equal(m1, m2)
    # the norm of h as it was stored is a rounding away from the one handed on: h's own (2^-8 of each
    # column, and of r_h at most as much again) and the results' two
    moe.norm_in(h1, w[2], nn)
    assert bool(((nn.double() - n1.double()).abs() <= 4.1 * 2.0 ** -8 * n1.double().abs()).all())
    xs, out = x.clone(), torch.empty_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = first(xs)
        second(a, b, out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, h2)


@pytest.mark.parametrize("bits", [32, 8])
def test_example_runs(moe, bits):
    """The example runs to its end, with finite losses (how far they fall is not tested)."""
    import math
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(__file__)), "examples"))
    import train_block
    losses = train_block.main(steps=4, bits=bits)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
