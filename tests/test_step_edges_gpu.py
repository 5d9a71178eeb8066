"""Calls of the training step's operators that their documentation allows and that lie at its edges."""
import ctypes
import dataclasses
import threading

import numpy as np
import pytest
import torch

import synth
from test_step_gpu import (BF, F32, adam_tensors, check_route, copy_of, e4m3_table, hold_reference,
                           mix, normal, route_cfg, route_inputs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def whole_scales(x):
    """x with the blocks as zeros whose scale, amax * fp32(1/448), is no normal number."""
    f = np.float32
    pad = np.concatenate([np.abs(x), np.zeros(-x.size % 128, f)]).reshape(-1, 128)
    scale = pad.max(1) * (f(1) / f(448))
    return np.where(np.repeat(scale >= f(2.0 ** -126), 128)[:x.size], x, f(0))


def check_steps(a, b, steps):
    """a: a tensor after `steps` steps of AdamW in 8 bits, betas 0.9 and 0.99, from step 1 on; b: before
    them, with the same gradients. The codes and scales of the definition, each one."""
    f = np.float32
    tab = np.concatenate([e4m3_table(), [np.nan]]).astype(f)
    tab = np.concatenate([tab, -tab])
    n = b["p"].numel()
    g = b["g"].float().cpu().numpy()
    codes = {k: b[k].cpu().numpy() for k in ("m", "v", "m_scale", "v_scale")}
    old = np.seterr(over="ignore", under="ignore")
    for step in range(1, steps + 1):
        sm, sv = (np.repeat(codes[k], 128)[:n] for k in ("m_scale", "v_scale"))
        m, v = tab[codes["m"]] * sm, tab[codes["v"]] * sv
        v = v * v
        m = f(0.9) * m + f(1 - 0.9) * g
        v = f(0.99) * v + f(1 - 0.99) * (g * g)
        root = np.sqrt(v)
        key = mix(np.array([(b["seed"] ^ (step * 0x9E3779B9)) & 0xFFFFFFFF], np.uint32))
        key = mix(key ^ np.arange((n + 127) // 128, dtype=np.uint32))
        place = (np.arange(128, dtype=np.uint64) * 0x9E3779B9).astype(np.uint32)
        r = mix(key[:, None] + place[None, :]).reshape(-1)
        for name, x, r16 in (("m", m, r >> np.uint32(16)), ("v", root, r & np.uint32(0xFFFF))):
            codes[name], codes[name + "_scale"] = hold_reference(whole_scales(x), r16, name == "v")
    np.seterr(**old)
    for name in ("m", "v"):
        assert np.array_equal(a[name + "_scale"].cpu().numpy(), codes[name + "_scale"]), name
        assert np.array_equal(a[name].cpu().numpy() & 127, codes[name] & 127), name
    assert bool(torch.isfinite(a["p"]).all())


def many(large, small):
    """250 tensors, the even ones about twice as large as the odd ones: 2125 whole chunks of 4096
    elements, three or four to each of the kernel's 608 CTAs, which so meet borders of tensors."""
    return [(4096 * (2 + i % 20) + large * i if i % 2 == 0 else 4096 * (1 + i % 10) + small * i)
            for i in range(250)]


@pytest.mark.parametrize("sizes,gtypes", [([5_000_011], [F32]), ([5_000_011], [BF]),
                                          (many(1, 3), [F32, BF]), (many(3, 1), [BF, F32])],
                         ids=["fp32", "bf16", "mostly fp32", "mostly bf16"])
def test_adamw_8_bit_chunk_after_chunk(moe, sizes, gtypes):
    """CTAs that take several chunks, of tensors with gradients of the other type beside: a tensor
    gets the codes of the definition, each of many what it gets alone."""
    A = adam_tensors(sizes, 8, gtypes, seed=5)
    B = copy_of(A)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    plan, state = moe.AdamTensors(A, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    steps = 2 if len(sizes) == 1 else 4
    for _ in range(steps):
        moe.adamw(cfg, plan, state)
    if len(sizes) == 1:
        check_steps(A[0], B[0], steps)
        return
    for i, (a, b) in enumerate(zip(A, B)):
        own, st = moe.AdamTensors([b], state_bits=8), moe.adam_state(0, 0.9, 0.99)
        for _ in range(steps):
            moe.adamw(cfg, own, st)
        for k in ("p", "m", "v", "m_scale", "v_scale"):
            assert torch.equal(a[k], b[k]), (i, k)
        assert b["w"] is None or torch.equal(a["w"], b["w"])


@pytest.mark.parametrize("n", [4096 * 700 + 1000, 3000])
def test_adamw_8_bit_scales_near_the_end_of_the_range(moe, n):
    """Moments whose block scales are 2^-149 to 2^-60, few codes above 0, and no gradient: codes and
    scales as defined, code by code."""
    T = adam_tensors([n], 8, [F32], seed=2, copies=False)
    t = T[0]
    blocks = (n + 127) // 128
    t["m"].copy_(torch.randint(0, 127, (n,), device="cuda") *
                 (torch.rand(n, device="cuda") < 0.1)).to(torch.uint8)
    t["m_scale"].copy_(torch.exp2(torch.linspace(-149, -60, blocks, dtype=torch.float64,
                                                 device="cuda")))
    t["v"].fill_(0x38)
    t["v_scale"].fill_(1e-5)
    t["g"].zero_()
    before = copy_of(T)[0]
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    plan, state = moe.AdamTensors(T, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    for _ in range(2):
        moe.adamw(cfg, plan, state)
    check_steps(t, before, 2)


def test_adamw_8_bit_moments_die_out(moe):
    """No gradient for a thousand steps (an expert without tokens): the first moment's scales pass the
    end of the fp32 range. The parameters stay finite, and the moment ends at 0."""
    T = adam_tensors([128 * 9000 + 77], 8, [F32], seed=3, copies=False)
    t = T[0]
    t["g"].mul_(torch.rand(t["g"].shape, device="cuda") < 0.02)   # mostly zeros, a few a block
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8)
    plan, state = moe.AdamTensors(T, state_bits=8), moe.adam_state(0, 0.9, 0.95)
    moe.adamw(cfg, plan, state)
    t["g"].zero_()
    for _ in range(1000):
        moe.adamw(cfg, plan, state)
    assert bool(torch.isfinite(t["p"]).all())
    assert int((t["m"] & 127).max()) == 0 and bool((t["m_scale"] == 1).all())


def test_adamw_8_bit_scales_that_underflow(moe):
    """Ten million elements, nearly all codes 0, scales of 1 to 512 times 2^-149, no gradient."""
    n = 128 * 80_000
    T = adam_tensors([n], 8, [BF], seed=4, copies=False)
    t = T[0]
    t["m"][::128] = 0x7e
    t["m_scale"].copy_(torch.arange(80_000, device="cuda", dtype=torch.float64) % 512 + 1)
    t["m_scale"].mul_(2.0 ** -100).mul_(2.0 ** -49)
    assert float(t["m_scale"][0]) == 2.0 ** -149 and float(t["m_scale"][511]) == 2.0 ** -140
    t["v"].fill_(0x38)
    t["v_scale"].fill_(1e-5)
    t["g"].zero_()
    plan, state = moe.AdamTensors(T, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    for _ in range(3):
        moe.adamw(cfg, plan, state)
        assert bool(torch.isfinite(t["p"]).all())
        assert int((t["m"] & 127).max()) == 0 and bool((t["m_scale"] == 1).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_adamw_8_bit_what_spoils_a_block(moe, bad):
    """A NaN or an infinity spoils its block (in whole chunks and past them) and no other: no value of
    its moments is left, and the next step leaves no parameter of it."""
    n = 3 * 4096 + 300
    A = adam_tensors([n], 8, [F32], seed=6)
    B = copy_of(A)
    at = [5, 4096 + 128 * 7 + 127, 3 * 4096 + 128, n - 1]
    spoilt = torch.zeros(n, dtype=torch.bool, device="cuda")
    for i in at:
        A[0]["g"][i] = bad
        spoilt[i // 128 * 128:i // 128 * 128 + 128] = True
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    pa, sa = moe.AdamTensors(A, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    pb, sb = moe.AdamTensors(B, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    a, b = A[0], B[0]
    for step in range(3):
        moe.adamw(cfg, pa, sa)
        moe.adamw(cfg, pb, sb)
        for k in ("m", "v"):
            x = a[k].view(torch.float8_e4m3fn).float() * a[k + "_scale"].repeat_interleave(128)[:n]
            assert torch.equal(~torch.isfinite(x), spoilt), (step, k)
            assert torch.equal(a[k][~spoilt], b[k][~spoilt])
        hit = spoilt if step else ~torch.isfinite(a["g"])
        if step == 0:
            a["g"].copy_(b["g"])
        assert torch.equal(~torch.isfinite(a["p"]), hit), step
        assert torch.equal(a["p"][~spoilt], b["p"][~spoilt])


@pytest.mark.parametrize("accumulate", [0, 1])
def test_norm_gradient_of_no_rows(moe, accumulate):
    """Without rows the weights' and the channel gate's gradients are 0 (or stay, accumulated), with
    the gate or, since none of it is read, without."""
    d = 192
    w, gate = normal(0, d, dtype=F32), normal(1, d, dtype=F32)
    ws = torch.empty(moe.norm_ws_bytes(0, d), dtype=torch.uint8, device="cuda")
    cfg = moe.NormCfg(rows=0, d=d, eps=1e-6, res_scale=1.0, out_scale=1.0,
                      stream_dtype=moe.MOE_BF16, gate=moe.MOE_GATE_CHANNEL)
    for g in (gate.data_ptr(), None):
        out = [torch.full((d,), 7.0 if accumulate else float("nan"), device="cuda")
               for _ in range(3)]
        dgate, dw_post, dw_next = [t.data_ptr() for t in out]
        rc = moe._lib.moe_norm_out_grad(
            ctypes.byref(cfg), None, None, None, None, w.data_ptr(), g, w.data_ptr(), None, None,
            None, None, dgate, dw_post, dw_next, accumulate, ws.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        for t in out:
            assert bool((t == (7.0 if accumulate else 0.0)).all())


def serving_blocks(moe, T=24):
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], T=T, d_ff_shared=128)
    inp = synth.make_router_inputs(cfg, "cuda")
    W = synth.make_expert_weights(cfg, "cuda")
    w = [normal(i, cfg.d, std=0.1, mean=1.0, dtype=F32) for i in range(5)]
    layers = [moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W) for _ in range(2)]
    A = moe.MoEBlock(layers[0], w[0], w_out=w[1], w_next=w[2])
    B = moe.MoEBlock(layers[1], w[2], w_out=w[3], w_next=w[4])
    return cfg, A, B


@pytest.mark.parametrize("given", ["another's n", "no n", "its own n", "its own n of before"])
def test_serving_block_keeps_the_n_it_returned(moe, given):
    """The n that a block returned is as it was after the block's next call, whatever n that is
    given, and what the call gives does not depend on the buffer."""
    cfg, A, _ = serving_blocks(moe)
    xs = [normal(10 + i, cfg.T, cfg.d) for i in range(6)]
    outside = [normal(20 + i, cfg.T, cfg.d) for i in range(6)]
    kept, copies = [], []
    for i in range(6):
        n = {"another's n": outside[i], "no n": None,
             "its own n": kept[-1] if kept else None,
             "its own n of before": kept[-2] if i > 1 else None}[given]
        fresh = None if n is None else n.clone()
        h, m = A(xs[i], n)
        if kept:
            assert torch.equal(kept[-1], copies[-1]), i
        _, other, _ = serving_blocks(moe)
        h2, m2 = other(xs[i], fresh)
        assert torch.equal(h, h2) and torch.equal(m, m2), i
        kept.append(m)
        copies.append(m.clone())


def test_serving_two_batches_through_two_blocks(moe):
    """Block A takes both micro-batches before block B takes the first."""
    cfg, A, B = serving_blocks(moe)
    xs = [normal(10 + i, cfg.T, cfg.d) for i in range(2)]
    ns = [normal(20 + i, cfg.T, cfg.d) for i in range(2)]
    want = []
    for x, n in zip(xs, ns):
        h, m = A(x, n)
        h, m = B(h, m)
        want.append((h.clone(), m.clone()))
    mid = [A(x, n) for x, n in zip(xs, ns)]
    for (h, m), (wh, wm) in zip(mid, want):
        h, m = B(h, m)
        assert torch.equal(h, wh) and torch.equal(m, wm)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_parameters(moe, bits):
    """Weights that require gradients: stepped, saved, loaded; and a load that is refused changes
    nothing."""
    from combine_grouped_gemm_gb300.train import AdamW

    def make():
        P = {"a": torch.nn.Parameter(normal(1, 40, 64, std=0.02, dtype=F32)),
             "b": torch.nn.Parameter(normal(2, 8, 128, std=0.02))}
        G = {n: normal(7, *p.shape, std=1e-3, dtype=p.dtype) for n, p in P.items()}
        return P, AdamW({n: (p, G[n]) for n, p in P.items()}, lr=1e-3, state_bits=bits)
    P, opt = make()
    opt.step()
    saved = opt.state_dict()
    assert not any(v.requires_grad for t in saved["tensors"].values() for v in t.values())
    opt.step()
    after = {n: p.detach().clone() for n, p in P.items()}
    opt.load_state_dict(saved)
    opt.step()
    Q, other = make()
    other.load_state_dict(saved)
    other.step()
    for n in P:
        assert torch.equal(P[n], after[n]) and torch.equal(Q[n], after[n])
        assert P[n].requires_grad and P[n].is_leaf

    def everything(o):
        return [o.state] + [v for t in o.tensors for v in t.values() if isinstance(v, torch.Tensor)]
    before = [v.clone() for v in everything(opt)]
    less = {n: dict(t) for n, t in saved["tensors"].items()}
    less["b"].pop("v")
    short = {n: dict(t) for n, t in saved["tensors"].items()}
    short["b"]["p"] = short["b"]["p"][:4]
    for bad in (dict(saved, tensors=less), dict(saved, tensors=short),
                dict(saved, state=saved["state"][:16])):
        with pytest.raises(ValueError, match="load_state_dict"):
            opt.load_state_dict(bad)
        assert all(torch.equal(a, b) for a, b in zip(before, everything(opt)))


@pytest.mark.parametrize("which", ["MoELayer", "MoEBlock", "MoETrainLayer", "MoETrainBlock"])
def test_outputs_belong_to_the_stream_of_the_call(moe, which):
    """An output that a call makes comes from the memory of the stream that it is given: not from what
    the current stream has given back, which work of that stream may still read."""
    from test_block_gpu import setup
    cfg, inp, W, block, x, dh = setup(48)
    make = {"MoELayer": lambda: moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W),
            "MoEBlock": lambda: moe.MoEBlock(moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W),
                                             block.w_in, w_next=block.w_in),
            "MoETrainLayer": lambda: block.layer.forward, "MoETrainBlock": lambda: block.forward}
    call = make[which]()
    assert moe._output((3,), F32, "cuda", 0).shape == (3,)   # the default stream's handle
    first = lambda out: out[0] if isinstance(out, tuple) else out   # noqa: E731
    want = first(call(x)).clone()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):   # object and handle
        torch.cuda.synchronize()
        freed = [torch.empty_like(x) for _ in range(64)]
        places = {t.data_ptr() for t in freed}
        del freed
        got = first(call(x, stream=stream))
        torch.cuda.synchronize()
        assert got.data_ptr() not in places
        assert torch.equal(got, want)


def test_host_call_on_another_stream(moe):
    from test_block_gpu import setup
    cfg, inp, W, block, x, dh = setup(48)
    layer = moe.MoELayer(cfg, inp["w_gate"], inp["bias"], W)
    want = layer(x).cpu()
    x_host, y_host = x.cpu().pin_memory(), torch.empty_like(want).pin_memory()
    torch.cuda.synchronize()
    places = {t.data_ptr() for t in [torch.empty_like(x) for _ in range(64)]}
    for s in (torch.cuda.Stream(), None):
        y_host.zero_()
        layer.run_host(x_host, y_host, s)
        torch.cuda.synchronize()
        assert torch.equal(y_host, want)
    assert layer._x_dev.data_ptr() not in places and layer._y_dev.data_ptr() not in places


def test_adamw_leaves_its_configuration(moe):
    """One AdamCfg for several plans and threads: a call writes nothing into it."""
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    was = bytes(cfg)
    lr = torch.full((1,), 5e-4, device="cuda")
    runs = []
    for bits, rate in ((32, lr), (8, None), (32, None), (8, lr)):
        T = adam_tensors([5000], bits, [F32], seed=bits)
        runs.append((moe.AdamTensors(T, state_bits=bits), moe.adam_state(0, 0.9, 0.99), rate, T))
    errors = []

    def work(plan, state, rate, stream):
        try:
            for _ in range(200):
                moe.adamw(cfg, plan, state, stream=stream, lr=rate)
        except Exception as e:   # noqa: BLE001
            errors.append(e)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(*r[:3], torch.cuda.Stream())) for r in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and bytes(cfg) == was
    for plan, state, rate, T in runs:
        U = adam_tensors([5000], plan.state_bits, [F32], seed=plan.state_bits)
        p, s = moe.AdamTensors(U, state_bits=plan.state_bits), moe.adam_state(0, 0.9, 0.99)
        for _ in range(200):
            moe.adamw(cfg, p, s, lr=rate)
        assert torch.equal(T[0]["p"], U[0]["p"])


@pytest.mark.parametrize("T,k", [(40, 4), (400, 4), (1500, 1)])
def test_route_grad_of_scores_near_zero(moe, T, k):
    """Chosen experts with scores of 1e-42 to 1e-36 (logits near -90): the quotients s / sum s are what
    they are for larger ones, as in the forward pass, though 1 / sum s has left the fp32 range."""
    d, E = 256, 24
    q = route_inputs(T, d, E, k, 0.0, seed=11)
    q["s"] = torch.exp(normal(12, T, k, std=3.0, mean=-90.0, dtype=F32).double()).to(F32)
    c = route_cfg(moe, T, d, E, k)
    ws = torch.zeros(moe.route_grad_ws_bytes(c), dtype=torch.uint8, device="cuda")
    check_route(moe, q, T, d, E, k, c, ws)
