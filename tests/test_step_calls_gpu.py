"""Calls of the training step's operators at the borders of their kernels, captured, back to back and
with values that spoil: the router's gradient, AdamW over more tensors than a call takes, the block."""
import math

import pytest
import torch

from test_block_gpu import setup
from test_step_gpu import (ADAM_SIZES, BF, F32, adam_tensors, check_route, copy_of, normal,
                           route_cfg, route_inputs, route_reference)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def route_ws(moe, c):
    return torch.zeros(moe.route_grad_ws_bytes(c), dtype=torch.uint8, device="cuda")


# 512 choices: the last in one launch; 1024 tokens: the first with slabs, of 128 columns up to 437
# experts, 64 up to 875; lists whose last 32 choices are few; chunks of other lengths; the widest row
BORDERS = [(64, 256, 16, 8), (65, 256, 16, 8), (128, 256, 16, 8), (512, 128, 8, 1),
           (513, 128, 8, 1), (17, 256, 40, 32), (33, 256, 40, 32), (511, 384, 24, 3),
           (1023, 384, 24, 3), (1024, 384, 24, 3), (1030, 384, 437, 2), (1030, 384, 438, 2),
           (1100, 384, 875, 3), (1100, 384, 876, 3), (1025, 128, 8, 1), (600, 640, 1024, 32),
           (4097, 256, 64, 2), (5200, 128, 9, 7), (21000, 128, 12, 3),
           (520, 65536, 4, 2), (2, 65536, 1024, 32)]


@pytest.mark.parametrize("T,d,E,k", BORDERS)
def test_route_grad_at_borders(moe, T, d, E, k):
    q = route_inputs(T, d, E, k, 0.5, seed=T)
    c = route_cfg(moe, T, d, E, k)
    check_route(moe, q, T, d, E, k, c, route_ws(moe, c))


@pytest.mark.parametrize("T", [40, 300, 1500])
def test_route_grad_captured(moe, T):
    """Replayed with other inputs each time it gives what an eager call gives, on one workspace."""
    d, E, k = 384, 24, 4
    c = route_cfg(moe, T, d, E, k)
    ws = route_ws(moe, c)
    q = route_inputs(T, d, E, k, 0.0, seed=1)
    dx, dw = torch.empty_like(q["x"]), torch.empty_like(q["w"])
    args = [q[n] for n in ("x", "w", "idx", "s", "dw", "dx_in")]
    moe.route_grad(c, *args, dx, dw, ws)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.route_grad(c, *args, dx, dw, ws)
    for seed in (2, 3, 4):
        other = route_inputs(T, d, E, k, 1.0, seed=seed)
        for n, t in q.items():
            t.copy_(other[n])
        graph.replay()
        got = dx.clone(), dw.clone()
        moe.route_grad(c, *args, dx, dw, ws)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("T", [40, 300, 1500])
def test_route_grad_keeps_what_spoils_to_its_own(moe, T):
    """A token that is not finite reaches the experts that it chose, an expert's weights that are not
    the tokens that chose it, and nothing else: not the tokens before and behind, not an expert
    without choices."""
    d, E, k = 256, 24, 4
    c = route_cfg(moe, T, d, E, k)
    q = route_inputs(T, d, E, k, 0.0, seed=9)
    q["idx"][q["idx"] == 5] = -1          # expert 5 has no choices
    bad = {0, T // 2, T - 1}
    for t in bad:
        q["x"][t] = float("nan") if t else float("inf")
    q["w"][7] = float("nan")
    q["w"][5] = float("inf")
    dx, dw = torch.empty_like(q["x"]), torch.empty_like(q["w"])
    moe.route_grad(c, q["x"], q["w"], q["idx"], q["s"], q["dw"], q["dx_in"], dx, dw, route_ws(moe, c))
    spoilt = set(q["idx"][sorted(bad)].flatten().tolist()) - {-1}
    for e in range(E):
        assert bool(torch.isfinite(dw[e]).all()) == (e not in spoilt), e
    assert bool((dw[5] == 0).all())
    chose = (q["idx"] == 7).any(1)
    assert torch.equal(torch.isfinite(dx).all(1), ~chose)


def test_adamw_8_bit_over_several_calls(moe):
    """600 tensors take three calls: each gets what a step of its own gives it."""
    sizes = [130 + 7 * (i % 40) for i in range(588)] + ADAM_SIZES
    A = adam_tensors(sizes, 8, [F32, BF], seed=2)
    B = copy_of(A)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8)
    plan, state = moe.AdamTensors(A, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    for _ in range(2):
        moe.adamw(cfg, plan, state)
    assert moe.adam_step(state) == 2
    for i in list(range(0, 600, 37)) + [255, 256, 511, 512, 599]:
        single, own = moe.AdamTensors([B[i]], state_bits=8), moe.adam_state(0, 0.9, 0.99)
        done = B[i].get("done")
        if not done:
            for _ in range(2):
                moe.adamw(cfg, single, own)
            B[i]["done"] = True
        for n in ("p", "m", "v", "m_scale", "v_scale"):
            assert torch.equal(A[i][n], B[i][n]), (i, n)


def test_adam_tensors_of_several_calls_that_meet(moe):
    T = adam_tensors([64] * 300, 32, [F32])
    moe.AdamTensors(T)
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamTensors(T[:299] + [dict(T[299], p=T[0]["p"])])
    long = torch.zeros(96, device="cuda")
    T[1]["m"], T[290]["v"] = long[:64], long[32:]
    with pytest.raises(ValueError, match="overlap"):
        moe.AdamTensors(T)


def test_adamw_behind_its_norm(moe):
    """The step is launched while the norm's kernel runs, and waits for it: many in a row without a
    pause, the gradients changed between, are what they are with pauses."""
    sizes = [3_000_001, 70_000, 5]
    A, B = adam_tensors(sizes, 32, [F32], seed=6), adam_tensors(sizes, 32, [F32], seed=6)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.05)
    norms = []
    for T, pause in ((A, False), (B, True)):
        plan, state = moe.AdamTensors(T), moe.adam_state(0, 0.9, 0.99)
        norm, kept = torch.zeros(1, device="cuda"), []
        for i in range(12):
            for t in T:
                t["g"].mul_(1.0 + 0.25 * math.cos(i))
            if pause:
                torch.cuda.synchronize()
            moe.grad_norm(plan, state, norm)
            if pause:
                torch.cuda.synchronize()
            moe.adamw(cfg, plan, state, norm)
            kept.append(norm.clone())
        norms.append(torch.cat(kept))
    assert torch.equal(*norms)
    for a, b in zip(A, B):
        for n in ("p", "m", "v"):
            assert torch.equal(a[n], b[n])


def test_adam_plan_keeps_its_memory(moe):
    """A tensor whose storage is replaced: the plan goes on with the one that it was made with."""
    T = adam_tensors([5000], 32, [F32])
    plan, state = moe.AdamTensors(T), moe.adam_state(0, 0.9, 0.99)
    p, old = T[0]["p"], T[0]["p"].clone()
    p.data = torch.full_like(p, 3.0)
    moe.adamw(moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8), plan, state)
    assert bool((p == 3.0).all())
    assert not torch.equal(plan.tensors[0]["p"], old)


def test_block_refuses_its_input_as_output(moe):
    _, _, _, block, x, _ = setup(32)
    with pytest.raises(ValueError, match="another"):
        block.forward(x, x.view(32, -1))


@pytest.mark.parametrize("gate,st", [("channel", BF), ("element", F32), ("token", BF)])
def test_norms_captured_beside_other_sizes(moe, gate, st):
    """A captured pair of calls, replayed while eager calls of other sizes come between."""
    rows, d = 300, 1536
    q = {n: normal(i, rows, d, dtype=t) for i, (n, t) in enumerate(
        dict(y=BF, x=st, dh=st, dn=BF).items())}
    gates = dict(channel=normal(8, d, dtype=F32), token=normal(8, rows, dtype=F32),
                 element=normal(8, rows, d))
    g, wp, wn = gates[gate], normal(9, d, dtype=F32), normal(10, d, dtype=F32)
    ws = torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8, device="cuda")

    def buffers():
        e = lambda *s, t=F32: torch.empty(s, dtype=t, device="cuda")   # noqa: E731
        return dict(h=e(rows, d, t=st), n=e(rows, d, t=BF), ry=e(rows), rh=e(rows),
                    dx=e(rows, d, t=st), dy=e(rows, d, t=BF), dg=torch.empty_like(g), dwp=e(d),
                    dwn=e(d))

    def run(b):
        moe.norm_out(q["y"], q["x"], wp, g, wn, b["h"], b["n"], b["ry"], b["rh"])
        moe.norm_out_grad(q["dh"], q["dn"], q["y"], b["h"], wp, g, wn, b["ry"], b["rh"], b["dx"],
                          b["dy"], b["dg"], b["dwp"], b["dwn"], ws)
    a, b = buffers(), buffers()
    run(a)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(a)
    small = normal(11, 5, 64, dtype=F32)
    for seed in (20, 30):
        for i, t in enumerate(q.values()):
            t.copy_(normal(seed + i, rows, d, dtype=t.dtype))
        moe.norm_in(small, wp[:64].clone(), torch.empty((5, 64), dtype=BF, device="cuda"))
        graph.replay()
        run(b)
        for n in a:
            assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("before", ["nothing", "fill", "copy", "join", "fork"])
def test_adamw_captured_behind_other_work(moe, before):
    """The step with a norm captured where the norm's kernel is not the node before it: first of the
    graph, behind a fill or a copy, behind two streams that meet, and on a stream of its own."""
    A = adam_tensors([70_000, 33], 32, [F32], seed=1)
    B = copy_of(A)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.05)
    pa, sa = moe.AdamTensors(A), moe.adam_state(0, 0.9, 0.99)
    pb, sb = moe.AdamTensors(B), moe.adam_state(0, 0.9, 0.99)
    norm, other = torch.full((1,), 0.5, device="cuda"), torch.zeros(1 << 22, device="cuda")
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        if before == "nothing":
            moe.adamw(cfg, pa, sa, norm)
        elif before in ("fill", "copy"):
            if before == "fill":
                other.zero_()
            A[0]["g"].copy_(B[0]["g"])
            moe.adamw(cfg, pa, sa, norm)
        else:
            side.wait_stream(main)
            with torch.cuda.stream(side):
                A[0]["g"].copy_(B[0]["g"])
                other.add_(1.0)
                if before == "fork":
                    moe.adamw(cfg, pa, sa, norm)
            if before == "join":
                norm.add_(0.0)
                main.wait_stream(side)
                moe.adamw(cfg, pa, sa, norm)
            else:
                main.wait_stream(side)
    for step in range(3):
        B[0]["g"].copy_(normal(step, 70_000, std=1e-3, dtype=F32))
        if before == "nothing":
            A[0]["g"].copy_(B[0]["g"])
        graph.replay()
        moe.adamw(cfg, pb, sb, norm)
        for a, b in zip(A, B):
            for n in ("p", "m", "v"):
                assert torch.equal(a[n], b[n]), (step, n)
    assert moe.adam_step(sa) == 3


def test_norms_past_2_31_elements(moe):
    """Rows whose offsets do not fit 31 bits of elements, nor 32 of bytes: the first and last rows are
    what calls of these rows alone give, the weights' gradients those of a sum over parts."""
    rows, d, part = 270_000, 8192, 3000
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    one = torch.randn((part, d), generator=g, device="cuda").to(BF)
    x, dn = one.repeat(rows // part, 1), one.flip(0).repeat(rows // part, 1)
    w = normal(4, d, std=0.2, mean=1.0, dtype=F32)
    n, r = torch.empty_like(x), torch.empty(rows, device="cuda")
    moe.norm_in(x, w, n, r)
    n1, r1 = torch.empty_like(one), torch.empty(part, device="cuda")
    moe.norm_in(one, w, n1, r1)
    for k in (0, rows // part // 2, rows // part - 1):
        assert torch.equal(n[k * part:(k + 1) * part], n1)
        assert torch.equal(r[k * part:(k + 1) * part], r1)
    dw, ws = torch.empty_like(w), torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8,
                                              device="cuda")
    moe.norm_in_grad(dn, x, w, r, x, n, dw, ws)
    dx1, dw1 = torch.empty_like(one), torch.empty_like(w)
    moe.norm_in_grad(dn[:part], one, w, r1, one, dx1, dw1, ws)
    for k in (0, rows // part // 2, rows // part - 1):
        assert torch.equal(n[k * part:(k + 1) * part], dx1)
    xh = one.double() * r1.double()[:, None]
    ref, mag = (one.flip(0).double() * xh).sum(0), (one.flip(0).double() * xh).abs().sum(0)
    # each of 152 CTAs' 1800 rows in fp32, then 152 sums
    assert bool(((dw.double() - ref * (rows // part)).abs()
                 <= 2000 * 2.0 ** -24 * mag * (rows // part)).all())


def test_route_grad_past_2_31_elements(moe):
    T, d, E, k = 300_032, 7168, 16, 2
    q = route_inputs(T, 128, E, k, 0.5, seed=3)
    part = normal(5, 1024, d)
    x = part.repeat(T // 1024, 1)
    w = normal(6, E, d, std=0.05, dtype=F32)
    c = route_cfg(moe, T, d, E, k)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    moe.route_grad(c, x, w, q["idx"], q["s"], q["dw"], x, dx, dw, route_ws(moe, c))
    for t0 in (0, T // 2, T - 1000):
        few = slice(t0, t0 + 1000)
        cf = route_cfg(moe, 1000, d, E, k)
        dxf, dwf = torch.empty_like(x[few]), torch.empty_like(w)
        moe.route_grad(cf, x[few], w, q["idx"][few], q["s"][few], q["dw"][few], x[few], dxf, dwf,
                       route_ws(moe, cf))
        assert torch.equal(dx[few], dxf)
    Z, M = route_reference(q, 2.5, E)
    X = part.double()
    folded = Z.view(-1, 1024, E).sum(0), M.view(-1, 1024, E).sum(0)
    ref, mag = folded[0].t() @ X, folded[1].t() @ X.abs()
    # segments of at most 1024 choices in fp32, then at most 600 of them, and dz's own k + 9 roundings
    assert bool(((dw.double() - ref).abs() <= 1700 * 2.0 ** -24 * mag + 1e-30).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_past_2_31_elements(moe, bits):
    """A tensor of more than 2^31 elements: its ends are what a step over them alone gives (in 8 bits
    the random numbers go by the block, so there only the first end has the same)."""
    n, end = 2 ** 31 + 128 * 1000 + 5, 128 * 1000 + 5
    big = adam_tensors([end], bits, [BF], seed=4, copies=False)[0]

    def repeated(t):   # the tensor's last `end` elements, and its first ones, are t's
        out = torch.zeros(n * t.numel() // end if t.numel() == end else (n + 127) // 128,
                          dtype=t.dtype, device="cuda")
        out[:t.numel()] = t
        out[-t.numel():] = t
        return out
    long = {k: repeated(v) if isinstance(v, torch.Tensor) else v for k, v in big.items()}
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=1e9)
    pa, sa = moe.AdamTensors([long], state_bits=bits), moe.adam_state(0, 0.9, 0.99)
    pb, sb = moe.AdamTensors([big], state_bits=bits), moe.adam_state(0, 0.9, 0.99)
    norm = torch.zeros(1, device="cuda")
    moe.grad_norm(pa, sa, norm)
    exact = math.sqrt(2 * float(big["g"].double().square().sum()))
    assert abs(float(norm) - exact) <= 4 * 2.0 ** -24 * exact
    moe.adamw(cfg, pa, sa, norm)
    moe.adamw(cfg, pb, sb, norm)
    for k in ("p", "m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
        a, b = long[k], big[k]
        assert torch.equal(a[:b.numel()], b), k
        if bits == 32 or k not in ("m", "v"):
            assert torch.equal(a[-b.numel():], b), k
        assert bool((a[b.numel() + 128:b.numel() + 10 ** 6] == (1.0 if "scale" in k else 0)).all())
