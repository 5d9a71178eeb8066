"""Calls of the training step's operators at the borders of their kernels, captured, back to back and
with values that spoil: the router's gradient, AdamW over more tensors than a call takes, the block."""
import math

import pytest
import torch

from test_block_gpu import setup
from test_step_gpu import (ADAM_SIZES, BF, F32, adam_tensors, check_route, copy_of, normal,
                           route_cfg, route_inputs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def route_ws(moe, c):
    return torch.zeros(moe.route_grad_ws_bytes(c), dtype=torch.uint8, device="cuda")


# 1024 choices: the last in one launch; 512 tokens: the first with a slab, whose columns are 128, 64
# or 32 by the experts; lists whose last 32 choices are few; chunks of other lengths; the widest row
BORDERS = [(128, 256, 16, 8), (129, 256, 16, 8), (1024, 128, 8, 1), (1025, 128, 8, 1),
           (33, 256, 40, 32), (511, 384, 24, 3), (512, 384, 24, 3), (513, 384, 440, 2),
           (600, 384, 460, 3), (600, 640, 1024, 32), (4097, 256, 64, 2), (5200, 128, 9, 7),
           (21000, 128, 12, 3), (520, 65536, 4, 2), (2, 65536, 1024, 32)]


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
