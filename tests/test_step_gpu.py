"""The norms around a block, the router's gradient and AdamW on the GPU against their formulas in 64
bits.

Tolerances. A stored result is off by its own rounding, at most half a step: 2^-8 of its size in bf16,
2^-24 in fp32. Before it, sums in fp32: a sum of m products is off by at most (m + 1) 2^-24 S, S the sum
of their magnitudes, for any order. The kernels add a row of d columns in chains of at most 16 terms
and 10 levels of a tree (26 additions), so with the few roundings before and after it each quantity of
a row is off by less than EPS = 2^-18 of the magnitudes that it is made of.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
EPS = 2.0 ** -18


@pytest.fixture(scope="module")
def moe():
    import combine_grouped_gemm_gb300 as m
    return m


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(seed, *shape, std=1.0, mean=0.0, dtype=BF):
    return (torch.randn(shape, generator=gen_of(seed), device="cuda") * std + mean).to(dtype)


def within(got, ref, slack):
    """|got - ref| <= got's own rounding + slack, element by element; every element finite."""
    got64 = got.double()
    own = ref.abs() * (2.0 ** -8 if got.dtype is BF else 2.0 ** -24)
    assert bool(torch.isfinite(got64).all())
    over = (got64 - ref).abs() - (own + slack + 1e-37)
    assert float(over.max() if over.numel() else -1.0) <= 0.0


def rms(x, eps):
    return (x.square().mean(1) + eps) ** -0.5


# ---------------------------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------------------------
SIZES = [(1, 8), (1, 7168), (3, 264), (5, 16384), (64, 7168), (70, 1000), (200, 8192), (33, 8200),
         (1000, 64), (400, 2048), (5000, 256), (1, 16)]


@pytest.mark.parametrize("st", [BF, F32])
@pytest.mark.parametrize("rows,d", SIZES)
def test_norm_in_and_its_gradient(moe, rows, d, st):
    x, w = normal(1, rows, d, std=3.0, dtype=st), normal(2, d, std=0.2, mean=1.0, dtype=F32)
    if rows > 2:
        x[rows // 2] = 0   # a row of padding
    n = torch.full((rows, d), float("nan"), dtype=BF, device="cuda")
    r = torch.full((rows,), float("nan"), device="cuda")
    moe.norm_in(x, w, n, r, eps=1e-5)
    X, W = x.double(), w.double()
    R = rms(X, 1e-5)
    within(r, R, EPS * R)
    N = X * R[:, None] * W
    within(n, N, EPS * N.abs())
    n2 = torch.empty_like(n)
    moe.norm_in(x, w, n2, eps=1e-5)
    assert torch.equal(n, n2)

    dn, dres = normal(3, rows, d, std=0.05), normal(4, rows, d, std=0.05, dtype=st)
    ws = torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8, device="cuda").fill_(255)
    dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
    moe.norm_in_grad(dn, x, w, r, dres, dx, dw, ws)
    R, A = r.double(), dn.double() * W
    H = X * R[:, None]
    ref = dres.double() + R[:, None] * (A - H * (A * H).mean(1, keepdim=True))
    mag = dres.double().abs() + R[:, None] * (A.abs() + H.abs() * (A * H).abs().mean(1, keepdim=True))
    within(dx, ref, EPS * mag)
    terms = dn.double() * H
    col = (rows + 64) * 2.0 ** -24 * terms.abs().sum(0)
    within(dw, terms.sum(0), col)
    # without the residual's gradient, in place of nothing; the weight's added to what is there
    dx2, dw2 = torch.empty_like(x), dw.clone()
    moe.norm_in_grad(dn, x, w, r, None, dx2, dw2, ws, accumulate=True)
    within(dx2, ref - dres.double(), EPS * mag)
    within(dw2, 2 * terms.sum(0), 3 * col)
    # in the residual's place, no weight gradient
    moe.norm_in_grad(dn, x, w, r, dres, dres, None, ws)
    assert torch.equal(dres, dx)


def gate_of(kind, rows, d):
    g = gen_of(9)
    if kind == "none":
        return None
    if kind == "channel":
        return torch.rand((d,), generator=g, device="cuda") - 0.3
    if kind == "token":
        return torch.rand((rows, 1), generator=g, device="cuda")
    return (torch.rand((rows, d), generator=g, device="cuda") - 0.3).to(BF)


FORMS = [(g, p, n) for g in ("none", "channel", "token", "element") for p in (True, False)
         for n in (True, False)]
OUT_SIZES = [(1, 7168, BF), (3, 264, F32), (70, 1000, BF), (5, 16384, F32), (33, 8200, BF),
             (400, 2048, F32), (3000, 64, BF), (300, 7168, BF), (160, 7168, F32), (4, 16384, BF)]


def wide(t):
    return None if t is None else t.double()


@pytest.mark.parametrize("gate,post,nxt", FORMS)
@pytest.mark.parametrize("rows,d,st", OUT_SIZES)
def test_norm_out_and_its_gradient(moe, rows, d, st, gate, post, nxt):
    eps, res, out = 1e-6, 0.9, 0.7
    y, x = normal(1, rows, d, std=0.6), normal(2, rows, d, std=2.0, dtype=st)
    if rows > 2:
        y[rows // 3], x[rows // 3] = 0, 0
    wp = normal(3, d, std=0.2, mean=1.0, dtype=F32) if post else None
    wn = normal(4, d, std=0.2, mean=1.0, dtype=F32) if nxt else None
    g = gate_of(gate, rows, d)
    h = torch.full_like(x, float("nan"))
    n = torch.full_like(y, float("nan")) if nxt else None
    ry = torch.empty(rows, device="cuda") if post else None
    rh = torch.empty(rows, device="cuda") if nxt else None
    moe.norm_out(y, x, wp, g, wn, h, n, ry, rh, eps=eps, res_scale=res, out_scale=out)

    Y, X = y.double(), x.double()
    G = torch.ones((), dtype=torch.float64, device="cuda") if g is None else g.double()
    S = Y
    if post:
        RY = rms(Y, eps)
        within(ry, RY, EPS * RY)
        S = Y * RY[:, None] * wp.double()
    res32, out32 = (float(torch.tensor(v, dtype=F32)) for v in (res, out))
    H = res32 * X + out32 * G * S
    dH = EPS * ((res32 * X).abs() + (out32 * G * S).abs())
    within(h, H, dH)
    if nxt:
        RH = rms(H, eps)
        # r_h moves with the error of h at most as its norm does
        rel = EPS + dH.norm(dim=1) * (H.square().sum(1) + d * eps) ** -0.5
        within(rh, RH, RH * rel)
        within(n, H * RH[:, None] * wn.double(),
               (RH[:, None] * wn.double()).abs() * (dH + H.abs() * rel[:, None]))

    # gradients, from what the forward pass stored
    dh = normal(5, rows, d, std=0.05, dtype=st)
    dn = normal(6, rows, d, std=0.05) if nxt else None
    ws = torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8, device="cuda").fill_(255)
    nan = float("nan")

    def outputs():
        return (torch.full_like(x, nan), torch.full_like(y, nan),
                None if g is None else torch.full_like(g, nan),
                None if wp is None else torch.full_like(wp, nan),
                None if wn is None else torch.full_like(wn, nan))
    need_y = post or gate != "none"
    args = (dh, dn, y if need_y else None, h if nxt else None, wp, g, wn, ry, rh)
    dx, dy, dg, dwp, dwn = o = outputs()
    moe.norm_out_grad(*args, *o, ws, res_scale=res, out_scale=out)

    T = dh.double()
    mag = T.abs()
    if nxt:
        R, A = rh.double()[:, None], dn.double() * wn.double()
        HH = h.double() * R
        T = T + R * (A - HH * (A * HH).mean(1, keepdim=True))
        mag = mag + R * (A.abs() + HH.abs() * (A * HH).abs().mean(1, keepdim=True))
        terms = dn.double() * HH
        within(dwn, terms.sum(0), (rows + 64) * 2.0 ** -24 * terms.abs().sum(0))
    within(dx, res32 * T, EPS * res32 * mag)
    U, mU = out32 * T, out32 * mag
    YH = Y * ry.double()[:, None] if post else Y
    S = YH * wp.double() if post else Y
    DS, mDS = U * G, (mU * G).abs()
    if post:
        R, P = ry.double()[:, None], DS * wp.double()
        mP = mDS * wp.double().abs()
        ref = R * (P - YH * (P * YH).mean(1, keepdim=True))
        within(dy, ref, 2 * EPS * R * (mP + YH.abs() * (mP * YH.abs()).mean(1, keepdim=True)))
        terms = DS * YH
        within(dwp, terms.sum(0), EPS * (mDS * YH).abs().sum(0)
               + (rows + 64) * 2.0 ** -24 * (mDS * YH).abs().sum(0))
    else:
        within(dy, DS, EPS * mDS)
    if gate == "channel":
        m = (mU * S).abs().sum(0)
        within(dg, (U * S).sum(0), (EPS + (rows + 64) * 2.0 ** -24) * m)
    elif gate == "token":
        within(dg, (U * S).sum(1, keepdim=True), 2 * EPS * (mU * S).abs().sum(1, keepdim=True))
    elif gate == "element":
        within(dg, U * S, EPS * (mU * S).abs())
    # again: the same bits
    o2 = outputs()
    moe.norm_out_grad(*args, *o2, ws, res_scale=res, out_scale=out)
    for a, b in zip(o, o2):
        assert a is None or torch.equal(a, b)
    # outputs in their inputs' places, nothing else wanted
    dh2, dn2 = dh.clone(), None if dn is None else dn.clone()
    moe.norm_out_grad(dh2, dn2, *args[2:], dh2, dy if dn2 is None else dn2, None, None, None, ws,
                      res_scale=res, out_scale=out)
    assert torch.equal(dh2, dx) and (dn2 is None or torch.equal(dn2, dy))
    x2, y2 = x.clone(), y.clone()
    moe.norm_out(y2, x2, wp, g, wn, x2, y2 if nxt else None, eps=eps, res_scale=res, out_scale=out)
    assert torch.equal(x2, h) and (not nxt or torch.equal(y2, n))
    # accumulated sums; no gradient from the residual's side
    if nxt:
        sums = [None if t is None else t.clone() for t in (dg if gate == "channel" else None, dwp, dwn)]
        other = dg.clone() if gate in ("token", "element") else sums[0]
        moe.norm_out_grad(*args, dx, dy, other, sums[1], sums[2], ws, res_scale=res,
                          out_scale=out, accumulate=True)
        for a, b in zip(sums, (dg, dwp, dwn)):
            assert a is None or torch.equal(a, b + b)
        if gate in ("token", "element"):
            assert torch.equal(other, dg)
        moe.norm_out_grad(None, dn, *args[2:], dx2 := torch.empty_like(x), dy, None, None, None, ws,
                          res_scale=res, out_scale=out)
        within(dx2, res32 * (T - dh.double()), EPS * res32 * mag)


def test_norm_gradient_against_differences(moe):
    """norm_out's gradients against central differences of a 64-bit loss."""
    rows, d, eps, res, out = 4, 40, 1e-3, 0.9, 0.7
    t = dict(y=normal(1, rows, d), x=normal(2, rows, d, dtype=F32),
             wp=normal(3, d, std=0.2, mean=1.0, dtype=F32), g=normal(4, d, std=0.3, dtype=F32),
             wn=normal(5, d, std=0.2, mean=1.0, dtype=F32))
    ch, cn = normal(6, rows, d, dtype=F32), normal(7, rows, d)

    def loss(y, x, wp, g, wn):
        h = res * x + out * g * (y * rms(y, eps)[:, None] * wp)
        return float((h * ch.double()).sum() + (h * rms(h, eps)[:, None] * wn * cn.double()).sum())
    h, n = torch.empty_like(t["x"]), torch.empty_like(t["y"])
    ry, rh = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.norm_out(t["y"], t["x"], t["wp"], t["g"], t["wn"], h, n, ry, rh, eps=eps, res_scale=res,
                 out_scale=out)
    o = dict(x=torch.empty_like(t["x"]), y=torch.empty_like(t["y"]), g=torch.empty_like(t["g"]),
             wp=torch.empty_like(t["wp"]), wn=torch.empty_like(t["wn"]))
    ws = torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8, device="cuda")
    moe.norm_out_grad(ch, cn, t["y"], h, t["wp"], t["g"], t["wn"], ry, rh, o["x"], o["y"], o["g"],
                      o["wp"], o["wn"], ws, res_scale=res, out_scale=out)
    base = {k: v.double() for k, v in t.items()}
    for name, at in (("y", (1, 7)), ("y", (3, 39)), ("x", (0, 0)), ("x", (2, 20)), ("g", (5,)),
                     ("wp", (17,)), ("wn", (30,))):
        step = 1e-5
        lo, hi = ({**base, name: base[name].clone()} for _ in range(2))
        lo[name][at] -= step
        hi[name][at] += step
        slope = (loss(**hi) - loss(**lo)) / (2 * step)
        got = float(o[name][at])
        # 2^-8 for dy in bf16; differences of order step^2; a loss of ~100 in 64 bits / step
        assert abs(got - slope) <= 2.0 ** -8 * abs(slope) + 1e-4, (name, at, got, slope)


def test_norm_no_rows(moe):
    d = 64
    x = torch.empty((0, d), dtype=F32, device="cuda")
    y = torch.empty((0, d), dtype=BF, device="cuda")
    w, dw = torch.ones(d, device="cuda"), torch.full((d,), 3.0, device="cuda")
    ws = torch.empty(moe.norm_ws_bytes(0, d), dtype=torch.uint8, device="cuda")
    r = torch.empty(0, device="cuda")
    moe.norm_in(x, w, y, r)
    moe.norm_in_grad(y, x, w, r, None, torch.empty_like(x), dw, ws, accumulate=True)
    assert bool((dw == 3.0).all())
    moe.norm_in_grad(y, x, w, r, None, torch.empty_like(x), dw, ws)
    assert bool((dw == 0.0).all())


# ---------------------------------------------------------------------------------------------
# Router
# ---------------------------------------------------------------------------------------------
def route_inputs(T, d, E, k, skew, seed=0):
    g = gen_of(seed)
    pop = torch.arange(1, E + 1, device="cuda").float() ** -skew
    race = torch.empty((T, E), device="cuda").exponential_(generator=g) / pop
    idx = race.topk(k, 1, largest=False).indices.to(torch.int32)
    s = torch.sigmoid(torch.randn((T, k), generator=g, device="cuda") * 2)
    return dict(x=normal(seed + 1, T, d), w=normal(seed + 2, E, d, std=0.05, dtype=F32), idx=idx, s=s,
                dw=torch.randn((T, k), generator=g, device="cuda") * 0.1,
                dx_in=normal(seed + 3, T, d, std=0.1))


def route_reference(q, scale, E):
    s, dw = q["s"].double(), q["dw"].double()
    p = s / s.sum(1, keepdim=True)
    live = (q["idx"] >= 0) & (q["idx"] < E)
    dz = scale * p * (1 - s) * (dw - (p * dw).sum(1, keepdim=True)) * live
    mag = scale * p * (1 - s) * (dw.abs() + (p * dw).abs().sum(1, keepdim=True)) * live
    out = []
    for z in (dz, mag):
        Z = torch.zeros((s.shape[0], E), dtype=torch.float64, device="cuda")
        Z.scatter_add_(1, q["idx"].clamp(0, E - 1).long(), z)
        out.append(Z)
    return out


def route_cfg(moe, T, d, E, k, scale=2.5):
    return moe.Cfg(T, d, E, k, 1, 1, 128, 0, 1, scale, moe.MOE_BF16, moe.MOE_BF16)


def check_route(moe, q, T, d, E, k, c, ws, bits=0):
    dx, dwg = torch.full_like(q["x"], float("nan")), torch.full_like(q["w"], float("nan"))
    moe.route_grad(c, q["x"], q["w"], q["idx"], q["s"], q["dw"], q["dx_in"], dx, dwg, ws)
    Z, M = route_reference(q, 2.5, E)
    W, X, B = q["w"].double(), q["x"].double(), q["dx_in"].double()
    # dz: sums of k terms and 8 roundings; then k + 1 (tokens) or at most T (gate weights) additions
    ez = (k + 9) * 2.0 ** -24
    within(dx, B + Z @ W, (ez + (k + 2) * 2.0 ** -24) * (B.abs() + M @ W.abs()))
    within(dwg, Z.t() @ X, (ez + (T + 16) * 2.0 ** -24) * (M.t() @ X.abs()))
    assert moe.read_status(ws) == bits
    return dx, dwg


ROUTES = [(1, 128, 8, 1, 0.0), (1, 7168, 256, 8, 0.0), (3, 256, 16, 2, 0.0), (64, 7168, 256, 8, 0.0),
          (257, 384, 1024, 32, 0.8), (300, 640, 7, 7, 0.0), (1000, 1152, 64, 6, 1.2),
          (2500, 512, 8, 1, 3.0), (513, 2048, 300, 5, 0.8), (1024, 7168, 256, 8, 0.8),
          (700, 128, 1, 1, 0.0), (5000, 256, 33, 4, 1.2)]


@pytest.mark.parametrize("T,d,E,k,skew", ROUTES)
def test_route_grad(moe, T, d, E, k, skew):
    q = route_inputs(T, d, E, k, skew)
    c = route_cfg(moe, T, d, E, k)
    ws = torch.empty(moe.route_grad_ws_bytes(c), dtype=torch.uint8, device="cuda").fill_(255)
    moe.clear_status(ws)
    dx, dwg = check_route(moe, q, T, d, E, k, c, ws)
    # again: the same bits; in place, the gate weights' gradient added to
    dx2, dwg2 = q["dx_in"].clone(), dwg.clone()
    moe.route_grad(c, q["x"], q["w"], q["idx"], q["s"], q["dw"], dx2, dx2, dwg2, ws, accumulate=True)
    assert torch.equal(dx2, dx) and torch.equal(dwg2, dwg + dwg)
    # no gradient from elsewhere
    zero = torch.zeros_like(q["x"])
    moe.route_grad(c, q["x"], q["w"], q["idx"], q["s"], q["dw"], zero, dx2, dwg2, ws)
    moe.route_grad(c, q["x"], q["w"], q["idx"], q["s"], q["dw"], None, dx, dwg2, ws)
    assert torch.equal(dx, dx2) and torch.equal(dwg, dwg2)


@pytest.mark.parametrize("T", [5, 400, 3000])
def test_route_grad_of_odd_choices(moe, T):
    """Dropped choices (-1), choices of experts that there are not, one expert twice, all tokens on
    one expert."""
    d, E, k = 256, 24, 4
    q = route_inputs(T, d, E, k, 0.0, seed=5)
    c = route_cfg(moe, T, d, E, k)
    ws = torch.zeros(moe.route_grad_ws_bytes(c), dtype=torch.uint8, device="cuda")
    q["idx"][::3, 1] = -1
    check_route(moe, q, T, d, E, k, c, ws)
    q["idx"][1::2, 2] = q["idx"][1::2, 0]
    q["idx"][2] = -1
    check_route(moe, q, T, d, E, k, c, ws)
    q["idx"][1::4, 3] = E
    q["idx"][2::4, 3] = -7
    q["idx"][3::4, 3] = 2 ** 31 - 1
    check_route(moe, q, T, d, E, k, c, ws, bits=moe.MOE_DEV_BOUNDS)
    moe.clear_status(ws)
    q["idx"][:] = E - 1
    check_route(moe, q, T, d, E, k, c, ws)


@pytest.mark.parametrize("T", [16, 200, 1100, 2100])
def test_route_save_keeps_the_scores(moe, T):
    """The chosen experts' scores, with route's own choices and weights, in each of the router's
    kernels."""
    import dataclasses

    import synth
    for base in (synth.CONFIGS["tiny"], synth.CONFIGS["dsv3_decode"]):
        cfg = dataclasses.replace(base, T=T, R=1, d=512)
        inp = synth.make_router_inputs(cfg, "cuda")
        b = moe.Buffers(cfg)
        moe.route(cfg, inp["x"], inp["w_gate"], inp["bias"], b["topk_idx"], b["topk_w"], b["ws"])
        idx, w = torch.empty_like(b["topk_idx"]), torch.empty_like(b["topk_w"])
        s = torch.full_like(w, float("nan"))
        moe.route_save(cfg, inp["x"], inp["w_gate"], inp["bias"], idx, w, s, b["ws"])
        assert torch.equal(idx, b["topk_idx"]) and torch.equal(w, b["topk_w"])
        z = inp["x"].double() @ inp["w_gate"].double().t()
        mag = inp["x"].double().abs() @ inp["w_gate"].double().abs().t()
        ref = torch.sigmoid(z).gather(1, idx.long())
        # sigmoid's slope is at most 1/4; the logit is a sum of d products
        within(s, ref, (cfg.d + 8) * 2.0 ** -26 * mag.gather(1, idx.long()) + 2.0 ** -21)


# ---------------------------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------------------------
def adam_tensors(sizes, bits, gtypes, seed=0, copies=True):
    out = []
    for i, n in enumerate(sizes):
        gt = gtypes[i % len(gtypes)]
        p = normal(seed + 10 * i, n, std=0.02, dtype=F32)
        t = dict(p=p, g=normal(seed + 10 * i + 1, n, std=1e-3, dtype=gt),
                 w=torch.zeros(n, dtype=BF, device="cuda") if copies and i % 2 == 0 else None,
                 weight_decay=0.1 * (i % 3), seed=seed + i)
        if bits == 32:
            t.update(m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda"))
        else:
            b = (n + 127) // 128
            t.update(m=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                     v=torch.zeros(n, dtype=torch.uint8, device="cuda"),
                     m_scale=torch.zeros(b, device="cuda"), v_scale=torch.zeros(b, device="cuda"))
        out.append(t)
    return out


ADAM_SIZES = [1, 2, 3, 5, 127, 128, 129, 1000, 4095, 4096, 4097, 70001]


def copy_of(tensors):
    return [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
            for t in tensors]


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("sizes", [ADAM_SIZES, [300] * 300 + ADAM_SIZES, [2_500_003]])
def test_adamw_32(moe, sizes, clip):
    T = adam_tensors(sizes, 32, [F32, BF])
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.01 if clip else 0.0)
    plan, state = moe.AdamTensors(T), moe.adam_state(0, 0.9, 0.99)
    norm = torch.zeros(1, device="cuda")
    for step in (1, 2, 3):
        before = copy_of(T)
        for i, t in enumerate(T):
            t["g"].copy_(normal(1000 * step + i, t["g"].numel(), std=1e-3, dtype=t["g"].dtype))
        f = 1.0
        if clip:
            moe.grad_norm(plan, state, norm)
            exact = sum(float(t["g"].double().square().sum()) for t in T) ** 0.5
            # four squares in fp32 a sum, all positive, then fp64: 5 roundings, half in the root
            assert abs(float(norm) - exact) <= 4 * 2.0 ** -24 * exact
            f = min(1.0, 0.01 / float(norm))
            moe.adamw(cfg, plan, state, norm)
        else:
            moe.adamw(cfg, plan, state)
        assert moe.adam_step(state) == step
        for a, b in zip(before, T):
            g = b["g"].double() * f
            m = 0.9 * a["m"].double() + (1 - 0.9) * g
            v = 0.99 * a["v"].double() + (1 - 0.99) * g * g
            # fp32 constants, the factor and three roundings each
            within(b["m"], m, 6 * 2.0 ** -24 * (0.9 * a["m"].double().abs() + 0.1 * g.abs()))
            within(b["v"], v, 8 * 2.0 ** -24 * v)
            mh, vh = b["m"].double() / (1 - 0.9 ** step), b["v"].double() / (1 - 0.99 ** step)
            P = a["p"].double()
            move = 1e-3 * mh / (vh.sqrt() + 1e-8)
            ref = P * (1 - 1e-3 * b["weight_decay"]) - move
            within(b["p"], ref, 2.0 ** -23 * P.abs() + 2.0 ** -20 * move.abs())
            if b["w"] is not None:
                assert torch.equal(b["w"], b["p"].to(BF))
    assert moe.read_status(state) == 0


def mix(x):
    import numpy as np
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x7FEB352D)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x846CA68B)
    return x ^ (x >> np.uint32(16))


def e4m3_table():
    import numpy as np
    return torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()


def hold_reference(x, r16, root):
    """Codes and scales of x from the definition: the code below, or the one above by the odds and
    the random number (in numpy fp32, whose operations are IEEE's)."""
    import numpy as np
    n, f = x.size, np.float32
    nb = (n + 127) // 128
    b = np.zeros(nb * 128, f)
    b[:n] = x
    b = b.reshape(nb, 128)
    mag = np.abs(b)
    amax = mag.max(1, keepdims=True)
    scale = np.where(amax > 0, amax * (f(1) / f(448)), f(1)).astype(f)
    q = np.minimum((mag / scale).astype(f), f(448))
    r = r16.reshape(nb, 128).astype(np.int64)
    tab = np.concatenate([e4m3_table(), [f(480)]]).astype(f)
    # below 2^-6, q counts as rounded to multiples of 2^-29, which 2^-6 + q has
    at = np.where(q < f(2.0 ** -6), (q + f(2.0 ** -6)).astype(f) - f(2.0 ** -6), q).astype(f)
    low = np.searchsorted(tab, at, side="right") - 1
    lo, hi = tab[low], tab[low + 1]
    if root:
        up = r.astype(f) * ((hi - lo) * (hi + lo)) < ((q - lo) * (q + lo)) * f(65536)
    else:   # the distance to lo in 2^-20 of a step, and the random bits, pass a whole step together
        frac = np.round((at - lo).astype(np.float64) / (hi - lo) * 2 ** 20).astype(np.int64)
        up = frac + (r << 4) >= 2 ** 20
    code = low + up
    if root:
        code = np.where((b > 0) & (code == 0), 1, code)
    code = code | np.where(np.signbit(b), 128, 0)
    return code.reshape(-1)[:n].astype(np.uint8), scale.reshape(-1)


@pytest.mark.parametrize("clip", [False, True])
@pytest.mark.parametrize("sizes", [ADAM_SIZES, [300_007]])
def test_adamw_8_bit_code_by_code(moe, sizes, clip):
    import numpy as np
    f = np.float32
    T = adam_tensors(sizes, 8, [F32, BF], seed=3)
    for t in T:   # gradients that differ widely inside a block
        t["g"].mul_(torch.exp(normal(77, t["g"].numel(), std=3.0, dtype=F32)).to(t["g"].dtype))
        t["g"][t["g"].numel() // 2:t["g"].numel() // 2 + 200] = 0
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.01 if clip else 0.0)
    plan, state = moe.AdamTensors(T, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    norm = torch.zeros(1, device="cuda")
    tab = np.concatenate([e4m3_table(), [np.nan]]).astype(f)
    tab = np.concatenate([tab, -tab])
    old = np.seterr(over="ignore")
    for step in (1, 2, 3):
        before = copy_of(T)
        factor = None
        if clip:
            moe.grad_norm(plan, state, norm)
            factor = min(f(0.01) * (f(1) / norm.cpu().numpy()[0]), f(1))
        moe.adamw(cfg, plan, state, norm if clip else None)
        for a, b in zip(before, T):
            n = a["p"].numel()
            g = b["g"].float().cpu().numpy()
            if factor is not None:
                g = g * factor
            sm, sv = (np.repeat(a[k].cpu().numpy(), 128)[:n] for k in ("m_scale", "v_scale"))
            m = tab[a["m"].cpu().numpy()] * sm
            v = tab[a["v"].cpu().numpy()] * sv
            v = v * v
            m = f(0.9) * m + f(1 - 0.9) * g
            v = f(0.99) * v + f(1 - 0.99) * (g * g)
            root = np.sqrt(v)
            key = mix(np.array([(b["seed"] ^ (step * 0x9E3779B9)) & 0xFFFFFFFF], np.uint32))
            nb = (n + 127) // 128
            key = mix(key ^ np.arange(nb, dtype=np.uint32))
            place = (np.arange(128, dtype=np.uint64) * 0x9E3779B9).astype(np.uint32)
            r = mix(key[:, None] + place[None, :]).reshape(-1)
            for name, x, r16 in (("m", m, r >> np.uint32(16)), ("v", root, r & np.uint32(0xFFFF))):
                code, scale = hold_reference(x, r16, name == "v")
                assert np.array_equal(b[name + "_scale"].cpu().numpy(), scale)
                got = b[name].cpu().numpy()
                assert np.array_equal(got & 127, code & 127), (n, name, step)
                assert np.array_equal((got >> 7)[code & 127 > 0], (code >> 7)[code & 127 > 0])
            c1, c2 = 1 - 0.9 ** step, 1 - 0.99 ** step
            move = 1e-3 * (m.astype(np.float64) / c1) / (np.sqrt(v.astype(np.float64) / c2) + 1e-8)
            P = a["p"].double().cpu().numpy()
            ref = P * (1 - 1e-3 * b["weight_decay"]) - move
            err = np.abs(b["p"].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -23 * np.abs(P) + 2.0 ** -20 * np.abs(move) + 1e-37).all()
            if b["w"] is not None:
                assert torch.equal(b["w"], b["p"].to(BF))
    np.seterr(**old)


def test_8_bit_moments_follow_32_bit_ones(moe):
    """A second moment that changes by 0.1 % a step moves in 8 bits too, without a bias: after 400
    steps from a tenth of its final size the mean over the elements is that of 32 bits. (An element
    is off by some codes' steps, 1/8 of it each; the mean over 2^17 elements by 2^-8.5 of that, below
    0.002.)"""
    n = 1 << 17
    cfg = moe.AdamCfg(lr=0.0, beta1=0.9, beta2=0.999, eps=1e-8)
    runs = {}
    for bits in (32, 8):
        T = adam_tensors([n], bits, [F32], copies=False)
        plan, state = moe.AdamTensors(T, state_bits=bits), moe.adam_state(0, 0.9, 0.999)
        for step in range(400):
            size = 1e-4 if step < 100 else 1e-3
            T[0]["g"].copy_(normal(step, n, std=size, dtype=F32).abs() + size)
            moe.adamw(cfg, plan, state)
        t = T[0]
        if bits == 8:
            v = t["v"].view(torch.float8_e4m3fn).double() * t["v_scale"].double().repeat_interleave(128)
            m = t["m"].view(torch.float8_e4m3fn).double() * t["m_scale"].double().repeat_interleave(128)
            runs[bits] = (float(m.mean()), float((v * v).mean()))
        else:
            runs[bits] = (float(t["m"].double().mean()), float(t["v"].double().mean()))
    assert abs(runs[8][0] / runs[32][0] - 1) < 0.005
    assert abs(runs[8][1] / runs[32][1] - 1) < 0.005


def test_adamw_norm_that_is_not_finite_leaves_the_step_out(moe):
    for bits in (32, 8):
        T = adam_tensors([1000, 77], bits, [F32])
        cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=1.0)
        plan, state = moe.AdamTensors(T, state_bits=bits), moe.adam_state(0, 0.9, 0.99)
        norm = torch.zeros(1, device="cuda")
        moe.grad_norm(plan, state, norm)
        moe.adamw(cfg, plan, state, norm)
        before = copy_of(T)
        for bad in (float("inf"), float("nan")):
            T[0]["g"][500] = bad
            moe.grad_norm(plan, state, norm)
            moe.adamw(cfg, plan, state, norm)
            assert moe.adam_step(state) == 1
            assert moe.read_status(state) == moe.MOE_DEV_NONFINITE
            moe.clear_status(state)
            for a, b in zip(before, T):
                for k in ("p", "m", "v", "w"):
                    assert a.get(k) is None or torch.equal(a[k], b[k])
        T[0]["g"][500] = 0.0
        moe.grad_norm(plan, state, norm)
        moe.adamw(cfg, plan, state, norm)
        assert moe.adam_step(state) == 2 and moe.read_status(state) == 0


def test_adamw_captured_with_a_rate_that_changes(moe):
    """A captured step, replayed with another rate each time, gives what eager steps give; its step
    count goes on between replays."""
    sizes = [5000, 128, 33]
    A, B = adam_tensors(sizes, 8, [F32], seed=8), adam_tensors(sizes, 8, [F32], seed=8)
    cfg = moe.AdamCfg(lr=9.0, beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.02)
    lr, norm = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    norm2 = torch.zeros(1, device="cuda")
    pa, sa = moe.AdamTensors(A, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    pb, sb = moe.AdamTensors(B, state_bits=8), moe.adam_state(0, 0.9, 0.99)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        moe.grad_norm(pa, sa, norm)
        moe.adamw(cfg, pa, sa, norm, lr=lr)
    for step, rate in enumerate((1e-3, 2e-3, 0.0, 5e-4)):
        for i, (a, b) in enumerate(zip(A, B)):
            a["g"].copy_(normal(50 * step + i, a["g"].numel(), std=1e-3, dtype=F32))
            b["g"].copy_(a["g"])
        lr.fill_(rate)
        graph.replay()
        moe.grad_norm(pb, sb, norm2)
        c = moe.AdamCfg(lr=float(lr), beta1=0.9, beta2=0.99, eps=1e-8, max_norm=0.02)
        moe.adamw(c, pb, sb, norm2)
        torch.cuda.synchronize()
        assert torch.equal(norm, norm2)
        for a, b in zip(A, B):
            for k in ("p", "m", "v", "m_scale", "v_scale"):
                assert torch.equal(a[k], b[k]), (step, k)
    assert moe.adam_step(sa) == 4


def test_adam_state_resumes(moe):
    """A state made for a step count goes on as the one that has made the steps."""
    A, B = adam_tensors([3000], 32, [F32], seed=4), adam_tensors([3000], 32, [F32], seed=4)
    cfg = moe.AdamCfg(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)
    pa, sa = moe.AdamTensors(A), moe.adam_state(0, 0.9, 0.999)
    for _ in range(5):
        moe.adamw(cfg, pa, sa)
    for k in ("p", "m", "v"):
        B[0][k].copy_(A[0][k])
    pb, sb = moe.AdamTensors(B), moe.adam_state(5, 0.9, 0.999)
    moe.adamw(cfg, pa, sa)
    moe.adamw(cfg, pb, sb)
    assert torch.equal(A[0]["p"], B[0]["p"])   # the corrections differ by 1e-16
    moe.adamw(cfg, moe.AdamTensors([]), sa)    # no tensors: the step counts
    assert moe.adam_step(sa) == 7 and moe.adam_step(sb) == 6


def test_calls_on_two_streams(moe):
    """The calls run on the stream that they are given, with scratch of their own."""
    rows, d = 500, 2048
    s = [torch.cuda.Stream() for _ in range(2)]
    x = [normal(i, rows, d, dtype=F32) for i in range(2)]
    w = normal(5, d, std=0.2, mean=1.0, dtype=F32)
    ws = [torch.empty(moe.norm_ws_bytes(rows, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dn = normal(6, rows, d)
    out = []
    torch.cuda.synchronize()
    for i in range(2):
        n, r = torch.empty((rows, d), dtype=BF, device="cuda"), torch.empty(rows, device="cuda")
        dx, dw = torch.empty_like(x[i]), torch.empty_like(w)
        torch.cuda.synchronize()
        for _ in range(5):
            moe.norm_in(x[i], w, n, r, stream=s[i])
            moe.norm_in_grad(dn, x[i], w, r, None, dx, dw, ws[i], stream=s[i])
        out.append((n, r, dx, dw))
    torch.cuda.synchronize()
    for i in range(2):
        n, r = torch.empty((rows, d), dtype=BF, device="cuda"), torch.empty(rows, device="cuda")
        dx, dw = torch.empty_like(x[i]), torch.empty_like(w)
        moe.norm_in(x[i], w, n, r)
        moe.norm_in_grad(dn, x[i], w, r, None, dx, dw, ws[0])
        for a, b in zip(out[i], (n, r, dx, dw)):
            assert torch.equal(a, b)
