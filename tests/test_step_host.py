"""Refusals of the calls around the layer (norms, router's gradient, optimiser), checked on the host:
nothing here launches GPU work."""
import ctypes

import pytest
import torch

# the addresses are made up, so a check that let one through must not find a device
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="host checks, run without a GPU")

OK = 1 << 20


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__.build()
    import combine_grouped_gemm_gb300 as m
    return m


def norm_cfg(moe, **kw):
    return ctypes.byref(moe.NormCfg(**{**dict(rows=16, d=64, eps=1e-6, res_scale=1.0, out_scale=1.0,
                                              stream_dtype=moe.MOE_BF16, gate=0), **kw}))


def far(n):
    """n addresses 1 TB apart"""
    return [(i + 1) << 40 for i in range(n)]


@pytest.mark.parametrize("rows,d,code", [(-1, 64, 1), (4, 0, 1), (4, 60, 2), (4, 16392, 2),
                                         (2 ** 31 - 1, 128, 2), (0, 8, 0), (5, 16384, 0)])
def test_norm_sizes(moe, rows, d, code):
    L, n = moe._lib, ctypes.c_size_t(0)
    assert L.moe_norm_query(rows, d, ctypes.byref(n)) == code
    assert (n.value > 0) == (code == 0)
    if code:
        c = norm_cfg(moe, rows=rows, d=d)
        assert L.moe_norm_in(c, *far(4), None) == code
        assert L.moe_norm_in_grad(c, *far(7), 0, OK, None) == code
        assert L.moe_norm_out(c, *far(2), OK, None, OK, *far(4), None) == code
        assert L.moe_norm_out_grad(c, *far(4), OK, None, OK, *far(4), None, OK, OK, 0, OK,
                                   None) == code
    assert L.moe_norm_query(4, 64, None) == 1


@pytest.mark.parametrize("change", [dict(eps=-1.0), dict(eps=float("nan")), dict(stream_dtype=1),
                                    dict(res_scale=float("inf")), dict(out_scale=float("nan")),
                                    dict(gate=4), dict(gate=-1)])
def test_norm_configurations(moe, change):
    L, c = moe._lib, norm_cfg(moe, **change)
    a = far(9)
    assert L.moe_norm_out(c, a[0], a[1], None, a[2] if "gate" in change else None, None, a[3], None,
                          None, None, None) == 1
    if not set(change) & {"res_scale", "out_scale", "gate"}:   # norm_in does not read those
        assert L.moe_norm_in(c, *a[:4], None) == 1
    assert L.moe_norm_in(None, *a[:4], None) == 1


def test_norm_pointers(moe):
    L, c = moe._lib, norm_cfg(moe)
    a = far(4)
    for i in range(3):
        b = list(a)
        b[i] = None
        assert L.moe_norm_in(c, *b, None) == 1
    for i in range(4):
        b = list(a)
        b[i] += 8
        assert L.moe_norm_in(c, *b, None) == 3
    names = ["dn", "x", "w", "rstd", "dres", "dx", "dw"]
    for i, name in enumerate(names):
        b = far(7)
        b[i] = None
        if name not in ("dres", "dw"):
            assert L.moe_norm_in_grad(c, *b, 0, 1 << 50, None) == 1, name
        b[i] = OK + 4
        assert L.moe_norm_in_grad(c, *b, 0, 1 << 50, None) == 3, name
    assert L.moe_norm_in_grad(c, *far(7), 0, None, None) == 1   # scratch
    # a gate without its kind and a kind without its gate; a next norm without its output; factors
    # kept of a norm that there is not
    y, x, wp, g, wn, h, n, ry, rh = far(9)
    ch = norm_cfg(moe, gate=moe.MOE_GATE_CHANNEL)
    assert L.moe_norm_out(c, y, x, wp, g, wn, h, n, ry, rh, None) == 1
    assert L.moe_norm_out(ch, y, x, wp, None, wn, h, n, ry, rh, None) == 1
    assert L.moe_norm_out(c, y, x, wp, None, wn, h, None, ry, rh, None) == 1
    assert L.moe_norm_out(c, y, x, wp, None, None, h, n, ry, None, None) == 1
    assert L.moe_norm_out(c, y, x, None, None, wn, h, n, ry, rh, None) == 1
    assert L.moe_norm_out(c, y, x, wp, None, None, h, None, ry, rh, None) == 1
    names = ["dh", "dn", "y", "h", "wp", "g", "wn", "ry", "rh", "dx", "dy", "dg", "dwp", "dwn"]
    base = dict(zip(names, far(14)))

    def grad(cfg=ch, ws=1 << 50, **kw):
        p = {**base, **kw}
        return L.moe_norm_out_grad(cfg, *[p[n] for n in names], 0, ws, None)
    for n in ("dn", "y", "h", "g", "ry", "rh", "dy"):
        assert grad(**{n: None}) == 1, n
    for n in names:
        assert grad(**{n: OK + 8}) == 3, n
    assert grad(ws=None) == 1
    assert grad(wn=None, dwn=None, dh=None) == 1     # nothing to go back from
    assert grad(wn=None) == 1                        # a weight's gradient without the weight
    assert grad(wp=None) == 1
    assert grad(cfg=c, g=None) == 1                  # a gate's gradient without the gate
    assert grad(cfg=c) == 1


def meets(call, sizes, out, instead=()):
    base = {n: (i + 1) << 40 for i, n in enumerate(sizes)}
    for other in sizes:
        if other == out:
            continue
        at = [base[other] + sizes[other] - 16, base[other] - sizes[out] + 16]
        if other not in instead:
            at.append(base[other])
        for p in at:
            assert call(**{**base, out: p}) == 1, (out, other)


def test_norm_outputs_that_meet_an_input(moe):
    L, rows, d = moe._lib, 16, 64
    c, ch = norm_cfg(moe), norm_cfg(moe, gate=moe.MOE_GATE_CHANNEL)
    e, v, r = 2 * rows * d, 4 * d, 4 * rows
    s = dict(x=e, w=v, n=e, rstd=r)
    for out, instead in (("n", ("x",)), ("rstd", ())):
        meets(lambda **p: L.moe_norm_in(c, *p.values(), None), s, out, instead)
    ws = moe.norm_ws_bytes(rows, d) // 16 * 16
    s = dict(dn=e, x=e, w=v, rstd=r, dres=e, dx=e, dw=v, ws=ws)
    for out, instead in (("dx", ("dres",)), ("dw", ()), ("ws", ())):
        meets(lambda dn, x, w, rstd, dres, dx, dw, ws: L.moe_norm_in_grad(
            c, dn, x, w, rstd, dres, dx, dw, 0, ws, None), s, out, instead)
    s = dict(y=e, x=e, wp=v, g=v, wn=v, h=e, n=e, ry=r, rh=r)
    for out, instead in (("h", ("x",)), ("n", ("y",)), ("ry", ()), ("rh", ())):
        meets(lambda **p: L.moe_norm_out(ch, *p.values(), None), s, out, instead)
    s = dict(dh=e, dn=e, y=e, h=e, wp=v, g=v, wn=v, ry=r, rh=r, dx=e, dy=e, dg=v, dwp=v, dwn=v, ws=ws)
    for out, instead in (("dx", ("dh",)), ("dy", ("dn",)), ("dg", ()), ("dwp", ()), ("dwn", ()),
                         ("ws", ())):
        meets(lambda ws, **p: L.moe_norm_out_grad(ch, *p.values(), 0, ws, None), s, out, instead)


def route_cfg(moe, **kw):
    return moe.Cfg(**{**dict(T=16, d=128, E=8, k=2, n_group=1, topk_group=1, d_ff=128, d_ff_shared=0,
                             R=1, route_scale=1.0, act_dtype=0, w_dtype=0), **kw})


def test_route_grad_checks(moe):
    L, n = moe._lib, ctypes.c_size_t(0)
    for change, code in ((dict(k=9), 1), (dict(d=200), 2), (dict(E=2048, k=1), 2),
                         (dict(d=65664), 2), (dict(T=2 ** 21, d=65536, k=1), 2),
                         (dict(route_scale=float("nan")), 1), (dict(), 0)):
        c = ctypes.byref(route_cfg(moe, **change))
        assert L.moe_route_grad_query(c, ctypes.byref(n)) == code, change
        if code:
            assert L.moe_route_grad(c, *far(8), 0, 1 << 50, None) == code
    c = ctypes.byref(route_cfg(moe))
    assert L.moe_route_grad_query(c, None) == 1
    assert L.moe_route_grad_query(None, ctypes.byref(n)) == 1
    names = ["x", "w", "idx", "s", "dw", "dx_in", "dx", "dwg"]
    for i, name in enumerate(names):
        a = far(8)
        a[i] = None
        if name != "dx_in":
            assert L.moe_route_grad(c, *a, 0, 1 << 50, None) == 1, name
        a[i] = OK + 8
        assert L.moe_route_grad(c, *a, 0, 1 << 50, None) == 3, name
    assert L.moe_route_grad(c, *far(8), 0, None, None) == 1
    T, d, E, k = 16, 128, 8, 2
    ws = moe.route_grad_ws_bytes(route_cfg(moe)) // 16 * 16
    sizes = dict(x=2 * T * d, w=4 * E * d, idx=4 * T * k, s=4 * T * k, dw=4 * T * k, dx_in=2 * T * d,
                 dx=2 * T * d, dwg=4 * E * d, ws=ws)
    for out, instead in (("dx", ("dx_in",)), ("dwg", ()), ("ws", ())):
        meets(lambda ws, **p: L.moe_route_grad(c, *p.values(), 0, ws, None), sizes, out, instead)
    # route_save: the scores are an output like the others
    need = moe.query_sizes(route_cfg(moe))["ws_bytes"] // 16 * 16
    sizes = dict(x=2 * T * d, w=4 * E * d, b=4 * E, idx=4 * T * k, tw=4 * T * k, ts=4 * T * k, ws=need)
    for out in ("idx", "tw", "ts", "ws"):
        meets(lambda **p: L.moe_route_save(c, *p.values(), None), sizes, out)
    a = far(7)
    a[5] = None
    assert L.moe_route_save(c, *a, None) == 1


def tensor_c(moe, **kw):
    a = dict(zip(("p", "g", "w", "m", "v"), far(5)))
    return moe.AdamTensorC(**{**a, **dict(n=1000, weight_decay=0.1, g_dtype=moe.MOE_F32), **kw})


def adam(moe, tensors, bits=32, state=1 << 52, norm=None, **kw):
    arr = (moe.AdamTensorC * max(len(tensors), 1))(*tensors)
    c = moe.AdamCfg(**{**dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, state_bits=bits), **kw})
    return moe._lib.moe_adamw(ctypes.byref(c), arr, len(tensors), 0, state, norm, None)


def test_adamw_checks(moe):
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(beta1=1.0), dict(beta2=-0.1), dict(beta2=nan),
                dict(eps=0.0), dict(eps=1e-50), dict(eps=inf), dict(max_norm=-1.0),
                dict(max_norm=inf), dict(max_norm=1.0), dict(state_bits=16), dict(reserved=1)):
        assert adam(moe, [tensor_c(moe)], **bad) == 1, bad   # (max_norm alone: no norm given)
    for bad, code in ((dict(n=-1), 1), (dict(n=2 ** 39), 2), (dict(g_dtype=1), 1),
                      (dict(weight_decay=-1.0), 1), (dict(weight_decay=nan), 1), (dict(p=None), 1),
                      (dict(g=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(p=OK + 4), 3),
                      (dict(w=OK + 4), 3), (dict(reserved=3), 1), (dict(m_scale=1 << 45), 1),
                      (dict(v_scale=1 << 45), 1)):
        assert adam(moe, [tensor_c(moe, **bad)]) == code, bad
    held = dict(m_scale=1 << 45, v_scale=1 << 46)
    for bad, code in ((dict(held, m_scale=None), 1), (dict(held, v_scale=None), 1),
                      (dict(held, m_scale=OK + 4), 3)):
        assert adam(moe, [tensor_c(moe, **bad)], bits=8) == code, bad
    assert adam(moe, [tensor_c(moe)], state=None) == 1
    assert adam(moe, [tensor_c(moe)], state=OK + 8) == 3
    assert adam(moe, [tensor_c(moe)], norm=OK + 2) == 3
    assert adam(moe, [tensor_c(moe)], lr_dev=OK + 1) == 3
    assert adam(moe, [tensor_c(moe, n=0)] * 257) == 2
    L = moe._lib
    assert L.moe_adamw(None, None, 0, 0, OK, None, None) == 1
    assert L.moe_adam_query(None) == 1
    assert L.moe_grad_norm(None, 1, 0, OK, OK, None) == 1
    assert L.moe_grad_norm(None, -1, 0, OK, OK, None) == 1
    arr = (moe.AdamTensorC * 1)(tensor_c(moe))
    assert L.moe_grad_norm(arr, 1, 0, 1 << 52, None, None) == 1
    assert L.moe_grad_norm(arr, 1, 0, 1 << 52, OK + 1, None) == 3
    assert L.moe_grad_norm(arr, 1, 0, None, OK, None) == 1
    assert L.moe_grad_norm(arr, 1, 0, 1 << 52, (1 << 52) + 32, None) == 1   # inside the state
    assert L.moe_grad_norm(arr, 1, 0, 1 << 52, arr[0].g + 3996, None) == 1  # inside a gradient


def test_adamw_arrays_that_meet(moe):
    size = dict(p=4000, g=4000, w=2000, m=4000, v=4000)
    for bits in (32, 8):
        one = dict(zip(size, far(5)))
        n = dict(size, m=1000, v=1000, m_scale=32, v_scale=32) if bits == 8 else size
        if bits == 8:
            one.update(m_scale=1 << 45, v_scale=1 << 46)
        two = {k: p + (1 << 47) for k, p in one.items()}
        for k in n:
            for other in n:
                for at in {two[other] + n[other] // 16 * 16 - 16, two[other]} - {two[k]}:
                    a, b = dict(one, **{k: at}), dict(two)
                    assert adam(moe, [tensor_c(moe, **a), tensor_c(moe, **b)], bits) == 1, (k, other)
        assert adam(moe, [tensor_c(moe, **one), tensor_c(moe, **one)], bits) == 1
        for k in n:
            assert adam(moe, [tensor_c(moe, **dict(one, **{k: 1 << 52}))], bits) == 1   # the state
            assert adam(moe, [tensor_c(moe, **one)], bits, norm=one[k] + 16) == 1


def test_binding_refuses_other_tensors(moe):
    bf = torch.bfloat16
    x, w = torch.zeros(16, 64, dtype=bf), torch.zeros(64)
    with pytest.raises(ValueError, match="CUDA"):
        moe.norm_in(x, w, torch.zeros_like(x))
    with pytest.raises(ValueError, match="x must be"):
        moe.norm_in(x.double(), w, x)
    with pytest.raises(ValueError, match="2-D"):
        moe.norm_in(x[0], w, x)
    with pytest.raises(ValueError, match="gate must be"):
        moe.norm_out(x, x, w, torch.zeros(5), w, x, x)
    with pytest.raises(ValueError, match="gate must be"):
        moe.norm_out(x, x, w, x.float(), w, x, x)
    cfg = route_cfg(moe)
    with pytest.raises(ValueError, match="ws must be"):
        moe.route_grad(cfg, x, w, x, x, x, None, x, w, torch.zeros(4))
    t = dict(p=w, g=w, m=w, v=w)
    with pytest.raises(ValueError, match="CUDA"):
        moe.AdamTensors([t])
    with pytest.raises(ValueError, match="state_bits"):
        moe.AdamTensors([t], state_bits=4)
    with pytest.raises(ValueError, match="g must be"):
        moe.AdamTensors([dict(t, g=w.double())])
    with pytest.raises(ValueError, match="p must be"):
        moe.AdamTensors([dict(t, p=w.to(bf))])
    assert len(moe.AdamTensors([]).parts) == 1     # a step of no tensors still counts
    s = moe.adam_state(7, 0.9, 0.99, device="cpu")
    assert moe.adam_step(s) == 7
    c1, c2 = s[16:32].view(torch.float64)
    assert float(c1) == 1 - 0.9 ** 7 and float(c2) == 1 - 0.99 ** 7


def test_train_block_checks_its_weights():
    import dataclasses

    import synth
    from combine_grouped_gemm_gb300.train import MoETrainBlock
    cfg = dataclasses.replace(synth.CONFIGS["tiny"], R=1)
    good = torch.ones(cfg.d)
    for name, w in (("w_in", None), ("w_in", good.bfloat16()), ("w_out", torch.ones(cfg.d + 1)),
                    ("gate", torch.ones(cfg.T, 1)), ("gate", 0.5)):
        kw = {"w_in": good, "w_out": good, "gate": good, name: w}
        with pytest.raises(ValueError, match=name):
            MoETrainBlock(cfg, None, None, {}, kw["w_in"], kw["w_out"], kw["gate"])


def test_norm_factors_are_numbers():
    """A tensor as a factor would be kept by its identity, with the value that it had first."""
    import combine_grouped_gemm_gb300 as moe
    x, w = torch.zeros(2, 8), torch.ones(8)
    n = torch.empty(2, 8, dtype=torch.bfloat16)
    for name in ("res_scale", "out_scale", "eps"):
        for value in (torch.tensor(0.5), "1", None):
            with pytest.raises(ValueError, match="numbers"):
                moe.norm_out(n, x, w, None, None, x, None, **{name: value})
    with pytest.raises(ValueError, match="numbers"):
        moe.norm_in(x, w, n, eps=torch.tensor(1e-6))
