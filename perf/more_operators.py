"""Timed cases of the operators around the expert path in a training or serving step of an MoE block.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the framework's calls:

* RMS norms before and after a block: the norm of the residual stream (``norm_in``); the norm of
  the block's output fused with its gate, the residual's scale and the next block's norm
  (``norm_out``); the gradients of both (``norm_in_grad``, ``norm_out_grad``);
* the gradient of the router, from the routing weights' gradient to the gate weights and the
  tokens (``route_grad``);
* a step of AdamW over many tensors at once with moments in 32 or 8 bits, after the norm of all
  the gradients where it clips by it (``adamw``).
"""
import math

import torch

own = False

_E4M3_MAX = 448.0
_BLOCK = 128
_EPS = 1e-6
_ADAM = dict(lr=2e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1000)
_M32 = 0xFFFFFFFF


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    """Shapes are those of the framework's own workloads: d 7168, d_ff 2048, 256 experts, top 8;
    batches of 1, 64, 2048 and 16384 tokens."""
    return [
        # one token between two blocks while it is decoded: the smallest call, launch latency
        dict(name="norm_token", op="norm_out", rows=1, d=7168, stream="bf16", gate="none",
             post=False, next=True),
        # a decode batch through a block with a norm on both sides and a learned gate
        dict(name="norm_decode", op="norm_out", rows=64, d=7168, stream="bf16", gate="channel",
             post=True, next=True),
        # a prefill through the same block
        dict(name="norm_prefill", op="norm_out", rows=16384, d=7168, stream="bf16",
             gate="channel", post=True, next=True),
        # a training micro-batch's first norm, residual stream in fp32
        dict(name="norm_in_micro", op="norm_in", rows=2048, d=7168, stream="fp32"),
        # the backward pass of that first norm, the residual's gradient joined
        dict(name="norm_in_grad", op="norm_in_grad", rows=2048, d=7168, stream="fp32"),
        # the backward pass behind a block for a training batch
        dict(name="norm_grad_batch", op="norm_out_grad", rows=16384, d=7168, stream="bf16",
             gate="channel", post=True, next=True),
        # the router's gradient for a small batch: latency, and the gate weights' own gradient
        dict(name="route_grad_64", op="route_grad", T=64, d=7168, E=256, k=8, skew=0.0),
        # for a training micro-batch
        dict(name="route_grad_micro", op="route_grad", T=2048, d=7168, E=256, k=8, skew=0.0),
        # for a long batch with unevenly loaded experts
        dict(name="route_grad_batch", op="route_grad", T=16384, d=7168, E=256, k=8, skew=0.8),
        # the gate and four norms: what every rank updates beside its experts
        dict(name="adamw_small", op="adamw", experts=0, f=0, d=7168, gate=256, norms=4, odd=0,
             grad="fp32", bits=32, clip=True),
        # the experts of one rank (8 of 256, and the shared one), moments in 32 bits, with clipping
        dict(name="adamw_rank", op="adamw", experts=9, f=2048, d=7168, gate=256, norms=2, odd=0,
             grad="fp32", bits=32, clip=True),
        # the same with gradients in bf16 and moments in 8 bits
        dict(name="adamw_rank_8bit", op="adamw", experts=9, f=2048, d=7168, gate=256, norms=2,
             odd=0, grad="bf16", bits=8, clip=False),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(min(max(step, step * round(v / step)), hi // step * step))


def draw(rng):
    """Another case of the listed ranges: any of the operators, log-uniform sizes, odd ones too."""
    op = rng.choice(["norm_in", "norm_in_grad", "norm_out", "norm_out", "norm_out_grad",
                     "norm_out_grad", "route_grad", "route_grad", "route_grad", "adamw", "adamw",
                     "adamw"])
    if op.startswith("norm"):
        c = dict(op=op, rows=_log_int(rng, 1, 16384), d=_log_int(rng, 64, 7168, 8),
                 stream=rng.choice(["bf16", "fp32"]))
        if op.startswith("norm_out"):
            c.update(gate=rng.choice(["none", "channel", "token", "element"]),
                     post=rng.random() < 0.7, next=rng.random() < 0.8)
        return c
    if op == "route_grad":
        E = _log_int(rng, 8, 1024)
        return dict(op=op, T=_log_int(rng, 1, 16384), d=_log_int(rng, 128, 7168, 128), E=E,
                    k=rng.randint(1, 8), skew=rng.choice([0.0, 0.8, 1.2]))
    return dict(op=op, experts=rng.randint(1, 9), f=_log_int(rng, 64, 2048, 8),
                d=_log_int(rng, 64, 7168, 8), gate=_log_int(rng, 4, 256), norms=rng.randint(0, 6),
                odd=_log_int(rng, 1, 100001), grad=rng.choice(["fp32", "bf16"]),
                bits=rng.choice([32, 8]), clip=rng.random() < 0.5)


def _sizes(case):
    """Elements of each tensor of an optimiser's case, and whether it is an expert's (a bf16 copy,
    gradient of the case's type, weight decay) or not (fp32 only, no decay)."""
    e, f, d = case["experts"], case["f"], case["d"]
    big = [2 * f * d * e, d * f * e] if e else []
    rest = [case["gate"] * d] + [d] * case["norms"] + ([case["odd"]] if case["odd"] else [])
    return [(n, True) for n in big] + [(n, False) for n in rest]


def work(case):
    """Bytes each pass must read and write once, and its floating-point operations."""
    op = case["op"]
    if op.startswith("norm"):
        rows, d = case["rows"], case["d"]
        n, st = rows * d, 4.0 if case["stream"] == "fp32" else 2.0
        if op == "norm_in":
            return dict(bytes=n * (st + 2) + 4.0 * (d + rows), flops=4.0 * n)
        if op == "norm_in_grad":
            return dict(bytes=n * (3 * st + 2) + 4.0 * (2 * d + rows), flops=10.0 * n)
        gate = dict(none=0.0, channel=4.0 * d, token=4.0 * rows, element=2.0 * n)[case["gate"]]
        nx, post = case["next"], case["post"]
        small = 4.0 * (d + rows) * (post + nx)
        if op == "norm_out":
            return dict(bytes=n * (2 + 2 * st + 2 * nx) + gate + small,
                        flops=n * (3.0 + 4 * post + 4 * nx))
        # the block's output is needed for the gradients of its norm and its gate only, the stream
        # for that of the next norm
        reads_y = post or case["gate"] != "none"
        return dict(bytes=n * (2 * st + 2 + 2 * reads_y + (2 + st) * nx) + 2 * gate
                    + small + 4.0 * d * (post + nx),
                    flops=n * (4.0 + 9 * post + 9 * nx))
    if op == "route_grad":
        T, d, E, k = case["T"], case["d"], case["E"], case["k"]
        return dict(bytes=6.0 * T * d + 8.0 * E * d + 12.0 * T * k, flops=4.0 * T * k * d)
    total, flops = 0.0, 0.0
    for n, big in _sizes(case):
        grad = 2 if big and case["grad"] == "bf16" else 4
        state = 16.0 if case["bits"] == 32 else 4.0 + 16.0 / _BLOCK
        total += n * (grad + 8 + state + (2 if big else 0))
        flops += n * (15.0 + (2 if case["clip"] else 0))
    return dict(bytes=total, flops=flops)


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def _normal(gen, shape, std=1.0, dtype=torch.bfloat16, mean=0.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(mean, std, generator=gen)


def _uniform(gen, shape, lo, hi):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(lo, hi, generator=gen)


def _rstd(x):
    return 1.0 / torch.sqrt(x.float().square().mean(1) + _EPS)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    if op.startswith("norm"):
        return _prepare_norm(case, gen)
    if op == "route_grad":
        return _prepare_route(case, gen)
    return _prepare_adamw(case, gen, seed)


def _prepare_norm(case, gen):
    rows, d, op = case["rows"], case["d"], case["op"]
    st = torch.float32 if case["stream"] == "fp32" else torch.bfloat16
    f32 = dict(dtype=torch.float32, device="cuda")
    s = dict(case=case, res_scale=1.0, out_scale=0.5, rstd_y=None, rstd_h=None)
    # the stream grows through the layers: a few times the size of one block's output
    s["x"] = _normal(gen, (rows, d), 3.0, st)
    if op.startswith("norm_in"):
        s["w"] = _normal(gen, (d,), 0.2, torch.float32, 1.0)
        s["n"] = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
        s["rstd"] = torch.empty((rows,), **f32)
        if op == "norm_in_grad":
            s["rstd"].copy_(_rstd(s["x"]))
            s["dn"] = _normal(gen, (rows, d), 0.02)
            s["dres"] = _normal(gen, (rows, d), 0.02, st)
            s["dx"] = torch.empty((rows, d), dtype=st, device="cuda")
            s["dw"] = torch.empty((d,), **f32)
        return s
    s["y"] = _normal(gen, (rows, d), 0.6)
    s["w_post"] = _normal(gen, (d,), 0.2, torch.float32, 1.0) if case["post"] else None
    s["w_next"] = _normal(gen, (d,), 0.2, torch.float32, 1.0) if case["next"] else None
    kind = case["gate"]
    s["gate"] = {"none": lambda: None, "channel": lambda: _uniform(gen, (d,), 0.1, 1.0),
                 "token": lambda: _uniform(gen, (rows,), 0.0, 1.0),
                 "element": lambda: _uniform(gen, (rows, d), 0.0, 1.0).to(torch.bfloat16)}[kind]()
    if case["post"]:
        s["rstd_y"] = torch.empty((rows,), **f32)
    if case["next"]:
        s["rstd_h"] = torch.empty((rows,), **f32)
    if op == "norm_out":
        s["h"] = torch.empty((rows, d), dtype=st, device="cuda")
        s["n"] = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda") if case["next"] \
            else None
        return s
    s["h"] = s.pop("x")   # the stream behind the block, as the forward pass left it
    if case["post"]:
        s["rstd_y"].copy_(_rstd(s["y"]))
    if case["next"]:
        s["rstd_h"].copy_(_rstd(s["h"]))
    s["dh"] = _normal(gen, (rows, d), 0.02, st)
    s["dn"] = _normal(gen, (rows, d), 0.02) if case["next"] else None
    s["dx"] = torch.empty((rows, d), dtype=st, device="cuda")
    s["dy"] = torch.empty((rows, d), dtype=torch.bfloat16, device="cuda")
    s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
    s["dw_post"] = torch.empty((d,), **f32) if case["post"] else None
    s["dw_next"] = torch.empty((d,), **f32) if case["next"] else None
    return s


def _prepare_route(case, gen):
    T, d, E, k = case["T"], case["d"], case["E"], case["k"]
    s = dict(case=case, scale=2.5)
    s["x"] = _normal(gen, (T, d))
    s["w_gate"] = _normal(gen, (E, d), 0.02, torch.float32)
    # k distinct experts a token, drawn by popularity rank^-skew (the exponential race)
    pop = torch.arange(1, E + 1, device="cuda", dtype=torch.float32).pow(-case["skew"])
    pop = pop[torch.randperm(E, generator=gen, device="cuda")]
    race = torch.empty((T, E), device="cuda").exponential_(generator=gen) / pop
    s["idx"] = race.topk(k, dim=1, largest=False).indices.to(torch.int32)
    s["score"] = torch.sigmoid(_normal(gen, (T, k), 1.0, torch.float32, 1.5))
    s["dtopk_w"] = _normal(gen, (T, k), 0.05, torch.float32)
    s["dx_in"] = _normal(gen, (T, d), 0.02)
    s["dx"] = torch.empty((T, d), dtype=torch.bfloat16, device="cuda")
    s["dw_gate"] = torch.empty((E, d), dtype=torch.float32, device="cuda")
    return s


def _prepare_adamw(case, gen, seed):
    tensors = []
    for i, (n, big) in enumerate(_sizes(case)):
        p = _normal(gen, (n,), 0.02, torch.float32)
        gtype = torch.bfloat16 if big and case["grad"] == "bf16" else torch.float32
        # gradients whose size differs from block to block and element to element
        g = _normal(gen, (n,), 1e-3, torch.float32)
        g *= _uniform(gen, (n,), 0.0, 2.0)
        t = dict(p=p, g=g.to(gtype), w=p.to(torch.bfloat16) if big else None,
                 weight_decay=_ADAM["weight_decay"] if big else 0.0, seed=(seed + 977 * i) & _M32)
        m = _normal(gen, (n,), 2e-4, torch.float32)
        v = _uniform(gen, (n,), 0.1, 2.0).square_().mul_(1e-6)
        if case["bits"] == 32:
            t.update(m=m, v=v)
        else:
            t["m"], t["m_scale"] = _codes(m)
            t["v"], t["v_scale"] = _codes(torch.sqrt(v))
        tensors.append(t)
    return dict(case=case, tensors=tensors, step=_ADAM["step"],
                norm=torch.zeros(1, dtype=torch.float32, device="cuda"),
                max_norm=1.0 if case["clip"] else 0.0)


def _blocks(x):
    """x [n] as rows of 128, the last one filled up with zeros."""
    n = x.numel()
    if n % _BLOCK:
        x = torch.cat([x, x.new_zeros(_BLOCK - n % _BLOCK)])
    return x.view(-1, _BLOCK)


def _codes(x):
    """A moment as a training run would hold it: e4m3 codes (nearest) and their scales."""
    b = _blocks(x)
    amax = b.abs().amax(1)
    scale = torch.where(amax > 0, amax / _E4M3_MAX, torch.ones_like(amax))
    q = (b / scale.unsqueeze(1)).clamp_(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).flatten()[:x.numel()].clone(), scale


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    return _framework(state) if own else _PLAIN[state["case"]["op"]](state)


def _framework(s):
    import combine_grouped_gemm_gb300 as moe

    c = s["case"]
    op = c["op"]
    if op == "norm_in":
        moe.norm_in(s["x"], s["w"], s["n"], s["rstd"], eps=_EPS)
        return s["n"], s["rstd"]
    gate, dgate = s.get("gate"), s.get("dgate")
    if c.get("gate") == "token":   # [rows][1]: one factor a row, whatever the width
        gate = gate.view(-1, 1)
        dgate = None if dgate is None else dgate.view(-1, 1)
    if op == "norm_out":
        moe.norm_out(s["y"], s["x"], s["w_post"], gate, s["w_next"], s["h"], s["n"],
                     s["rstd_y"], s["rstd_h"], eps=_EPS, res_scale=s["res_scale"],
                     out_scale=s["out_scale"])
        return [t for t in (s["h"], s["n"], s["rstd_y"], s["rstd_h"]) if t is not None]
    if op.startswith("norm"):
        if "ws" not in s:   # the workspace that a program keeps for a shape
            s["ws"] = torch.zeros(moe.norm_ws_bytes(c["rows"], c["d"]), dtype=torch.uint8,
                                  device="cuda")
        if op == "norm_in_grad":
            moe.norm_in_grad(s["dn"], s["x"], s["w"], s["rstd"], s["dres"], s["dx"], s["dw"],
                             s["ws"])
            return s["dx"], s["dw"]
        moe.norm_out_grad(s["dh"], s["dn"], s["y"], s["h"], s["w_post"], gate, s["w_next"],
                          s["rstd_y"], s["rstd_h"], s["dx"], s["dy"], dgate, s["dw_post"],
                          s["dw_next"], s["ws"], res_scale=s["res_scale"],
                          out_scale=s["out_scale"])
        return [t for t in (s["dx"], s["dy"], s["dgate"], s["dw_post"], s["dw_next"])
                if t is not None]
    if op == "route_grad":
        if "cfg" not in s:
            s["cfg"] = moe.Cfg(c["T"], c["d"], c["E"], c["k"], 1, 1, 128, 0, 1, s["scale"],
                               moe.MOE_BF16, moe.MOE_BF16)
            s["ws"] = torch.zeros(moe.route_grad_ws_bytes(s["cfg"]), dtype=torch.uint8,
                                  device="cuda")
        moe.route_grad(s["cfg"], s["x"], s["w_gate"], s["idx"], s["score"], s["dtopk_w"],
                       s["dx_in"], s["dx"], s["dw_gate"], s["ws"])
        return s["dx"], s["dw_gate"]
    if "plan" not in s:
        s["plan"] = moe.AdamTensors(s["tensors"], state_bits=c["bits"])
        s["cfg"] = moe.AdamCfg(lr=_ADAM["lr"], beta1=_ADAM["beta1"], beta2=_ADAM["beta2"],
                               eps=_ADAM["eps"], max_norm=s["max_norm"])
        s["state"] = moe.adam_state(s["step"], _ADAM["beta1"], _ADAM["beta2"])
    if c["clip"]:
        moe.grad_norm(s["plan"], s["state"], s["norm"])
        moe.adamw(s["cfg"], s["plan"], s["state"], s["norm"])
    else:
        moe.adamw(s["cfg"], s["plan"], s["state"])
    return _adam_outputs(s)


def _adam_outputs(s):
    out = [s["norm"]] if s["case"]["clip"] else []
    for t in s["tensors"]:
        out.append(t["p"])
        if t["w"] is not None:
            out.append(t["w"])
        if s["case"]["bits"] == 32:
            out += [t["m"], t["v"]]
        else:
            out += [t["m"].view(torch.float8_e4m3fn), t["m_scale"],
                    t["v"].view(torch.float8_e4m3fn), t["v_scale"]]
    return out


# -------------------------------------- the plain forms --------------------------------------
def _plain_norm_in(s):
    x = s["x"].float()
    r = 1.0 / torch.sqrt((x * x).mean(1) + _EPS)
    return (x * r.unsqueeze(1) * s["w"]).to(torch.bfloat16), r


def _gate(s):
    g = s["gate"]
    if g is None:
        return 1.0
    return g.unsqueeze(1) if s["case"]["gate"] == "token" else g.float()


def _plain_norm_out(s):
    y, x = s["y"].float(), s["x"].float()
    out = []
    if s["w_post"] is not None:
        ry = 1.0 / torch.sqrt((y * y).mean(1) + _EPS)
        out.append(ry)
        y = y * ry.unsqueeze(1) * s["w_post"]
    h = s["res_scale"] * x + s["out_scale"] * _gate(s) * y
    if s["w_next"] is None:
        return [h.to(s["x"].dtype)] + out
    rh = 1.0 / torch.sqrt((h * h).mean(1) + _EPS)
    n = h * rh.unsqueeze(1) * s["w_next"]
    return [h.to(s["x"].dtype), n.to(torch.bfloat16)] + out + [rh]


def _plain_norm_grad(dn, x, r, w):
    """Gradients of x r w with respect to x and w."""
    xh = x * r.unsqueeze(1)
    a = dn * w
    dx = r.unsqueeze(1) * (a - xh * (a * xh).mean(1, keepdim=True))
    return dx, (dn * xh).sum(0)


def _plain_norm_in_grad(s):
    dx, dw = _plain_norm_grad(s["dn"].float(), s["x"].float(), s["rstd"], s["w"])
    return (s["dres"].float() + dx).to(s["dx"].dtype), dw


def _plain_norm_out_grad(s):
    c = s["case"]
    grad, y = s["dh"].float(), s["y"].float()
    tail = []
    if c["next"]:
        d, dw_next = _plain_norm_grad(s["dn"].float(), s["h"].float(), s["rstd_h"], s["w_next"])
        grad = grad + d
        tail = [dw_next]
    out = [(s["res_scale"] * grad).to(s["dx"].dtype)]
    part = s["out_scale"] * grad
    ds = part * _gate(s)
    if c["post"]:
        dy, dw_post = _plain_norm_grad(ds, y, s["rstd_y"], s["w_post"])
        tail.insert(0, dw_post)
        y = y * s["rstd_y"].unsqueeze(1) * s["w_post"]
    else:
        dy = ds
    out.append(dy.to(torch.bfloat16))
    if c["gate"] != "none":
        dg = part * y
        if c["gate"] != "element":
            dg = dg.sum(0 if c["gate"] == "channel" else 1)
        out.append(dg.to(s["dgate"].dtype))
    return out + tail


def _plain_route_grad(s):
    score, dw, idx = s["score"], s["dtopk_w"], s["idx"].long()
    p = score / score.sum(1, keepdim=True)
    dz = s["scale"] * p * (1.0 - score) * (dw - (p * dw).sum(1, keepdim=True))
    dense = torch.zeros((idx.shape[0], s["w_gate"].shape[0]), device=idx.device)
    dense.scatter_(1, idx, dz)
    dx = s["dx_in"].float() + dense @ s["w_gate"]
    return dx.to(torch.bfloat16), dense.t() @ s["x"].float()


def _mix(x):
    """The 32-bit integer hash "lowbias32" (C. Wellons, 2018) on int64 tensors."""
    x = x ^ (x >> 16)
    x = (x * 0x7FEB352D) & _M32
    x = x ^ (x >> 15)
    x = (x * 0x846CA68B) & _M32
    return x ^ (x >> 16)


def _noise(n, seed, step, device):
    """Two 16-bit random numbers an element, [blocks][128]: the upper and the lower half of a hash
    of the tensor's seed, the step, the block and the place in the block."""
    i64 = dict(dtype=torch.int64, device=device)
    key = _mix(torch.tensor((seed ^ (step * 0x9E3779B9)) & _M32, **i64))
    blocks = torch.arange((n + _BLOCK - 1) // _BLOCK, **i64)
    key = _mix(key ^ blocks)
    place = (torch.arange(_BLOCK, **i64) * 0x9E3779B9) & _M32
    r = _mix((key.unsqueeze(1) + place) & _M32)
    return r >> 16, r & 0xFFFF


def _round_e4m3(q, r16):
    """Magnitudes q <= 448 rounded up or down to e4m3 as the 16-bit random number says: the odds of
    rounding up are the distance from the lower neighbour. (Below 2^-6 the steps are 2^-9: adding
    2^-6 puts them at the same bits of the fp32 number.)"""
    small = q < 2.0 ** -6
    y = torch.where(small, q + 2.0 ** -6, q)
    bits = (y.view(torch.int32) + (r16.to(torch.int32) << 4)) & ~0xFFFFF
    y = bits.view(torch.float32)
    return torch.where(small, y - 2.0 ** -6, y)


def _round_root_e4m3(q, r16):
    """The same for the root of a second moment, with odds that keep the mean of its square:
    (q^2 - lo^2) / (hi^2 - lo^2) between the neighbours lo and hi."""
    small = q < 2.0 ** -6
    y = torch.where(small, q + 2.0 ** -6, q)
    bits = y.view(torch.int32) & ~0xFFFFF
    shift = torch.where(small, torch.full_like(q, 2.0 ** -6), torch.zeros_like(q))
    lo, hi = bits.view(torch.float32) - shift, (bits + 0x100000).view(torch.float32) - shift
    up = r16.float() * ((hi - lo) * (hi + lo)) < (q - lo) * (q + lo) * 65536.0
    return torch.where(up, hi, lo)


def _plain_hold(x, r16, root):
    """A moment x [n] in 8 bits: codes and scales. root: x is the root of the second one, which
    keeps a code above 0 where it is above 0."""
    n = x.numel()
    b = _blocks(x)
    mag = b.abs()
    amax = mag.amax(1, keepdim=True)
    scale = torch.where(amax > 0, amax / _E4M3_MAX, torch.ones_like(amax))
    q = mag / scale
    q = torch.where(q > _E4M3_MAX, torch.full_like(q, _E4M3_MAX), q)
    q = _round_root_e4m3(q, r16) if root else _round_e4m3(q, r16)
    if root:
        q = torch.where((b > 0) & (q < 2.0 ** -9), torch.full_like(q, 2.0 ** -9), q)
    code = torch.copysign(q, b).to(torch.float8_e4m3fn).view(torch.uint8)
    return code.flatten()[:n], scale.flatten()


def _restore(code, scale):
    n = code.numel()
    v = _blocks(code.view(torch.float8_e4m3fn).float()) * scale.unsqueeze(1)
    return v.flatten()[:n]


def _plain_adamw(s):
    a, c = _ADAM, s["case"]
    s["step"] += 1
    step = s["step"]
    factor = 1.0
    if c["clip"]:
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for t in s["tensors"]:
            total += t["g"].double().square().sum()
        s["norm"].copy_(total.sqrt())
        factor = torch.clamp(s["max_norm"] / s["norm"], max=1.0)
    c1, c2 = 1.0 - a["beta1"] ** step, 1.0 - a["beta2"] ** step
    for t in s["tensors"]:
        g = t["g"].float()
        if c["clip"]:
            g = g * factor
        held = c["bits"] == 8
        m = _restore(t["m"], t["m_scale"]) if held else t["m"]
        v = _restore(t["v"], t["v_scale"]).square() if held else t["v"]
        m = a["beta1"] * m + (1.0 - a["beta1"]) * g
        v = a["beta2"] * v + (1.0 - a["beta2"]) * (g * g)
        root = torch.sqrt(v)
        move = m / (root / math.sqrt(c2) + a["eps"])
        t["p"].mul_(1.0 - a["lr"] * t["weight_decay"]).sub_(move * (a["lr"] / c1))
        if t["w"] is not None:
            t["w"].copy_(t["p"])
        if held:
            rm, rv = _noise(m.numel(), t["seed"], step, m.device)
            for name, x, r in (("m", m, rm), ("v", root, rv)):
                code, scale = _plain_hold(x, r, name == "v")
                t[name].copy_(code)
                t[name + "_scale"].copy_(scale)
        else:
            t["m"].copy_(m)
            t["v"].copy_(v)
    return _adam_outputs(s)


_PLAIN = dict(norm_in=_plain_norm_in, norm_in_grad=_plain_norm_in_grad, norm_out=_plain_norm_out,
              norm_out_grad=_plain_norm_out_grad, route_grad=_plain_route_grad,
              adamw=_plain_adamw)


# --------------------------------------------------------------------------------------------
# In 64 bits, from the definitions
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](s)


def _wide(t):
    return None if t is None else t.double()


def _exact_norm_in(s):
    x, d = s["x"].double(), s["x"].shape[1]
    r = (torch.einsum("td,td->t", x, x) / d + _EPS) ** -0.5
    return torch.einsum("td,t,d->td", x, r, s["w"].double()), r


def _gated(t, s, kind):
    """t times the gate."""
    g = _wide(s["gate"])
    return t if g is None else torch.einsum(
        {"channel": "td,d->td", "token": "td,t->td", "element": "td,td->td"}[kind], t, g)


def _exact_norm_out(s):
    y, x, kind, d = s["y"].double(), s["x"].double(), s["case"]["gate"], s["y"].shape[1]
    rs = []
    if s["w_post"] is not None:
        rs.append((torch.einsum("td,td->t", y, y) / d + _EPS) ** -0.5)
        y = torch.einsum("td,t,d->td", y, rs[0], s["w_post"].double())
    h = s["res_scale"] * x + s["out_scale"] * _gated(y, s, kind)
    if s["w_next"] is None:
        return [h] + rs
    r = (torch.einsum("td,td->t", h, h) / d + _EPS) ** -0.5
    return [h, torch.einsum("td,t,d->td", h, r, s["w_next"].double())] + rs + [r]


def _exact_norm_back(dn, x, r, w):
    """The gradient through n_j = x_j r w_j, r a function of x: d n_j / d x_i = r w_j (i = j)
    - x_j w_j r^3 x_i / d."""
    d = x.shape[1]
    along = torch.einsum("td,td,d->t", dn, x, w) * r ** 3 / d
    return dn * w * r[:, None] - along[:, None] * x, torch.einsum("td,td,t->d", dn, x, r)


def _exact_norm_in_grad(s):
    dx, dw = _exact_norm_back(s["dn"].double(), s["x"].double(), s["rstd"].double(),
                              s["w"].double())
    return s["dres"].double() + dx, dw


def _exact_norm_out_grad(s):
    kind = s["case"]["gate"]
    total, y = s["dh"].double(), s["y"].double()
    dw_post = dw_next = None
    if s["w_next"] is not None:
        more, dw_next = _exact_norm_back(s["dn"].double(), s["h"].double(), s["rstd_h"].double(),
                                         s["w_next"].double())
        total = total + more
    ds = s["out_scale"] * _gated(total, s, kind)
    normed = y
    if s["w_post"] is not None:
        ry, w = s["rstd_y"].double(), s["w_post"].double()
        normed = torch.einsum("td,t,d->td", y, ry, w)
        dy, dw_post = _exact_norm_back(ds, y, ry, w)
    else:
        dy = ds
    dgate = None
    if kind != "none":
        dgate = s["out_scale"] * torch.einsum(
            {"channel": "td,td->d", "token": "td,td->t", "element": "td,td->td"}[kind], total,
            normed)
    return [t for t in (s["res_scale"] * total, dy, dgate, dw_post, dw_next) if t is not None]


def _exact_route_grad(s):
    T, k = s["idx"].shape
    score, dw = s["score"].double(), s["dtopk_w"].double()
    # topk_w_i = scale s_i / S: its derivative by s_j is scale ((i = j) / S - s_i / S^2)
    S = score.sum(1)
    ds = s["scale"] * (dw / S[:, None] - (torch.einsum("tk,tk->t", dw, score) / S ** 2)[:, None])
    dz = ds * score * (1.0 - score)
    dx = s["dx_in"].double()
    dgate = torch.zeros(s["w_gate"].shape, dtype=torch.float64, device="cuda")
    rows = torch.arange(T, device="cuda")
    w, x = s["w_gate"].double(), s["x"].double()
    for i in range(k):
        e = s["idx"][:, i].long()
        one = torch.zeros((T, w.shape[0]), dtype=torch.float64, device="cuda")
        one[rows, e] = dz[:, i]
        dx = dx + one @ w
        dgate += one.t() @ x
    return dx, dgate


def _exact_adamw(s):
    a, held = _ADAM, s["case"]["bits"] == 8
    step = s["step"] + 1
    out, factor = [], 1.0
    if s["case"]["clip"]:
        norm = math.sqrt(sum(float(t["g"].double().pow(2).sum()) for t in s["tensors"]))
        out.append(torch.tensor([norm], dtype=torch.float64, device="cuda"))
        factor = min(1.0, s["max_norm"] / norm) if norm > 0 else 1.0
    for t in s["tensors"]:
        m, v = t["m"], t["v"]
        if held:
            n = m.numel()
            m, v = (c.view(torch.float8_e4m3fn).double() *
                    t[name].double().repeat_interleave(_BLOCK)[:n]
                    for c, name in ((m, "m_scale"), (v, "v_scale")))
            v = v * v
        g = t["g"].double() * factor
        m = torch.lerp(g, m.double(), a["beta1"])
        v = torch.lerp(g * g, v.double(), a["beta2"])
        mean, var = m / (1 - a["beta1"] ** step), v / (1 - a["beta2"] ** step)
        p = t["p"].double()
        p = p - a["lr"] * (t["weight_decay"] * p + mean / (var.sqrt() + a["eps"]))
        out.append(p)
        if t["w"] is not None:
            out.append(p)
        if not held:
            out += [m, v]
            continue
        # the codes are choices of a random rounding: they have no value beside their own
        out += [None, _exact_scale(m), None, _exact_scale(v.sqrt())]
    return out


def _exact_scale(x):
    top = _blocks(x).abs().max(dim=1).values
    return torch.where(top > 0, top / _E4M3_MAX, torch.ones_like(top))


_EXACT = dict(norm_in=_exact_norm_in, norm_in_grad=_exact_norm_in_grad, norm_out=_exact_norm_out,
              norm_out_grad=_exact_norm_out_grad, route_grad=_exact_route_grad,
              adamw=_exact_adamw)
