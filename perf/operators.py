"""Timed cases of the operators that train the expert path of the MoE layer.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once at
the end) and as the framework's calls:

* matrix products grouped by expert over ragged row counts: forward (``mm``), gradient of the
  rows (``mm_dx``) and gradient of the weights (``mm_dw``);
* activation checkpoints in 8 bits (e4m3 codes, one fp32 scale per 128 columns): token rows
  saved and loaded back per expert row (``rows``), the SwiGLU that saves its input
  (``swiglu_save``) and its gradient from the saved codes (``swiglu_grad``);
* the gradient of the weighted combine (``combine_grad``).
"""
import math
import random

import torch

own = False

_E4M3_MAX = 448.0
_BLOCK = 128


# --------------------------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------------------------
def listed():
    """Shapes are those of the framework's own workloads: d 7168, d_ff 2048, top 8 of 256 experts
    (decode), or of 32 experts with the same expert shapes (prefill stand-ins)."""
    return [
        # one token through the gate/up weights of its 8 experts: a decode step of one request
        dict(name="mm_token", op="mm", rows=8, E=256, n=4096, k=7168, skew=0.0),
        # 64 tokens over 256 experts: a decode batch, two rows an expert on average, some with none
        dict(name="mm_decode", op="mm", rows=512, E=256, n=4096, k=7168, skew=0.0),
        # 2048 tokens through the gate/up weights of 32 experts: the forward of a training batch
        dict(name="mm_batch", op="mm", rows=16384, E=32, n=4096, k=7168, skew=0.0),
        # the down projection's input gradient for the same batch, experts unevenly loaded
        dict(name="dx_batch", op="mm_dx", rows=16384, E=32, n=7168, k=2048, skew=0.8),
        # the gate/up weight gradient of a small micro-batch, kept in fp32 for accumulation
        dict(name="dw_micro", op="mm_dw", rows=4096, E=32, n=4096, k=7168, skew=0.8, out="fp32"),
        # the down projection's weight gradient of the full batch, in the weights' own bf16
        dict(name="dw_batch", op="mm_dw", rows=16384, E=32, n=7168, k=2048, skew=0.0, out="bf16"),
        # the SwiGLU of one token's 8 expert rows: the smallest call, launch latency
        dict(name="swiglu_token", op="swiglu_save", rows=8, f=2048),
        # the SwiGLU of a training batch's expert rows, its input saved in 8 bits
        dict(name="swiglu_batch", op="swiglu_save", rows=16384, f=2048),
        # the backward pass of that SwiGLU from the saved codes
        dict(name="swiglu_grad", op="swiglu_grad", rows=16384, f=2048),
        # 2048 token rows saved in 8 bits, then loaded back for each of their 8 expert rows
        dict(name="rows_batch", op="rows", T=2048, k=8, d=7168),
        # the combine's gradient for a decode-sized batch of 64 tokens
        dict(name="combine_grad_64", op="combine_grad", T=64, k=8, d=7168),
        # and for a training batch of 2048 tokens
        dict(name="combine_grad_batch", op="combine_grad", T=2048, k=8, d=7168),
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = int(min(max(step, step * round(v / step)), hi // step * step))
    return v + step if v == 3072 else v   # a size that belongs to other projects' benchmarks


def draw(rng):
    """Another case of the listed ranges: any of the operators, log-uniform sizes, odd ones too."""
    op = rng.choice(["mm", "mm", "mm_dx", "mm_dx", "mm_dw", "mm_dw", "swiglu_save",
                     "swiglu_grad", "rows", "combine_grad"])
    if op.startswith("mm"):
        while True:
            c = dict(op=op, rows=_log_int(rng, 1, 16384), E=_log_int(rng, 1, 256),
                     n=_log_int(rng, 64, 7168, 8), k=_log_int(rng, 64, 7168, 8),
                     skew=rng.choice([0.0, 0.8, 1.2]))
            if op == "mm_dw":
                c["out"] = rng.choice(["fp32", "bf16"])
            w = work(c)
            if w["flops"] <= 1e12 and w["bytes"] <= 15e9 and c["E"] * c["n"] * c["k"] <= 2 ** 32:
                return c
    if op.startswith("swiglu"):
        return dict(op=op, rows=_log_int(rng, 1, 16384), f=_log_int(rng, 128, 2048, 128))
    return dict(op=op, T=_log_int(rng, 1, 2048), k=rng.randint(1, 8),
                d=_log_int(rng, 128, 7168, 128))


def _counts(case):
    """Rows per group (before the seed permutes the groups): the rows dealt over E groups whose
    popularity falls as rank^-skew (0: evenly likely). Some groups of a small batch get none."""
    E, rows, skew = case["E"], case["rows"], case["skew"]
    rng = random.Random("%d %d %.2f" % (rows, E, skew))
    p = [(i + 1.0) ** -skew for i in range(E)]
    c = [0] * E
    for g in rng.choices(range(E), weights=p, k=rows):
        c[g] += 1
    return c


def work(case):
    """Bytes each pass must read and write once, and its floating-point operations."""
    op = case["op"]
    if op.startswith("mm"):
        rows, n, k = case["rows"], case["n"], case["k"]
        flops = 2.0 * rows * n * k
        if op == "mm_dw":
            size = 4 if case["out"] == "fp32" else 2
            return dict(bytes=2.0 * rows * (n + k) + size * case["E"] * n * k, flops=flops)
        active = sum(1 for c in _counts(case) if c)
        return dict(bytes=2.0 * rows * (n + k) + 2.0 * active * n * k, flops=flops)
    if op == "swiglu_save":
        rows, f = case["rows"], case["f"]
        return dict(bytes=rows * f * (4.0 + 2 + 2 + 8 / _BLOCK), flops=12.0 * rows * f)
    if op == "swiglu_grad":
        rows, f = case["rows"], case["f"]
        return dict(bytes=rows * f * (2.0 + 8 / _BLOCK + 2 + 4 + 2), flops=16.0 * rows * f)
    T, k, d = case["T"], case["k"], case["d"]
    if op == "rows":
        saved = T * d * (1.0 + 4 / _BLOCK)
        return dict(bytes=2.0 * T * d + 2 * saved + 2.0 * T * k * d + 4.0 * T * k,
                    flops=2.0 * T * d + 1.0 * T * k * d)
    return dict(bytes=2.0 * T * d + 2 * 2.0 * T * k * d + 12.0 * T * k, flops=3.0 * T * k * d)


# --------------------------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------------------------
def _normal(gen, shape, std=1.0):
    t = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return t.normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op.startswith("mm"):
        rows, E, n, k = case["rows"], case["E"], case["n"], case["k"]
        c = _counts(case)
        random.Random(seed).shuffle(c)
        s["counts"] = torch.tensor(c, dtype=torch.int32, device="cuda")
        if op != "mm_dw":
            s["w"] = _normal(gen, (E, n, k), 0.02)
        if op != "mm_dx":
            s["x"] = _normal(gen, (rows, k))
        if op != "mm":
            s["dy"] = _normal(gen, (rows, n), 0.1)
        if op == "mm_dw":
            dt = torch.float32 if case["out"] == "fp32" else torch.bfloat16
            s["out"] = torch.empty((E, n, k), dtype=dt, device="cuda")
        else:
            s["out"] = torch.empty((rows, n if op == "mm" else k), dtype=torch.bfloat16,
                                   device="cuda")
    elif op.startswith("swiglu"):
        rows, f = case["rows"], case["f"]
        gu = _normal(gen, (rows, 2 * f), 1.7)   # |x| of 7168 unit values times weights of 0.02
        s["a"] = torch.empty((rows, f), dtype=torch.bfloat16, device="cuda")
        s["q"] = torch.empty((rows, 2 * f), dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty((2 * f // _BLOCK, rows), dtype=torch.float32, device="cuda")
        if op == "swiglu_save":
            s["gu"] = gu
        else:
            q, sc = _quantise(gu.float())
            s["q"].copy_(q.view(torch.uint8))
            s["scales"].copy_(sc)
            s["da"] = _normal(gen, (rows, f), 0.1)
            s["dgu"] = torch.empty((rows, 2 * f), dtype=torch.bfloat16, device="cuda")
    else:
        T, k, d = case["T"], case["k"], case["d"]
        order = torch.randperm(T * k, generator=gen, device="cuda")   # an expert-sorted batch's
        if op == "rows":
            s["x"] = _normal(gen, (T, d))
            s["index"] = (order // k).to(torch.int32)
            s["q"] = torch.empty((T, d), dtype=torch.uint8, device="cuda")
            s["scales"] = torch.empty((d // _BLOCK, T), dtype=torch.float32, device="cuda")
            s["out"] = torch.empty((T * k, d), dtype=torch.bfloat16, device="cuda")
        else:
            s["ebuf"] = _normal(gen, (T * k, d), 0.5)
            s["row_of"] = order.to(torch.int32).view(T, k)
            w = torch.rand((T, k), generator=gen, device="cuda")
            s["topk_w"] = (2.5 * w / w.sum(1, keepdim=True)).contiguous()
            s["dy"] = _normal(gen, (T, d), 0.1)
            s["debuf"] = torch.empty((T * k, d), dtype=torch.bfloat16, device="cuda")
            s["dtopk_w"] = torch.empty((T, k), dtype=torch.float32, device="cuda")
    return s


# --------------------------------------------------------------------------------------------
# One pass
# --------------------------------------------------------------------------------------------
def run(state):
    return _framework(state) if own else _PLAIN[state["case"]["op"]](state)


def _framework(s):
    import combine_grouped_gemm_gb300 as moe

    c = s["case"]
    op = c["op"]
    if op.startswith("mm"):
        if "ws" not in s:   # the plan that a program keeps for a shape
            s["cfg"] = moe.GroupCfg(rows=c["rows"], E=c["E"], n=c["n"], k=c["k"])
            s["ws"] = torch.zeros(moe.grouped_ws_bytes(s["cfg"]), dtype=torch.uint8,
                                  device="cuda")
        if op == "mm":
            moe.grouped_mm(s["cfg"], s["x"], s["counts"], s["w"], s["out"], s["ws"])
        elif op == "mm_dx":
            moe.grouped_mm_dx(s["cfg"], s["dy"], s["counts"], s["w"], s["out"], s["ws"])
        else:
            moe.grouped_mm_dw(s["cfg"], s["dy"], s["x"], s["counts"], s["out"], s["ws"])
        return s["out"]
    if op == "swiglu_save":
        moe.swiglu_save(s["gu"], s["a"], s["q"], s["scales"])
        return s["a"], s["q"].view(torch.float8_e4m3fn), s["scales"]
    if op == "swiglu_grad":
        moe.swiglu_grad(s["q"], s["scales"], s["da"], s["dgu"], s["a"])
        return s["dgu"], s["a"]
    if op == "rows":
        moe.act_save(s["x"], s["q"], s["scales"])
        moe.act_load(s["q"], s["scales"], s["index"], s["out"])
        return s["out"], s["q"].view(torch.float8_e4m3fn), s["scales"]
    moe.combine_grad(s["ebuf"], s["row_of"], s["topk_w"], s["dy"], s["debuf"], s["dtopk_w"])
    return s["debuf"], s["dtopk_w"]


# -------------------------------------- the plain forms --------------------------------------
def _slots(counts, rows):
    """The groups that have rows, and each row's place: (its group among those, its number in
    the group), and the most rows of a group."""
    ends = torch.cumsum(counts.long(), 0)
    r = torch.arange(rows, device=counts.device)
    group = torch.searchsorted(ends, r, right=True)
    pos = r - (ends - counts)[group]
    active = torch.nonzero(counts).flatten()
    rank = torch.zeros_like(ends)
    rank[active] = torch.arange(active.numel(), device=counts.device)
    return active, rank[group], pos, int(counts.max())


def _padded(t, n_groups, group, pos, most):
    p = torch.zeros((n_groups, most, t.shape[1]), dtype=torch.float32, device=t.device)
    p[group, pos] = t.float()
    return p


def _plain_mm(s):
    active, group, pos, most = _slots(s["counts"], s["x"].shape[0])
    xp = _padded(s["x"], active.numel(), group, pos, most)
    y = torch.bmm(xp, s["w"][active].float().transpose(1, 2))
    return y[group, pos].to(torch.bfloat16)


def _plain_mm_dx(s):
    active, group, pos, most = _slots(s["counts"], s["dy"].shape[0])
    dyp = _padded(s["dy"], active.numel(), group, pos, most)
    dx = torch.bmm(dyp, s["w"][active].float())
    return dx[group, pos].to(torch.bfloat16)


def _plain_mm_dw(s):
    active, group, pos, most = _slots(s["counts"], s["x"].shape[0])
    dyp = _padded(s["dy"], active.numel(), group, pos, most)
    xp = _padded(s["x"], active.numel(), group, pos, most)
    dw = torch.zeros(s["out"].shape, dtype=s["out"].dtype, device=s["out"].device)
    dw[active] = torch.bmm(dyp.transpose(1, 2), xp).to(dw.dtype)
    return dw


def _quantise(x):
    """e4m3 codes of x [rows][c] in blocks of 128 columns, and their scales [c / 128][rows]."""
    b = x.view(x.shape[0], -1, _BLOCK)
    amax = b.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / _E4M3_MAX, torch.ones_like(amax))
    q = (b / scale).to(torch.float8_e4m3fn).view(x.shape)
    return q, scale.squeeze(-1).t().contiguous()


def _restore(q, scales):
    b = q.float().view(q.shape[0], -1, _BLOCK) * scales.t().unsqueeze(-1)
    return b.view(q.shape)


def _plain_swiglu_save(s):
    gu = s["gu"].float()
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    a = g / (1.0 + torch.exp(-g)) * u
    q, scales = _quantise(gu)
    return a.to(torch.bfloat16), q, scales


def _plain_swiglu_grad(s):
    gu = _restore(s["q"].view(torch.float8_e4m3fn), s["scales"])
    f = gu.shape[1] // 2
    g, u, da = gu[:, :f], gu[:, f:], s["da"].float()
    sig = 1.0 / (1.0 + torch.exp(-g))
    dg = da * u * sig * (1.0 + g * (1.0 - sig))
    du = da * g * sig
    a = g * sig * u
    return torch.cat([dg, du], 1).to(torch.bfloat16), a.to(torch.bfloat16)


def _plain_rows(s):
    q, scales = _quantise(s["x"].float())
    out = _restore(q, scales)[s["index"].long()].to(torch.bfloat16)
    return out, q, scales


def _plain_combine_grad(s):
    rows = s["row_of"].long()
    dy = s["dy"].float().unsqueeze(1)
    dw = (s["ebuf"][rows].float() * dy).sum(-1)
    de = torch.zeros(s["ebuf"].shape, dtype=torch.bfloat16, device=rows.device)
    de[rows.flatten()] = (s["topk_w"].unsqueeze(-1) * dy).to(torch.bfloat16).flatten(0, 1)
    return de, dw


_PLAIN = dict(mm=_plain_mm, mm_dx=_plain_mm_dx, mm_dw=_plain_mm_dw,
              swiglu_save=_plain_swiglu_save, swiglu_grad=_plain_swiglu_grad,
              rows=_plain_rows, combine_grad=_plain_combine_grad)


# --------------------------------------------------------------------------------------------
# In 64 bits, from the definitions
# --------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("mm"):
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        first = 0
        for e, c in enumerate(s["counts"].tolist()):
            rows = slice(first, first + c)
            first += c
            if c == 0:
                continue
            if op == "mm":
                out[rows] = s["x"][rows].double() @ s["w"][e].double().t()
            elif op == "mm_dx":
                out[rows] = s["dy"][rows].double() @ s["w"][e].double()
            else:
                out[e] = s["dy"][rows].double().t() @ s["x"][rows].double()
        return out
    if op == "swiglu_save":
        g, u = s["gu"].double().chunk(2, dim=1)
        # the codes are whole choices of a rounding: they have no value beside their own
        return g * torch.sigmoid(g) * u, None, _exact_scales(s["gu"].double())
    if op == "swiglu_grad":
        v = s["q"].view(torch.float8_e4m3fn).double()
        v = v * s["scales"].double().t().repeat_interleave(_BLOCK, dim=1)
        g, u = v.chunk(2, dim=1)
        sig = torch.sigmoid(g)
        da = s["da"].double()
        slope = sig + g * sig * torch.sigmoid(-g)
        return torch.cat((da * u * slope, da * g * sig), dim=1), g * sig * u
    if op == "rows":
        x = s["x"].double()
        sc = _exact_scales(x)
        wide = sc.t().repeat_interleave(_BLOCK, dim=1)
        v = x / wide
        # the e4m3 grid: steps of 2^(e-3) with the exponent e at least -6, ties to even
        _, e = torch.frexp(v)
        step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(min=-6) - 3)
        v = (torch.round(v / step) * step).clamp(-_E4M3_MAX, _E4M3_MAX)
        return (v * wide)[s["index"].long()], None, sc
    e = s["ebuf"].double()
    dy, w, row_of = s["dy"].double(), s["topk_w"].double(), s["row_of"].long()
    de = torch.zeros_like(e)
    dw = torch.zeros_like(w)
    for i in range(case["k"]):
        de[row_of[:, i]] = w[:, i:i + 1] * dy
        dw[:, i] = torch.einsum("td,td->t", dy, e[row_of[:, i]])
    return de, dw


def _exact_scales(x):
    amax = x.abs().reshape(x.shape[0], -1, _BLOCK).max(dim=-1).values
    return torch.where(amax > 0, amax / _E4M3_MAX, torch.ones_like(amax)).t().contiguous()
