"""A training step of the layer: forward with 8-bit activation checkpoints, backward to the gradients
of the input, the expert weights, the routing weights and (train_router) the gate; the block around it
(MoETrainBlock: norms, gate, residual); its optimiser (AdamW).

Composed of the library's calls only (include/moe.h, "Training of the expert path" and "The rest of a
training step of an MoE block"). Without train_router the gradients stop at the routing weights
dtopk_w.
"""
from __future__ import annotations

import torch

from . import (AdamCfg, AdamTensors, Buffers, GroupCfg, MOE_BF16, _output, act_load, act_save,
               adam_state, adam_step, adamw, combine, combine_grad, dispatch, grad_norm, grouped_mm,
               grouped_mm_dw, grouped_mm_dx, grouped_ws_bytes, make_cfg, norm_in, norm_in_grad,
               norm_out, norm_out_grad, norm_ws_bytes, route, route_grad, route_grad_ws_bytes,
               route_save, swiglu_grad, swiglu_save)


class _Experts:
    """SwiGLU experts over rows in group order: the buffers and the calls of both directions.
    Between the two passes it keeps the 8-bit codes of the gate/up product only."""

    def __init__(self, rows, E, d, f, device):
        self.up = GroupCfg(rows=rows, E=E, n=2 * f, k=d)
        self.down = GroupCfg(rows=rows, E=E, n=d, k=f)
        size = max(grouped_ws_bytes(self.up), grouped_ws_bytes(self.down))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=device)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.gu = torch.empty((rows, 2 * f), **bf)     # gate/up product; its gradient
        self.a = torch.empty((rows, f), **bf)
        self.da = torch.empty((rows, f), **bf)
        self.q = torch.empty((rows, 2 * f), dtype=torch.uint8, device=device)
        self.scales = torch.empty((2 * f // 128, rows), dtype=torch.float32, device=device)

    def forward(self, x, counts, w13, w2, y, stream=None):
        grouped_mm(self.up, x, counts, w13, self.gu, self.ws, stream=stream)
        swiglu_save(self.gu, self.a, self.q, self.scales, stream=stream)
        grouped_mm(self.down, self.a, counts, w2, y, self.ws, stream=stream)

    def backward_hidden(self, dy, counts, w13, w2, dw2, dx, accumulate, stream=None):
        """Down to the gate/up product's gradient (kept in gu), the rows' and dw2."""
        grouped_mm_dx(self.down, dy, counts, w2, self.da, self.ws, stream=stream)
        swiglu_grad(self.q, self.scales, self.da, self.gu, self.a, stream=stream)
        grouped_mm_dw(self.down, dy, self.a, counts, dw2, self.ws, accumulate, stream=stream)
        grouped_mm_dx(self.up, self.gu, counts, w13, dx, self.ws, stream=stream)

    def backward_up(self, x, counts, dw13, accumulate, stream=None):
        grouped_mm_dw(self.up, self.gu, x, counts, dw13, self.ws, accumulate, stream=stream)


class MoETrainLayer:
    """One MoE layer whose experts are trained: ``y = layer.forward(x)`` routes, dispatches, runs
    the experts and combines; ``grads = layer.backward(dy)`` then fills ``layer.grads``.

    cfg: a bf16 configuration with R = 1 (expert-contiguous rows). weights: w13, w2 and, with a
    shared expert, ws13 and ws2, as MoELayer takes them. grad_dtype: torch.float32 (gradients
    may be summed over micro-batches, ``backward(dy, accumulate=True)``; they start at zero) or
    torch.bfloat16. train_router: the gate is trained too; dx then holds the router's part, and grads
    has dw_gate (fp32), from x as the 8-bit checkpoint keeps it.
    Between forward and backward the layer keeps x once per token and the gate/up products in 8
    bits, and the expert outputs (for dtopk_w) in bf16. backward writes over the latter two, so
    it runs once for each forward: another one is a RuntimeError."""

    def __init__(self, cfg, w_gate, bias, weights: dict, device="cuda",
                 grad_dtype=torch.float32, train_router=False):
        mc = make_cfg(cfg)
        if mc.R != 1 or mc.act_dtype != MOE_BF16:
            raise ValueError("MoETrainLayer takes a bf16 configuration with R == 1")
        self.cfg, self.w_gate, self.bias, self.weights = cfg, w_gate, bias, weights
        self._saved = False   # whether the buffers hold a forward's values
        T, k, d, E, f, fs = cfg.T, cfg.k, cfg.d, cfg.E, cfg.d_ff, cfg.d_ff_shared
        rows = T * k
        bf = dict(dtype=torch.bfloat16, device=device)
        self.bufs = Buffers(cfg, device)
        self.src_tok = torch.empty((rows,), dtype=torch.int32, device=device)
        self.xq = torch.empty((T, d), dtype=torch.uint8, device=device)
        self.x_scales = torch.empty((d // 128, T), dtype=torch.float32, device=device)
        self.routed = _Experts(rows, E, d, f, device)
        self.drows = torch.empty((rows, d), **bf)
        self.ones = torch.ones((T, k), dtype=torch.float32, device=device)
        g = dict(dtype=grad_dtype, device=device)
        self.grads = dict(dx=torch.empty((T, d), **bf),
                          dtopk_w=torch.empty((T, k), dtype=torch.float32, device=device),
                          dw13=torch.zeros((E, 2 * f, d), **g), dw2=torch.zeros((E, d, f), **g))
        self.shared = None
        if fs or train_router:
            self.xs = torch.empty((T, d), **bf)
        self.train_router = train_router
        if train_router:
            self.topk_s = torch.empty((T, k), dtype=torch.float32, device=device)
            self.router_ws = torch.zeros(route_grad_ws_bytes(cfg), dtype=torch.uint8,
                                         device=device)
            self.grads["dw_gate"] = torch.zeros((E, d), dtype=torch.float32, device=device)
        if fs:
            self.shared = _Experts(T, 1, d, fs, device)
            self.all_rows = torch.full((1,), T, dtype=torch.int32, device=device)
            self.dxs = torch.empty((T, d), **bf)
            self.grads.update(dws13=torch.zeros((1, 2 * fs, d), **g),
                              dws2=torch.zeros((1, d, fs), **g))

    def forward(self, x, y=None, stream=None):
        b, w = self.bufs, self.weights
        shape = (self.cfg.T, self.cfg.d)
        for name, t in (("x", x), ("y", x if y is None else y)):
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.bfloat16 or t.shape != shape:
                raise ValueError(f"MoETrainLayer.forward: {name} must be a bf16 tensor {shape}")
        self._saved = False
        if y is None:
            y = _output(shape, torch.bfloat16, x.device, stream)
        if self.train_router:
            route_save(self.cfg, x, self.w_gate, self.bias, b["topk_idx"], b["topk_w"],
                       self.topk_s, b["ws"], stream)
        else:
            route(self.cfg, x, self.w_gate, self.bias, b["topk_idx"], b["topk_w"], b["ws"], stream)
        dispatch(self.cfg, x, b["topk_idx"], b["recv"], None, b["counts"], b["row_of"],
                 self.src_tok, stream, status=b["ws"])
        act_save(x, self.xq, self.x_scales, stream=stream)
        self.routed.forward(b["recv"], b["counts"].view(-1), w["w13"], w["w2"], b["ebuf"], stream)
        if self.shared is not None:
            self.shared.forward(x, self.all_rows, w["ws13"].unsqueeze(0), w["ws2"].unsqueeze(0),
                                b["shared_out"], stream)
        combine(self.cfg, b["ebuf"], b["row_of"], b["topk_w"], b["shared_out"], y, stream,
                status=b["ws"])
        self._saved = True
        return y

    def backward(self, dy, accumulate=False, stream=None):
        """Gradients for the last forward: dx and dtopk_w (replaced), dw13, dw2, the shared expert's
        dws13, dws2 and the gate's dw_gate (accumulate: added to). Once for each forward."""
        if not self._saved:
            raise RuntimeError("MoETrainLayer.backward: needs a forward of its own")
        b, w, g = self.bufs, self.weights, self.grads
        if accumulate and g["dw13"].dtype is not torch.float32:
            raise ValueError("MoETrainLayer.backward: accumulate needs grad_dtype torch.float32")
        self._saved = False
        counts = b["counts"].view(-1)
        de = self.drows
        combine_grad(b["ebuf"], b["row_of"], b["topk_w"], dy, de, g["dtopk_w"], stream=stream,
                     status=b["ws"])
        # ebuf has been read: it takes the rows' gradient
        self.routed.backward_hidden(de, counts, w["w13"], w["w2"], g["dw2"], b["ebuf"],
                                    accumulate, stream)
        act_load(self.xq, self.x_scales, self.src_tok, b["recv"], stream=stream, status=b["ws"])
        self.routed.backward_up(b["recv"], counts, g["dw13"], accumulate, stream)
        if self.shared is not None:
            self.shared.backward_hidden(dy, self.all_rows, w["ws13"].unsqueeze(0),
                                        w["ws2"].unsqueeze(0), g["dws2"], self.dxs, accumulate,
                                        stream)
        if self.shared is not None or self.train_router:
            act_load(self.xq, self.x_scales, None, self.xs, stream=stream)
        if self.shared is not None:
            self.shared.backward_up(self.xs, self.all_rows, g["dws13"], accumulate, stream)
        combine(self.cfg, b["ebuf"], b["row_of"], self.ones,
                self.dxs if self.shared is not None else None, g["dx"], stream, status=b["ws"])
        if self.train_router:
            route_grad(self.cfg, self.xs, self.w_gate, b["topk_idx"], self.topk_s, g["dtopk_w"],
                       g["dx"], g["dx"], g["dw_gate"], self.router_ws, accumulate, stream)
        return g


class MoETrainBlock:
    """A block of the residual stream around a MoETrainLayer whose gate is trained too:

        h = res_scale x + out_scale gate norm(layer(norm(x) w_in)) w_out

    ``h = block.forward(x)``, then ``grads = block.backward(dh)``: the layer's gradients with the
    block's own (dx, dw_in, dw_out, dgate) among them; dx is that of the block's x.

    w_in, w_out (None: no norm behind the layer): fp32 [d]. gate: None or fp32 [d] (a layer scale).
    stream_dtype: of x, h, dh and dx. Between the passes the block keeps the layer's output and x
    itself, which must not change until backward. The other arguments are MoETrainLayer's."""

    def __init__(self, cfg, w_gate, bias, weights: dict, w_in, w_out=None, gate=None, eps=1e-6,
                 res_scale=1.0, out_scale=1.0, stream_dtype=torch.bfloat16, device="cuda",
                 grad_dtype=torch.float32):
        for name, w in (("w_in", w_in), ("w_out", w_out), ("gate", gate)):
            if (name == "w_in" or w is not None) and (
                    not isinstance(w, torch.Tensor) or w.dtype is not torch.float32
                    or w.shape != (cfg.d,)):
                raise ValueError(f"MoETrainBlock: {name} must be an fp32 tensor ({cfg.d},)")
        self.layer = MoETrainLayer(cfg, w_gate, bias, weights, device, grad_dtype,
                                   train_router=True)
        self.w_in, self.w_out, self.gate = w_in, w_out, gate
        self.eps, self.scales = eps, dict(res_scale=res_scale, out_scale=out_scale)
        T, d = cfg.T, cfg.d
        f32 = dict(dtype=torch.float32, device=device)
        bf = dict(dtype=torch.bfloat16, device=device)
        self.stream_dtype, self.shape = stream_dtype, (T, d)
        self.n, self.y = torch.empty((T, d), **bf), torch.empty((T, d), **bf)
        self.rstd_in = torch.empty((T,), **f32)
        self.rstd_out = torch.empty((T,), **f32) if w_out is not None else None
        self.dres = torch.empty((T, d), dtype=stream_dtype, device=device)
        self.ws = torch.zeros(norm_ws_bytes(T, d), dtype=torch.uint8, device=device)
        zeros = lambda w: None if w is None else torch.zeros((d,), **f32)   # noqa: E731
        self.own = dict(dx=torch.empty((T, d), dtype=stream_dtype, device=device),
                        dw_in=zeros(w_in), dw_out=zeros(w_out), dgate=zeros(gate))
        self.grads = {**self.layer.grads, **{k: v for k, v in self.own.items() if v is not None}}
        self._x = None

    def parameters(self):
        """name -> (weight, gradient), for AdamW."""
        w = dict(self.layer.weights, w_gate=self.layer.w_gate, w_in=self.w_in, w_out=self.w_out,
                 gate=self.gate)
        return {n: (w[n], self.grads["d" + n].view(w[n].shape)) for n in
                ("w13", "w2", "ws13", "ws2", "w_gate", "w_in", "w_out", "gate")
                if w.get(n) is not None and "d" + n in self.grads}

    def forward(self, x, h=None, stream=None):
        for name, t in (("x", x), ("h", x if h is None else h)):
            if (not isinstance(t, torch.Tensor) or t.dtype is not self.stream_dtype
                    or t.shape != self.shape):
                raise ValueError(f"MoETrainBlock.forward: {name} must be a {self.stream_dtype} "
                                 f"tensor {self.shape}")
        if h is not None and h.data_ptr() == x.data_ptr():
            raise ValueError("MoETrainBlock.forward: x is kept for backward: h must be another")
        self._x = None
        if h is None:
            h = _output(x.shape, x.dtype, x.device, stream)
        norm_in(x, self.w_in, self.n, self.rstd_in, eps=self.eps, stream=stream)
        self.layer.forward(self.n, self.y, stream)
        norm_out(self.y, x, self.w_out, self.gate, None, h, None, self.rstd_out, None,
                 eps=self.eps, stream=stream, **self.scales)
        self._x = x
        return h

    def backward(self, dh, accumulate=False, stream=None):
        """Gradients for the last forward (accumulate: the weights' are added to). Once for each
        forward."""
        if self._x is None:
            raise RuntimeError("MoETrainBlock.backward: needs a forward of its own")
        if accumulate and self.layer.grads["dw13"].dtype is not torch.float32:
            raise ValueError("MoETrainBlock.backward: accumulate needs grad_dtype torch.float32")
        o, x = self.own, self._x
        # n and y's gradient share a buffer: n has been read (the layer keeps its own copy)
        norm_out_grad(dh, None, self.y, None, self.w_out, self.gate, None, self.rstd_out, None,
                      self.dres, self.n, o["dgate"], o["dw_out"], None, self.ws,
                      accumulate=accumulate, stream=stream, **self.scales)
        self._x = None
        self.layer.backward(self.n, accumulate, stream)
        norm_in_grad(self.layer.grads["dx"], x, self.w_in, self.rstd_in, self.dres, o["dx"],
                     o["dw_in"], self.ws, accumulate=accumulate, stream=stream)
        return self.grads


class AdamW:
    """AdamW over named weights: ``AdamW(block.parameters(), lr)``, then ``step()`` after each
    backward, one launch for all of them (and one for the gradients' norm, with max_norm).

    params: name -> (weight, gradient), each kept as the very tensors. A bf16 weight gets an fp32
    master copy, which the step updates and rounds into the weight; an fp32 one is updated itself.
    weight_decay: of the weights of two dimensions and more (norms and layer scales have none).
    state_bits: 32, or 8: both moments as e4m3 codes with a scale per 128 elements, rounded at random
    from the seed. A step whose norm is not finite is left out (max_norm; MOE_DEV_NONFINITE in the
    state's status word)."""

    def __init__(self, params, lr, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, max_norm=0.0,
                 state_bits=32, seed=0):
        self.tensors, self.names = [], list(params)
        for i, (weight, grad) in enumerate(params.values()):
            if weight.requires_grad:   # (the same memory: a step is written into a leaf in place)
                weight = weight.detach()
            own = weight.dtype is torch.float32
            p = weight if own else weight.float()
            n, dev = weight.numel(), weight.device
            t = dict(p=p, g=grad, w=None if own else weight, seed=(seed + 0x9E3779B1 * i),
                     weight_decay=weight_decay if weight.dim() > 1 else 0.0)
            kind = torch.float32 if state_bits == 32 else torch.uint8
            for m in ("m", "v"):
                t[m] = torch.zeros(weight.shape, dtype=kind, device=dev)
                if state_bits == 8:
                    t[m + "_scale"] = torch.zeros(((n + 127) // 128,), device=dev)
            self.tensors.append(t)
        self.plan = AdamTensors(self.tensors, state_bits)
        self.cfg = AdamCfg(lr=lr, beta1=betas[0], beta2=betas[1], eps=eps, max_norm=max_norm)
        dev = self.tensors[0]["p"].device if self.tensors else "cuda"
        self.state = adam_state(0, *betas, device=dev)
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev) if max_norm > 0 else None

    @property
    def steps(self):
        """Steps made (synchronises)."""
        return adam_step(self.state)

    def step(self, lr=None, stream=None):
        """One step. lr: None, a number (from now on), or an fp32 device tensor read by this call."""
        if lr is not None and not isinstance(lr, torch.Tensor):
            self.cfg.lr, lr = float(lr), None
        if self.norm is not None:
            grad_norm(self.plan, self.state, self.norm, stream=stream)
        adamw(self.cfg, self.plan, self.state, self.norm, stream=stream, lr=lr)

    def state_dict(self):
        """Copies of everything a later load_state_dict needs."""
        return dict(state=self.state.clone(),
                    tensors={n: {k: t[k].clone() for k in self._kept(t)}
                             for n, t in zip(self.names, self.tensors)})

    @staticmethod
    def _kept(t):
        return [k for k in ("p", "m", "v", "m_scale", "v_scale") if k in t]

    def load_state_dict(self, saved):
        """What state_dict gave, of an optimiser of the same weights and state_bits. One that does not
        fit is a ValueError, before anything is written."""
        if set(saved["tensors"]) != set(self.names):
            raise ValueError("AdamW.load_state_dict: saved for other weights")
        if saved["state"].shape != self.state.shape or saved["state"].dtype != self.state.dtype:
            raise ValueError("AdamW.load_state_dict: state is of another kind")
        for n, t in zip(self.names, self.tensors):
            s = saved["tensors"][n]
            if set(s) != set(self._kept(t)):
                raise ValueError(f"AdamW.load_state_dict: {n}: saved with other moments")
            for k, v in s.items():
                if t[k].shape != v.shape or t[k].dtype != v.dtype:
                    raise ValueError(f"AdamW.load_state_dict: {n}: {k} is of another kind")
        for n, t in zip(self.names, self.tensors):
            for k, v in saved["tensors"][n].items():
                t[k].copy_(v)
            if t["w"] is not None:
                t["w"].copy_(t["p"])
        self.state.copy_(saved["state"])
