"""A training step of the layer's experts: forward with 8-bit activation checkpoints, backward to
the gradients of the input, the expert weights and the routing weights.

Composed of the library's calls only (include/moe.h, "Training of the expert path"); the
gradients stop at the routing weights dtopk_w, which the caller carries on into the gate.
"""
from __future__ import annotations

import torch

from . import (Buffers, GroupCfg, MOE_BF16, act_load, act_save, combine, combine_grad, dispatch,
               grouped_mm, grouped_mm_dw, grouped_mm_dx, grouped_ws_bytes, make_cfg, route,
               swiglu_grad, swiglu_save)


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
    torch.bfloat16.
    Between forward and backward the layer keeps x once per token and the gate/up products in 8
    bits, and the expert outputs (for dtopk_w) in bf16. backward writes over the latter two, so
    it runs once for each forward: another one is a RuntimeError."""

    def __init__(self, cfg, w_gate, bias, weights: dict, device="cuda",
                 grad_dtype=torch.float32):
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
        if fs:
            self.shared = _Experts(T, 1, d, fs, device)
            self.all_rows = torch.full((1,), T, dtype=torch.int32, device=device)
            self.xs = torch.empty((T, d), **bf)
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
            y = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
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
        """Gradients for the last forward: dx and dtopk_w (replaced), dw13, dw2 and the shared
        expert's dws13, dws2 (accumulate: added to). Once for each forward."""
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
            act_load(self.xq, self.x_scales, None, self.xs, stream=stream)
            self.shared.backward_up(self.xs, self.all_rows, g["dws13"], accumulate, stream)
        combine(self.cfg, b["ebuf"], b["row_of"], self.ones,
                self.dxs if self.shared is not None else None, g["dx"], stream, status=b["ws"])
        return g
