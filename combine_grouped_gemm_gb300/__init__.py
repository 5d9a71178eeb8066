"""Python binding of libmoe, the GB300 (sm_103a) MoE-layer hot path.

Argument marshalling only: every function below passes device pointers of torch CUDA tensors
and the current CUDA stream to the C ABI declared in include/moe.h, and raises MoEError on a
non-zero return code. All the work runs in the library's CUDA kernels; there is no fallback.
If the shared library is missing, importing this package raises at once: build it with
``python combine_grouped_gemm_gb300/build.py``.

A call runs on ``stream`` (None: the current one), and an output that it makes itself belongs to that
stream, as if it had been made with the stream current. The buffers of a layer or block belong to the
stream that was current when it was made: another one waits for that once, before its first call.
"""
from __future__ import annotations

import ctypes
import numbers
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe.so")

MOE_BF16, MOE_FP8_E4M3, MOE_FP8_E4M3_POW2 = 0, 1, 2
MOE_F32 = 3   # dtype of a weight gradient, the norms' residual stream or an optimiser's gradient
MOE_DEV_TIMEOUT, MOE_DEV_BOUNDS, MOE_DEV_SCALE, MOE_DEV_NONFINITE = 1, 2, 4, 8
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN, MOE_GATE_ELEMENT = 0, 1, 2, 3
MOE_ADAM_TENSORS = 256   # tensors of one moe_adamw or moe_grad_norm call
MOE_LAYER_EVENTS = 7
STAGE_NAMES = ["route", "dispatch", "ffn_setup", "ffn_gate_up", "ffn_down", "combine"]


class MoEError(RuntimeError):
    def __init__(self, fn, code, msg, cuda_err=0):
        super().__init__(f"{fn}: {msg} (code {code}" + (f", cudaError {cuda_err})" if cuda_err else ")"))
        self.code = code
        self.cuda_error = cuda_err


class Cfg(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("d_ff_shared", ctypes.c_int32), ("R", ctypes.c_int32),
                ("route_scale", ctypes.c_float), ("act_dtype", ctypes.c_int32),
                ("w_dtype", ctypes.c_int32)]


class Sizes(ctypes.Structure):
    _fields_ = [("recv_rows", ctypes.c_int64), ("cap", ctypes.c_int32),
                ("recv_bytes", ctypes.c_size_t), ("recv_scale_bytes", ctypes.c_size_t),
                ("ebuf_bytes", ctypes.c_size_t), ("ws_bytes", ctypes.c_size_t)]


MOE_OPT_GATHER_X, MOE_OPT_SHARED_SIDE_STREAM, MOE_OPT_FUSED_FFN = 1, 2, 4


class PlacementC(ctypes.Structure):
    _fields_ = [("slots_per_rank", ctypes.c_int32), ("max_copies", ctypes.c_int32),
                ("slot_expert", ctypes.c_void_p), ("n_copies", ctypes.c_void_p),
                ("copy_slot", ctypes.c_void_p)]


class LayerOpts(ctypes.Structure):
    _fields_ = [("flags", ctypes.c_uint32), ("side_stream", ctypes.c_void_p),
                ("fork_event", ctypes.c_void_p), ("join_event", ctypes.c_void_p),
                ("side_ctas", ctypes.c_int32), ("placement", ctypes.POINTER(PlacementC))]


class GroupCfg(ctypes.Structure):
    """moe_group_cfg: the shape of one grouped product (rows in all, groups, weights [n][k])."""
    _fields_ = [("rows", ctypes.c_int32), ("E", ctypes.c_int32), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32)]


class NormCfg(ctypes.Structure):
    """moe_norm_cfg: rows, width, scales and types of the norms around a block."""
    _fields_ = [("rows", ctypes.c_int32), ("d", ctypes.c_int32), ("eps", ctypes.c_float),
                ("res_scale", ctypes.c_float), ("out_scale", ctypes.c_float),
                ("stream_dtype", ctypes.c_int32), ("gate", ctypes.c_int32)]


class AdamTensorC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "g", "w", "m", "v", "m_scale", "v_scale")] + [
        ("n", ctypes.c_int64), ("weight_decay", ctypes.c_float), ("seed", ctypes.c_uint32),
        ("g_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class AdamCfg(ctypes.Structure):
    """moe_adam_cfg: an AdamW step's rates. adamw takes state_bits from the tensors' plan and lr_dev
    from its own argument, and writes nothing into the one that it is given."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("max_norm", ctypes.c_double),
                ("lr_dev", ctypes.c_void_p), ("state_bits", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("w13", "w13_scales", "w2", "w2_scales", "ws13", "ws13_scales", "ws2",
                 "ws2_scales")]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmoe.so not found at {LIB_PATH}; build it with "
                          "`python combine_grouped_gemm_gb300/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p
    sigs = {
        "moe_validate": [P],
        "moe_query_sizes": [P, P],
        "moe_route": [P, P, P, P, P, P, P, S],
        "moe_route_noalloc": [P, P, P, P, P, P, S],
        "moe_dispatch": [P, P, P, P, P, P, P, P, P, S],
        "moe_expert_ffn": [P, P, P, P, P, P, P, P, P, S],
        "moe_combine": [P, P, P, P, P, P, P, S],
        "moe_layer": [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P],
        "moe_layer_ex": [P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, P, S, P],
        "moe_dispatch_index": [P, P, P, P, P, P, S],
        "moe_place_experts": [I, I, I, P, I, P, P, P],
        "moe_query_sizes_placed": [P, I, P],
        "moe_expert_ffn_gather": [P, P, P, P, P, P, P, P, S],
        "moe_grouped_query": [P, P],
        "moe_grouped_mm": [P, P, P, P, P, P, S],
        "moe_grouped_mm_dx": [P, P, P, P, P, P, S],
        "moe_grouped_mm_dw": [P, P, P, P, P, I, I, P, S],
        "moe_act_save": [I, I, P, P, P, S],
        "moe_act_load": [I, I, I, P, P, P, P, P, S],
        "moe_swiglu_save": [I, I, P, P, P, P, S],
        "moe_swiglu_grad": [I, I, P, P, P, P, P, S],
        "moe_combine_grad": [I, I, I, I, P, P, P, P, P, P, P, S],
        "moe_norm_query": [I, I, P],
        "moe_norm_in": [P, P, P, P, P, S],
        "moe_norm_in_grad": [P, P, P, P, P, P, P, P, I, P, S],
        "moe_norm_out": [P, P, P, P, P, P, P, P, P, P, S],
        "moe_norm_out_grad": [P] * 15 + [I, P, S],
        "moe_route_save": [P, P, P, P, P, P, P, P, S],
        "moe_route_grad": [P, P, P, P, P, P, P, P, P, I, P, S],
        "moe_route_grad_query": [P, P],
        "moe_adamw": [P, P, I, I, P, P, S],
        "moe_grad_norm": [P, I, I, P, P, S],
        "moe_adam_query": [P],
        "moe_clear_status": [P, S],
        "moe_read_status": [P, P, S],
        "moe_selftest_wait": [P, ctypes.c_int64, S],
        "moe_strerror": [I],
        "moe_abi_version": [],
        "moe_last_cuda_error": [],
    }
    for name, args in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_char_p if name == "moe_strerror" else ctypes.c_int
    return L


_lib = _load()

EXPORTED = ["moe_validate", "moe_query_sizes", "moe_route", "moe_route_noalloc", "moe_dispatch",
            "moe_expert_ffn", "moe_combine", "moe_layer", "moe_layer_ex", "moe_dispatch_index",
            "moe_expert_ffn_gather", "moe_place_experts", "moe_query_sizes_placed",
            "moe_grouped_query", "moe_grouped_mm", "moe_grouped_mm_dx", "moe_grouped_mm_dw",
            "moe_act_save", "moe_act_load", "moe_swiglu_save", "moe_swiglu_grad",
            "moe_combine_grad", "moe_norm_query", "moe_norm_in", "moe_norm_in_grad",
            "moe_norm_out", "moe_norm_out_grad", "moe_route_save", "moe_route_grad",
            "moe_route_grad_query", "moe_adamw", "moe_grad_norm", "moe_adam_query",
            "moe_clear_status", "moe_read_status", "moe_selftest_wait",
            "moe_strerror", "moe_abi_version", "moe_last_cuda_error"]


def _check(fn, rc):
    if rc != 0:
        err = _lib.moe_last_cuda_error() if rc == 4 else 0
        raise MoEError(fn, rc, _lib.moe_strerror(rc).decode(), err)


def _dtype_code(v):
    if isinstance(v, str):
        return MOE_FP8_E4M3 if v in ("fp8", "e4m3") else MOE_BF16
    return int(v)


def make_cfg(c) -> Cfg:
    """Cfg from any object with the moe_cfg fields (act / w may be "bf16" / "fp8"; an e4m3
    configuration with scales == "pow2" takes the power-of-two recipe)."""
    act = _dtype_code(getattr(c, "act_dtype", getattr(c, "act", MOE_BF16)))
    w = _dtype_code(getattr(c, "w_dtype", getattr(c, "w", act)))
    if getattr(c, "scales", "amax") == "pow2":
        act = MOE_FP8_E4M3_POW2 if act == MOE_FP8_E4M3 else act
        w = MOE_FP8_E4M3_POW2 if w == MOE_FP8_E4M3 else w
    return Cfg(c.T, c.d, c.E, c.k, c.n_group, c.topk_group, c.d_ff, c.d_ff_shared, c.R,
               float(c.route_scale), act, w)


def _p(t):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors")
    return t.data_ptr()


# The handle of a device's current stream without building a Stream object (3 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _s(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _output(shape, dtype, device, stream):
    """An output that a call on this stream makes. (From the current stream's memory it could be what
    that stream has given back while its work still reads it.)"""
    handle = None if stream is None else _s(stream)
    if handle is None or handle == _s(None):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle > 1 else
                  torch.cuda.default_stream(device))   # (0 and 1 are that one's names)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


_WEIGHT_KEYS = ("w13", "w13_s", "w2", "w2_s", "ws13", "ws13_s", "ws2", "ws2_s")


def _weights(w: dict) -> Weights:
    """moe_weights from a dict with keys w13, w13_s, w2, w2_s, ws13, ws13_s, ws2, ws2_s."""
    return Weights(*[_p(w.get(n)) for n in _WEIGHT_KEYS])


def validate(cfg) -> int:
    return _lib.moe_validate(ctypes.byref(make_cfg(cfg)))


def query_sizes(cfg) -> dict:
    s = Sizes()
    _check("moe_query_sizes", _lib.moe_query_sizes(ctypes.byref(make_cfg(cfg)), ctypes.byref(s)))
    return {n: getattr(s, n) for n, _ in Sizes._fields_}


def query_sizes_placed(cfg, slots_per_rank) -> dict:
    s = Sizes()
    _check("moe_query_sizes_placed", _lib.moe_query_sizes_placed(
        ctypes.byref(make_cfg(cfg)), int(slots_per_rank), ctypes.byref(s)))
    return {n: getattr(s, n) for n, _ in Sizes._fields_}


def place_experts(load, R, slots_per_rank, max_copies=8):
    """moe_place_experts on the host: (slot_expert [R*S], n_copies [E], copy_slot [E][max])
    as numpy int32 arrays, from estimated loads [E]."""
    import numpy as np
    ld = np.ascontiguousarray(load, dtype=np.float64)
    E = ld.size
    se = np.empty(R * slots_per_rank, dtype=np.int32)
    nc = np.empty(E, dtype=np.int32)
    cs = np.empty((E, max_copies), dtype=np.int32)
    ptr = lambda a: a.ctypes.data_as(ctypes.c_void_p)   # noqa: E731
    _check("moe_place_experts", _lib.moe_place_experts(E, R, slots_per_rank, ptr(ld), max_copies,
                                                       ptr(se), ptr(nc), ptr(cs)))
    return se, nc, cs


class Placement:
    """A placement of the experts on slots (see moe_placement), held on the device."""

    def __init__(self, slot_expert, n_copies, copy_slot, slots_per_rank, device="cuda"):
        self.slots_per_rank = int(slots_per_rank)
        self.slot_expert = torch.as_tensor(slot_expert, dtype=torch.int32).to(device).contiguous()
        self.n_copies = torch.as_tensor(n_copies, dtype=torch.int32).to(device).contiguous()
        self.copy_slot = torch.as_tensor(copy_slot, dtype=torch.int32).to(device).contiguous()
        self.c = PlacementC(self.slots_per_rank, self.copy_slot.shape[1],
                            self.slot_expert.data_ptr(), self.n_copies.data_ptr(),
                            self.copy_slot.data_ptr())

    @classmethod
    def from_loads(cls, load, R, slots_per_rank, max_copies=8, device="cuda"):
        se, nc, cs = place_experts(load, R, slots_per_rank, max_copies)
        return cls(se, nc, cs, slots_per_rank, device)


def route(cfg, x, w_gate, bias, topk_idx, topk_w, ws, stream=None):
    _check("moe_route", _lib.moe_route(ctypes.byref(make_cfg(cfg)), _p(x), _p(w_gate), _p(bias),
                                       _p(topk_idx), _p(topk_w), _p(ws), _s(stream)))


def route_noalloc(cfg, x, w_gate, bias, topk_idx, topk_w, stream=None):
    """moe_route for callers that cannot supply a workspace: the library's own fixed device
    array holds the router's scratch (see moe_route_noalloc in include/moe.h)."""
    _check("moe_route_noalloc", _lib.moe_route_noalloc(ctypes.byref(make_cfg(cfg)), _p(x),
                                                       _p(w_gate), _p(bias), _p(topk_idx),
                                                       _p(topk_w), _s(stream)))


def dispatch(cfg, x, topk_idx, recv, recv_scales, counts, row_of, src_tok=None, stream=None,
             status=None):
    """status: None or a device tensor whose first 4 bytes receive MOE_DEV_* bits (e.g. ws)."""
    _check("moe_dispatch", _lib.moe_dispatch(ctypes.byref(make_cfg(cfg)), _p(x), _p(topk_idx),
                                             _p(recv), _p(recv_scales), _p(counts), _p(row_of),
                                             _p(src_tok), _p(status), _s(stream)))


def expert_ffn(cfg, recv, recv_scales, counts, x, weights: dict, ebuf, shared_out, ws,
               stream=None):
    w = _weights(weights)
    _check("moe_expert_ffn", _lib.moe_expert_ffn(ctypes.byref(make_cfg(cfg)), _p(recv),
                                                 _p(recv_scales), _p(counts), _p(x),
                                                 ctypes.byref(w), _p(ebuf), _p(shared_out),
                                                 _p(ws), _s(stream)))


def combine(cfg, ebuf, row_of, topk_w, shared_out, y, stream=None, status=None):
    _check("moe_combine", _lib.moe_combine(ctypes.byref(make_cfg(cfg)), _p(ebuf), _p(row_of),
                                           _p(topk_w), _p(shared_out), _p(y), _p(status),
                                           _s(stream)))


def layer(cfg, x, w_gate, bias, weights: dict, bufs: dict, y, stream=None, events=None):
    """The whole layer. bufs holds topk_idx, topk_w, recv, recv_scales, counts, row_of, ebuf,
    shared_out and ws (see Buffers). events: None or MOE_LAYER_EVENTS torch.cuda.Event that
    have been recorded once (so their handles exist)."""
    w = _weights(weights)
    ev = None
    if events is not None:
        arr = (ctypes.c_void_p * MOE_LAYER_EVENTS)(*[e.cuda_event for e in events])
        ev = ctypes.cast(arr, ctypes.c_void_p)
    b = bufs
    _check("moe_layer", _lib.moe_layer(ctypes.byref(make_cfg(cfg)), _p(x), _p(w_gate), _p(bias),
                                       ctypes.byref(w), _p(b["topk_idx"]), _p(b["topk_w"]),
                                       _p(b["recv"]), _p(b.get("recv_scales")), _p(b["counts"]),
                                       _p(b["row_of"]), _p(b["ebuf"]), _p(b.get("shared_out")),
                                       _p(y), _p(b["ws"]), _s(stream), ev))


def layer_ex(cfg, opts: LayerOpts | None, x, w_gate, bias, weights: dict, bufs: dict, y,
             stream=None, events=None):
    """moe_layer_ex: the layer with the variants of opts (None: moe_layer)."""
    w = _weights(weights)
    ev = None
    if events is not None:
        arr = (ctypes.c_void_p * MOE_LAYER_EVENTS)(*[e.cuda_event for e in events])
        ev = ctypes.cast(arr, ctypes.c_void_p)
    b = bufs
    _check("moe_layer_ex", _lib.moe_layer_ex(ctypes.byref(make_cfg(cfg)),
                                             ctypes.byref(opts) if opts is not None else None,
                                             _p(x), _p(w_gate), _p(bias), ctypes.byref(w),
                                             _p(b["topk_idx"]), _p(b["topk_w"]), _p(b.get("recv")),
                                             _p(b.get("recv_scales")), _p(b["counts"]),
                                             _p(b["row_of"]), _p(b["ebuf"]),
                                             _p(b.get("shared_out")), _p(y), _p(b["ws"]),
                                             _s(stream), ev))


def dispatch_index(cfg, topk_idx, counts, row_of, src_tok, stream=None, status=None):
    _check("moe_dispatch_index", _lib.moe_dispatch_index(ctypes.byref(make_cfg(cfg)), _p(topk_idx),
                                                         _p(counts), _p(row_of), _p(src_tok),
                                                         _p(status), _s(stream)))


def expert_ffn_gather(cfg, x, counts, src_tok, weights: dict, ebuf, shared_out, ws, stream=None):
    w = _weights(weights)
    _check("moe_expert_ffn_gather",
           _lib.moe_expert_ffn_gather(ctypes.byref(make_cfg(cfg)), _p(x), _p(counts), _p(src_tok),
                                      ctypes.byref(w), _p(ebuf), _p(shared_out), _p(ws),
                                      _s(stream)))


# ---------------------------------------------------------------------------------------------
# Training of the expert path (see include/moe.h). Row counts and widths are taken from the
# tensors; a tensor of another type or size than the call needs, or of another device than the
# current one, is a ValueError.
# ---------------------------------------------------------------------------------------------
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _device():
    """The number of the current device, which no tensor has where there is none."""
    try:
        return _get_device()
    except (RuntimeError, AssertionError):
        return -2


def _here(fn, dev, name, t):
    """_p(t), for a tensor that must be device dev's."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{fn}: {name} must be on the current device, cuda:{dev}")
    return _p(t)


def _stream(stream, dev):
    """_s(stream), where the current device's number is known."""
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _s(stream)


def _need(fn, dev, name, t, dtype, *shape):
    """_p(t), for a tensor of device dev that must have this element type and shape. int8 and
    e4m3 tensors count as bytes."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{fn}: {name} must be a CUDA tensor")
    if t.dtype is not dtype and not (dtype is torch.uint8 and t.dtype in
                                     (torch.int8, torch.float8_e4m3fn)):
        raise ValueError(f"{fn}: {name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{fn}: {name} must have shape {shape}, got {tuple(t.shape)}")
    return _here(fn, dev, name, t)


_ws_need = {}   # (rows, E, n, k) -> bytes: a host-side size, asked for once per shape


def grouped_ws_bytes(g: GroupCfg) -> int:
    """Bytes of the grouped products' workspace for this shape; zero it once before its first
    use."""
    n = ctypes.c_size_t(0)
    _check("moe_grouped_query", _lib.moe_grouped_query(ctypes.byref(g), ctypes.byref(n)))
    return n.value


def _need_ws(fn, dev, g, shape, ws):
    need = _ws_need.get(shape)
    if need is None:
        need = _ws_need[shape] = grouped_ws_bytes(g)
    if not isinstance(ws, torch.Tensor) or ws.nbytes < need:
        raise ValueError(f"{fn}: ws must be a CUDA tensor of grouped_ws_bytes(cfg) bytes")
    return _here(fn, dev, "ws", ws)


def grouped_mm(g: GroupCfg, x, counts, w, y, ws, stream=None):
    """y[r] = x[r] . w[e]^T for every row r of group e (counts rows each, in group order)."""
    fn, bf, dev = "moe_grouped_mm", torch.bfloat16, _device()
    rows, E, n, k = shape = g.rows, g.E, g.n, g.k
    _check(fn, _lib.moe_grouped_mm(ctypes.byref(g), _need(fn, dev, "x", x, bf, rows, k),
                                   _need(fn, dev, "counts", counts, torch.int32, E),
                                   _need(fn, dev, "w", w, bf, E, n, k),
                                   _need(fn, dev, "y", y, bf, rows, n),
                                   _need_ws(fn, dev, g, shape, ws), _stream(stream, dev)))


def grouped_mm_dx(g: GroupCfg, dy, counts, w, dx, ws, stream=None):
    """dx[r] = dy[r] . w[e]: the gradient of grouped_mm's rows."""
    fn, bf, dev = "moe_grouped_mm_dx", torch.bfloat16, _device()
    rows, E, n, k = shape = g.rows, g.E, g.n, g.k
    _check(fn, _lib.moe_grouped_mm_dx(ctypes.byref(g), _need(fn, dev, "dy", dy, bf, rows, n),
                                      _need(fn, dev, "counts", counts, torch.int32, E),
                                      _need(fn, dev, "w", w, bf, E, n, k),
                                      _need(fn, dev, "dx", dx, bf, rows, k),
                                      _need_ws(fn, dev, g, shape, ws), _stream(stream, dev)))


def grouped_mm_dw(g: GroupCfg, dy, x, counts, dw, ws, accumulate=False, stream=None):
    """dw[e] = sum of dy[r]^T x[r] over group e's rows (accumulate: added to dw, fp32 only): the
    gradient of grouped_mm's weights. dw bf16 or fp32."""
    fn, bf, dev = "moe_grouped_mm_dw", torch.bfloat16, _device()
    rows, E, n, k = shape = g.rows, g.E, g.n, g.k
    f32 = isinstance(dw, torch.Tensor) and dw.dtype is torch.float32
    _check(fn, _lib.moe_grouped_mm_dw(ctypes.byref(g), _need(fn, dev, "dy", dy, bf, rows, n),
                                      _need(fn, dev, "x", x, bf, rows, k),
                                      _need(fn, dev, "counts", counts, torch.int32, E),
                                      _need(fn, dev, "dw", dw, torch.float32 if f32 else bf,
                                            E, n, k),
                                      MOE_F32 if f32 else MOE_BF16, 1 if accumulate else 0,
                                      _need_ws(fn, dev, g, shape, ws), _stream(stream, dev)))


def _rows_cols(fn, name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{fn}: {name} must be a 2-D CUDA tensor")
    return t.shape


def act_save(x, q, scales, stream=None):
    """Keeps bf16 rows x [rows][d] as e4m3 codes q (bytes [rows][d]) and fp32 scales
    [d/128][rows]."""
    fn, dev = "moe_act_save", _device()
    rows, d = _rows_cols(fn, "x", x)
    _check(fn, _lib.moe_act_save(rows, d, _need(fn, dev, "x", x, torch.bfloat16, rows, d),
                                 _need(fn, dev, "q", q, torch.uint8, rows, d),
                                 _need(fn, dev, "scales", scales, torch.float32, d // 128, rows),
                                 _stream(stream, dev)))


def act_load(q, scales, index, out, stream=None, status=None):
    """out[i] = the saved row index[i] in bf16 (index None: row i; -1: zeros)."""
    fn, dev = "moe_act_load", _device()
    src, d = _rows_cols(fn, "q", q)
    rows = _rows_cols(fn, "out", out)[0]
    _check(fn, _lib.moe_act_load(rows, src, d, _need(fn, dev, "q", q, torch.uint8, src, d),
                                 _need(fn, dev, "scales", scales, torch.float32, d // 128, src),
                                 None if index is None else
                                 _need(fn, dev, "index", index, torch.int32, rows),
                                 _need(fn, dev, "out", out, torch.bfloat16, rows, d),
                                 _here(fn, dev, "status", status), _stream(stream, dev)))


def swiglu_save(gu, a, q, scales, stream=None):
    """a = silu(g) * u of gu = [g | u] [rows][2f], with gu kept as act_save keeps it."""
    fn, dev = "moe_swiglu_save", _device()
    rows, f2 = _rows_cols(fn, "gu", gu)
    f = f2 // 2
    _check(fn, _lib.moe_swiglu_save(rows, f, _need(fn, dev, "gu", gu, torch.bfloat16, rows, 2 * f),
                                    _need(fn, dev, "a", a, torch.bfloat16, rows, f),
                                    _need(fn, dev, "q", q, torch.uint8, rows, 2 * f),
                                    _need(fn, dev, "scales", scales, torch.float32, 2 * f // 128,
                                          rows),
                                    _stream(stream, dev)))


def swiglu_grad(q, scales, da, dgu, a=None, stream=None):
    """dgu [rows][2f], and a [rows][f] again (None: not wanted), from swiglu_save's codes."""
    fn, dev = "moe_swiglu_grad", _device()
    rows, f = _rows_cols(fn, "da", da)
    _check(fn, _lib.moe_swiglu_grad(rows, f, _need(fn, dev, "q", q, torch.uint8, rows, 2 * f),
                                    _need(fn, dev, "scales", scales, torch.float32, 2 * f // 128,
                                          rows),
                                    _need(fn, dev, "da", da, torch.bfloat16, rows, f),
                                    _need(fn, dev, "dgu", dgu, torch.bfloat16, rows, 2 * f),
                                    None if a is None else
                                    _need(fn, dev, "a", a, torch.bfloat16, rows, f),
                                    _stream(stream, dev)))


def combine_grad(ebuf, row_of, topk_w, dy, debuf, dtopk_w, stream=None, status=None):
    """The gradient of combine: debuf (rows of ebuf) and dtopk_w [T][k] from dy [T][d]."""
    fn, bf, dev = "moe_combine_grad", torch.bfloat16, _device()
    T, d = _rows_cols(fn, "dy", dy)
    k = _rows_cols(fn, "row_of", row_of)[1]
    rows = _rows_cols(fn, "ebuf", ebuf)[0]
    _check(fn, _lib.moe_combine_grad(T, k, d, rows, _need(fn, dev, "ebuf", ebuf, bf, rows, d),
                                     _need(fn, dev, "row_of", row_of, torch.int32, T, k),
                                     _need(fn, dev, "topk_w", topk_w, torch.float32, T, k),
                                     _need(fn, dev, "dy", dy, bf, T, d),
                                     _need(fn, dev, "debuf", debuf, bf, rows, d),
                                     _need(fn, dev, "dtopk_w", dtopk_w, torch.float32, T, k),
                                     _here(fn, dev, "status", status), _stream(stream, dev)))


# ---------------------------------------------------------------------------------------------
# The rest of a training step of an MoE block (see include/moe.h): the norms around the layer, the
# router's gradient and the optimiser. Sizes come from the tensors, checked as above.
# ---------------------------------------------------------------------------------------------
def _stream_type(fn, name, t):
    if not isinstance(t, torch.Tensor) or t.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"{fn}: {name} must be a bf16 or fp32 CUDA tensor")
    return t.dtype


_norm_cfgs = {}   # moe_norm_cfg's fields -> the struct by reference (calls only read it)


def _norm_cfg(*key):
    """rows, d, stream's type, eps, res_scale, out_scale, gate"""
    c = _norm_cfgs.get(key)
    if c is None:
        if len(_norm_cfgs) >= 4096:   # sizes that differ from call to call
            _norm_cfgs.clear()
        rows, d, st, eps, res, out, gate = key
        # (a tensor would be found again by its identity, whatever it holds by then)
        if not all(isinstance(v, numbers.Real) for v in (eps, res, out)):
            raise ValueError("moe_norm: eps, res_scale and out_scale must be numbers")
        c = _norm_cfgs[key] = ctypes.byref(NormCfg(
            rows, d, eps, res, out, MOE_F32 if st is torch.float32 else MOE_BF16, gate))
    return c


def _gate_of(fn, gate, rows, d):
    """The kind of a gate, from its type and shape, and that type and shape. fp32 [d] is a channel
    gate where rows == d: a token gate is then fp32 [rows][1]."""
    if gate is None:
        return MOE_GATE_NONE, None, ()
    if isinstance(gate, torch.Tensor):
        shape, f32 = tuple(gate.shape), gate.dtype is torch.float32
        if f32 and shape == (d,):
            return MOE_GATE_CHANNEL, torch.float32, shape
        if f32 and shape in ((rows,), (rows, 1)):
            return MOE_GATE_TOKEN, torch.float32, shape
        if gate.dtype is torch.bfloat16 and shape == (rows, d):
            return MOE_GATE_ELEMENT, torch.bfloat16, shape
    raise ValueError(f"{fn}: gate must be fp32 [d], fp32 [rows] or bf16 [rows][d]")


def _opt(fn, dev, name, t, dtype, *shape):
    if t is None:
        return None
    if (t.__class__ is torch.Tensor and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return t.data_ptr()
    return _need(fn, dev, name, t, dtype, *shape)


def norm_ws_bytes(rows, d) -> int:
    """Bytes of the norm gradients' scratch for rows of width d."""
    n = ctypes.c_size_t(0)
    _check("moe_norm_query", _lib.moe_norm_query(int(rows), int(d), ctypes.byref(n)))
    return n.value


_norm_need = {}   # (rows, d) -> bytes


def _norm_ws(fn, dev, rows, d, ws):
    need = _norm_need.get((rows, d))
    if need is None:
        need = _norm_need[rows, d] = norm_ws_bytes(rows, d)
    if not isinstance(ws, torch.Tensor) or ws.nbytes < need:
        raise ValueError(f"{fn}: ws must be a CUDA tensor of norm_ws_bytes(rows, d) bytes")
    return _here(fn, dev, "ws", ws)


def norm_in(x, w, n, rstd=None, eps=1e-6, stream=None):
    """n = bf16(x r w), r = 1/sqrt(mean x^2 + eps) of each row (kept in rstd if given). x bf16 or
    fp32 [rows][d], w fp32 [d], n bf16."""
    fn, dev, f32 = "moe_norm_in", _device(), torch.float32
    rows, d = _rows_cols(fn, "x", x)
    st = _stream_type(fn, "x", x)
    _check(fn, _lib.moe_norm_in(
        _norm_cfg(rows, d, st, eps, 1.0, 1.0, 0), _need(fn, dev, "x", x, st, rows, d),
        _need(fn, dev, "w", w, f32, d), _need(fn, dev, "n", n, torch.bfloat16, rows, d),
        _opt(fn, dev, "rstd", rstd, f32, rows), _stream(stream, dev)))


def norm_in_grad(dn, x, w, rstd, dres, dx, dw, ws, accumulate=False, stream=None):
    """dx = dres + the gradient of norm_in's rows (dres None: without it), dw (None: not wanted;
    accumulate: added to) that of its weight."""
    fn, dev, f32 = "moe_norm_in_grad", _device(), torch.float32
    rows, d = _rows_cols(fn, "x", x)
    st = _stream_type(fn, "x", x)
    _check(fn, _lib.moe_norm_in_grad(
        _norm_cfg(rows, d, st, 0.0, 1.0, 1.0, 0),
        _need(fn, dev, "dn", dn, torch.bfloat16, rows, d), _need(fn, dev, "x", x, st, rows, d),
        _need(fn, dev, "w", w, f32, d),
        _need(fn, dev, "rstd", rstd, f32, rows), _opt(fn, dev, "dres", dres, st, rows, d),
        _need(fn, dev, "dx", dx, st, rows, d), _opt(fn, dev, "dw", dw, f32, d),
        1 if accumulate else 0, _norm_ws(fn, dev, rows, d, ws), _stream(stream, dev)))


def norm_out(y, x, w_post, gate, w_next, h, n, rstd_y=None, rstd_h=None, eps=1e-6, res_scale=1.0,
             out_scale=1.0, stream=None):
    """h = res_scale x + out_scale gate s, s the norm of y with weight w_post (None: y itself), and
    n the norm of h with weight w_next (None: no n). gate: None, fp32 [d], fp32 [rows] or bf16
    [rows][d]. x, h bf16 or fp32 [rows][d]."""
    fn, dev, f32, bf = "moe_norm_out", _device(), torch.float32, torch.bfloat16
    rows, d = _rows_cols(fn, "y", y)
    st = _stream_type(fn, "x", x)
    kind, gt, gs = _gate_of(fn, gate, rows, d)
    _check(fn, _lib.moe_norm_out(
        _norm_cfg(rows, d, st, eps, res_scale, out_scale, kind),
        _need(fn, dev, "y", y, bf, rows, d), _need(fn, dev, "x", x, st, rows, d),
        _opt(fn, dev, "w_post", w_post, f32, d), _opt(fn, dev, "gate", gate, gt, *gs),
        _opt(fn, dev, "w_next", w_next, f32, d), _need(fn, dev, "h", h, st, rows, d),
        _opt(fn, dev, "n", n, bf, rows, d), _opt(fn, dev, "rstd_y", rstd_y, f32, rows),
        _opt(fn, dev, "rstd_h", rstd_h, f32, rows), _stream(stream, dev)))


def norm_out_grad(dh, dn, y, h, w_post, gate, w_next, rstd_y, rstd_h, dx, dy, dgate, dw_post,
                  dw_next, ws, res_scale=1.0, out_scale=1.0, accumulate=False, stream=None):
    """The gradient of norm_out from dh (None: none) and dn: dy, and dx, dgate, dw_post, dw_next
    (None: not wanted). y, h, rstd_y, rstd_h, dn: None where norm_out's form does not need them."""
    fn, dev, f32, bf = "moe_norm_out_grad", _device(), torch.float32, torch.bfloat16
    rows, d = _rows_cols(fn, "dy", dy)
    st = next((_stream_type(fn, name, t) for name, t in (("dh", dh), ("h", h), ("dx", dx))
               if t is not None), bf)
    kind, gt, gs = _gate_of(fn, gate, rows, d)
    _check(fn, _lib.moe_norm_out_grad(
        _norm_cfg(rows, d, st, 0.0, res_scale, out_scale, kind),
        _opt(fn, dev, "dh", dh, st, rows, d), _opt(fn, dev, "dn", dn, bf, rows, d),
        _opt(fn, dev, "y", y, bf, rows, d), _opt(fn, dev, "h", h, st, rows, d),
        _opt(fn, dev, "w_post", w_post, f32, d), _opt(fn, dev, "gate", gate, gt, *gs),
        _opt(fn, dev, "w_next", w_next, f32, d), _opt(fn, dev, "rstd_y", rstd_y, f32, rows),
        _opt(fn, dev, "rstd_h", rstd_h, f32, rows), _opt(fn, dev, "dx", dx, st, rows, d),
        _need(fn, dev, "dy", dy, bf, rows, d), _opt(fn, dev, "dgate", dgate, gt, *gs),
        _opt(fn, dev, "dw_post", dw_post, f32, d), _opt(fn, dev, "dw_next", dw_next, f32, d),
        1 if accumulate else 0, _norm_ws(fn, dev, rows, d, ws), _stream(stream, dev)))


def route_save(cfg, x, w_gate, bias, topk_idx, topk_w, topk_s, ws, stream=None):
    """route that also keeps the chosen experts' sigmoid scores topk_s [T][k] for route_grad."""
    fn, dev, c = "moe_route_save", _device(), make_cfg(cfg)
    f32 = torch.float32
    _check(fn, _lib.moe_route_save(
        ctypes.byref(c), _need(fn, dev, "x", x, torch.bfloat16, c.T, c.d),
        _need(fn, dev, "w_gate", w_gate, f32, c.E, c.d), _need(fn, dev, "bias", bias, f32, c.E),
        _need(fn, dev, "topk_idx", topk_idx, torch.int32, c.T, c.k),
        _need(fn, dev, "topk_w", topk_w, f32, c.T, c.k),
        _need(fn, dev, "topk_s", topk_s, f32, c.T, c.k), _here(fn, dev, "ws", ws),
        _stream(stream, dev)))


def route_grad_ws_bytes(cfg) -> int:
    """Bytes of route_grad's workspace; zero its first word once before its first use."""
    n = ctypes.c_size_t(0)
    c = cfg if isinstance(cfg, Cfg) else make_cfg(cfg)
    _check("moe_route_grad_query", _lib.moe_route_grad_query(ctypes.byref(c), ctypes.byref(n)))
    return n.value


_route_need = {}   # (T, E, k, d) -> bytes


def route_grad(cfg, x, w_gate, topk_idx, topk_s, dtopk_w, dx_in, dx, dw_gate, ws,
               accumulate=False, stream=None):
    """The router's gradient from that of its weights: dx = dx_in (None: 0) + the tokens' part,
    dw_gate fp32 [E][d] (accumulate: added to)."""
    fn, dev = "moe_route_grad", _device()
    c = cfg if isinstance(cfg, Cfg) else make_cfg(cfg)
    T, d, E, k = c.T, c.d, c.E, c.k
    f32, bf = torch.float32, torch.bfloat16
    need = _route_need.get((T, E, k, d))
    if need is None:
        need = _route_need[T, E, k, d] = route_grad_ws_bytes(c)
    if not isinstance(ws, torch.Tensor) or ws.nbytes < need:
        raise ValueError(f"{fn}: ws must be a CUDA tensor of route_grad_ws_bytes(cfg) bytes")
    _check(fn, _lib.moe_route_grad(
        ctypes.byref(c), _need(fn, dev, "x", x, bf, T, d),
        _need(fn, dev, "w_gate", w_gate, f32, E, d),
        _need(fn, dev, "topk_idx", topk_idx, torch.int32, T, k),
        _need(fn, dev, "topk_s", topk_s, f32, T, k), _need(fn, dev, "dtopk_w", dtopk_w, f32, T, k),
        _opt(fn, dev, "dx_in", dx_in, bf, T, d), _need(fn, dev, "dx", dx, bf, T, d),
        _need(fn, dev, "dw_gate", dw_gate, f32, E, d), 1 if accumulate else 0,
        _here(fn, dev, "ws", ws), _stream(stream, dev)))


class AdamTensors:
    """The tensors of an AdamW step, checked once and held: a list of dicts with p (fp32), g (fp32
    or bf16), w (bf16 copy of p, or None), m, v (fp32; 8 bits: bytes) and, with state_bits 8,
    m_scale and v_scale (fp32, one per 128 elements); optional weight_decay (0) and seed (the
    tensor's place in the list). All contiguous, on one device, and no two may overlap. The plan
    keeps these very arrays: another one put into a dict or under a tensor (``t.data = ...``) later
    is not seen."""

    def __init__(self, tensors, state_bits=32):
        fn, dev = "AdamTensors", _device()
        if state_bits not in (32, 8):
            raise ValueError(f"{fn}: state_bits must be 32 or 8")
        self.state_bits, self.device = state_bits, dev
        # (references of its own to the memory: the pointers stay valid)
        self.tensors = [{k: v.detach() if isinstance(v, torch.Tensor) else v for k, v in t.items()}
                        for t in tensors]
        f32, n = torch.float32, len(self.tensors)
        self.array = (AdamTensorC * n)()
        for i, (t, c) in enumerate(zip(self.tensors, self.array)):
            p, g = t["p"], t["g"]
            gt = _stream_type(fn, "g", g)
            if not isinstance(p, torch.Tensor):
                raise ValueError(f"{fn}: p must be a CUDA tensor")
            shape, c.n = tuple(p.shape), p.numel()
            held = state_bits == 8
            st = torch.uint8 if held else f32
            c.p = _need(fn, dev, "p", p, f32, *shape)
            c.g = _need(fn, dev, "g", g, gt, *shape)
            c.w = _opt(fn, dev, "w", t.get("w"), torch.bfloat16, *shape)
            c.m = _need(fn, dev, "m", t["m"], st, *shape)
            c.v = _need(fn, dev, "v", t["v"], st, *shape)
            if held:
                blocks = (c.n + 127) // 128
                c.m_scale = _need(fn, dev, "m_scale", t["m_scale"], f32, blocks)
                c.v_scale = _need(fn, dev, "v_scale", t["v_scale"], f32, blocks)
            c.weight_decay = float(t.get("weight_decay", 0.0))
            c.seed = int(t.get("seed", i)) & 0xFFFFFFFF
            c.g_dtype = MOE_F32 if gt is f32 else MOE_BF16
        # the calls a step is made of: (first tensor, tensors, whether another call follows)
        size = ctypes.sizeof(AdamTensorC)
        base = ctypes.addressof(self.array)
        self.parts = [(base + i * size, min(MOE_ADAM_TENSORS, n - i), i + MOE_ADAM_TENSORS < n)
                      for i in range(0, max(n, 1), MOE_ADAM_TENSORS)]
        if len(self.parts) > 1:   # (each call of a step checks its own arrays)
            spans = sorted((v.data_ptr(), v.data_ptr() + v.nbytes) for t in self.tensors
                           for v in t.values() if isinstance(v, torch.Tensor) and v.numel())
            if any(a[1] > b[0] for a, b in zip(spans, spans[1:])):
                raise ValueError(f"{fn}: two of the arrays overlap")


_adam_bytes = []


def _adam_state(fn, dev, state):
    if not _adam_bytes:
        n = ctypes.c_size_t(0)
        _check("moe_adam_query", _lib.moe_adam_query(ctypes.byref(n)))
        _adam_bytes.append(n.value)
    if not isinstance(state, torch.Tensor) or state.nbytes < _adam_bytes[0]:
        raise ValueError(f"{fn}: state must be a tensor of adam_state")
    return _here(fn, dev, "state", state)


def adam_state(step=0, beta1=0.9, beta2=0.999, device="cuda"):
    """The state of an optimiser that has made `step` steps with these betas."""
    n = ctypes.c_size_t(0)
    _check("moe_adam_query", _lib.moe_adam_query(ctypes.byref(n)))
    host = torch.zeros(n.value, dtype=torch.uint8)
    host[8:16].view(torch.int64)[0] = step
    host[16:32].view(torch.float64).copy_(
        torch.tensor([1.0 - beta1 ** step, 1.0 - beta2 ** step], dtype=torch.float64))
    return host.to(device)


def adam_step(state) -> int:
    """The number of steps that a state counts (synchronises)."""
    return int(state[8:16].cpu().view(torch.int64))


def _same_device(fn, plan):
    dev = _device()
    if plan.device != dev:
        raise ValueError(f"{fn}: the tensors must be on the current device, cuda:{dev}")
    return dev


def grad_norm(plan: AdamTensors, state, norm, stream=None):
    """norm (fp32, one element) = the root of the sum of all gradients' squares."""
    fn = "moe_grad_norm"
    dev = _same_device(fn, plan)
    if not isinstance(norm, torch.Tensor) or norm.dtype is not torch.float32 or norm.numel() != 1:
        raise ValueError(f"{fn}: norm must be an fp32 CUDA tensor of one element")
    st, out, s = _adam_state(fn, dev, state), _here(fn, dev, "norm", norm), _stream(stream, dev)
    for at, n, more in plan.parts:
        _check(fn, _lib.moe_grad_norm(at, n, more, st, out, s))


def adamw(cfg: AdamCfg, plan: AdamTensors, state, norm=None, stream=None, lr=None):
    """One AdamW step over the plan's tensors. norm: grad_norm's result (needed where the cfg clips;
    a norm that is not finite leaves the step out). lr: None, or an fp32 CUDA tensor of one element
    that is read in place of cfg.lr."""
    fn = "moe_adamw"
    dev = _same_device(fn, plan)
    for name, t in (("norm", norm), ("lr", lr)):
        if t is not None and (not isinstance(t, torch.Tensor) or t.dtype is not torch.float32
                              or t.numel() != 1):
            raise ValueError(f"{fn}: {name} must be an fp32 CUDA tensor of one element")
    cfg = AdamCfg.from_buffer_copy(cfg)   # (the caller's may be another call's, too)
    cfg.state_bits = plan.state_bits
    cfg.lr_dev = None if lr is None else _here(fn, dev, "lr", lr)
    st, s = _adam_state(fn, dev, state), _stream(stream, dev)
    nm = None if norm is None else _here(fn, dev, "norm", norm)
    for at, n, more in plan.parts:
        _check(fn, _lib.moe_adamw(ctypes.byref(cfg), at, n, more, st, nm, s))


def clear_status(ws, stream=None):
    _check("moe_clear_status", _lib.moe_clear_status(_p(ws), _s(stream)))


def read_status(ws, stream=None) -> int:
    st = ctypes.c_uint32(0)
    _check("moe_read_status", _lib.moe_read_status(_p(ws), ctypes.byref(st), _s(stream)))
    return st.value


def selftest_wait(ws, limit_ns, stream=None):
    """Launches the library's wait diagnostic (see moe_selftest_wait): a kernel whose bounded
    waits run out after about limit_ns and set MOE_DEV_TIMEOUT in ws's status word."""
    _check("moe_selftest_wait", _lib.moe_selftest_wait(_p(ws), int(limit_ns), _s(stream)))


def abi_version() -> int:
    return _lib.moe_abi_version()


class Buffers(dict):
    """Device buffers of one layer configuration, allocated once with torch (the library itself
    allocates nothing)."""

    def __init__(self, cfg, device="cuda", with_recv=True, slots_per_rank=0):
        super().__init__()
        s = query_sizes_placed(cfg, slots_per_rank) if slots_per_rank else query_sizes(cfg)
        T, k, d, R, E = cfg.T, cfg.k, cfg.d, cfg.R, cfg.E
        if slots_per_rank:
            E = R * slots_per_rank     # counts are over the slots
        self.sizes = s
        fp8 = make_cfg(cfg).act_dtype != MOE_BF16
        self["topk_idx"] = torch.empty((T, k), dtype=torch.int32, device=device)
        self["topk_w"] = torch.empty((T, k), dtype=torch.float32, device=device)
        self["recv"] = (torch.empty((s["recv_rows"], d),
                                    dtype=torch.uint8 if fp8 else torch.bfloat16, device=device)
                        if with_recv else None)
        self["recv_scales"] = (torch.empty((d // 128, s["recv_rows"]), dtype=torch.float32,
                                           device=device) if fp8 and with_recv else None)
        self["counts"] = torch.empty((R, E), dtype=torch.int32, device=device)
        self["row_of"] = torch.empty((T, k), dtype=torch.int32, device=device)
        self["ebuf"] = torch.empty((s["recv_rows"], d), dtype=torch.bfloat16, device=device)
        self["shared_out"] = (torch.empty((T, d), dtype=torch.bfloat16, device=device)
                              if cfg.d_ff_shared else None)
        self["ws"] = torch.zeros(s["ws_bytes"], dtype=torch.uint8, device=device)


class MoELayer:
    """One MoE layer with resident weights: ``y = layer(x)`` runs router, dispatch, expert
    FFNs and combine on the current stream through ``moe_layer`` (``moe_layer_ex`` when a
    variant is asked for).

    gather: the expert GEMMs read routed rows from x by token (no receive-buffer copy; the
    receive buffers are not allocated). side_stream: the shared expert runs on a second stream
    of its own, limited to side_ctas CTAs per GEMM. placement: redundant experts on slots
    (Placement); the dispatch splits each expert's rows over its copies. fused: both expert
    GEMMs and the combine in one persistent launch (bf16)."""

    def __init__(self, cfg, w_gate, bias, weights: dict, device="cuda", gather=False,
                 side_stream=False, side_ctas=0, placement: Placement | None = None,
                 fused=False):
        self.cfg = cfg
        self.w_gate = w_gate
        self.bias = bias
        self.weights = weights
        self.placement = placement
        self.bufs = Buffers(cfg, device, with_recv=not gather,
                            slots_per_rank=placement.slots_per_rank if placement else 0)
        self.opts = None
        if gather or side_stream or fused or placement is not None:
            self.opts = LayerOpts(flags=(MOE_OPT_GATHER_X if gather else 0)
                                  | (MOE_OPT_SHARED_SIDE_STREAM if side_stream else 0)
                                  | (MOE_OPT_FUSED_FFN if fused else 0),
                                  side_ctas=int(side_ctas))
            if placement is not None:
                self.opts.placement = ctypes.pointer(placement.c)
            if side_stream:
                # the stream and events live as long as the layer object
                self._side = torch.cuda.Stream(device=device)
                self._fork = torch.cuda.Event()
                self._join = torch.cuda.Event()
                cur = torch.cuda.current_stream(device)
                self._fork.record(cur)      # gives the events their handles
                self._join.record(cur)
                torch.cuda.synchronize(device)
                self.opts.side_stream = self._side.cuda_stream
                self.opts.fork_event = self._fork.cuda_event
                self.opts.join_event = self._join.cuda_event

    def _run(self, x, y, stream, events):
        if self.opts is None:
            layer(self.cfg, x, self.w_gate, self.bias, self.weights, self.bufs, y, stream, events)
        else:
            layer_ex(self.cfg, self.opts, x, self.w_gate, self.bias, self.weights, self.bufs, y,
                     stream, events)

    def __call__(self, x, y=None, stream=None, events=None):
        if y is None:
            y = _output((self.cfg.T, self.cfg.d), torch.bfloat16, x.device, stream)
        self._run(x, y, stream, events)
        return y

    def run_host(self, x_host, y_host, stream=None):
        """Host-to-host call: copies x_host (pinned bf16 [T][d]) to the device, runs the layer
        and copies the output back into y_host (pinned), all enqueued on the stream. The caller
        synchronises before reading y_host."""
        s = stream or torch.cuda.current_stream()
        with torch.cuda.stream(s):
            if not hasattr(self, "_x_dev"):
                self._x_dev = torch.empty((self.cfg.T, self.cfg.d), dtype=torch.bfloat16,
                                          device=self.w_gate.device)
                self._y_dev = torch.empty_like(self._x_dev)
            self._x_dev.copy_(x_host, non_blocking=True)
            self._run(self._x_dev, self._y_dev, s, None)
            y_host.copy_(self._y_dev, non_blocking=True)
        return y_host


class MoEBlock:
    """A block of the residual stream around a MoELayer, for serving:

        h = res_scale x + out_scale gate norm(layer(norm(x) w_in)) w_out

    ``h = block(x)``; with w_next (the weight of the next block's first norm) ``h, n = block(x, n)``:
    n is what the next block's layer takes, normed in the pass that ends this block, and n given is
    that of the block before (None: normed here). w_in, w_out (None: no norm behind the layer),
    w_next: fp32 [d]; gate: None, fp32 [d], fp32 [T][1] or bf16 [T][d]; x bf16 or fp32 [T][d]."""

    def __init__(self, layer: MoELayer, w_in, w_out=None, gate=None, w_next=None, eps=1e-6,
                 res_scale=1.0, out_scale=1.0):
        self.layer, self.w_in, self.w_out = layer, w_in, w_out
        self.gate, self.w_next, self.eps = gate, w_next, eps
        self.scales = dict(res_scale=res_scale, out_scale=out_scale)
        shape, dev = (layer.cfg.T, layer.cfg.d), layer.w_gate.device
        # the layer's input and output, and the n that the last call returned
        self.rows = [torch.empty(shape, dtype=torch.bfloat16, device=dev)
                     for _ in range(2 if w_next is None else 3)]
        self._last = None

    def __call__(self, x, n=None, h=None, stream=None):
        """h may be x itself. The n that is returned is a buffer of the block's own: the block's next
        call leaves it as it is, whatever n that is given, and the one after it may write over it."""
        free = [t for t in self.rows if t is not self._last]
        if n is None:
            n = free.pop()
            norm_in(x, self.w_in, n, eps=self.eps, stream=stream)
        if h is None:
            h = _output(x.shape, x.dtype, x.device, stream)
        # (not n's place, where n is the block's own of an earlier call: layers that share weights)
        y = next(t for t in free if t.data_ptr() != n.data_ptr())
        self.layer(n, y, stream)
        if self.w_next is None:
            norm_out(y, x, self.w_out, self.gate, None, h, None, eps=self.eps, stream=stream,
                     **self.scales)
            return h
        # the layer's output has been read where the next norm's takes its place
        norm_out(y, x, self.w_out, self.gate, self.w_next, h, y, eps=self.eps, stream=stream,
                 **self.scales)
        self._last = y
        return h, y
