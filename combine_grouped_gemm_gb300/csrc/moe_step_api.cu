// C ABI of the calls around the layer in a training step (declared in include/moe.h): the norms,
// the router's gradient and the optimiser. Argument checks only; nothing here allocates or waits.
#include <math.h>

#include <algorithm>

#include "moe_check.h"

using namespace moe;

namespace {

int check_norm_size(int32_t rows, int32_t d) {
  if (rows < 0 || d < 1) return MOE_ERR_INVALID_ARG;
  if (d % 8 || d > 16384 || (long long)rows * d >= 1ll << 37) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_norm(const moe_norm_cfg* c, bool out) {
  if (!c) return MOE_ERR_INVALID_ARG;
  const int rc = check_norm_size(c->rows, c->d);
  if (rc != MOE_OK) return rc;
  if (!isfinite(c->eps) || c->eps < 0.0f) return MOE_ERR_INVALID_ARG;
  if (c->stream_dtype != MOE_BF16 && c->stream_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  if (!out) return MOE_OK;
  if (!isfinite(c->res_scale) || !isfinite(c->out_scale)) return MOE_ERR_INVALID_ARG;
  return c->gate < MOE_GATE_NONE || c->gate > MOE_GATE_ELEMENT ? MOE_ERR_INVALID_ARG : MOE_OK;
}

// The same configuration for the norm before a block, which has no output, gate or scales.
moe_norm_cfg norm_in_cfg(const moe_norm_cfg& c) {
  moe_norm_cfg n = c;
  n.res_scale = n.out_scale = 1.0f;
  n.gate = MOE_GATE_NONE;
  return n;
}

// Whether two arrays are the same one: an output in an input's place.
bool same(const Span& a, const Span& b) { return a.p && a.p == b.p && a.n == b.n; }

// An output against all arrays of a call but itself (by its address in the list) and the one whose
// place it may take.
template <size_t N>
bool clashes(const Span (&all)[N], size_t out, size_t instead = N) {
  for (size_t i = 0; i < N; ++i) {
    if (i == out || (i == instead && same(all[out], all[i]))) continue;
    if (meets(all[out], {all[i]})) return true;
  }
  return false;
}

}  // namespace

extern "C" {

int moe_norm_query(int32_t rows, int32_t d, size_t* ws_bytes) {
  const int rc = check_norm_size(rows, d);
  if (rc != MOE_OK) return rc;
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  *ws_bytes = norm_ws_bytes(rows, d);
  return MOE_OK;
}

int moe_norm_in(const moe_norm_cfg* cfg, const void* x, const float* w, void* n, float* rstd,
                cudaStream_t stream) {
  const int rc = check_norm(cfg, false);
  if (rc != MOE_OK || cfg->rows == 0) return rc;
  MOE_NEED(x);
  MOE_NEED(w);
  MOE_NEED(n);
  MOE_OPT(rstd);
  const size_t el = (size_t)cfg->rows * cfg->d, sz = cfg->stream_dtype == MOE_F32 ? 4 : 2;
  const Span all[] = {{x, sz * el}, {w, 4 * (size_t)cfg->d}, {n, 2 * el},
                      {rstd, 4 * (size_t)cfg->rows}};
  if (clashes(all, 2, 0) || clashes(all, 3)) return MOE_ERR_INVALID_ARG;
  NormFwd a{};
  a.x = x;
  a.w_next = w;
  a.n = n;
  a.rstd_h = rstd;
  const cudaError_t e = launch_norm(norm_in_cfg(*cfg), a, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

int moe_norm_in_grad(const moe_norm_cfg* cfg, const void* dn, const void* x, const float* w,
                     const float* rstd, const void* dres, void* dx, float* dw, int32_t accumulate,
                     void* ws, cudaStream_t stream) {
  const int rc = check_norm(cfg, false);
  if (rc != MOE_OK) return rc;
  if (cfg->rows > 0) {
    MOE_NEED(dn);
    MOE_NEED(x);
    MOE_NEED(rstd);
    MOE_NEED(dx);
  }
  MOE_NEED(w);
  MOE_OPT(dres);
  MOE_OPT(dw);
  MOE_NEED(ws);
  const size_t el = (size_t)cfg->rows * cfg->d, sz = cfg->stream_dtype == MOE_F32 ? 4 : 2;
  const size_t wb = 4 * (size_t)cfg->d;
  const Span all[] = {{dn, 2 * el}, {x, sz * el}, {w, wb}, {rstd, 4 * (size_t)cfg->rows},
                      {dres, sz * el}, {dx, sz * el}, {dw, wb},
                      {ws, norm_ws_bytes(cfg->rows, cfg->d)}};
  if (clashes(all, 5, 4) || clashes(all, 6) || clashes(all, 7)) return MOE_ERR_INVALID_ARG;
  NormGrad a{};
  a.dh = dres;
  a.dn = dn;
  a.h = x;
  a.w_next = w;
  a.rstd_h = rstd;
  a.dx = dx;
  a.dw_next = dw;
  const cudaError_t e = launch_norm_grad(norm_in_cfg(*cfg), a, accumulate != 0, ws, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

namespace {
size_t gate_bytes(const moe_norm_cfg& c) {
  switch (c.gate) {
    case MOE_GATE_CHANNEL: return 4 * (size_t)c.d;
    case MOE_GATE_TOKEN: return 4 * (size_t)c.rows;
    case MOE_GATE_ELEMENT: return 2 * (size_t)c.rows * c.d;
    default: return 0;
  }
}
}  // namespace

int moe_norm_out(const moe_norm_cfg* cfg, const void* y, const void* x, const float* w_post,
                 const void* gate, const float* w_next, void* h, void* n, float* rstd_y,
                 float* rstd_h, cudaStream_t stream) {
  const int rc = check_norm(cfg, true);
  if (rc != MOE_OK) return rc;
  // a gate with its kind, a next norm with its output
  if (!gate != (cfg->gate == MOE_GATE_NONE) || !w_next != !n) {
    if (cfg->rows > 0) return MOE_ERR_INVALID_ARG;
  }
  if ((!w_post && rstd_y) || (!w_next && rstd_h)) return MOE_ERR_INVALID_ARG;
  if (cfg->rows == 0) return MOE_OK;
  MOE_NEED(y);
  MOE_NEED(x);
  MOE_OPT(w_post);
  MOE_OPT(gate);
  MOE_OPT(w_next);
  MOE_NEED(h);
  MOE_OPT(n);
  MOE_OPT(rstd_y);
  MOE_OPT(rstd_h);
  const size_t el = (size_t)cfg->rows * cfg->d, sz = cfg->stream_dtype == MOE_F32 ? 4 : 2;
  const size_t wb = 4 * (size_t)cfg->d, rb = 4 * (size_t)cfg->rows;
  const Span all[] = {{y, 2 * el}, {x, sz * el}, {w_post, wb}, {gate, gate_bytes(*cfg)},
                      {w_next, wb}, {h, sz * el}, {n, 2 * el}, {rstd_y, rb}, {rstd_h, rb}};
  if (clashes(all, 5, 1) || clashes(all, 6, 0) || clashes(all, 7) || clashes(all, 8))
    return MOE_ERR_INVALID_ARG;
  const NormFwd a{y, x, w_post, w_next, gate, h, n, rstd_y, rstd_h};
  const cudaError_t e = launch_norm(*cfg, a, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

int moe_norm_out_grad(const moe_norm_cfg* cfg, const void* dh, const void* dn, const void* y,
                      const void* h, const float* w_post, const void* gate, const float* w_next,
                      const float* rstd_y, const float* rstd_h, void* dx, void* dy, void* dgate,
                      float* dw_post, float* dw_next, int32_t accumulate, void* ws,
                      cudaStream_t stream) {
  const int rc = check_norm(cfg, true);
  if (rc != MOE_OK) return rc;
  const bool some = cfg->rows > 0, gated = cfg->gate != MOE_GATE_NONE;
  if (gated != (gate != nullptr) && (some || gate)) return MOE_ERR_INVALID_ARG;
  if ((dgate && !gated) || (dw_post && !w_post) || (dw_next && !w_next)) return MOE_ERR_INVALID_ARG;
  if (some) {
    if (!dh && !w_next) return MOE_ERR_INVALID_ARG;
    if (w_next) {
      MOE_NEED(dn);
      MOE_NEED(h);
      MOE_NEED(rstd_h);
    }
    if (w_post) MOE_NEED(rstd_y);
    if (w_post || gated) MOE_NEED(y);
    MOE_NEED(dy);
  }
  MOE_OPT(dh);
  MOE_OPT(w_post);
  MOE_OPT(gate);
  MOE_OPT(w_next);
  MOE_OPT(dx);
  MOE_OPT(dgate);
  MOE_OPT(dw_post);
  MOE_OPT(dw_next);
  MOE_NEED(ws);
  const size_t el = (size_t)cfg->rows * cfg->d, sz = cfg->stream_dtype == MOE_F32 ? 4 : 2;
  const size_t wb = 4 * (size_t)cfg->d, rb = 4 * (size_t)cfg->rows, gb = gate_bytes(*cfg);
  const bool has_y = w_post || gated;
  const Span all[] = {{dh, sz * el}, {w_next ? dn : nullptr, 2 * el}, {has_y ? y : nullptr, 2 * el},
                      {w_next ? h : nullptr, sz * el}, {w_post, wb}, {gate, gb}, {w_next, wb},
                      {w_post ? rstd_y : nullptr, rb}, {w_next ? rstd_h : nullptr, rb},
                      {dx, sz * el}, {dy, 2 * el}, {dgate, gb}, {dw_post, wb}, {dw_next, wb},
                      {ws, norm_ws_bytes(cfg->rows, cfg->d)}};
  if (clashes(all, 9, 0) || clashes(all, 10, 1)) return MOE_ERR_INVALID_ARG;
  for (size_t i = 11; i < 15; ++i)
    if (clashes(all, i)) return MOE_ERR_INVALID_ARG;
  const NormGrad a{dh, dn, y, h, w_post, w_next, gate, rstd_y, rstd_h, dx, dy, dgate, dw_post,
                   dw_next};
  const cudaError_t e = launch_norm_grad(*cfg, a, accumulate != 0, ws, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

// ------------------------------------------------------------------------------------------
// The router's gradient
// ------------------------------------------------------------------------------------------
namespace {
int check_route_grad(const moe_cfg* cfg) {
  MOE_CHECK_CFG(cfg);
  if (cfg->d > 65536 || (long long)cfg->T * cfg->d >= 1ll << 37) return MOE_ERR_UNSUPPORTED;
  // (the kernels' 32-bit places in the lists run up to a segment past the last choice)
  if ((long long)cfg->T * cfg->k > (1ll << 31) - 2048) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
}  // namespace

int moe_route_grad_query(const moe_cfg* cfg, size_t* ws_bytes) {
  const int rc = check_route_grad(cfg);
  if (rc != MOE_OK) return rc;
  if (!ws_bytes) return MOE_ERR_INVALID_ARG;
  *ws_bytes = route_grad_ws_bytes(*cfg);
  return MOE_OK;
}

int moe_route_grad(const moe_cfg* cfg, const void* x, const float* w_gate, const int32_t* topk_idx,
                   const float* topk_s, const float* dtopk_w, const void* dx_in, void* dx,
                   float* dw_gate, int32_t accumulate, void* ws, cudaStream_t stream) {
  const int rc = check_route_grad(cfg);
  if (rc != MOE_OK) return rc;
  MOE_NEED(x);
  MOE_NEED(w_gate);
  MOE_NEED(topk_idx);
  MOE_NEED(topk_s);
  MOE_NEED(dtopk_w);
  MOE_OPT(dx_in);
  MOE_NEED(dx);
  MOE_NEED(dw_gate);
  MOE_NEED(ws);
  const size_t xb = 2 * (size_t)cfg->T * cfg->d, wb = 4 * (size_t)cfg->E * cfg->d;
  const size_t tk = 4 * (size_t)cfg->T * cfg->k;
  const Span all[] = {{x, xb}, {w_gate, wb}, {topk_idx, tk}, {topk_s, tk}, {dtopk_w, tk},
                      {dx_in, xb}, {dx, xb}, {dw_gate, wb}, {ws, route_grad_ws_bytes(*cfg)}};
  if (clashes(all, 6, 5) || clashes(all, 7) || clashes(all, 8)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_route_grad(*cfg, x, w_gate, topk_idx, topk_s, dtopk_w, dx_in, dx,
                                          dw_gate, accumulate != 0, ws, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

// ------------------------------------------------------------------------------------------
// The optimiser
// ------------------------------------------------------------------------------------------
namespace {

constexpr size_t kMostSpans = MOE_ADAM_TENSORS * 7 + 3;

// Whether any two of the arrays overlap. (Sorted by address, an overlap shows between neighbours or
// with an array that reaches past its successor.)
bool any_overlap(Span* s, size_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) {
    return reinterpret_cast<uintptr_t>(a.p) < reinterpret_cast<uintptr_t>(b.p);
  });
  uintptr_t end = 0;
  for (size_t i = 0; i < n; ++i) {
    const auto b = reinterpret_cast<uintptr_t>(s[i].p);
    if (i > 0 && b < end) return true;
    end = b + s[i].n;
  }
  return false;
}

int check_tensors(const moe_adam_tensor* t, int32_t n, bool step, int bits, Span* spans,
                  size_t* used) {
  if (n < 0 || (n > 0 && !t)) return MOE_ERR_INVALID_ARG;
  if (n > MOE_ADAM_TENSORS) return MOE_ERR_UNSUPPORTED;
  long long chunks = 0;
  const auto add = [&](const void* p, size_t bytes) { spans[(*used)++] = Span{p, bytes}; };
  for (int i = 0; i < n; ++i) {
    const moe_adam_tensor& e = t[i];
    if (e.n < 0 || e.reserved != 0) return MOE_ERR_INVALID_ARG;
    if (e.g_dtype != MOE_F32 && e.g_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (step && (!isfinite(e.weight_decay) || e.weight_decay < 0.0f)) return MOE_ERR_INVALID_ARG;
    if (step && bits == 32 && (e.m_scale || e.v_scale)) return MOE_ERR_INVALID_ARG;
    if (e.n >= 1ll << 39) return MOE_ERR_UNSUPPORTED;
    chunks += (e.n + 4095) / 4096;
    if (e.n == 0) continue;
    MOE_NEED(e.g);
    const size_t el = static_cast<size_t>(e.n);
    add(e.g, el * (e.g_dtype == MOE_F32 ? 4 : 2));
    if (!step) continue;
    MOE_NEED(e.p);
    MOE_OPT(e.w);
    MOE_NEED(e.m);
    MOE_NEED(e.v);
    add(e.p, 4 * el);
    if (e.w) add(e.w, 2 * el);
    add(e.m, bits == 8 ? el : 4 * el);
    add(e.v, bits == 8 ? el : 4 * el);
    if (bits == 8) {
      MOE_NEED(e.m_scale);
      MOE_NEED(e.v_scale);
      add(e.m_scale, (el + 127) / 128 * 4);
      add(e.v_scale, (el + 127) / 128 * 4);
    }
  }
  return chunks > INT32_MAX ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

bool rate(double v) { return isfinite(v) && v >= 0.0; }

}  // namespace

int moe_adam_query(size_t* state_bytes) {
  if (!state_bytes) return MOE_ERR_INVALID_ARG;
  *state_bytes = adam_state_bytes();
  return MOE_OK;
}

int moe_grad_norm(const moe_adam_tensor* tensors, int32_t n, int32_t more, void* state, float* norm,
                  cudaStream_t stream) {
  Span spans[kMostSpans];
  size_t used = 0;
  const int rc = check_tensors(tensors, n, false, 32, spans, &used);
  if (rc != MOE_OK) return rc;
  MOE_NEED(state);
  if (!norm) return MOE_ERR_INVALID_ARG;
  if (misaligned4(norm)) return MOE_ERR_MISALIGNED;
  const Span st{state, adam_state_bytes()}, out{norm, 4};
  if (meets(out, {st})) return MOE_ERR_INVALID_ARG;
  for (size_t i = 0; i < used; ++i)   // (gradients may overlap one another: they are read only)
    if (meets(st, {spans[i]}) || meets(out, {spans[i]})) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_grad_norm(tensors, n, more != 0, state, norm, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

int moe_adamw(const moe_adam_cfg* cfg, const moe_adam_tensor* tensors, int32_t n, int32_t more,
              void* state, const float* norm, cudaStream_t stream) {
  if (!cfg || cfg->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (!rate(cfg->lr) || !rate(cfg->beta1) || cfg->beta1 >= 1.0 || !rate(cfg->beta2) ||
      cfg->beta2 >= 1.0 || !rate(cfg->max_norm))
    return MOE_ERR_INVALID_ARG;
  if (!isfinite(cfg->eps) || !(static_cast<float>(cfg->eps) >= 1.17549435e-38f))
    return MOE_ERR_INVALID_ARG;
  if (cfg->state_bits != 32 && cfg->state_bits != 8) return MOE_ERR_INVALID_ARG;
  Span spans[kMostSpans];
  size_t used = 0;
  const int rc = check_tensors(tensors, n, true, cfg->state_bits, spans, &used);
  if (rc != MOE_OK) return rc;
  MOE_NEED(state);
  if (cfg->max_norm > 0.0 && !norm) return MOE_ERR_INVALID_ARG;
  if ((norm && misaligned4(norm)) || (cfg->lr_dev && misaligned4(cfg->lr_dev)))
    return MOE_ERR_MISALIGNED;
  spans[used++] = Span{state, adam_state_bytes()};
  if (norm) spans[used++] = Span{norm, 4};
  if (cfg->lr_dev && cfg->lr_dev != norm) spans[used++] = Span{cfg->lr_dev, 4};
  if (any_overlap(spans, used)) return MOE_ERR_INVALID_ARG;
  const cudaError_t e = launch_adamw(*cfg, tensors, n, more != 0, state, norm, stream);
  return e == cudaSuccess ? MOE_OK : cuda_fail(e);
}

}  // extern "C"
