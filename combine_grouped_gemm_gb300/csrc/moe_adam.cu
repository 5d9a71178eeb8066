// AdamW over a list of tensors in one launch, moments in 32 or 8 bits, and the norm of all their
// gradients. Both stream their arrays from HBM once: 30 bytes a parameter with fp32 gradients, fp32
// moments and a bf16 copy, 18.1 with 8-bit moments; the norm reads the gradients alone.
//
// The tensors are cut into chunks, which the CTAs of one grid take in turn; the table of the tensors
// travels as a kernel argument, so the step needs no device table and a captured one keeps its own.
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 4096;                // elements; a multiple of 128
constexpr int kMostCtas = 152 * 8;
constexpr int kBlock = 128;                 // elements that share a scale

// The head of the state, then the partial sums of the norm.
struct State {
  uint32_t status, ticket;
  long long step;
  double c1, c2;    // 1 - b^t
  double sum;       // of the squares, between the calls of one norm
  double partial[kMostCtas];
};

template <int CAP>
struct Table {
  moe_adam_tensor t[CAP];
  uint32_t first[CAP + 1];   // chunks before each tensor
  int n;
};

template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& tab, uint32_t chunk) {
  int lo = 0, hi = tab.n - 1;   // the last tensor whose first chunk is at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (tab.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Four values of a gradient from element i on (cnt of them exist; the others are 0).
__device__ __forceinline__ float4 load_grad(const void* g, bool f32, long long i, int cnt) {
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (f32) {
    const float* p = static_cast<const float*>(g) + i;
    if (cnt == 4) return __ldcs(reinterpret_cast<const float4*>(p));
    if (cnt > 0) v.x = p[0];
    if (cnt > 1) v.y = p[1];
    if (cnt > 2) v.z = p[2];
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(g) + i;
    if (cnt == 4) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
      return make_float4(bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y));
    }
    if (cnt > 0) v.x = __bfloat162float(p[0]);
    if (cnt > 1) v.y = __bfloat162float(p[1]);
    if (cnt > 2) v.z = __bfloat162float(p[2]);
  }
  return v;
}
__device__ __forceinline__ float4 load4(const float* p, int cnt) {
  if (cnt == 4) return __ldcs(reinterpret_cast<const float4*>(p));
  return make_float4(cnt > 0 ? p[0] : 0.0f, cnt > 1 ? p[1] : 0.0f, cnt > 2 ? p[2] : 0.0f, 0.0f);
}
__device__ __forceinline__ void store4(float* p, const float2 (&v)[2], int cnt) {
  if (cnt == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
    return;
  }
  if (cnt > 0) p[0] = v[0].x;
  if (cnt > 1) p[1] = v[0].y;
  if (cnt > 2) p[2] = v[1].x;
}
__device__ __forceinline__ void store4_bf16(void* w, long long i, const float2 (&v)[2], int cnt) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(w) + i;
  if (cnt == 4) {
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y)));
    return;
  }
  if (cnt > 0) p[0] = __float2bfloat16_rn(v[0].x);
  if (cnt > 1) p[1] = __float2bfloat16_rn(v[0].y);
  if (cnt > 2) p[2] = __float2bfloat16_rn(v[1].x);
}
__device__ __forceinline__ uint32_t load_codes(const void* q, long long i, int cnt) {
  const uint8_t* p = static_cast<const uint8_t*>(q) + i;
  if (cnt == 4) return __ldcs(reinterpret_cast<const uint32_t*>(p));
  uint32_t v = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) v |= static_cast<uint32_t>(p[j]) << (8 * j);
  return v;
}
__device__ __forceinline__ void store_codes(void* q, long long i, uint32_t v, int cnt) {
  uint8_t* p = static_cast<uint8_t*>(q) + i;
  if (cnt == 4) {
    __stcs(reinterpret_cast<uint32_t*>(p), v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) p[j] = static_cast<uint8_t>(v >> (8 * j));
}

// The last CTA of the grid to come here gets true (all threads). The ticket is left at 0.
__device__ __forceinline__ bool last_cta(uint32_t* ticket) {
  __shared__ bool last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    if (last) {
      *ticket = 0;
      __threadfence();
    }
  }
  __syncthreads();
  return last;
}

// ------------------------------------------------------------------------------------------
// Norm of the gradients: each thread adds its squares in fp32 four at a time, those sums in fp64
// (the result is then rounded once in effect); the CTAs' sums are joined in order by the last one.
// ------------------------------------------------------------------------------------------
template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table<CAP> tab,
                                                             uint32_t chunks, State* state,
                                                             float* norm, bool more) {
  double acc = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(tab, c);
    const moe_adam_tensor& e = tab.t[t];
    const long long base = (long long)(c - tab.first[t]) * kChunk;
    const bool f32 = e.g_dtype == MOE_F32;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk / (4 * kThreads); ++i) {
      const long long at = base + (i * kThreads + (int)threadIdx.x) * 4;
      const long long left = e.n - at;
      const float4 g = load_grad(e.g, f32, at, left >= 4 ? 4 : left > 0 ? (int)left : 0);
      s += __fmaf_rn(g.x, g.x, g.y * g.y) + __fmaf_rn(g.z, g.z, g.w * g.w);
    }
    acc += static_cast<double>(s);
  }
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    state->partial[blockIdx.x] = s;
  }
  if (!last_cta(&state->ticket)) return;
  acc = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kThreads) acc += __ldcg(&state->partial[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x != 0) return;
  double s = state->sum;
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  state->sum = more ? s : 0.0;
  if (!more) *norm = static_cast<float>(sqrt(s));
}

// ------------------------------------------------------------------------------------------
// The step
// ------------------------------------------------------------------------------------------
struct Hyper {
  double lr, beta1, beta2, max_norm;
  float eps;
  const float* lr_dev;
};
// What a CTA works with, from the state.
struct Scalars {
  float b1, n1, b2, n2;   // beta, 1 - beta
  float factor;           // of the gradients
  float move;             // lr / (1 - b1^t)
  float root;             // 1 / sqrt(1 - b2^t)
  float lr, eps;
  uint32_t step;
  bool skip, clip;
};

// "lowbias32" (C. Wellons, 2018)
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  x *= 0x846ca68bu;
  return x ^ (x >> 16);
}
constexpr uint32_t kGolden = 0x9e3779b9u;

__device__ __forceinline__ Scalars scalars(const Hyper& h, const State* state, const float* norm) {
  __shared__ Scalars sc;
  if (threadIdx.x == 0) {
    const double c1 = h.beta1 * state->c1 + (1.0 - h.beta1);
    const double c2 = h.beta2 * state->c2 + (1.0 - h.beta2);
    const double lr = h.lr_dev ? static_cast<double>(*h.lr_dev) : h.lr;
    sc.b1 = static_cast<float>(h.beta1);
    sc.n1 = static_cast<float>(1.0 - h.beta1);
    sc.b2 = static_cast<float>(h.beta2);
    sc.n2 = static_cast<float>(1.0 - h.beta2);
    sc.move = static_cast<float>(lr / c1);
    sc.root = static_cast<float>(1.0 / sqrt(c2));
    sc.lr = static_cast<float>(lr);
    sc.eps = h.eps;
    sc.step = static_cast<uint32_t>(state->step + 1);
    const float total = norm ? *norm : 0.0f;
    sc.skip = !(fabsf(total) < INFINITY);
    sc.factor = h.max_norm > 0.0
                    ? fminf(__fmul_rn(static_cast<float>(h.max_norm), __frcp_rn(total)), 1.0f)
                    : 1.0f;
    sc.clip = sc.factor < 1.0f;
  }
  __syncthreads();
  return sc;
}

// Two fp32 operations in one instruction. (The assembler joins a mul2 and an add2 of its result into
// one operation of one rounding, .rn or not: sums of products that have to be rounded twice are
// written one by one, which it leaves as they are.)
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(float2 v) { return make_float2(-v.x, -v.y); }

// A pair of elements: the new moments and the parameters. Each product and sum of the moments is
// rounded by itself, so that 8-bit moments can be checked code by code; the parameter's quotient
// takes the hardware's reciprocal (1 ulp).
__device__ __forceinline__ float recip(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void update(const Scalars& sc, float decay, float2 g, float2& p, float2& m,
                                       float2& v, float2& root) {
  if (sc.clip) g = mul2(g, both(sc.factor));
  const auto mean = [](float b, float old, float n, float now) {
    return __fadd_rn(__fmul_rn(b, old), __fmul_rn(n, now));
  };
  const float2 gg = mul2(g, g);
  m = make_float2(mean(sc.b1, m.x, sc.n1, g.x), mean(sc.b1, m.y, sc.n1, g.y));
  v = make_float2(mean(sc.b2, v.x, sc.n2, gg.x), mean(sc.b2, v.y, sc.n2, gg.y));
  root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 den = fma2(root, both(sc.root), both(sc.eps));
  const float2 quot = mul2(m, make_float2(recip(den.x), recip(den.y)));
  p = fma2(both(-decay), p, p);
  p = fma2(both(-sc.move), quot, p);
}

// The largest of a warp's non-negative numbers (their order is that of their bits).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// |x| / scale, the IEEE quotients, at most 448. By the correctly rounded reciprocal and one
// correction step (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) where nothing of it can leave the fp32 range, by division otherwise.
__device__ __forceinline__ float2 quotients(float2 x, float scale, float r, bool plain) {
  float2 a = make_float2(fabsf(x.x), fabsf(x.y)), q;
  if (plain) {
    const float2 q0 = mul2(a, both(r));
    q = fma2(fma2(q0, both(scale), minus(a)), both(-r), q0);
  } else {
    q = make_float2(__fdiv_rn(a.x, scale), __fdiv_rn(a.y, scale));
  }
  return make_float2(q.x > 448.0f ? 448.0f : q.x, q.y > 448.0f ? 448.0f : q.y);
}

// A pair of quotients rounded up or down to e4m3 by 16 random bits each (the upper half of r). With
// the random bits added below the code's last bit, cutting off what is below it rounds up with odds
// of the distance from the lower code. Below 2^-6 the steps are 2^-9: with 2^-6 added they lie at the
// same bits.
__device__ __forceinline__ float2 shift_of(float2 q) {
  return make_float2(q.x < 0x1p-6f ? 0x1p-6f : 0.0f, q.y < 0x1p-6f ? 0x1p-6f : 0.0f);
}
__device__ __forceinline__ float cut(float v, uint32_t more = 0) {
  return __uint_as_float((__float_as_uint(v) + more) & 0xfff00000u);
}
__device__ __forceinline__ float2 round_e4m3(float2 q, uint32_t r0, uint32_t r1) {
  const float2 shift = shift_of(q), y = add2(q, shift);
  return add2(make_float2(cut(y.x, (r0 >> 12) & 0xffff0u), cut(y.y, (r1 >> 12) & 0xffff0u)),
              minus(shift));
}
// The same for the root of a second moment (by the lower half of r), with odds that keep the mean of
// its square, (q^2 - lo^2) / (hi^2 - lo^2): odds linear in q would add the rounding's variance to v
// each step, several percent of v in the long run.
__device__ __forceinline__ float2 round_root_e4m3(float2 q, uint32_t r0, uint32_t r1) {
  const float2 shift = shift_of(q), y = add2(q, shift);
  const float2 cx = make_float2(cut(y.x), cut(y.y));
  const float2 cy = make_float2(__uint_as_float(__float_as_uint(cx.x) + 0x100000u),
                                __uint_as_float(__float_as_uint(cx.y) + 0x100000u));
  const float2 lo = add2(cx, minus(shift)), hi = add2(cy, minus(shift));   // exact, and so are
  const float2 odds = mul2(add2(q, minus(lo)), add2(q, lo));
  const float2 whole = mul2(add2(hi, minus(lo)), add2(hi, lo));            // hi - lo and hi + lo
  // r / 2^16 as the fraction of a number between 1 and 2
  const float2 r = add2(make_float2(__uint_as_float(0x3f800000u | ((r0 << 7) & 0x7fff80u)),
                                    __uint_as_float(0x3f800000u | ((r1 << 7) & 0x7fff80u))),
                        both(-1.0f));
  const float2 at = mul2(r, whole);
  return make_float2(at.x < odds.x ? hi.x : lo.x, at.y < odds.y ? hi.y : lo.y);
}
__device__ __forceinline__ uint32_t pack_codes(float2 a, float2 b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
}
__device__ __forceinline__ float2 codes2(uint32_t c, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3);
  return mul2(__half22float2(__half2(h)), both(s));
}
__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
}
__device__ __forceinline__ bool plain_scale(float s) { return s > 0x1p-60f && s < 0x1p100f; }

// What a lane has loaded of its four elements of a block.
template <int BITS>
struct Loaded {
  float4 g, p, m, v;
  uint32_t qm, qv;
  float sm, sv;
};
template <int BITS>
__device__ __forceinline__ Loaded<BITS> load_block(const moe_adam_tensor& e, bool f32,
                                                   long long block, int lane, int cnt) {
  const long long at = block * kBlock + lane * 4;
  Loaded<BITS> l;
  l.g = load_grad(e.g, f32, at, cnt);
  l.p = load4(e.p + at, cnt);
  if (BITS == 32) {
    l.m = load4(static_cast<const float*>(e.m) + at, cnt);
    l.v = load4(static_cast<const float*>(e.v) + at, cnt);
  } else {
    l.qm = load_codes(e.m, at, cnt);
    l.qv = load_codes(e.v, at, cnt);
    l.sm = __ldcs(e.m_scale + block);
    l.sv = __ldcs(e.v_scale + block);
  }
  return l;
}
template <int BITS>
__device__ __forceinline__ void step_block(const Scalars& sc, const moe_adam_tensor& e, float decay,
                                           uint32_t key, long long block, int lane, int cnt,
                                           const Loaded<BITS>& l) {
  const long long at = block * kBlock + lane * 4;
  float2 p[2] = {make_float2(l.p.x, l.p.y), make_float2(l.p.z, l.p.w)}, m[2], v[2], root[2];
  if (BITS == 32) {
    m[0] = make_float2(l.m.x, l.m.y), m[1] = make_float2(l.m.z, l.m.w);
    v[0] = make_float2(l.v.x, l.v.y), v[1] = make_float2(l.v.z, l.v.w);
  } else {
    m[0] = codes2(l.qm, l.sm), m[1] = codes2(l.qm >> 16, l.sm);
    v[0] = codes2(l.qv, l.sv), v[1] = codes2(l.qv >> 16, l.sv);
    v[0] = mul2(v[0], v[0]), v[1] = mul2(v[1], v[1]);
  }
  update(sc, decay, make_float2(l.g.x, l.g.y), p[0], m[0], v[0], root[0]);
  update(sc, decay, make_float2(l.g.z, l.g.w), p[1], m[1], v[1], root[1]);
  store4(e.p + at, p, cnt);
  if (e.w) store4_bf16(e.w, at, p, cnt);
  if (BITS == 32) {
    store4(static_cast<float*>(e.m) + at, m, cnt);
    store4(static_cast<float*>(e.v) + at, v, cnt);
    return;
  }
  // (fmaxf leaves a NaN out)
  const float am = warp_max(fmaxf(fmaxf(fabsf(m[0].x), fabsf(m[0].y)),
                                  fmaxf(fabsf(m[1].x), fabsf(m[1].y))));
  const float av = warp_max(fmaxf(fmaxf(root[0].x, root[0].y), fmaxf(root[1].x, root[1].y)));
  const float sm = block_scale(am), sv = block_scale(av);
  const float rm = __frcp_rn(sm), rv = __frcp_rn(sv);
  const bool pm = plain_scale(sm), pv = plain_scale(sv);
  const uint32_t from = mix(key ^ static_cast<uint32_t>(block)) + lane * 4 * kGolden;
  float2 cm[2], cv[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t r0 = mix(from + 2 * j * kGolden), r1 = mix(from + (2 * j + 1) * kGolden);
    const float2 q = round_e4m3(quotients(m[j], sm, rm, pm), r0, r1);
    cm[j] = make_float2(copysignf(q.x, m[j].x), copysignf(q.y, m[j].y));
    const float2 u = round_root_e4m3(quotients(root[j], sv, rv, pv), r0, r1);
    // a second moment above 0 stays above 0 (its place in the quotient m / sqrt(v) must not)
    cv[j] = make_float2(root[j].x > 0.0f && u.x < 0x1p-9f ? 0x1p-9f : u.x,
                        root[j].y > 0.0f && u.y < 0x1p-9f ? 0x1p-9f : u.y);
  }
  store_codes(e.m, at, pack_codes(cm[0], cm[1]), cnt);
  store_codes(e.v, at, pack_codes(cv[0], cv[1]), cnt);
  if (lane == 0) {
    e.m_scale[block] = sm;
    e.v_scale[block] = sv;
  }
}

template <int CAP, int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Table<CAP> tab,
                                                         const Hyper hyper, uint32_t chunks,
                                                         State* state, const float* norm,
                                                         bool more) {
  const Scalars sc = scalars(hyper, state, norm);
  if (sc.skip) {   // the same in every CTA: nothing is written, the step does not count
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(&state->status, MOE_DEV_NONFINITE);
    return;
  }
  constexpr int kWarps = kThreads / 32, kSteps = kChunk / (4 * kThreads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(tab, c);
    const moe_adam_tensor& e = tab.t[t];
    const long long chunk = c - tab.first[t];
    const bool f32 = e.g_dtype == MOE_F32;
    const float decay = sc.lr * e.weight_decay;
    const uint32_t key = BITS == 8 ? mix(e.seed ^ (sc.step * kGolden)) : 0;
    // a warp's four elements a lane are one block of 128
    const long long first = chunk * (kChunk / kBlock) + warp;
    if ((chunk + 1) * kChunk <= e.n) {
      Loaded<BITS> next = load_block<BITS>(e, f32, first, lane, 4);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const Loaded<BITS> now = next;
        if (i + 1 < kSteps) next = load_block<BITS>(e, f32, first + (i + 1) * kWarps, lane, 4);
        step_block<BITS>(sc, e, decay, key, first + i * kWarps, lane, 4, now);
      }
      continue;
    }
    for (int i = 0; i < kSteps; ++i) {
      const long long block = first + i * kWarps, left = e.n - block * kBlock - lane * 4;
      if (e.n <= block * kBlock) break;   // whole warps
      const int cnt = left >= 4 ? 4 : left > 0 ? (int)left : 0;
      step_block<BITS>(sc, e, decay, key, block, lane, cnt,
                       load_block<BITS>(e, f32, block, lane, cnt));
    }
  }
  if (more || !last_cta(&state->ticket) || threadIdx.x != 0) return;
  // every CTA has read the state before it took its ticket
  state->step += 1;
  state->c1 = hyper.beta1 * state->c1 + (1.0 - hyper.beta1);
  state->c2 = hyper.beta2 * state->c2 + (1.0 - hyper.beta2);
}

template <int CAP>
uint32_t fill(Table<CAP>& tab, const moe_adam_tensor* t, int n) {
  uint32_t chunks = 0;
  tab.n = n;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.first[i] = chunks;
    chunks += static_cast<uint32_t>((t[i].n + kChunk - 1) / kChunk);
  }
  tab.first[n] = chunks;
  return chunks;
}
unsigned grid_of(uint32_t chunks) {
  return chunks < 1 ? 1 : chunks > (uint32_t)kMostCtas ? kMostCtas : chunks;
}

template <int CAP>
cudaError_t norm_cap(const moe_adam_tensor* t, int n, bool more, State* state, float* norm,
                     cudaStream_t st) {
  Table<CAP> tab;
  const uint32_t chunks = fill(tab, t, n);
  return launch_kernel(grad_norm_kernel<CAP>, dim3(grid_of(chunks)), dim3(kThreads), 0, st, false,
                       tab, chunks, state, norm, more);
}
template <int CAP>
cudaError_t adam_cap(const moe_adam_cfg& c, const moe_adam_tensor* t, int n, bool more, State* state,
                     const float* norm, cudaStream_t st) {
  Table<CAP> tab;
  const uint32_t chunks = fill(tab, t, n);
  const Hyper h{c.lr, c.beta1, c.beta2, c.max_norm, static_cast<float>(c.eps), c.lr_dev};
  auto kern = c.state_bits == 8 ? adamw_kernel<CAP, 8> : adamw_kernel<CAP, 32>;
  return launch_kernel(kern, dim3(grid_of(chunks)), dim3(kThreads), 0, st, false, tab, h, chunks,
                       state, norm, more);
}

// a short table for the few tensors of one layer, so that the launch carries less
constexpr int kFew = 16;

}  // namespace

size_t adam_state_bytes() { return sizeof(State); }

cudaError_t launch_grad_norm(const moe_adam_tensor* t, int n, bool more, void* state, float* norm,
                             cudaStream_t st) {
  State* s = static_cast<State*>(state);
  return n <= kFew ? norm_cap<kFew>(t, n, more, s, norm, st)
                   : norm_cap<MOE_ADAM_TENSORS>(t, n, more, s, norm, st);
}

cudaError_t launch_adamw(const moe_adam_cfg& c, const moe_adam_tensor* t, int n, bool more,
                         void* state, const float* norm, cudaStream_t st) {
  State* s = static_cast<State*>(state);
  return n <= kFew ? adam_cap<kFew>(c, t, n, more, s, norm, st)
                   : adam_cap<MOE_ADAM_TENSORS>(c, t, n, more, s, norm, st);
}

}  // namespace moe
