// AdamW over a list of tensors in one launch, moments in 32 or 8 bits, and the norm of all their
// gradients. Both stream their arrays from HBM once: 30 bytes a parameter with fp32 gradients, fp32
// moments and a bf16 copy, 18.1 with 8-bit moments; the norm reads the gradients alone.
//
// The tensors are cut into chunks, which the CTAs of one grid take in turn; the table of the tensors
// travels as a kernel argument, so the step needs no device table and a captured one keeps its own.
#include "moe_device.cuh"
#include "moe_f32x2.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kStep = 4 * kThreads;         // elements that a CTA takes at once; a multiple of 128
constexpr int kSteps = 4;
constexpr int kChunk = kSteps * kStep;
constexpr int kGpuSms = 152;                // grids are sized for GB300
constexpr int kMostCtas = kGpuSms * 8;
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
__device__ __forceinline__ uint32_t load_codes(const char* q, int cnt) {
  if (cnt == 4) return __ldcs(reinterpret_cast<const uint32_t*>(q));
  uint32_t v = 0;
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) v |= static_cast<uint32_t>(static_cast<uint8_t>(q[j])) << (8 * j);
  return v;
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
__device__ __forceinline__ void store4_bf16(__nv_bfloat16* p, const float2 (&v)[2], int cnt) {
  if (cnt == 4) {
    __stcs(reinterpret_cast<uint2*>(p),
           make_uint2(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y)));
    return;
  }
  if (cnt > 0) p[0] = __float2bfloat16_rn(v[0].x);
  if (cnt > 1) p[1] = __float2bfloat16_rn(v[0].y);
  if (cnt > 2) p[2] = __float2bfloat16_rn(v[1].x);
}
__device__ __forceinline__ void store_codes(char* q, uint32_t v, int cnt) {
  if (cnt == 4) {
    __stcs(reinterpret_cast<uint32_t*>(q), v);
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) q[j] = static_cast<char>(v >> (8 * j));
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
// Norm of the gradients: each thread adds 16 squares in fp32, those sums in fp64
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
    const long long base = (long long)(c - tab.first[t]) * kChunk + threadIdx.x * 4;
    const bool f32 = e.g_dtype == MOE_F32;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const long long at = base + i * kStep, left = e.n - at;
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

// "lowbias32" (C. Wellons, 2018), and the same without its last step
__device__ __forceinline__ uint32_t premix(uint32_t x) {
  x ^= x >> 16;
  x *= 0x7feb352du;
  x ^= x >> 15;
  return x * 0x846ca68bu;
}
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = premix(x);
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

// A pair of elements: the new moments and the parameters. Each product and sum of the moments is
// rounded by itself, so that 8-bit moments can be checked code by code. (They are written one by one:
// the assembler joins a mul2 and an add2 of its result into one operation of one rounding, .rn or
// not.) The parameter's quotient takes the hardware's reciprocal (1 ulp).
__device__ __forceinline__ float recip(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void update(const Scalars& sc, float decay, f32x2 g2, f32x2& p, float2& m,
                                       float2& v, float2& root) {
  if (sc.clip) g2 = mul2(g2, both(sc.factor));
  const auto mean = [](float b, float old, float n, float now) {
    return __fadd_rn(__fmul_rn(b, old), __fmul_rn(n, now));
  };
  const float2 g = halves(g2), gg = halves(mul2(g2, g2));
  m = make_float2(mean(sc.b1, m.x, sc.n1, g.x), mean(sc.b1, m.y, sc.n1, g.y));
  v = make_float2(mean(sc.b2, v.x, sc.n2, gg.x), mean(sc.b2, v.y, sc.n2, gg.y));
  root = make_float2(__fsqrt_rn(v.x), __fsqrt_rn(v.y));
  const float2 den = halves(fma2(pair(root.x, root.y), both(sc.root), both(sc.eps)));
  const f32x2 quot = mul2(pair(m.x, m.y), pair(recip(den.x), recip(den.y)));
  p = fma2(both(-decay), p, p);
  p = fma2(both(-sc.move), quot, p);
}

// The largest of a warp's non-negative numbers (their order is that of their bits).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// |x| / scale, the IEEE quotients (up to 448 and a rounding). By the correctly rounded reciprocal and
// one correction step (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990) where nothing of it can leave the fp32 range, by division otherwise.
__device__ __forceinline__ f32x2 quotients(float2 x, float scale, f32x2 r, bool plain) {
  const f32x2 a = pair(fabsf(x.x), fabsf(x.y));
  if (plain) {
    const f32x2 q0 = mul2(a, r);
    return fma2(fma2(q0, both(scale), minus(a)), minus(r), q0);
  }
  return pair(__fdiv_rn(fabsf(x.x), scale), __fdiv_rn(fabsf(x.y), scale));
}

// The steps below choose by saturation (0 or 1 on the FMA pipe) rather than by comparison and select
// (two operations of the ALU pipe, which has half its rate and the integer work beside it).
__device__ __forceinline__ float is_positive(float v, float big) {   // v * big >= 1 where v > 0
  float r;
  asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(big));
  return r;
}

// A pair of quotients rounded up or down to e4m3 by 16 random bits each. With the random bits added
// below the code's last bit, cutting off what is below it rounds up with odds of the distance from the
// lower code. Below 2^-6 the steps are 2^-9: with 2^-6 added they lie at the same bits. (What is past
// 448 by a rounding is cut or, as a code, saturated.)
__device__ __forceinline__ f32x2 shift_of(f32x2 q) {   // 2^-6 where q < 2^-6, else 0
  const float2 f = halves(fma2(q, both(-0x1p40f), both(0x1p34f)));
  return mul2(pair(__saturatef(f.x), __saturatef(f.y)), both(0x1p-6f));
}
__device__ __forceinline__ float cut(uint32_t bits) { return __uint_as_float(bits & 0xfff00000u); }
__device__ __forceinline__ f32x2 round_e4m3(f32x2 q, uint32_t r0, uint32_t r1) {
  const f32x2 shift = shift_of(q);
  const float2 y = halves(add2(q, shift));
  return add2(pair(cut(__float_as_uint(y.x) + r0 * 16), cut(__float_as_uint(y.y) + r1 * 16)),
              minus(shift));
}
// The same for the root of a second moment, with odds that keep the mean of its square, (q^2 - lo^2)
// / (hi^2 - lo^2): odds linear in q would add the rounding's variance to v each step, several percent
// of v in the long run. A root above 0 keeps a code above 0.
__device__ __forceinline__ f32x2 round_root_e4m3(f32x2 q, float2 root, uint32_t r0, uint32_t r1) {
  const f32x2 back = minus(shift_of(q));
  const float2 y = halves(add2(q, minus(back)));
  const float cx = cut(__float_as_uint(y.x)), cy = cut(__float_as_uint(y.y));
  const f32x2 lo = add2(pair(cx, cy), back);   // exact, and so are hi, hi - lo and hi + lo
  const f32x2 hi = add2(pair(__uint_as_float(__float_as_uint(cx) + 0x100000u),
                             __uint_as_float(__float_as_uint(cy) + 0x100000u)),
                        back);
  const f32x2 gap = add2(hi, minus(lo));
  const f32x2 odds = mul2(add2(q, minus(lo)), add2(q, lo)), whole = mul2(gap, add2(hi, lo));
  // r / 2^16 as the fraction of a number between 1 and 2
  const f32x2 r = add2(pair(__uint_as_float(0x3f800000u + r0 * 128),
                            __uint_as_float(0x3f800000u + r1 * 128)),
                       both(-1.0f));
  // up where r whole, rounded, < odds. (A difference that is no multiple of 2^-100 leaves a value
  // below the lowest code, which the next line makes that code.)
  const float2 rr = halves(r), w = halves(whole), o = halves(odds);
  const float2 ahead = make_float2(__fadd_rn(o.x, -__fmul_rn(rr.x, w.x)),
                                   __fadd_rn(o.y, -__fmul_rn(rr.y, w.y)));
  const float2 u = halves(fma2(pair(is_positive(ahead.x, 0x1p100f), is_positive(ahead.y, 0x1p100f)),
                               gap, lo));
  const float2 least = halves(mul2(pair(is_positive(root.x, 0x1p100f), is_positive(root.y, 0x1p100f)),
                                   both(0x1p-9f)));
  float2 v;   // (a NaN stays one)
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.x) : "f"(u.x), "f"(least.x));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(v.y) : "f"(u.y), "f"(least.y));
  return pair(v.x, v.y);
}
__device__ __forceinline__ uint32_t pack_codes(float2 a, float2 b) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3)) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
}
__device__ __forceinline__ f32x2 codes2(uint32_t c, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(c & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return mul2(pair(f.x, f.y), both(s));
}
__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
}
// (the reciprocal, its correction and the quotient stay inside the fp32 range)
__device__ __forceinline__ bool plain_scale(float s) { return s > 0x1p-60f && s < 0x1p100f; }

// The last call of a step: the last CTA to end counts it. (Every CTA has read the state before it
// took its ticket.)
__device__ __forceinline__ void finish(const Hyper& h, State* state, bool more) {
  if (more || !last_cta(&state->ticket) || threadIdx.x != 0) return;
  state->step += 1;
  state->c1 = h.beta1 * state->c1 + (1.0 - h.beta1);
  state->c2 = h.beta2 * state->c2 + (1.0 - h.beta2);
}

// A lane's four elements of a block, and the step on them. The pointers are the lane's own; cnt of
// the elements exist.
struct Pointers {
  const char* g;
  char *p, *w, *m, *v;
  float *ms, *vs;   // of the warp's block
};
template <int BITS>
__device__ __forceinline__ Pointers pointers(const moe_adam_tensor& e, long long block) {
  const long long at = block * kBlock + (threadIdx.x & 31) * 4;
  constexpr int kMoment = BITS == 8 ? 1 : 4;
  Pointers r;
  r.g = static_cast<const char*>(e.g) + at * (e.g_dtype == MOE_F32 ? 4 : 2);
  r.p = reinterpret_cast<char*>(e.p) + at * 4;
  r.w = e.w ? static_cast<char*>(e.w) + at * 2 : nullptr;
  r.m = static_cast<char*>(e.m) + at * kMoment;
  r.v = static_cast<char*>(e.v) + at * kMoment;
  r.ms = BITS == 8 ? e.m_scale + block : nullptr;
  r.vs = BITS == 8 ? e.v_scale + block : nullptr;
  return r;
}
struct Four {
  f32x2 g[2], p[2];
  float2 m[2], v[2];
};

__device__ __forceinline__ void from_codes(Four& f, uint32_t qm, uint32_t qv, float sm, float sv) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    f.m[j] = halves(codes2(qm >> (16 * j), sm));
    const f32x2 u = codes2(qv >> (16 * j), sv);
    f.v[j] = halves(mul2(u, u));
  }
}

template <int BITS>
__device__ __forceinline__ void step_four(const Scalars& sc, float decay, uint32_t key, long long block,
                                          const Pointers& to, int i, int cnt, Four& f) {
  float2 root[2];
  update(sc, decay, f.g[0], f.p[0], f.m[0], f.v[0], root[0]);
  update(sc, decay, f.g[1], f.p[1], f.m[1], f.v[1], root[1]);
  const float2 p[2] = {halves(f.p[0]), halves(f.p[1])};
  // i: steps of the CTA past the pointers
  store4(reinterpret_cast<float*>(to.p) + i * kStep, p, cnt);
  if (to.w) store4_bf16(reinterpret_cast<__nv_bfloat16*>(to.w) + i * kStep, p, cnt);
  if (BITS == 32) {
    store4(reinterpret_cast<float*>(to.m) + i * kStep, f.m, cnt);
    store4(reinterpret_cast<float*>(to.v) + i * kStep, f.v, cnt);
    return;
  }
  const int lane = threadIdx.x & 31;
  // (fmaxf leaves a NaN out)
  const float am = warp_max(fmaxf(fmaxf(fabsf(f.m[0].x), fabsf(f.m[0].y)),
                                  fmaxf(fabsf(f.m[1].x), fabsf(f.m[1].y))));
  const float av = warp_max(fmaxf(fmaxf(root[0].x, root[0].y), fmaxf(root[1].x, root[1].y)));
  const float sm = block_scale(am), sv = block_scale(av);
  const f32x2 rm = both(__frcp_rn(sm)), rv = both(__frcp_rn(sv));
  const bool plain = plain_scale(sm) && plain_scale(sv);
  const uint32_t from = mix(key ^ static_cast<uint32_t>(block)) + lane * 4 * kGolden;
  float2 cm[2], cv[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    // the halves of the hash x ^ (x >> 16)
    const uint32_t x0 = premix(from + 2 * j * kGolden), x1 = premix(from + (2 * j + 1) * kGolden);
    const uint32_t h0 = x0 >> 16, h1 = x1 >> 16;
    const float2 q = halves(round_e4m3(quotients(f.m[j], sm, rm, plain), h0, h1));
    cm[j] = make_float2(copysignf(q.x, f.m[j].x), copysignf(q.y, f.m[j].y));
    cv[j] = halves(round_root_e4m3(quotients(root[j], sv, rv, plain), root[j], (x0 ^ h0) & 0xffffu,
                                   (x1 ^ h1) & 0xffffu));
  }
  store_codes(to.m + i * kStep, pack_codes(cm[0], cm[1]), cnt);
  store_codes(to.v + i * kStep, pack_codes(cv[0], cv[1]), cnt);
  if (lane == 0) {
    to.ms[i * (kStep / kBlock)] = sm;
    to.vs[i * (kStep / kBlock)] = sv;
  }
}

// Loads straight from memory: a step ahead with 32-bit moments, and where a tensor ends.
template <int BITS>
__device__ __forceinline__ Four load_four(const Pointers& from, bool g_f32, int i, int cnt) {
  Four f;
  const float4 g = load_grad(from.g, g_f32, (long long)i * kStep, cnt);
  const float4 p = load4(reinterpret_cast<const float*>(from.p) + i * kStep, cnt);
  f.g[0] = pair(g.x, g.y), f.g[1] = pair(g.z, g.w);
  f.p[0] = pair(p.x, p.y), f.p[1] = pair(p.z, p.w);
  if (BITS == 32) {
    const float4 m = load4(reinterpret_cast<const float*>(from.m) + i * kStep, cnt);
    const float4 v = load4(reinterpret_cast<const float*>(from.v) + i * kStep, cnt);
    f.m[0] = make_float2(m.x, m.y), f.m[1] = make_float2(m.z, m.w);
    f.v[0] = make_float2(v.x, v.y), f.v[1] = make_float2(v.z, v.w);
  } else {
    from_codes(f, load_codes(from.m + i * kStep, cnt), load_codes(from.v + i * kStep, cnt),
               from.ms[i * (kStep / kBlock)], from.vs[i * (kStep / kBlock)]);
  }
  return f;
}

// The elements past a tensor's last whole chunk, tensor by tensor a CTA.
template <int CAP, int BITS>
__device__ __forceinline__ void tails(const Table<CAP>& tab, const Scalars& sc) {
  const int lane = threadIdx.x & 31;
  // (the first whole chunks go to the first CTAs: the tails to the last ones)
  for (int t = gridDim.x - 1 - blockIdx.x; t < tab.n; t += gridDim.x) {
    const moe_adam_tensor& e = tab.t[t];
    const uint32_t key = BITS == 8 ? mix(e.seed ^ (sc.step * kGolden)) : 0;
    for (long long block = e.n / kChunk * (kChunk / kBlock) + (threadIdx.x >> 5);
         block * kBlock < e.n; block += kThreads / 32) {   // whole warps
      const long long left = e.n - block * kBlock - lane * 4;
      const int cnt = left >= 4 ? 4 : left > 0 ? (int)left : 0;
      const Pointers at = pointers<BITS>(e, block);
      Four f = load_four<BITS>(at, e.g_dtype == MOE_F32, 0, cnt);
      step_four<BITS>(sc, sc.lr * e.weight_decay, key, block, at, 0, cnt, f);
    }
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Table<CAP> tab,
                                                            const Hyper hyper, uint32_t chunks,
                                                            State* state, const float* norm,
                                                            bool more) {
  const Scalars sc = scalars(hyper, state, norm);
  if (sc.skip) {   // the same in every CTA: nothing is written, the step does not count
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(&state->status, MOE_DEV_NONFINITE);
    return;
  }
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(tab, c);
    const moe_adam_tensor& e = tab.t[t];
    const long long first =
        (long long)(c - tab.first[t]) * (kChunk / kBlock) + (threadIdx.x >> 5);
    const Pointers at = pointers<32>(e, first);
    const bool f32 = e.g_dtype == MOE_F32;
    const float decay = sc.lr * e.weight_decay;
    Four next = load_four<32>(at, f32, 0, 4);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      Four now = next;
      if (i + 1 < kSteps) next = load_four<32>(at, f32, i + 1, 4);
      step_four<32>(sc, decay, 0, first, at, i, 4, now);
    }
  }
  tails<CAP, 32>(tab, sc);
  finish(hyper, state, more);
}

// 8-bit moments: the arithmetic of the rounding bounds it, not memory. Each thread's elements come
// through stages of its own in shared memory, a chunk ahead, and a CTA takes neighbouring chunks, so
// that addresses are constants past a chunk's pointers. 398 M parameters, bf16 gradients: 1.59 ms
// (4.0 TB/s); with loads to registers a step ahead 1.93 ms, waiting for memory half of the time; with
// the ring but its addresses computed for each step 1.88 ms, 145 instructions an element.
struct Stage8 {
  float4 g[kThreads];    // bf16 gradients: 8 bytes used
  float4 p[kThreads];
  uint32_t m[kThreads], v[kThreads];
};
template <int BYTES>
__device__ __forceinline__ void copy_in(void* to, const void* from) {
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_addr(to)), "l"(from),
                 "n"(BYTES)
                 : "memory");
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, 4) adamw8_kernel(const __grid_constant__ Table<CAP> tab,
                                                             const Hyper hyper, uint32_t chunks,
                                                             State* state, const float* norm,
                                                             bool more) {
  extern __shared__ __align__(16) char raw[];
  Stage8* ring = reinterpret_cast<Stage8*>(raw);
  const Scalars sc = scalars(hyper, state, norm);
  if (sc.skip) {
    if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(&state->status, MOE_DEV_NONFINITE);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31;
  constexpr int kBlocks = kChunk / kBlock, kWarps = kThreads / 32;
  uint32_t c = (uint32_t)((unsigned long long)chunks * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((unsigned long long)chunks * (blockIdx.x + 1) / gridDim.x);
  // the chunk that is copied, one before the one that is worked on
  int t_in = 0;
  Pointers in;
  float scale_in = 0.0f;   // lanes 0-3: of m, steps 0-3; lanes 4-7: of v
  bool f32_in = true;
  const auto enter = [&](uint32_t chunk) {
    if (chunk >= end) return;
    t_in = tensor_of(tab, chunk);
    const moe_adam_tensor& e = tab.t[t_in];
    in = pointers<8>(e, (long long)(chunk - tab.first[t_in]) * kBlocks + (tid >> 5));
    f32_in = e.g_dtype == MOE_F32;
    if (lane < 8) scale_in = (lane < 4 ? in.ms : in.vs)[(lane & 3) * kWarps];
  };
  const auto copy = [&](uint32_t chunk, int i) {
    if (chunk < end) {
      Stage8& st = ring[i];
      if (f32_in)
        copy_in<16>(&st.g[tid], in.g + (size_t)i * kStep * 4);
      else
        copy_in<8>(&st.g[tid], in.g + (size_t)i * kStep * 2);
      copy_in<16>(&st.p[tid], in.p + (size_t)i * kStep * 4);
      copy_in<4>(&st.m[tid], in.m + (size_t)i * kStep);
      copy_in<4>(&st.v[tid], in.v + (size_t)i * kStep);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  enter(c);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) copy(c, i);
  for (; c < end; ++c) {
    const int t = t_in;
    const Pointers at = in;
    const float scales = scale_in;
    const bool f32 = f32_in;
    const moe_adam_tensor& e = tab.t[t];
    const float decay = sc.lr * e.weight_decay;
    const uint32_t key = mix(e.seed ^ (sc.step * kGolden));
    const long long first = (long long)(c - tab.first[t]) * kBlocks + (tid >> 5);
    enter(c + 1);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSteps - 1) : "memory");
      const Stage8& st = ring[i];
      Four f;
      const float4 p = st.p[tid];
      f.p[0] = pair(p.x, p.y), f.p[1] = pair(p.z, p.w);
      if (f32) {
        const float4 g = st.g[tid];
        f.g[0] = pair(g.x, g.y), f.g[1] = pair(g.z, g.w);
      } else {
        const uint2 g = *reinterpret_cast<const uint2*>(&st.g[tid]);
        f.g[0] = pair_of_bf16(g.x), f.g[1] = pair_of_bf16(g.y);
      }
      from_codes(f, st.m[tid], st.v[tid], __shfl_sync(0xffffffffu, scales, i),
                 __shfl_sync(0xffffffffu, scales, 4 + i));
      copy(c + 1, i);   // into the place that has just been read
      step_four<8>(sc, decay, key, first + i * kWarps, at, i, 4, f);
    }
  }
  tails<CAP, 8>(tab, sc);
  finish(hyper, state, more);
}

// whole: chunks that a tensor fills, else all of them
template <int CAP>
uint32_t fill(Table<CAP>& tab, const moe_adam_tensor* t, int n, bool whole) {
  uint32_t chunks = 0;
  tab.n = n;
  for (int i = 0; i < n; ++i) {
    tab.t[i] = t[i];
    tab.first[i] = chunks;
    chunks += static_cast<uint32_t>((t[i].n + (whole ? 0 : kChunk - 1)) / kChunk);
  }
  tab.first[n] = chunks;
  return chunks;
}
unsigned grid_of(uint32_t chunks, int per_sm) {
  const uint32_t most = kGpuSms * per_sm;
  return chunks < 1 ? 1 : chunks > most ? most : chunks;
}

template <int CAP>
cudaError_t norm_cap(const moe_adam_tensor* t, int n, bool more, State* state, float* norm,
                     cudaStream_t st) {
  Table<CAP> tab;
  const uint32_t chunks = fill(tab, t, n, false);
  return launch_kernel(grad_norm_kernel<CAP>, dim3(grid_of(chunks, 8)), dim3(kThreads), 0, st, false,
                       tab, chunks, state, norm, more);
}
template <int CAP>
cudaError_t adam_cap(const moe_adam_cfg& c, const moe_adam_tensor* t, int n, bool more, State* state,
                     const float* norm, cudaStream_t st) {
  Table<CAP> tab;
  const uint32_t chunks = fill(tab, t, n, true);
  const Hyper h{c.lr, c.beta1, c.beta2, c.max_norm, static_cast<float>(c.eps), c.lr_dev};
  const bool held = c.state_bits == 8;
  auto kern = held ? adamw8_kernel<CAP> : adamw_kernel<CAP>;
  const size_t smem = held ? kSteps * sizeof(Stage8) : 0;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem + 1024);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid_of(chunks + n, 4)), dim3(kThreads), smem, st, false, tab, h,
                       chunks, state, norm, more);
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
