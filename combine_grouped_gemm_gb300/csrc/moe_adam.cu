// AdamW over a list of tensors in one launch, moments in 32 or 8 bits, and the norm of all their
// gradients:
//   g' = g min(1, max_norm / |g|)    m = b1 m + (1 - b1) g'    v = b2 v + (1 - b2) g'^2
//   p -= lr wd p + lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
// Both stream their arrays from HBM once: 30 bytes a parameter with fp32 gradients, fp32 moments
// and a bf16 copy, 18.1 with 8-bit moments; the norm reads the gradients alone.
//
// The tensors are cut into chunks, which the CTAs of one grid take in turn; the table of the
// tensors travels as a kernel argument, so the step needs no device table and a captured one keeps
// its own.
#include "moe_device.cuh"

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

// Four values from element i on, of which cnt exist (none, if it is negative); the others are 0.
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
__device__ __forceinline__ void store4(float* p, const float4& v, int cnt) {
  if (cnt >= 4) {
    __stcs(reinterpret_cast<float4*>(p), v);
    return;
  }
  if (cnt > 0) p[0] = v.x;
  if (cnt > 1) p[1] = v.y;
  if (cnt > 2) p[2] = v.z;
}
__device__ __forceinline__ void store4_bf16(__nv_bfloat16* p, const float4& v, int cnt) {
  if (cnt >= 4) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)));
    return;
  }
  if (cnt > 0) p[0] = __float2bfloat16_rn(v.x);
  if (cnt > 1) p[1] = __float2bfloat16_rn(v.y);
  if (cnt > 2) p[2] = __float2bfloat16_rn(v.z);
}
__device__ __forceinline__ void store_codes(char* q, uint32_t v, int cnt) {
  if (cnt >= 4) {
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
  pdl_trigger();
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
  bool skip;
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
  pdl_wait();
  if (threadIdx.x == 0) {
    const double c1 = h.beta1 * state->c1 + (1.0 - h.beta1);
    const double c2 = h.beta2 * state->c2 + (1.0 - h.beta2);
    const double lr = h.lr_dev ? static_cast<double>(*h.lr_dev) : h.lr;
    sc.b1 = static_cast<float>(h.beta1);
    sc.n1 = static_cast<float>(1.0 - h.beta1);
    sc.b2 = static_cast<float>(h.beta2);
    sc.n2 = static_cast<float>(1.0 - h.beta2);
    // (the corrections themselves need fp64, as sums of small parts; quotient and root do not, and
    // fp64 division and root take microseconds here)
    sc.lr = static_cast<float>(lr);
    sc.move = __fdiv_rn(sc.lr, static_cast<float>(c1));
    sc.root = __frsqrt_rn(static_cast<float>(c2));
    sc.eps = h.eps;
    sc.step = static_cast<uint32_t>(state->step + 1);
    const float total = norm ? *norm : 0.0f;
    sc.skip = !(fabsf(total) < INFINITY);
    sc.factor = h.max_norm > 0.0
                    ? fminf(__fmul_rn(static_cast<float>(h.max_norm), __frcp_rn(total)), 1.0f)
                    : 1.0f;
  }
  __syncthreads();
  return sc;
}

// One element: the new moments and the parameter. Each product and sum of the moments is rounded by
// itself, so that 8-bit moments can be checked code by code; the parameter's quotient takes the
// hardware's reciprocal (1 ulp).
__device__ __forceinline__ float recip(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ void update(const Scalars& sc, float decay, float g, float& p, float& m,
                                       float& v, float& root) {
  g = __fmul_rn(g, sc.factor);   // (1 where nothing is clipped)
  m = __fadd_rn(__fmul_rn(sc.b1, m), __fmul_rn(sc.n1, g));
  v = __fadd_rn(__fmul_rn(sc.b2, v), __fmul_rn(sc.n2, __fmul_rn(g, g)));
  root = __fsqrt_rn(v);
  const float quot = m * recip(__fmaf_rn(root, sc.root, sc.eps));
  p = __fmaf_rn(-sc.move, quot, __fmaf_rn(-decay, p, p));
}

__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The largest of 16 lanes' non-negative numbers (their order is that of their bits, a NaN last).
__device__ __forceinline__ float half_warp_max(float v) {
  const uint32_t lanes = (threadIdx.x & 16) ? 0xffff0000u : 0xffffu;
  return __uint_as_float(__reduce_max_sync(lanes, __float_as_uint(v)));
}

// 1 where v > 0 (and v * big >= 1), else 0; a NaN gives 0. (By saturation on the FMA pipe:
// comparison and select are two operations of the ALU pipe, which the integer work beside them
// fills.)
__device__ __forceinline__ float is_positive(float v, float big) {
  float r;
  asm("mul.rn.sat.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(big));
  return r;
}
__device__ __forceinline__ float below_2_6(float q) {
  return __saturatef(__fmaf_rn(q, -0x1p40f, 0x1p34f));
}
__device__ __forceinline__ float cut(uint32_t bits) { return __uint_as_float(bits & 0xfff00000u); }

// A quotient rounded up or down to e4m3 by 16 random bits. With the random bits added below the
// code's last bit, cutting off what is below it rounds up with odds of the distance from the lower
// code. Below 2^-6 the steps are 2^-9: with 2^-6 added they lie at the same bits. (What is past 448
// by a rounding is cut or, as a code, saturated.)
__device__ __forceinline__ float round_e4m3(float q, uint32_t r16) {
  const float s = below_2_6(q), y = __fmaf_rn(s, 0x1p-6f, q);
  return __fmaf_rn(s, -0x1p-6f, cut(__float_as_uint(y) + r16 * 16));
}
// The same for the root of a second moment, with odds that keep the mean of its square, (q^2 -
// lo^2) / (hi^2 - lo^2): odds linear in q would add the rounding's variance to v each step, several
// percent of v in the long run. A root above 0 keeps a code above 0.
__device__ __forceinline__ float round_root_e4m3(float q, float root, uint32_t r16) {
  const float s = below_2_6(q), y = __fmaf_rn(s, 0x1p-6f, q), c = cut(__float_as_uint(y));
  const float lo = __fmaf_rn(s, -0x1p-6f, c);   // exact, as are hi - lo (a step) and hi + lo
  const float gap = __uint_as_float((__float_as_uint(c) & 0x7f800000u) - 0x01800000u);
  const float odds = __fmul_rn(__fadd_rn(q, -lo), __fadd_rn(q, lo));
  const float whole = __fmul_rn(gap, __fmaf_rn(2.0f, lo, gap));
  // r / 2^16 as the fraction of a number between 1 and 2
  const float r = __fadd_rn(__uint_as_float(0x3f800000u + r16 * 128), -1.0f);
  // up where r whole, rounded, < odds. (A difference that is no multiple of 2^-100 leaves a value
  // below the lowest code, which the next lines make that code.)
  const float up = is_positive(__fadd_rn(odds, -__fmul_rn(r, whole)), 0x1p100f);
  const float u = __fmaf_rn(up, gap, lo), least = is_positive(root, 0x1p100f) * 0x1p-9f;
  return max_or_nan(u, least);
}
__device__ __forceinline__ uint32_t pack_codes(const float* v) {
  return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v[0], v[1]), __NV_SATFINITE,
                                                        __NV_E4M3)) |
         static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(v[2], v[3]), __NV_SATFINITE,
                                                        __NV_E4M3))
             << 16;
}
__device__ __forceinline__ void codes4(uint32_t c, float s, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((c >> (16 * i)) & 0xffffu), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = __fmul_rn(v.x, s);
    f[2 * i + 1] = __fmul_rn(v.y, s);
  }
}

// The last call of a step: the last CTA to end counts it. (Every CTA has read the state before it
// took its ticket.)
__device__ __forceinline__ void finish(const Hyper& h, State* state, bool more) {
  if (more || !last_cta(&state->ticket) || threadIdx.x != 0) return;
  state->step += 1;
  state->c1 = h.beta1 * state->c1 + (1.0 - h.beta1);
  state->c2 = h.beta2 * state->c2 + (1.0 - h.beta2);
}

// ------------------------------------------------------------------------------------------
// Moments in 32 bits: four elements a lane at once, loads a step ahead. 398 M parameters with fp32
// gradients and their norm: 2.05 ms for 13.5 GB, 6.6 TB/s: bound by memory.
// ------------------------------------------------------------------------------------------
struct Four {
  float4 g, p, m, v;
};
__device__ __forceinline__ Four load_four(const moe_adam_tensor& e, long long at, int cnt) {
  return Four{load_grad(e.g, e.g_dtype == MOE_F32, at, cnt), load4(e.p + at, cnt),
              load4(static_cast<const float*>(e.m) + at, cnt),
              load4(static_cast<const float*>(e.v) + at, cnt)};
}
__device__ __forceinline__ void step_four(const Scalars& sc, const moe_adam_tensor& e, float decay,
                                          long long at, int cnt, Four f) {
  float root;
  update(sc, decay, f.g.x, f.p.x, f.m.x, f.v.x, root);
  update(sc, decay, f.g.y, f.p.y, f.m.y, f.v.y, root);
  update(sc, decay, f.g.z, f.p.z, f.m.z, f.v.z, root);
  update(sc, decay, f.g.w, f.p.w, f.m.w, f.v.w, root);
  store4(e.p + at, f.p, cnt);
  if (e.w) store4_bf16(static_cast<__nv_bfloat16*>(e.w) + at, f.p, cnt);
  store4(static_cast<float*>(e.m) + at, f.m, cnt);
  store4(static_cast<float*>(e.v) + at, f.v, cnt);
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
    const long long first = (long long)(c - tab.first[t]) * kChunk + threadIdx.x * 4;
    const float decay = sc.lr * e.weight_decay;
    Four next = load_four(e, first, 4);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const Four now = next;
      if (i + 1 < kSteps) next = load_four(e, first + (i + 1) * kStep, 4);
      step_four(sc, e, decay, first + i * kStep, 4, now);
    }
  }
  // the elements past the whole chunks, tensor by tensor a CTA (the last CTAs: the first ones have
  // had the odd chunks)
  for (int t = gridDim.x - 1 - blockIdx.x; t < tab.n; t += gridDim.x) {
    const moe_adam_tensor& e = tab.t[t];
    for (long long at = e.n / kChunk * kChunk + threadIdx.x * 4; at < e.n; at += kStep) {
      const int cnt = e.n - at >= 4 ? 4 : (int)(e.n - at);
      step_four(sc, e, sc.lr * e.weight_decay, at, cnt, load_four(e, at, cnt));
    }
  }
  finish(hyper, state, more);
}

// ------------------------------------------------------------------------------------------
// Moments in 8 bits: eight elements a lane at once, so that 16 lanes hold a block and what is done
// once for it (scales, reciprocals, the key of its random numbers) is shared by eight elements.
// Each thread's elements come through two stages of its own in shared memory, and a CTA takes
// neighbouring chunks. 398 M parameters, bf16 gradients, no norm: 1.32 ms, 4.9 TB/s. Some 100
// instructions an element bound it, beside the update's the hash, the quotients and the rounding of
// two codes: the issue slots are four fifths full. (Four elements a lane 1.93 ms; loads through
// shared memory 1.59; eight a lane 1.41; one branch a block 1.32.)
// ------------------------------------------------------------------------------------------
constexpr int kStep8 = 8 * kThreads, kSteps8 = kChunk / kStep8;
struct Stage8 {
  uint4 g[2 * kThreads];   // bf16 gradients: half of it
  float4 p[2 * kThreads];
  uint2 m[kThreads], v[kThreads];
};
struct Eight {
  float g[8], p[8], m[8], v[8];
};
__device__ __forceinline__ void put4(float* f, const float4& v) {
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ float4 get4(const float* f) {
  return make_float4(f[0], f[1], f[2], f[3]);
}

// at: of the lane's first element, whose block is the lane's; cnt: how many exist
__device__ __forceinline__ void step_eight(const Scalars& sc, const moe_adam_tensor& e, float decay,
                                           uint32_t key, long long at, int cnt, Eight& f) {
  const long long block = at / kBlock;
  const int place = threadIdx.x & 15;
  float root[8], am = 0.0f, av = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    update(sc, decay, f.g[j], f.p[j], f.m[j], f.v[j], root[j]);
    am = max_or_nan(am, fabsf(f.m[j]));
    av = max_or_nan(av, root[j]);
  }
  __nv_bfloat16* w = static_cast<__nv_bfloat16*>(e.w) + at;
  if (cnt == 8) {
    __stcs(reinterpret_cast<float4*>(e.p + at), get4(f.p));
    __stcs(reinterpret_cast<float4*>(e.p + at) + 1, get4(f.p + 4));
    if (e.w)
      __stcs(reinterpret_cast<uint4*>(w),
             make_uint4(pack_bf16x2(f.p[0], f.p[1]), pack_bf16x2(f.p[2], f.p[3]),
                        pack_bf16x2(f.p[4], f.p[5]), pack_bf16x2(f.p[6], f.p[7])));
  } else {
    store4(e.p + at, get4(f.p), cnt);
    store4(e.p + at + 4, get4(f.p + 4), cnt - 4);
    if (e.w) {
      store4_bf16(w, get4(f.p), cnt);
      store4_bf16(w + 4, get4(f.p + 4), cnt - 4);
    }
  }
  // scale and reciprocal of the one moment in the even lanes, of the other in the odd ones
  const float sm0 = half_warp_max(am), sv0 = half_warp_max(av);
  const float amax = (threadIdx.x & 1) ? sv0 : sm0;
  // (A block whose scale would be no normal number, an amax below 5e-36, counts as zeros: its quotients
  // by 1 get code 0. Moments without gradients get there: 0.9 a step from 1e-4, 680 steps. The product
  // by 1/448 reaches 0 before amax does, and a quotient 0/0 is none. A NaN or an infinity in the block
  // becomes the scale, whatever the codes are.)
  const float part = __fmul_rn(amax, 1.0f / 448.0f), scale = part < 0x1p-126f ? 1.0f : part;
  const float inv = __frcp_rn(scale);
  // where the reciprocal, its correction and the quotient stay inside the fp32 range
  const bool plain = __all_sync(0xffffffffu, scale > 0x1p-60f && scale < 0x1p100f);
  const auto of_half = [](float v, int lane) { return __shfl_sync(0xffffffffu, v, lane, 16); };
  const float sm = of_half(scale, 0), sv = of_half(scale, 1);
  const float rm = of_half(inv, 0), rv = of_half(inv, 1);
  const uint32_t from = mix(key ^ static_cast<uint32_t>(block)) + place * 8 * kGolden;
  const auto hold = [&](auto quotient) {   // |x| / scale, the IEEE quotient
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // the halves of the hash x ^ (x >> 16)
      const uint32_t x = premix(from + j * kGolden), h = x >> 16;
      const float q = round_e4m3(quotient(fabsf(f.m[j]), sm, rm), h);
      f.m[j] = copysignf(q, f.m[j]);
      f.v[j] = round_root_e4m3(quotient(root[j], sv, rv), root[j], (x ^ h) & 0xffffu);
    }
  };
  // By the correctly rounded reciprocal and one correction step (P. Markstein, "Computation of
  // elementary functions on the IBM RISC System/6000 processor", 1990).
  if (plain)
    hold([](float x, float s, float r) {
      const float q = __fmul_rn(x, r);
      return __fmaf_rn(__fmaf_rn(-q, s, x), r, q);
    });
  else
    hold([](float x, float s, float) { return __fdiv_rn(x, s); });
  char *qm = static_cast<char*>(e.m) + at, *qv = static_cast<char*>(e.v) + at;
  if (cnt == 8) {
    __stcs(reinterpret_cast<uint2*>(qm), make_uint2(pack_codes(f.m), pack_codes(f.m + 4)));
    __stcs(reinterpret_cast<uint2*>(qv), make_uint2(pack_codes(f.v), pack_codes(f.v + 4)));
  } else {
    store_codes(qm, pack_codes(f.m), cnt);
    store_codes(qm + 4, pack_codes(f.m + 4), cnt - 4);
    store_codes(qv, pack_codes(f.v), cnt);
    store_codes(qv + 4, pack_codes(f.v + 4), cnt - 4);
  }
  if (place < 2 && (cnt == 8 || block * kBlock < e.n))
    (place ? e.v_scale : e.m_scale)[block] = scale;
}

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

// LINES: parameters and fp32 gradients, 32 bytes a lane, come to the warp by whole lines (neighbouring
// lanes copy neighbouring 16 bytes, then read two others, in an order free of bank conflicts): 127 M
// parameters with fp32 gradients 460 us, 541 where each lane copies its own 32 bytes. With bf16
// gradients the warp's two barriers cost more than this gives: 467 us against 455. So it goes by the
// type that most gradients have.
template <int CAP, bool LINES>
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
  uint32_t c = (uint32_t)((unsigned long long)chunks * blockIdx.x / gridDim.x);
  const uint32_t end = (uint32_t)((unsigned long long)chunks * (blockIdx.x + 1) / gridDim.x);
  // the chunk that is copied, one before the one that is worked on
  int t_in = 0;
  long long at_in = 0;     // of this thread's first element
  float scale_in = 0.0f;   // lanes 0-3: of m, steps 0 and 1, the warp's two blocks; lanes 4-7: of v
  const auto enter = [&](uint32_t chunk) {
    if (chunk >= end) return;
    t_in = tensor_of(tab, chunk);
    const moe_adam_tensor& e = tab.t[t_in];
    const long long first = (long long)(chunk - tab.first[t_in]) * kChunk;
    at_in = first + tid * 8;
    if (lane < 8)
      scale_in = (lane < 4 ? e.m_scale : e.v_scale)[first / kBlock + (tid >> 5) * 2 +
                                                    (lane & 1) + (lane & 2) * (kStep8 / kBlock / 2)];
  };
  // places of what this thread copies and of what it reads, in a stage's arrays of 16 bytes
  const int warp0 = (tid & ~31) * 2;
  const int put0 = LINES ? warp0 + (lane ^ ((lane >> 3) & 1)) : tid;
  const int put1 = LINES ? put0 + 32 : tid + kThreads;
  const int get0 = LINES ? warp0 + ((2 * lane) ^ ((lane >> 2) & 1)) : tid;
  const int get1 = LINES ? get0 ^ 1 : tid + kThreads;
  // bf16 gradients: inside the places of the same warp (LINES: whose barriers order its lanes) or
  // thread. A warp may be a chunk ahead of another, in a tensor of the other type.
  const int own_bf16 = LINES ? warp0 + lane : tid;
  const auto copy = [&](uint32_t chunk, int i) {
    if (chunk < end) {
      const moe_adam_tensor& e = tab.t[t_in];
      const long long at = at_in + i * kStep8;
      Stage8& st = ring[i];
      const long long at0 = LINES ? at - lane * 4 : at;
      constexpr int kNext = LINES ? 128 : 4;
      if (e.g_dtype == MOE_F32) {
        copy_in<16>(st.g + put0, static_cast<const float*>(e.g) + at0);
        copy_in<16>(st.g + put1, static_cast<const float*>(e.g) + at0 + kNext);
      } else {
        copy_in<16>(st.g + own_bf16, static_cast<const __nv_bfloat16*>(e.g) + at);
      }
      copy_in<16>(st.p + put0, e.p + at0);
      copy_in<16>(st.p + put1, e.p + at0 + kNext);
      copy_in<8>(&st.m[tid], static_cast<const char*>(e.m) + at);
      copy_in<8>(&st.v[tid], static_cast<const char*>(e.v) + at);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  enter(c);
#pragma unroll
  for (int i = 0; i < kSteps8; ++i) copy(c, i);
  for (; c < end; ++c) {
    const moe_adam_tensor& e = tab.t[t_in];
    const long long at = at_in;
    const float scales = scale_in;
    const float decay = sc.lr * e.weight_decay;
    const uint32_t key = mix(e.seed ^ (sc.step * kGolden));
    enter(c + 1);
#pragma unroll 1
    for (int i = 0; i < kSteps8; ++i) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kSteps8 - 1) : "memory");
      if (LINES) __syncwarp();
      const Stage8& st = ring[i];
      Eight f;
      if (e.g_dtype == MOE_F32) {
        put4(f.g, *reinterpret_cast<const float4*>(st.g + get0));
        put4(f.g + 4, *reinterpret_cast<const float4*>(st.g + get1));
      } else {
        const uint4 g = st.g[own_bf16];
        put4(f.g, make_float4(bf16_lo(g.x), bf16_hi(g.x), bf16_lo(g.y), bf16_hi(g.y)));
        put4(f.g + 4, make_float4(bf16_lo(g.z), bf16_hi(g.z), bf16_lo(g.w), bf16_hi(g.w)));
      }
      put4(f.p, st.p[get0]);
      put4(f.p + 4, st.p[get1]);
      const uint2 qm = st.m[tid], qv = st.v[tid];
      const int of = 2 * i + (lane >> 4);
      const float sm = __shfl_sync(0xffffffffu, scales, of);
      const float sv = __shfl_sync(0xffffffffu, scales, 4 + of);
      if (LINES) __syncwarp();
      copy(c + 1, i);   // into the place that has just been read
      codes4(qm.x, sm, f.m);
      codes4(qm.y, sm, f.m + 4);
      codes4(qv.x, sv, f.v);
      codes4(qv.y, sv, f.v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] = __fmul_rn(f.v[j], f.v[j]);
      step_eight(sc, e, decay, key, at + i * kStep8, 8, f);
    }
  }
  for (int t = gridDim.x - 1 - blockIdx.x; t < tab.n; t += gridDim.x) {   // as above
    const moe_adam_tensor& e = tab.t[t];
    const uint32_t key = mix(e.seed ^ (sc.step * kGolden));
    const bool f32 = e.g_dtype == MOE_F32;
    long long at = e.n / kChunk * kChunk + tid * 8;
    for (; at - lane * 8 < e.n; at += kStep8) {   // whole warps
      const int cnt = e.n - at >= 8 ? 8 : e.n > at ? (int)(e.n - at) : 0;
      Eight f;
      put4(f.g, load_grad(e.g, f32, at, cnt < 4 ? cnt : 4));
      put4(f.g + 4, load_grad(e.g, f32, at + 4, cnt - 4));
      put4(f.p, load4(e.p + at, cnt < 4 ? cnt : 4));
      put4(f.p + 4, load4(e.p + at + 4, cnt - 4));
      const char *qm = static_cast<const char*>(e.m) + at, *qv = static_cast<const char*>(e.v) + at;
      const float sm = cnt > 0 ? e.m_scale[at / kBlock] : 0.0f;
      const float sv = cnt > 0 ? e.v_scale[at / kBlock] : 0.0f;
      codes4(load_codes(qm, cnt < 4 ? cnt : 4), sm, f.m);
      codes4(load_codes(qm + 4, cnt - 4), sm, f.m + 4);
      codes4(load_codes(qv, cnt < 4 ? cnt : 4), sv, f.v);
      codes4(load_codes(qv + 4, cnt - 4), sv, f.v + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) f.v[j] = __fmul_rn(f.v[j], f.v[j]);
      step_eight(sc, e, sc.lr * e.weight_decay, key, at, cnt, f);
    }
  }
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
  long long wide = 0;   // fp32 gradients less bf16 ones
  for (int i = 0; i < n; ++i) wide += t[i].g_dtype == MOE_F32 ? t[i].n : -t[i].n;
  auto kern = !held      ? adamw_kernel<CAP>
              : wide > 0 ? adamw8_kernel<CAP, true>
                         : adamw8_kernel<CAP, false>;
  const size_t smem = held ? kSteps8 * sizeof(Stage8) : 0;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem + 1024);
  if (e != cudaSuccess) return e;
  // with a norm: launched while its kernel, the one before, still runs (1.9 M parameters in fp32,
  // norm and step: 18.4 us, 20.7 one after the other)
  return launch_kernel(kern, dim3(grid_of(chunks + n, 4)), dim3(kThreads), smem, st, norm != nullptr,
                       tab, h, chunks, state, norm, more);
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
