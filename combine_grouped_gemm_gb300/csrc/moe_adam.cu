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
__device__ __forceinline__ void store4(float* p, const float (&v)[4], int cnt) {
  if (cnt == 4) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) p[j] = v[j];
}
__device__ __forceinline__ void store4_bf16(void* w, long long i, const float (&v)[4], int cnt) {
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(w) + i;
  if (cnt == 4) {
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
    return;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j)
    if (j < cnt) p[j] = __float2bfloat16_rn(v[j]);
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

// One element: the new moments and the parameter. Each product and sum of the moments is rounded by
// itself (no fused multiply-add), so that 8-bit moments can be checked code by code.
__device__ __forceinline__ void update(const Scalars& sc, float decay, float g, float& p, float& m,
                                       float& v, float& root) {
  if (sc.clip) g = __fmul_rn(g, sc.factor);
  m = __fadd_rn(__fmul_rn(sc.b1, m), __fmul_rn(sc.n1, g));
  v = __fadd_rn(__fmul_rn(sc.b2, v), __fmul_rn(sc.n2, __fmul_rn(g, g)));
  root = __fsqrt_rn(v);
  const float den = __fmaf_rn(root, sc.root, sc.eps);
  p = __fmaf_rn(-decay, p, p);
  p = __fmaf_rn(-sc.move, __fdividef(m, den), p);
}

// The largest of a warp's non-negative numbers (their order is that of their bits).
__device__ __forceinline__ float warp_max(float v) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v)));
}

// e4m3 codes of four values of a block, rounded up or down by 16 random bits each: with the random
// bits added below the code's last bit, cutting off what is below it rounds up with odds of the
// distance from the lower code. Below 2^-6 the steps are 2^-9: with 2^-6 added they lie at the same
// bits.
__device__ __forceinline__ float round_e4m3(float q, uint32_t r16) {
  const bool small = q < 0x1p-6f;
  float y = small ? __fadd_rn(q, 0x1p-6f) : q;
  y = __uint_as_float((__float_as_uint(y) + (r16 << 4)) & 0xfff00000u);
  return small ? __fadd_rn(y, -0x1p-6f) : y;
}
// The same for the root of a second moment, with odds that keep the mean of its square, (q^2 - lo^2)
// / (hi^2 - lo^2): odds linear in q would add the rounding's variance to v each step, several
// percent of v in the long run.
__device__ __forceinline__ float round_root_e4m3(float q, uint32_t r16) {
  const float shift = q < 0x1p-6f ? 0x1p-6f : 0.0f;
  const uint32_t bits = __float_as_uint(__fadd_rn(q, shift)) & 0xfff00000u;
  const float lo = __fadd_rn(__uint_as_float(bits), -shift);   // exact, as are hi, hi - lo, hi + lo
  const float hi = __fadd_rn(__uint_as_float(bits + 0x100000u), -shift);
  const float odds = __fmul_rn(__fadd_rn(q, -lo), __fadd_rn(q, lo));
  const float whole = __fmul_rn(__fadd_rn(hi, -lo), __fadd_rn(hi, lo));
  return __fmul_rn(static_cast<float>(r16), whole) < __fmul_rn(odds, 65536.0f) ? hi : lo;
}
template <bool ROOT>
__device__ __forceinline__ uint32_t hold4(const float (&x)[4], float scale, const uint32_t (&r)[4],
                                          int shift) {
  uint32_t code = 0;
#pragma unroll
  for (int j = 0; j < 4; j += 2) {
    float q[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = fabsf(x[j + i]);
      const uint32_t r16 = (r[j + i] >> shift) & 0xffffu;
      q[i] = __fdiv_rn(a, scale);
      q[i] = q[i] > 448.0f ? 448.0f : q[i];
      if (ROOT) {
        q[i] = round_root_e4m3(q[i], r16);
        q[i] = a > 0.0f && q[i] < 0x1p-9f ? 0x1p-9f : q[i];
      } else {
        q[i] = copysignf(round_e4m3(q[i], r16), x[j + i]);
      }
    }
    code |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE,
                                                           __NV_E4M3))
            << (8 * j);
  }
  return code;
}
__device__ __forceinline__ void codes4(uint32_t c, float s, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((c >> (16 * i)) & 0xffffu), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = __fmul_rn(v.x, s);
    f[2 * i + 1] = __fmul_rn(v.y, s);
  }
}
__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? __fmul_rn(amax, 1.0f / 448.0f) : 1.0f;
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
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(tab, c);
    const moe_adam_tensor& e = tab.t[t];
    const long long base = (long long)(c - tab.first[t]) * kChunk;
    const bool f32 = e.g_dtype == MOE_F32;
    const float decay = sc.lr * e.weight_decay;
    const uint32_t key = BITS == 8 ? mix(e.seed ^ (sc.step * kGolden)) : 0;
    // a warp's four elements a lane are one block of 128
#pragma unroll 2
    for (int i = 0; i < kChunk / (4 * kThreads); ++i) {
      const long long block = base / kBlock + i * (kThreads / 32) + warp;
      const long long at = block * kBlock + lane * 4;
      const long long left = e.n - at;
      if (e.n <= block * kBlock) break;   // whole warps
      const int cnt = left >= 4 ? 4 : left > 0 ? (int)left : 0;
      const float4 g4 = load_grad(e.g, f32, at, cnt);
      const float4 p4 = load4(e.p + at, cnt);
      float g[4] = {g4.x, g4.y, g4.z, g4.w}, p[4] = {p4.x, p4.y, p4.z, p4.w};
      float m[4], v[4], root[4];
      if (BITS == 32) {
        const float4 m4 = load4(static_cast<const float*>(e.m) + at, cnt);
        const float4 v4 = load4(static_cast<const float*>(e.v) + at, cnt);
        m[0] = m4.x, m[1] = m4.y, m[2] = m4.z, m[3] = m4.w;
        v[0] = v4.x, v[1] = v4.y, v[2] = v4.z, v[3] = v4.w;
      } else {
        const uint32_t qm = load_codes(e.m, at, cnt), qv = load_codes(e.v, at, cnt);
        codes4(qm, e.m_scale[block], m);
        codes4(qv, e.v_scale[block], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __fmul_rn(v[j], v[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) update(sc, decay, g[j], p[j], m[j], v[j], root[j]);
      store4(e.p + at, p, cnt);
      if (e.w) store4_bf16(e.w, at, p, cnt);
      if (BITS == 32) {
        store4(static_cast<float*>(e.m) + at, m, cnt);
        store4(static_cast<float*>(e.v) + at, v, cnt);
      } else {
        // (fmaxf leaves a NaN out)
        const float am = warp_max(fmaxf(fmaxf(fabsf(m[0]), fabsf(m[1])),
                                        fmaxf(fabsf(m[2]), fabsf(m[3]))));
        const float av = warp_max(fmaxf(fmaxf(root[0], root[1]), fmaxf(root[2], root[3])));
        const float sm = block_scale(am), sv = block_scale(av);
        const uint32_t bkey = mix(key ^ static_cast<uint32_t>(block));
        uint32_t r[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = mix(bkey + (lane * 4 + j) * kGolden);
        store_codes(e.m, at, hold4<false>(m, sm, r, 16), cnt);
        store_codes(e.v, at, hold4<true>(root, sv, r, 0), cnt);
        if (lane == 0) {
          e.m_scale[block] = sm;
          e.v_scale[block] = sv;
        }
      }
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
