// The element-wise operators of the expert path's training step: activation checkpoints in 8
// bits (loading them, the SwiGLU that saves its input and its gradient from the saved codes) and
// the gradient of the combine. Each reads its inputs once and writes its outputs once.
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// 8 bf16 values as floats
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Four e4m3 codes (exact in fp16) times a scale.
__device__ __forceinline__ void codes4(uint32_t c, float s, float* f) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((c >> (16 * i)) & 0xffffu), __NV_E4M3);
    const float2 v = __half22float2(__half2(h));
    f[2 * i] = v.x * s;
    f[2 * i + 1] = v.y * s;
  }
}
__device__ __forceinline__ void codes8(const uint2& c, float s, float (&f)[8]) {
  codes4(c.x, s, f);
  codes4(c.y, s, f + 4);
}

// A 128-column block of one row over 16 lanes, 8 values each: the block's scale (the dispatch's
// rule, with IEEE divisions so that the codes are the dispatch's) and this lane's codes.
__device__ __forceinline__ uint2 quantise8(const float (&f)[8], float* scale_out) {
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    w[h] = 0;
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      w[h] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                  make_float2(__fdiv_rn(f[4 * h + j], scale), __fdiv_rn(f[4 * h + j + 1], scale)),
                  __NV_SATFINITE, __NV_E4M3))
              << (8 * j);
  }
  *scale_out = scale;
  return make_uint2(w[0], w[1]);
}

// One thread: 8 columns of one output row. A row is d / 8 threads.
__global__ void __launch_bounds__(kThreads) act_load_kernel(
    const uint2* __restrict__ q, const float* __restrict__ scales,
    const int32_t* __restrict__ index, uint4* __restrict__ out, int rows, int src_rows, int vpr,
    uint32_t* status) {
  const long long total = (long long)rows * vpr;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const int r = static_cast<int>(i / vpr), v = static_cast<int>(i % vpr);
    int src = index ? index[r] : r;
    if (src < -1 || src >= src_rows) {
      if (v == 0) raise_status(status, MOE_DEV_BOUNDS);
      src = -1;
    }
    uint4 o = make_uint4(0, 0, 0, 0);
    if (src >= 0) {
      float f[8];
      codes8(q[(long long)src * vpr + v], scales[(long long)(v / 16) * src_rows + src], f);
      o = pack8(f);
    }
    out[i] = o;
  }
}

// One thread: 8 columns of one row's gate and of its up half. The 16 lanes of a 128-column block
// are in one half-warp (f / 8 is a multiple of 16), and whole half-warps leave the loop together.
__global__ void __launch_bounds__(kThreads) swiglu_save_kernel(const uint4* __restrict__ gu,
                                                               uint4* __restrict__ a,
                                                               uint2* __restrict__ q,
                                                               float* __restrict__ scales,
                                                               int rows, int vpr) {
  const long long total = (long long)rows * vpr;
  const long long step = (long long)gridDim.x * kThreads;
  // every lane of a warp runs the same number of iterations (the shuffles take whole warps)
  for (long long i0 = (long long)blockIdx.x * kThreads; i0 < total; i0 += step) {
    const long long i = i0 + threadIdx.x;
    const bool in = i < total;
    const long long r = in ? i / vpr : 0;
    const int v = in ? static_cast<int>(i % vpr) : 0;
    float g[8] = {}, u[8] = {}, o[8];
    if (in) {
      unpack8(gu[r * 2 * vpr + v], g);
      unpack8(gu[r * 2 * vpr + vpr + v], u);
    }
    float sg, su;
    const uint2 cg = quantise8(g, &sg), cu = quantise8(u, &su);
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = silu(g[j]) * u[j];
    if (!in) continue;
    a[i] = pack8(o);
    q[r * 2 * vpr + v] = cg;
    q[r * 2 * vpr + vpr + v] = cu;
    if ((v & 15) == 0) {
      scales[(long long)(v / 16) * rows + r] = sg;
      scales[(long long)((vpr + v) / 16) * rows + r] = su;
    }
  }
}

__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(
    const uint2* __restrict__ q, const float* __restrict__ scales, const uint4* __restrict__ da,
    uint4* __restrict__ dgu, uint4* __restrict__ a, int rows, int vpr) {
  const long long total = (long long)rows * vpr;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kThreads) {
    const long long r = i / vpr;
    const int v = static_cast<int>(i % vpr);
    float g[8], u[8], d[8], dg[8], du[8], o[8];
    codes8(q[r * 2 * vpr + v], scales[(long long)(v / 16) * rows + r], g);
    codes8(q[r * 2 * vpr + vpr + v], scales[(long long)((vpr + v) / 16) * rows + r], u);
    unpack8(da[i], d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = 1.0f / (1.0f + __expf(-g[j]));
      const float gs = g[j] * s;
      dg[j] = d[j] * u[j] * (s + gs * (1.0f - s));
      du[j] = d[j] * gs;
      o[j] = gs * u[j];
    }
    dgu[r * 2 * vpr + v] = pack8(dg);
    dgu[r * 2 * vpr + vpr + v] = pack8(du);
    if (a) a[i] = pack8(o);
  }
}

// One CTA per (token, choice): dy's row times the weight, and its dot product with the row.
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(
    const uint4* __restrict__ ebuf, const int32_t* __restrict__ row_of,
    const float* __restrict__ topk_w, const uint4* __restrict__ dy, uint4* __restrict__ debuf,
    float* __restrict__ dtopk_w, int k, int vpr, int rows, uint32_t* status) {
  __shared__ float part[kThreads / 32];
  const long long c = blockIdx.x;
  const long long t = c / k;
  const int row = row_of[c];
  const float w = topk_w[c];
  if (row < 0 || row >= rows) {
    if (threadIdx.x == 0) {
      if (row >= rows) raise_status(status, MOE_DEV_BOUNDS);
      dtopk_w[c] = 0.0f;
    }
    return;
  }
  float acc = 0.0f;
  for (int v = threadIdx.x; v < vpr; v += kThreads) {
    float y[8], e[8], o[8];
    unpack8(dy[t * vpr + v], y);
    unpack8(ebuf[(long long)row * vpr + v], e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc = __fmaf_rn(y[j], e[j], acc);
      o[j] = w * y[j];
    }
    debuf[(long long)row * vpr + v] = pack8(o);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    dtopk_w[c] = s;
  }
}

unsigned blocks_for(long long threads) {
  const long long b = (threads + kThreads - 1) / kThreads;
  return static_cast<unsigned>(b < (1 << 20) ? b : 1 << 20);
}

}  // namespace

cudaError_t launch_act_load(int rows, int src_rows, int d, const void* q, const float* scales,
                            const int32_t* index, void* out, uint32_t* status, cudaStream_t st) {
  return launch_kernel(act_load_kernel, dim3(blocks_for((long long)rows * (d / 8))),
                       dim3(kThreads), 0, st, false, static_cast<const uint2*>(q), scales, index,
                       static_cast<uint4*>(out), rows, src_rows, d / 8, status);
}

cudaError_t launch_swiglu_save(int rows, int f, const void* gu, void* a, void* q, float* scales,
                               cudaStream_t st) {
  return launch_kernel(swiglu_save_kernel, dim3(blocks_for((long long)rows * (f / 8))),
                       dim3(kThreads), 0, st, false, static_cast<const uint4*>(gu),
                       static_cast<uint4*>(a), static_cast<uint2*>(q), scales, rows, f / 8);
}

cudaError_t launch_swiglu_grad(int rows, int f, const void* q, const float* scales,
                               const void* da, void* dgu, void* a, cudaStream_t st) {
  return launch_kernel(swiglu_grad_kernel, dim3(blocks_for((long long)rows * (f / 8))),
                       dim3(kThreads), 0, st, false, static_cast<const uint2*>(q), scales,
                       static_cast<const uint4*>(da), static_cast<uint4*>(dgu),
                       static_cast<uint4*>(a), rows, f / 8);
}

cudaError_t launch_combine_grad(int T, int k, int d, int rows, const void* ebuf,
                                const int32_t* row_of, const float* topk_w, const void* dy,
                                void* debuf, float* dtopk_w, uint32_t* status, cudaStream_t st) {
  return launch_kernel(combine_grad_kernel, dim3((unsigned)T * k), dim3(kThreads), 0, st, false,
                       static_cast<const uint4*>(ebuf), row_of, topk_w,
                       static_cast<const uint4*>(dy), static_cast<uint4*>(debuf), dtopk_w, k,
                       d / 8, rows, status);
}

}  // namespace moe
