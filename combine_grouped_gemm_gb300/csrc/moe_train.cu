// The element-wise operators of the expert path's training step: activation checkpoints in 8
// bits (loading them, the SwiGLU that saves its input and its gradient from the saved codes) and
// the gradient of the combine. Each reads its inputs from HBM once and writes its outputs once.
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

__device__ __forceinline__ float sigmoid(float g) {   // 0 where exp(-g) passes the fp32 range
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));   // exp(-g)
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));                       // 1 ulp
  return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
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

// Largest magnitude of 8 bf16 values (a NaN does not count), in the low half of the result.
__device__ __forceinline__ __nv_bfloat162 amax8(const uint4& v) {
  const auto h = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)); };
  const __nv_bfloat162 m = __hmax2(__hmax2(h(v.x), h(v.y)), __hmax2(h(v.z), h(v.w)));
  return __hmax2(m, __lowhigh2highlow(m));
}

// Largest over the 16 lanes of a half-warp, both halves of the register at once.
__device__ __forceinline__ __nv_bfloat162 half_warp_max2(__nv_bfloat162 m) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const uint32_t other =
        __shfl_xor_sync(0xffffffffu, *reinterpret_cast<const uint32_t*>(&m), o);
    m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&other));
  }
  return m;
}

// The dispatch's rule: scale = amax / 448 (1 if amax is 0), codes e4m3(x / scale), both IEEE
// divisions, so that the codes are the dispatch's bit for bit. The quotients x / scale come from
// the correctly rounded reciprocal by one correction step (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990): q = x r, then q - r (q
// scale - x) with fused multiply-adds is the correctly rounded quotient as long as nothing
// underflows or overflows (in this form a zero keeps its sign). Scales outside 2^-60 .. 2^100
// (infinities among them) take the divisions. Two quotients an instruction: with one at a time,
// and with IEEE divisions, the SwiGLU of 16384 rows of 2048 took 50 and 59 us.
__device__ __forceinline__ float block_scale(float amax) {
  return amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
}
__device__ __forceinline__ uint2 codes_of8(const float (&f)[8], float scale) {
  float q[8];
  if (scale > 0x1p-60f && scale < 0x1p100f) {
    const float r = __frcp_rn(scale);
    const float2 r2 = make_float2(r, r), s2 = make_float2(scale, scale), n2 = make_float2(-r, -r);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const float2 x = make_float2(f[j], f[j + 1]);
      const float2 q0 = mul2(x, r2);
      const float2 v = fma2(fma2(q0, s2, make_float2(-x.x, -x.y)), n2, q0);
      q[j] = v.x;
      q[j + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fdiv_rn(f[j], scale);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; j += 2)
    w[j >> 2] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[j], q[j + 1]),
                                                                __NV_SATFINITE, __NV_E4M3))
                 << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

// What these kernels measured (whole calls replayed from a graph, copy rate 6.7 TB/s): swiglu_save
// of 16384 rows of 2048 45 us (6.0 TB/s, instruction issue 79 % busy), its gradient 50 us (6.7
// TB/s), 2048 rows of 7168 saved and loaded 8-fold 44 us (6.7 TB/s); 8 rows about 2 us, a launch.
//
// The kernels that read or write scales take tiles of 16 rows x 128 columns a CTA: a half-warp is
// one row's block (8 columns a lane), so a CTA's scales are 16 consecutive floats. CTA c: column
// block c % nb of row group c / nb.
constexpr int kTileRows = kThreads / 16;

__global__ void __launch_bounds__(kThreads) act_save_kernel(const uint4* __restrict__ x,
                                                            uint2* __restrict__ q,
                                                            float* __restrict__ scales, int rows,
                                                            int nb) {
  const int rg = blockIdx.x / nb, b = blockIdx.x - rg * nb;
  const int r = rg * kTileRows + (threadIdx.x >> 4), l = threadIdx.x & 15;
  const bool in = r < rows;
  const size_t at = ((size_t)r * nb + b) * 16 + l;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (in) v = x[at];
  const float scale = block_scale(__low2float(half_warp_max2(amax8(v))));
  float f[8];
  unpack8(v, f);
  if (!in) return;
  q[at] = codes_of8(f, scale);
  if (l == 0) scales[(size_t)b * rows + r] = scale;
}

// One warp: up to 8 column blocks of one output row, two at a time. part: ceil(nb / 8).
constexpr int kLoadBlocks = 8;
__global__ void __launch_bounds__(kThreads) act_load_kernel(
    const uint2* __restrict__ q, const float* __restrict__ scales,
    const int32_t* __restrict__ index, uint4* __restrict__ out, int rows, int src_rows, int nb,
    int parts, uint32_t* status) {
  const unsigned item = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const unsigned r = item / parts, part = item - r * parts;
  if (r >= static_cast<unsigned>(rows)) return;
  int src = index ? index[r] : static_cast<int>(r);
  if (src < -1 || src >= src_rows) {
    if (lane == 0 && part == 0) raise_status(status, MOE_DEV_BOUNDS);
    src = -1;
  }
  const int b0 = part * kLoadBlocks + (lane >> 4);
  uint2 c[kLoadBlocks / 2];
  float s[kLoadBlocks / 2];
#pragma unroll
  for (int i = 0; i < kLoadBlocks / 2; ++i) {
    const int b = b0 + 2 * i;
    const bool in = src >= 0 && b < nb;
    c[i] = in ? q[((size_t)src * nb + b) * 16 + (lane & 15)] : make_uint2(0, 0);
    s[i] = in ? scales[(size_t)b * src_rows + src] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kLoadBlocks / 2; ++i) {
    const int b = b0 + 2 * i;
    float f[8];
    codes8(c[i], s[i], f);
    if (b < nb) __stcs(out + ((size_t)r * nb + b) * 16 + (lane & 15), pack8(f));
  }
}

// per: row groups a CTA takes one after the other, the next one's loads issued before the present
// one is worked on.
__global__ void __launch_bounds__(kThreads) swiglu_save_kernel(const uint4* __restrict__ gu,
                                                               uint4* __restrict__ a,
                                                               uint2* __restrict__ q,
                                                               float* __restrict__ scales,
                                                               int rows, int nb, int per) {
  const int set = blockIdx.x / nb, b = blockIdx.x - set * nb;
  const int l = threadIdx.x & 15;
  int r = set * per * kTileRows + (threadIdx.x >> 4);
  size_t ga = ((size_t)r * 2 * nb + b) * 16 + l;
  const size_t up = (size_t)nb * 16, hop = up * 2 * kTileRows;
  uint4 gn = make_uint4(0, 0, 0, 0), un = gn;
  if (r < rows) {
    gn = gu[ga];
    un = gu[ga + up];
  }
  for (int i = 0; i < per; ++i) {
    const uint4 gv = gn, uv = un;
    const bool in = r < rows;
    if (i + 1 < per && r + kTileRows < rows) {
      gn = gu[ga + hop];
      un = gu[ga + hop + up];
    }
    // both halves' largest values through the same shuffles: gate low, up high
    const __nv_bfloat162 m = half_warp_max2(__lows2bfloat162(amax8(gv), amax8(uv)));
    const float sg = block_scale(__low2float(m)), su = block_scale(__high2float(m));
    if (in) {
      float g[8], u[8], o[8];
      unpack8(gv, g);
      unpack8(uv, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = g[j] * sigmoid(g[j]) * u[j];
      a[((size_t)r * nb + b) * 16 + l] = pack8(o);
      q[ga] = codes_of8(g, sg);
      q[ga + up] = codes_of8(u, su);
      if (l == 0) {
        scales[(size_t)b * rows + r] = sg;
        scales[(size_t)(nb + b) * rows + r] = su;
      }
    }
    r += kTileRows;
    ga += hop;
  }
}

__global__ void __launch_bounds__(kThreads) swiglu_grad_kernel(
    const uint2* __restrict__ q, const float* __restrict__ scales, const uint4* __restrict__ da,
    uint4* __restrict__ dgu, uint4* __restrict__ a, int rows, int nb) {
  const int rg = blockIdx.x / nb, b = blockIdx.x - rg * nb;
  const int r = rg * kTileRows + (threadIdx.x >> 4), l = threadIdx.x & 15;
  if (r >= rows) return;
  const size_t ga = ((size_t)r * 2 * nb + b) * 16 + l, ua = ga + (size_t)nb * 16;
  const size_t at = ((size_t)r * nb + b) * 16 + l;
  float g[8], u[8], d[8], dg[8], du[8], o[8];
  const uint2 cg = q[ga], cu = q[ua];
  const uint4 dv = da[at];
  codes8(cg, scales[(size_t)b * rows + r], g);
  codes8(cu, scales[(size_t)(nb + b) * rows + r], u);
  unpack8(dv, d);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = sigmoid(g[j]);
    const float gs = g[j] * s;
    dg[j] = d[j] * u[j] * (s + gs * (1.0f - s));
    du[j] = d[j] * gs;
    o[j] = gs * u[j];
  }
  __stcs(dgu + ga, pack8(dg));
  __stcs(dgu + ua, pack8(du));
  if (a) __stcs(a + at, pack8(o));
}

// One choice of one token: dy's row times the weight, and its dot product with the choice's row.
// LANES threads a choice: a warp where rows are short or choices fill the GPU's warps, else a whole
// CTA. Choices x columns, CTA and warp: 9625 x 128 8.5 and 3.0 us, 16384 x 2048 31 and 26 us, 16384
// x 7168 82.4 and 80.6 us; 5600 x 7168 31 and 33 us, 512 x 7168 3.6 and 8.1 us. dy's row is read k
// times, from L2 after the first (a CTA for all choices of a token, reading it once: 81.7 us).
// Bound by HBM: 16384 x 7168 moves 499 MB at 6.2 TB/s.
template <int LANES>
__global__ void __launch_bounds__(kThreads) combine_grad_kernel(
    const uint4* __restrict__ ebuf, const int32_t* __restrict__ row_of,
    const float* __restrict__ topk_w, const uint4* __restrict__ dy, uint4* __restrict__ debuf,
    float* __restrict__ dtopk_w, int choices, int k, int vpr, int rows, uint32_t* status) {
  __shared__ float part[kThreads / 32];
  const unsigned c = blockIdx.x * (kThreads / LANES) + threadIdx.x / LANES;
  const int l = threadIdx.x % LANES;
  if (c >= static_cast<unsigned>(choices)) return;
  const unsigned t = c / static_cast<unsigned>(k);
  const int row = row_of[c];
  const float w = topk_w[c];
  if (row < 0 || row >= rows) {
    if (l == 0) {
      if (row >= rows) raise_status(status, MOE_DEV_BOUNDS);
      dtopk_w[c] = 0.0f;
    }
    return;
  }
  const uint4* ys = dy + (size_t)t * vpr;
  const uint4* es = ebuf + (size_t)row * vpr;
  uint4* ds = debuf + (size_t)row * vpr;
  float acc = 0.0f;
  for (int v = l; v < vpr; v += LANES) {
    float y[8], e[8], o[8];
    unpack8(ys[v], y);
    unpack8(es[v], e);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      acc = __fmaf_rn(y[j], e[j], acc);
      o[j] = w * y[j];
    }
    ds[v] = pack8(o);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (LANES == 32) {
    if (l == 0) dtopk_w[c] = acc;
    return;
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    dtopk_w[c] = s;
  }
}

// CTAs of the 16-row tiles. (The callers keep rows * cols below 2^37: grids and row numbers fit 32
// bits.)
unsigned tiles_of(int rows, int nb) {
  return static_cast<unsigned>(((long long)rows + kTileRows - 1) / kTileRows * nb);
}

}  // namespace

cudaError_t launch_act_save(int rows, int d, const void* x, void* q, float* scales,
                            cudaStream_t st) {
  return launch_kernel(act_save_kernel, dim3(tiles_of(rows, d / 128)), dim3(kThreads), 0, st, false,
                       static_cast<const uint4*>(x), static_cast<uint2*>(q), scales, rows,
                       d / 128);
}

cudaError_t launch_act_load(int rows, int src_rows, int d, const void* q, const float* scales,
                            const int32_t* index, void* out, uint32_t* status, cudaStream_t st) {
  const int nb = d / 128, parts = (nb + kLoadBlocks - 1) / kLoadBlocks;
  const long long warps = (long long)rows * parts;
  constexpr int kWarps = kThreads / 32;
  return launch_kernel(act_load_kernel, dim3((unsigned)((warps + kWarps - 1) / kWarps)),
                       dim3(kThreads), 0, st, false, static_cast<const uint2*>(q), scales, index,
                       static_cast<uint4*>(out), rows, src_rows, nb, parts, status);
}

cudaError_t launch_swiglu_save(int rows, int f, const void* gu, void* a, void* q, float* scales,
                               cudaStream_t st) {
  // four row groups a CTA once that still leaves every SM several CTAs (16384 rows of 2048: 59 ->
  // 50 us), one below (8 rows: 2.0 us, 2.7 with four)
  const int per = tiles_of(rows, f / 128) >= 4u * 6 * 152 ? 4 : 1;
  return launch_kernel(swiglu_save_kernel, dim3(tiles_of((rows + per - 1) / per, f / 128)),
                       dim3(kThreads), 0, st, false, static_cast<const uint4*>(gu),
                       static_cast<uint4*>(a), static_cast<uint2*>(q), scales, rows, f / 128, per);
}

cudaError_t launch_swiglu_grad(int rows, int f, const void* q, const float* scales,
                               const void* da, void* dgu, void* a, cudaStream_t st) {
  return launch_kernel(swiglu_grad_kernel, dim3(tiles_of(rows, f / 128)), dim3(kThreads), 0, st,
                       false, static_cast<const uint2*>(q), scales, static_cast<const uint4*>(da),
                       static_cast<uint4*>(dgu), static_cast<uint4*>(a), rows, f / 128);
}

cudaError_t launch_combine_grad(int T, int k, int d, int rows, const void* ebuf,
                                const int32_t* row_of, const float* topk_w, const void* dy,
                                void* debuf, float* dtopk_w, uint32_t* status, cudaStream_t st) {
  const int choices = T * k;
  const bool warps = d <= 1024 || choices >= 64 * 152;
  const unsigned per = warps ? kThreads / 32 : 1;
  auto kern = warps ? combine_grad_kernel<32> : combine_grad_kernel<kThreads>;
  return launch_kernel(kern, dim3(((unsigned)choices + per - 1) / per), dim3(kThreads), 0, st,
                       false, static_cast<const uint4*>(ebuf), row_of, topk_w,
                       static_cast<const uint4*>(dy), static_cast<uint4*>(debuf), dtopk_w, choices,
                       k, d / 8, rows, status);
}

}  // namespace moe
