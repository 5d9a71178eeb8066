// Gradient of the router. With s the chosen experts' sigmoid scores, p = s / sum s and dw the gradient
// of the routing weights scale * p,
//   dz_i = scale p_i (1 - s_i) (dw_i - sum_j p_j dw_j)
// is the gradient of the k chosen logits, the only ones that the weights depend on: a sparse [T][E]
// matrix of k entries a row. Tokens take dz . w_gate, gate weights dz^T . x.
//
// 1. A CTA per chunk of tokens computes dz and lists the chunk's choices expert by expert, in the
//    order of the tokens (a counting sort).
// 2. Tokens: dx.  3. Gate weights: dw_gate, the chunks' lists one after another, so that sums have a
//    fixed order.
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 256;         // tokens of a chunk
constexpr int kMostK = 32, kMostE = 1024;

struct Layout {   // of the workspace; the status word comes first
  size_t dz, offsets, list_tok, list_dz, total;
  int chunks;
};
Layout layout(const moe_cfg& c) {
  const auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  Layout L;
  L.chunks = (c.T + kChunk - 1) / kChunk;
  const size_t tk = (size_t)c.T * c.k;
  size_t o = 256;
  L.dz = o;        o = up(o + sizeof(float) * tk);
  L.offsets = o;   o = up(o + sizeof(int32_t) * (size_t)L.chunks * (c.E + 1));
  L.list_tok = o;  o = up(o + sizeof(int32_t) * tk);
  L.list_dz = o;   o = up(o + sizeof(float) * tk);
  L.total = o;
  return L;
}

// dz of a chunk's choices, and the chunk's list: offsets[chunk][E + 1] into its part of the list
// (from chunk * kChunk * k on), the tokens and their dz. Choices outside [0, E) are in no list.
__global__ void __launch_bounds__(kThreads) route_grad_list_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ score, const float* __restrict__ dw,
    int T, int k, int E, float scale, float* __restrict__ dz, int32_t* __restrict__ offsets,
    int32_t* __restrict__ list_tok, float* __restrict__ list_dz, uint32_t* status) {
  extern __shared__ int hist[];            // [kWarps][E], then the starts of each warp's entries
  __shared__ int warp_sum[kWarps];
  const int t0 = blockIdx.x * kChunk, nt = min(kChunk, T - t0), n = nt * k;
  const size_t base = (size_t)t0 * k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  for (int t = threadIdx.x; t < nt; t += kThreads) {
    const size_t at = base + (size_t)t * k;
    float sum = 0.0f, dot = 0.0f;
    for (int i = 0; i < k; ++i) sum += score[at + i];
    const float inv = 1.0f / sum;
    for (int i = 0; i < k; ++i) dot = __fmaf_rn(score[at + i] * inv, dw[at + i], dot);
    for (int i = 0; i < k; ++i) {
      const float s = score[at + i];
      const int e = idx[at + i];
      const bool in = e >= 0 && e < E;
      if (!in && e != -1) raise_status(status, MOE_DEV_BOUNDS);
      dz[at + i] = in ? scale * (s * inv) * (1.0f - s) * (dw[at + i] - dot) : 0.0f;
    }
  }
  for (int i = threadIdx.x; i < kWarps * E; i += kThreads) hist[i] = 0;
  __syncthreads();
  // a warp counts a contiguous part of the choices
  const int per = ((n + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int lo = min(warp * per, n), hi = min(lo + per, n);
  int* mine = hist + warp * E;
  for (int b = lo; b < hi; b += 32) {
    const int i = b + lane;
    int e = i < hi ? idx[base + i] : -1;
    if (e < 0 || e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  // starts: experts in order, the warps' parts in order within each. Thread i: experts 4i .. 4i + 3
  int tot[4], own = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = threadIdx.x * 4 + q;
    tot[q] = 0;
    if (e < E)
      for (int w = 0; w < kWarps; ++w) tot[q] += hist[w * E + e];
    own += tot[q];
  }
  int incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int at = incl - own;
  for (int w = 0; w < warp; ++w) at += warp_sum[w];
  int32_t* off = offsets + (size_t)blockIdx.x * (E + 1);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = threadIdx.x * 4 + q;
    if (e >= E) break;
    off[e] = at;
    if (e == E - 1) off[E] = at + tot[q];
    int run = at;
    for (int w = 0; w < kWarps; ++w) {
      const int c = hist[w * E + e];
      hist[w * E + e] = run;
      run += c;
    }
    at = run;
  }
  __syncthreads();
  for (int b = lo; b < hi; b += 32) {
    const int i = b + lane;
    int e = i < hi ? idx[base + i] : -1;
    if (e < 0 || e >= E) e = -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const int pos = mine[e] + __popc(same & ((1u << lane) - 1u));
      list_tok[base + pos] = t0 + i / k;
      list_dz[base + pos] = dz[base + i];
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
}

// A warp: 256 columns of a token's dx.
__global__ void __launch_bounds__(kThreads) route_grad_dx_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ dz, const float* __restrict__ w_gate,
    const uint4* dx_in, uint4* dx, int T, int k, int E, int d) {
  const int vecs = d / 8, parts = (vecs + 31) / 32;
  const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long t = item / parts;
  const int v = static_cast<int>(item - t * parts) * 32 + (threadIdx.x & 31);
  if (t >= T || v >= vecs) return;
  float acc[8] = {};
  if (dx_in) {
    const uint4 u = dx_in[(size_t)t * vecs + v];
    acc[0] = bf16_lo(u.x), acc[1] = bf16_hi(u.x), acc[2] = bf16_lo(u.y), acc[3] = bf16_hi(u.y);
    acc[4] = bf16_lo(u.z), acc[5] = bf16_hi(u.z), acc[6] = bf16_lo(u.w), acc[7] = bf16_hi(u.w);
  }
  for (int i = 0; i < k; ++i) {
    const int e = idx[(size_t)t * k + i];
    if (e < 0 || e >= E) continue;
    const float z = dz[(size_t)t * k + i];
    const float4* w = reinterpret_cast<const float4*>(w_gate + (size_t)e * d) + 2 * v;
    const float4 a = w[0], b = w[1];
    acc[0] = __fmaf_rn(z, a.x, acc[0]), acc[1] = __fmaf_rn(z, a.y, acc[1]);
    acc[2] = __fmaf_rn(z, a.z, acc[2]), acc[3] = __fmaf_rn(z, a.w, acc[3]);
    acc[4] = __fmaf_rn(z, b.x, acc[4]), acc[5] = __fmaf_rn(z, b.y, acc[5]);
    acc[6] = __fmaf_rn(z, b.z, acc[6]), acc[7] = __fmaf_rn(z, b.w, acc[7]);
  }
  dx[(size_t)t * vecs + v] =
      make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                 pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
}

// A CTA: 2048 columns of one expert's dw_gate, over all chunks in order.
__global__ void __launch_bounds__(kThreads) route_grad_dw_kernel(
    const uint4* __restrict__ x, const int32_t* __restrict__ offsets,
    const int32_t* __restrict__ list_tok, const float* __restrict__ list_dz,
    float* __restrict__ dw_gate, int chunks, int k, int E, int d, bool accumulate) {
  const int vecs = d / 8, e = blockIdx.x, v = blockIdx.y * kThreads + threadIdx.x;
  if (v >= vecs) return;
  float acc[8] = {};
  for (int c = 0; c < chunks; ++c) {
    const int32_t* off = offsets + (size_t)c * (E + 1) + e;
    const size_t base = (size_t)c * kChunk * k;
    const int to = off[1];
    for (int i = off[0]; i < to; ++i) {
      const float z = list_dz[base + i];
      const uint4 u = x[(size_t)list_tok[base + i] * vecs + v];
      acc[0] = __fmaf_rn(z, bf16_lo(u.x), acc[0]), acc[1] = __fmaf_rn(z, bf16_hi(u.x), acc[1]);
      acc[2] = __fmaf_rn(z, bf16_lo(u.y), acc[2]), acc[3] = __fmaf_rn(z, bf16_hi(u.y), acc[3]);
      acc[4] = __fmaf_rn(z, bf16_lo(u.z), acc[4]), acc[5] = __fmaf_rn(z, bf16_hi(u.z), acc[5]);
      acc[6] = __fmaf_rn(z, bf16_lo(u.w), acc[6]), acc[7] = __fmaf_rn(z, bf16_hi(u.w), acc[7]);
    }
  }
  float4* o = reinterpret_cast<float4*>(dw_gate + (size_t)e * d) + 2 * v;
  float4 a = make_float4(acc[0], acc[1], acc[2], acc[3]);
  float4 b = make_float4(acc[4], acc[5], acc[6], acc[7]);
  if (accumulate) {
    const float4 p = o[0], q = o[1];
    a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    b.x += q.x, b.y += q.y, b.z += q.z, b.w += q.w;
  }
  o[0] = a;
  o[1] = b;
}

}  // namespace

size_t route_grad_ws_bytes(const moe_cfg& c) { return layout(c).total; }

cudaError_t launch_route_grad(const moe_cfg& c, const void* x, const float* w_gate,
                              const int32_t* topk_idx, const float* topk_s, const float* dtopk_w,
                              const void* dx_in, void* dx, float* dw_gate, bool accumulate,
                              void* ws, cudaStream_t st) {
  const Layout L = layout(c);
  char* w = static_cast<char*>(ws);
  float* dz = reinterpret_cast<float*>(w + L.dz);
  int32_t* offsets = reinterpret_cast<int32_t*>(w + L.offsets);
  int32_t* tok = reinterpret_cast<int32_t*>(w + L.list_tok);
  float* ldz = reinterpret_cast<float*>(w + L.list_dz);
  const int vecs = c.d / 8;
  cudaError_t e = launch_kernel(route_grad_list_kernel, dim3(L.chunks), dim3(kThreads),
                                sizeof(int) * kWarps * (size_t)c.E, st, false, topk_idx, topk_s,
                                dtopk_w, c.T, c.k, c.E, c.route_scale, dz, offsets, tok, ldz,
                                static_cast<uint32_t*>(ws));
  if (e != cudaSuccess) return e;
  const long long items = (long long)c.T * ((vecs + 31) / 32);
  e = launch_kernel(route_grad_dx_kernel, dim3((unsigned)((items + kWarps - 1) / kWarps)),
                    dim3(kThreads), 0, st, false, topk_idx, static_cast<const float*>(dz), w_gate,
                    static_cast<const uint4*>(dx_in), static_cast<uint4*>(dx), c.T, c.k, c.E, c.d);
  if (e != cudaSuccess) return e;
  return launch_kernel(route_grad_dw_kernel, dim3(c.E, (vecs + kThreads - 1) / kThreads),
                       dim3(kThreads), 0, st, false, static_cast<const uint4*>(x),
                       static_cast<const int32_t*>(offsets), static_cast<const int32_t*>(tok),
                       static_cast<const float*>(ldz), dw_gate, L.chunks, c.k, c.E, c.d, accumulate);
}

}  // namespace moe
