// Gradient of the router. With s the chosen experts' sigmoid scores, p = s / sum s and dw the
// gradient of the routing weights scale * p,
//   dz_i = scale p_i (1 - s_i) (dw_i - sum_j p_j dw_j)
// is the gradient of the k chosen logits, the only ones that the weights depend on: a sparse [T][E]
// matrix of k entries a row. Tokens take dz . w_gate, gate weights dz^T . x.
//
// 1. A CTA per chunk of tokens computes dz and lists the chunk's choices expert by expert, in the
//    order of the tokens (a counting sort).
// 2. Tokens: dx.  3. Gate weights: dw_gate.
// Both products do 2 T k d operations on operands that k choices share: their traffic to registers,
// T k d elements, is what bounds them, so long batches keep a slab of columns in shared memory (dx:
// the gate weights', dw: a chunk of the tokens') and short ones read through L2.
#include <algorithm>

#include "moe_device.cuh"
#include "moe_f32x2.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float4 four(f32x2 a, f32x2 b) {
  const float2 x = halves(a), y = halves(b);
  return make_float4(x.x, x.y, y.x, y.y);
}
__device__ __forceinline__ void copy16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------------------------------------
// Workspace
// ------------------------------------------------------------------------------------------
constexpr int kMostChunk = 320;      // tokens of a chunk
constexpr int kMostList = 2560;      // choices of a chunk
constexpr int kMostParts = 16;
constexpr int kDwCols = 64, kDwExperts = 256;   // of a CTA in dw's long form

// A choice in a chunk's list: its token in the chunk and dz. An expert's run of them starts at a
// multiple of 4 and is filled up to one with entries of token kMostChunk and dz 0, so that four
// entries have one expert; the first of the four says which, and whether they end the run.
//   at: token * 128 (the byte offset of 64 bf16 columns in a tile of x) | last | expert of the block
//   of kDwExperts << 16
struct Entry {
  uint32_t at;
  float dz;
};
__device__ __forceinline__ int entry_row(const Entry& e) { return e.at & 0xff80u; }

// A choice of a token: its expert (E: none, with dz 0), and dz. Tokens have an even number of them.
struct Pick {
  int32_t expert;
  float dz;
};

struct Layout {   // the status word comes first
  size_t picks, runs, list, partial, total;
  int chunk, chunks, kp;   // tokens of a chunk, chunks, choices of a token rounded up to even
  int stride;              // list entries of a chunk
  int parts;               // of the chunks in dw's long form; 0: the short one
};

// dw's long form: parts of the chunks, so that the last wave of CTAs is nearly full. Least waves
// times chunks of a part (one more for the sums, written and joined).
int parts_of(const moe_cfg& c, int chunks) {
  const long long units = (long long)(c.d / kDwCols) * ((c.E + kDwExperts - 1) / kDwExperts);
  int parts = 1;
  long long best = -1;
  for (int p = 1; p <= kMostParts && p <= chunks; ++p) {
    const long long waves = (units * p + kSms - 1) / kSms;
    const long long cost = waves * ((chunks + p - 1) / p + 1);
    if (best < 0 || cost < best) best = cost, parts = p;
  }
  return parts;
}

Layout layout(const moe_cfg& c) {
  const auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  Layout L;
  L.chunk = kMostList / c.k < kMostChunk ? kMostList / c.k / 8 * 8 : kMostChunk;
  L.chunks = (int)(((long long)c.T + L.chunk - 1) / L.chunk);
  L.kp = (c.k + 1) / 2 * 2;
  size_t o = 256;
  L.picks = o;     o = up(o + sizeof(Pick) * (size_t)c.T * L.kp);
  L.runs = o;      o = up(o + sizeof(int2) * (size_t)L.chunks * c.E);
  L.stride = (L.chunk * c.k + 3 * std::min(c.E, L.chunk * c.k) + 3) / 4 * 4;
  L.list = o;      o = up(o + sizeof(Entry) * (size_t)L.chunks * L.stride);
  // The long forms from 512 tokens on (7168 columns, 8 of 256 experts, us, short and long: 256 tokens
  // 27 and 36, 512 36 and 44, 1024 55 and 57, 2048 87 and 81, 4096 152 and 130, evenly loaded; with
  // one expert chosen by half of the tokens the short form takes twice as long, the long one does not).
  L.parts = c.T >= 512 ? parts_of(c, L.chunks) : 0;
  L.partial = o;   o = up(o + (L.parts > 1 ? sizeof(float) * (size_t)L.parts * c.E * c.d : 0));
  L.total = o;
  return L;
}

// ------------------------------------------------------------------------------------------
// 1. dz, the tokens' picks, and each chunk's list: runs[chunk][expert] is the start and the end of the
// expert's run. Choices outside [0, E) are in no list; a token's second choice of one expert is added
// to its first.
//
// The order inside a run is that of the tokens: a bit mask of them for each expert (set by atomic
// ORs, whose order does not matter) gives a choice's place by counting the bits below its own.
// ------------------------------------------------------------------------------------------
constexpr int kListThreads = 512, kListWarps = kListThreads / 32;
constexpr int kMaskWords = kMostChunk / 32, kMaskStride = kMaskWords + 1;   // (odd: bank conflicts)
struct ListSmem {
  int expert[kMostList];
  float dz[kMostList], grad[kMostList];
};
__global__ void __launch_bounds__(kListThreads) route_grad_list_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ score, const float* __restrict__ dw,
    int T, int k, int kp, int E, float scale, int chunk, int stride, Pick* __restrict__ picks,
    int2* __restrict__ runs, Entry* __restrict__ list, uint32_t* status) {
  extern __shared__ __align__(16) char raw[];
  __shared__ int warp_sum[kListWarps];
  ListSmem& sm = *reinterpret_cast<ListSmem*>(raw);
  int* expert = sm.expert;
  float *dz = sm.dz, *grad = sm.grad;
  uint32_t* mask = reinterpret_cast<uint32_t*>(raw + sizeof(ListSmem));   // [E][kMaskStride]
  int2* run = reinterpret_cast<int2*>(grad);                               // [E], from the scan on
  const int t0 = blockIdx.x * chunk, nt = min(chunk, T - t0), n = nt * k;
  const size_t base = (size_t)t0 * k;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  for (int i = threadIdx.x; i < n; i += kListThreads) {
    const int e = idx[base + i];
    const bool in = e >= 0 && e < E;
    if (!in && e != -1) raise_status(status, MOE_DEV_BOUNDS);
    expert[i] = in ? e : -1;
    dz[i] = score[base + i];
    grad[i] = dw[base + i];
  }
  for (int i = threadIdx.x; i < E * kMaskStride; i += kListThreads) mask[i] = 0;
  __syncthreads();
  pdl_trigger();
  bool twice = false;
  for (int i = threadIdx.x; i < n; i += kListThreads) {
    const int e = expert[i], t = i / k;
    if (e < 0) continue;
    const uint32_t bit = 1u << (t & 31);
    twice |= (atomicOr(&mask[e * kMaskStride + (t >> 5)], bit) & bit) != 0;
  }
  for (int t = threadIdx.x; t < nt; t += kListThreads) {
    float *s = dz + t * k, *g = grad + t * k;
    float sum = 0.0f, dot = 0.0f;
    for (int i = 0; i < k; ++i) sum += s[i];
    const float inv = 1.0f / sum;
    for (int i = 0; i < k; ++i) dot = __fmaf_rn(s[i] * inv, g[i], dot);
    for (int i = 0; i < k; ++i)
      s[i] = expert[t * k + i] >= 0 ? scale * (s[i] * inv) * (1.0f - s[i]) * (g[i] - dot) : 0.0f;
  }
  if (__syncthreads_or(twice)) {
    for (int t = threadIdx.x; t < nt; t += kListThreads)
      for (int i = t * k + 1; i < (t + 1) * k; ++i)
        for (int j = t * k; j < i && expert[i] >= 0; ++j)
          if (expert[j] == expert[i]) {
            dz[j] += dz[i];
            dz[i] = 0.0f;
            expert[i] = -1;
          }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < nt * kp; i += kListThreads) {
    const int t = i / kp, j = i - t * kp;
    const int e = j < k ? expert[t * k + j] : -1;
    picks[(size_t)(t0 + t) * kp + j] = e >= 0 ? Pick{e, dz[t * k + j]} : Pick{E, 0.0f};
  }
  // starts of the runs. Thread i: experts 2i, 2i + 1
  int count[2], own = 0;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = threadIdx.x * 2 + q;
    count[q] = 0;
    if (e < E)
      for (int w = 0; w < kMaskWords; ++w) count[q] += __popc(mask[e * kMaskStride + w]);
    own += (count[q] + 3) / 4 * 4;
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
  Entry* out = list + (size_t)blockIdx.x * stride;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int e = threadIdx.x * 2 + q;
    if (e >= E) break;
    run[e] = make_int2(at, at + count[q]);
    runs[(size_t)blockIdx.x * E + e] = run[e];
    for (int i = count[q]; i & 3; ++i) out[at + i] = Entry{(uint32_t)kMostChunk * 128, 0.0f};
    at += (count[q] + 3) / 4 * 4;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kListThreads) {
    const int e = expert[i], t = i / k;
    if (e < 0) continue;
    const uint32_t* m = mask + e * kMaskStride;
    int rank = __popc(m[t >> 5] & ((1u << (t & 31)) - 1u));
    for (int w = 0; w < t >> 5; ++w) rank += __popc(m[w]);
    const int2 r = run[e];
    const uint32_t last = r.x + rank + 4 >= r.y ? 1u : 0u;
    out[r.x + rank] = Entry{(uint32_t)(t * 128) | last | (uint32_t)(e % kDwExperts) << 16, dz[i]};
  }
}

// ------------------------------------------------------------------------------------------
// 2. dx
// ------------------------------------------------------------------------------------------
// A warp takes 256 columns of a token, the gate weights come from L2.
__device__ __forceinline__ void dx_short(const Pick* __restrict__ picks,
                                         const float* __restrict__ w_gate, const uint4* dx_in,
                                         uint4* dx, int T, int kp, int E, int d, long long item) {
  const int vecs = d / 8, parts = (vecs + 31) / 32;
  const long long t = item / parts;
  const int v = static_cast<int>(item - t * parts) * 32 + (threadIdx.x & 31);
  if (t >= T || v >= vecs) return;
  f32x2 acc[4] = {};
  if (dx_in) {
    const uint4 u = dx_in[(size_t)t * vecs + v];
    acc[0] = pair_of_bf16(u.x);
    acc[1] = pair_of_bf16(u.y);
    acc[2] = pair_of_bf16(u.z);
    acc[3] = pair_of_bf16(u.w);
  }
  const int4* two = reinterpret_cast<const int4*>(picks + (size_t)t * kp);
#pragma unroll 4
  for (int i = 0; i < kp / 2; ++i) {
    const int4 p = two[i];   // expert, dz, expert, dz
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = j ? p.z : p.x;
      const f32x2 z2 = both(__int_as_float(j ? p.w : p.y));
      if (e == E) continue;
      const float4* w = reinterpret_cast<const float4*>(w_gate + (size_t)e * d) + 2 * v;
      const float4 a = w[0], b = w[1];
      acc[0] = fma2(z2, pair(a.x, a.y), acc[0]);
      acc[1] = fma2(z2, pair(a.z, a.w), acc[1]);
      acc[2] = fma2(z2, pair(b.x, b.y), acc[2]);
      acc[3] = fma2(z2, pair(b.z, b.w), acc[3]);
    }
  }
  dx[(size_t)t * vecs + v] =
      make_uint4(bf16_of_pair(acc[0]), bf16_of_pair(acc[1]),
                 bf16_of_pair(acc[2]), bf16_of_pair(acc[3]));
}

// A warp takes 256 columns of one expert's gate weights, over all chunks in order; x comes from L2.
__device__ __forceinline__ void dw_short(const uint4* __restrict__ x,
                                         const int2* __restrict__ runs,
                                         const Entry* __restrict__ list,
                                         float* __restrict__ dw_gate, int chunk, int chunks,
                                         int stride, int E, int d, bool accumulate,
                                         long long item) {
  const int vecs = d / 8, parts = (vecs + 31) / 32;
  const int e = static_cast<int>(item / parts);
  const int v = static_cast<int>(item - (long long)e * parts) * 32 + (threadIdx.x & 31);
  if (e >= E || v >= vecs) return;
  f32x2 acc[4] = {};
  for (int c = 0; c < chunks; ++c) {
    const int2 run = runs[(size_t)c * E + e];
    const Entry* in = list + (size_t)c * stride;
    const uint4* rows = x + (size_t)c * chunk * vecs + v;
#pragma unroll 4
    for (int i = run.x; i < run.y; ++i) {
      const Entry q = in[i];
      const uint4 u = rows[(size_t)(entry_row(q) >> 7) * vecs];
      acc[0] = fma2(both(q.dz), pair_of_bf16(u.x), acc[0]);
      acc[1] = fma2(both(q.dz), pair_of_bf16(u.y), acc[1]);
      acc[2] = fma2(both(q.dz), pair_of_bf16(u.z), acc[2]);
      acc[3] = fma2(both(q.dz), pair_of_bf16(u.w), acc[3]);
    }
  }
  float4* o = reinterpret_cast<float4*>(dw_gate + (size_t)e * d) + 2 * v;
  float4 a = four(acc[0], acc[1]), b = four(acc[2], acc[3]);
  if (accumulate) {
    const float4 p = o[0], q = o[1];
    a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
    b.x += q.x, b.y += q.y, b.z += q.z, b.w += q.w;
  }
  o[0] = a;
  o[1] = b;
}

// Short batches: both products in one launch, dx by the first dx_ctas CTAs.
__global__ void __launch_bounds__(kThreads) route_grad_short_kernel(
    const Pick* __restrict__ picks, const int2* __restrict__ runs, const Entry* __restrict__ list, const float* __restrict__ w_gate, const uint4* __restrict__ x,
    const uint4* dx_in, uint4* dx, float* __restrict__ dw_gate, int T, int kp, int E, int d,
    int chunk, int chunks, int stride, bool accumulate, unsigned dx_ctas) {
  pdl_wait();
  const int warp = threadIdx.x >> 5;
  if (blockIdx.x < dx_ctas)
    dx_short(picks, w_gate, dx_in, dx, T, kp, E, d, (long long)blockIdx.x * kWarps + warp);
  else
    dw_short(x, runs, list, dw_gate, chunk, chunks, stride, E, d, accumulate,
             (long long)(blockIdx.x - dx_ctas) * kWarps + warp);
}

// Long batches: a CTA keeps C columns of all gate weights in shared memory, and a row of zeros for
// picks that are none. The (slab of columns, token) pairs, slab by slab, are dealt to the CTAs in
// equal runs, so that a CTA loads one slab or two. C / 16 lanes take a token, 16 columns a lane, so
// that the picks, which all of a token's lanes read, cost little beside the weights.
constexpr int kDxThreads = 512;
template <int C>
__global__ void __launch_bounds__(kDxThreads, 1) route_grad_dx_slab_kernel(
    const Pick* __restrict__ picks, const float* __restrict__ w_gate, const uint4* dx_in, uint4* dx,
    int T, int kp, int E, int d, long long per_cta) {
  extern __shared__ __align__(16) char slab[];
  // a row: the lanes' columns 0-3 one after another, then their columns 4-7, 8-11, 12-15
  constexpr int kLanes = C / 16, kAtOnce = kDxThreads / kLanes, kRow = C * 4, kQuarter = C;
  const long long work = (long long)(d / C) * T;
  long long at = blockIdx.x * per_cta;
  const long long end = min(at + per_cta, work);
  const int l = threadIdx.x % kLanes, mine = threadIdx.x / kLanes;
  for (int i = threadIdx.x; i < C; i += kDxThreads)
    reinterpret_cast<float*>(slab + (size_t)E * kRow)[i] = 0.0f;
  pdl_wait();
  pdl_trigger();
  while (at < end) {
    const int s = static_cast<int>(at / T), t0 = static_cast<int>(at - (long long)s * T);
    const int t1 = static_cast<int>(min((long long)T, t0 + (end - at)));
    __syncthreads();   // the slab before this one has been read
    for (int i = threadIdx.x; i < E * (C / 4); i += kDxThreads) {
      const int e = i / (C / 4), v = i % (C / 4);
      copy16(slab + (size_t)e * kRow + (v & 3) * kQuarter + (v >> 2) * 16,
             w_gate + (size_t)e * d + s * C + v * 4);
    }
    copies_commit();
    copies_wait<0>();
    __syncthreads();
    const char* w = slab + l * 16;
    const size_t col = (size_t)s * (C / 8) + l * 2;
    // a token's dx_in and first eight picks are loaded while the one before it is worked on
    uint4 u_next[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    int4 p_next[4];
    const auto fetch = [&](int t) {
      if (dx_in) {
        u_next[0] = dx_in[(size_t)t * (d / 8) + col];
        u_next[1] = dx_in[(size_t)t * (d / 8) + col + 1];
      }
      const int4* p = reinterpret_cast<const int4*>(picks + (size_t)t * kp);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < kp) p_next[i] = p[i];
    };
    if (t0 + mine < t1) fetch(t0 + mine);
    for (int t = t0 + mine; t < t1; t += kAtOnce) {
      f32x2 acc[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 u = u_next[i];
        acc[4 * i] = pair_of_bf16(u.x);
        acc[4 * i + 1] = pair_of_bf16(u.y);
        acc[4 * i + 2] = pair_of_bf16(u.z);
        acc[4 * i + 3] = pair_of_bf16(u.w);
      }
      int4 p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = p_next[i];
      if (t + kAtOnce < t1) fetch(t + kAtOnce);
      const auto add = [&](int e, float z) {
        const f32x2 z2 = both(z);
        const char* row = w + e * kRow;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(row + i * kQuarter);
          acc[2 * i] = fma2(z2, pair(x.x, x.y), acc[2 * i]);
          acc[2 * i + 1] = fma2(z2, pair(x.z, x.w), acc[2 * i + 1]);
        }
      };
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (2 * i < kp) {
          add(p[i].x, __int_as_float(p[i].y));
          add(p[i].z, __int_as_float(p[i].w));
        }
      for (int i = 4; i < kp / 2; ++i) {
        const int4 q = reinterpret_cast<const int4*>(picks + (size_t)t * kp)[i];
        add(q.x, __int_as_float(q.y));
        add(q.z, __int_as_float(q.w));
      }
      uint4* o = dx + (size_t)t * (d / 8) + col;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        o[i] = make_uint4(bf16_of_pair(acc[4 * i]),
                          bf16_of_pair(acc[4 * i + 1]),
                          bf16_of_pair(acc[4 * i + 2]),
                          bf16_of_pair(acc[4 * i + 3]));
    }
    at += t1 - t0;
  }
}

// ------------------------------------------------------------------------------------------
// 3. dw_gate, long batches: a CTA takes 64 columns of up to 256 experts over a part of the chunks;
// their sums are in shared memory, and so are, for the present chunk and the next, x's tile and the
// list. Each 8 lanes take an equal part of the list, however the experts are loaded: 8 columns a
// lane, a run of one expert's choices added up in registers and then added to the expert's sums. A
// part's first run may belong to the expert that the part before it ends with: its sum goes to a side
// row, and the side rows are added in order after the chunk.
// ------------------------------------------------------------------------------------------
constexpr int kDwThreads = 512, kDwSlices = kDwThreads / 8;
struct DwSmem {
  float sums[kDwExperts][kDwCols];   // columns 8j .. 8j + 3 at 4j, 8j + 4 .. 8j + 7 at 32 + 4j
  char tile[2][(kMostChunk + 1) * 128];   // the last row: zeros
  Entry list[2][kMostList + 3 * kDwExperts];
  float side[kDwSlices][kDwCols];    // as sums
  int side_expert[kDwSlices];
  int entries[2];                    // of the block's experts in the list
};
static_assert(sizeof(DwSmem) <= 227 * 1024, "one CTA an SM");

__global__ void __launch_bounds__(kDwThreads, 1) route_grad_dw_slab_kernel(
    const char* __restrict__ x, const int2* __restrict__ runs, const Entry* __restrict__ list,
    float* __restrict__ out, int T, int chunk, int chunks,
    int stride, int k, int E, int d, int parts, bool accumulate) {
  extern __shared__ __align__(16) char raw[];
  DwSmem& sm = *reinterpret_cast<DwSmem*>(raw);
  const int lane = threadIdx.x & 31, l = threadIdx.x & 7, slice = threadIdx.x >> 3;
  const int col0 = blockIdx.x * kDwCols, e0 = blockIdx.y * kDwExperts, ne = min(kDwExperts, E - e0);
  const int part = blockIdx.z;
  const int c0 = (int)((long long)chunks * part / parts);
  const int c1 = (int)((long long)chunks * (part + 1) / parts);
  for (int i = threadIdx.x; i < kDwExperts * kDwCols; i += kDwThreads) sm.sums[0][i] = 0.0f;
  if (threadIdx.x < 16)
    *reinterpret_cast<uint4*>(sm.tile[threadIdx.x >> 3] + kMostChunk * 128 + l * 16) =
        make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();

  const auto fetch = [&](int c, int b) {
    const int t0 = c * chunk, nt = min(chunk, T - t0);
    const int2* run = runs + (size_t)c * E + e0;
    const int from = run[0].x, to = (run[ne - 1].y + 3) / 4 * 4;
    if (threadIdx.x == 0) sm.entries[b] = to - from;
    for (int i = threadIdx.x; i < nt * 8; i += kDwThreads)
      copy16(sm.tile[b] + i * 16,
             x + ((size_t)(t0 + (i >> 3)) * d + col0) * 2 + (size_t)(i & 7) * 16);
    const Entry* in = list + (size_t)c * stride + from;
    for (int i = threadIdx.x; i < (to - from) / 2; i += kDwThreads)
      copy16(&sm.list[b][2 * i], in + 2 * i);
    copies_commit();
  };
  if (c0 < c1) fetch(c0, 0);
  for (int c = c0; c < c1; ++c) {
    const int b = (c - c0) & 1;
    if (c + 1 < c1)
      fetch(c + 1, b ^ 1);
    else
      copies_commit();
    copies_wait<1>();
    __syncthreads();
    // fours of entries of this slice
    const int n = sm.entries[b] / 4, per = (n + kDwSlices - 1) / kDwSlices;
    const int begin = min(slice * per, n), end = min(begin + per, n);
    const Entry* in = sm.list[b];
    const char* tile = sm.tile[b] + l * 16;
    // the run that comes in from the slice before, if it does: its sum goes to the side row
    bool head = begin > 0 && begin < end && !(in[4 * begin - 4].at & 1);
    int side = -1;
    f32x2 acc[4] = {};
    for (int at = begin; at < end; ++at) {
      Entry q[4];
      uint4 u[4];
      {
        const int4 a = *reinterpret_cast<const int4*>(in + 4 * at);
        const int4 h = *reinterpret_cast<const int4*>(in + 4 * at + 2);
        q[0] = Entry{(uint32_t)a.x, __int_as_float(a.y)};
        q[1] = Entry{(uint32_t)a.z, __int_as_float(a.w)};
        q[2] = Entry{(uint32_t)h.x, __int_as_float(h.y)};
        q[3] = Entry{(uint32_t)h.z, __int_as_float(h.w)};
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = *reinterpret_cast<const uint4*>(tile + entry_row(q[i]));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0] = fma2(both(q[i].dz), pair_of_bf16(u[i].x), acc[0]);
        acc[1] = fma2(both(q[i].dz), pair_of_bf16(u[i].y), acc[1]);
        acc[2] = fma2(both(q[i].dz), pair_of_bf16(u[i].z), acc[2]);
        acc[3] = fma2(both(q[i].dz), pair_of_bf16(u[i].w), acc[3]);
      }
      if ((q[0].at & 1) || at == end - 1) {   // the run ends here, or goes on in the next slice
        const int e = q[0].at >> 16;
        float4* to = reinterpret_cast<float4*>(head ? sm.side[slice] : sm.sums[e]) + l;
        float4 a = four(acc[0], acc[1]), h = four(acc[2], acc[3]);
        if (head) {
          side = e;
        } else {
          const float4 p = to[0], r = to[8];
          a.x += p.x, a.y += p.y, a.z += p.z, a.w += p.w;
          h.x += r.x, h.y += r.y, h.z += r.z, h.w += r.w;
        }
        to[0] = a;
        to[8] = h;
        head = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = 0;
      }
    }
    if (l == 0) sm.side_expert[slice] = side;
    __syncthreads();
    {   // the side rows of experts e % 8 = mine by the same threads, in order
      const int col = threadIdx.x % kDwCols, mine = threadIdx.x / kDwCols;
      const int ea = sm.side_expert[lane], eb = sm.side_expert[32 + lane];
      uint32_t ma = __ballot_sync(0xffffffffu, ea >= 0 && ea % 8 == mine);
      uint32_t mb = __ballot_sync(0xffffffffu, eb >= 0 && eb % 8 == mine);
      while (ma | mb) {
        const int w = ma ? __ffs(ma) - 1 : 31 + __ffs(mb);
        if (ma)
          ma &= ma - 1;
        else
          mb &= mb - 1;
        sm.sums[sm.side_expert[w]][col] += sm.side[w][col];
      }
    }
    __syncthreads();
  }
  __syncthreads();
  float* to = out + (size_t)part * E * d;
  for (int i = threadIdx.x; i < ne * (kDwCols / 4); i += kDwThreads) {
    const int e = i / (kDwCols / 4), v = i % (kDwCols / 4);
    float4 s = reinterpret_cast<const float4*>(sm.sums[e])[(v & 1) * 8 + (v >> 1)];
    float4* o = reinterpret_cast<float4*>(to + (size_t)(e0 + e) * d + col0) + v;
    if (accumulate) {
      const float4 p = *o;
      s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
    }
    *o = s;
  }
}

// The parts' sums, in order.
__global__ void __launch_bounds__(kThreads) route_grad_join_kernel(
    const float4* __restrict__ partial, float4* __restrict__ dw_gate, size_t n, int parts,
    bool accumulate) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  pdl_wait();
  if (i >= n) return;
  float4 s = partial[i];
  const auto add = [&](const float4& v) { s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w; };
#pragma unroll 4
  for (int p = 1; p < parts; ++p) add(partial[(size_t)p * n + i]);
  if (accumulate) add(dw_gate[i]);
  dw_gate[i] = s;
}

template <int C>
cudaError_t dx_slab(const moe_cfg& c, const Pick* picks, const float* w_gate, const void* dx_in,
                    void* dx, int kp, cudaStream_t st) {
  auto kern = route_grad_dx_slab_kernel<C>;
  const size_t smem = (size_t)(c.E + 1) * C * 4;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  const long long work = (long long)(c.d / C) * c.T;
  const long long per = (work + kSms - 1) / kSms;
  return launch_kernel(kern, dim3((unsigned)((work + per - 1) / per)), dim3(kDxThreads), smem, st,
                       true, picks, w_gate, static_cast<const uint4*>(dx_in),
                       static_cast<uint4*>(dx), c.T, kp, c.E, c.d, per);
}

}  // namespace

size_t route_grad_ws_bytes(const moe_cfg& c) { return layout(c).total; }

cudaError_t launch_route_grad(const moe_cfg& c, const void* x, const float* w_gate,
                              const int32_t* topk_idx, const float* topk_s, const float* dtopk_w,
                              const void* dx_in, void* dx, float* dw_gate, bool accumulate,
                              void* ws, cudaStream_t st) {
  const Layout L = layout(c);
  char* w = static_cast<char*>(ws);
  Pick* picks = reinterpret_cast<Pick*>(w + L.picks);
  int2* runs = reinterpret_cast<int2*>(w + L.runs);
  Entry* list = reinterpret_cast<Entry*>(w + L.list);
  float* partial = reinterpret_cast<float*>(w + L.partial);
  const size_t masks = sizeof(ListSmem) + sizeof(uint32_t) * kMaskStride * (size_t)c.E;
  cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(route_grad_list_kernel),
                                    masks + 1024);   // (the static array counts, too)
  if (e != cudaSuccess) return e;
  e = launch_kernel(route_grad_list_kernel, dim3(L.chunks), dim3(kListThreads), masks, st, false,
                    topk_idx, topk_s, dtopk_w, c.T, c.k, L.kp, c.E, c.route_scale, L.chunk, L.stride,
                    picks, runs, list, static_cast<uint32_t*>(ws));
  if (e != cudaSuccess) return e;
  const Pick* pk = picks;
  const int2* rn = runs;
  const Entry* ls = list;
  if (L.parts == 0) {
    const long long parts = (c.d / 8 + 31) / 32;
    const auto ctas = [](long long warps) { return (unsigned)((warps + kWarps - 1) / kWarps); };
    const unsigned dx_ctas = ctas(c.T * parts);
    return launch_kernel(route_grad_short_kernel, dim3(dx_ctas + ctas(c.E * parts)), dim3(kThreads),
                         0, st, true, pk, rn, ls, w_gate, static_cast<const uint4*>(x),
                         static_cast<const uint4*>(dx_in), static_cast<uint4*>(dx), dw_gate, c.T,
                         L.kp, c.E, c.d, L.chunk, L.chunks, L.stride, accumulate, dx_ctas);
  }
  const size_t row = 4 * (size_t)(c.E + 1);
  e = row * 128 <= 227 * 1024  ? dx_slab<128>(c, pk, w_gate, dx_in, dx, L.kp, st)
      : row * 64 <= 227 * 1024 ? dx_slab<64>(c, pk, w_gate, dx_in, dx, L.kp, st)
                               : dx_slab<32>(c, pk, w_gate, dx_in, dx, L.kp, st);
  if (e != cudaSuccess) return e;
  const int slabs = c.d / kDwCols, blocks = (c.E + kDwExperts - 1) / kDwExperts;
  e = ensure_smem_limit(reinterpret_cast<const void*>(route_grad_dw_slab_kernel), sizeof(DwSmem));
  if (e != cudaSuccess) return e;
  e = launch_kernel(route_grad_dw_slab_kernel, dim3(slabs, blocks, L.parts), dim3(kDwThreads),
                    sizeof(DwSmem), st, true, static_cast<const char*>(x), rn, ls,
                    L.parts > 1 ? partial : dw_gate, c.T, L.chunk, L.chunks, L.stride, c.k, c.E, c.d,
                    L.parts, L.parts == 1 && accumulate);
  if (e != cudaSuccess || L.parts == 1) return e;
  const size_t n = (size_t)c.E * c.d / 4;
  return launch_kernel(route_grad_join_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, st, true, reinterpret_cast<const float4*>(partial),
                       reinterpret_cast<float4*>(dw_gate), n, L.parts, accumulate);
}

}  // namespace moe
