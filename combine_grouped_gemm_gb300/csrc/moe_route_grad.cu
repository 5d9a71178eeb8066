// Gradient of the router. With s the chosen experts' sigmoid scores, p = s / sum s and dw the
// gradient of the routing weights scale * p,
//   dz_i = scale p_i (1 - s_i) (dw_i - sum_j p_j dw_j)
// is the gradient of the k chosen logits, the only ones that the weights depend on: a sparse [T][E]
// matrix of k entries a row. Tokens take dz . w_gate, gate weights dz^T . x. Both products do 2 T k
// d operations on operands that several choices share, so what bounds them is the operands' way
// into registers: T k d elements each, fp32 for the tokens and bf16 for the gate weights. (As dense
// products on the tensor cores, fp32 factors as sums of two or three bf16 ones, they would be six
// products of 2 T E d operations, 190 us at the rate of the library's for the batch below, without
// the rest.)
//
// 1. Counts: a CTA per chunk of tokens computes dz and counts the chunk's choices of each expert.
// 2. Lists: the choices expert by expert, in the order of the tokens, cut into segments.
// 3. Products: the tokens' dx from the gate weights (long batches: from a slab of their columns in
//    shared memory), the segments' sums of x from L2, at the same time.
// 4. The segments' sums are joined in order: the result does not depend on the order of work.
// A short batch takes one launch for all of it.
//
// Measured, d = 7168, 256 experts, 8 choices: 16384 tokens 247 us, 2048 tokens 51 (count 4, lists 3,
// products 42, join 2), 64 tokens 8.6. The 16384 tokens' operands are 5.6 GB on their way through
// the SMs' shared memory and L1, 155 us at 128 bytes a clock and SM, of which L2 hands out the
// segments' rows at some 8 TB/s. (Tokens and gate weights one after the other, the latter summed
// chunk by chunk in shared memory: 370 us; first form 3431.)
#include <algorithm>

#include "moe_device.cuh"
#include "moe_f32x2.cuh"

namespace moe {
namespace {

constexpr int kSms = 152;

__device__ __forceinline__ void copy16(void* smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem)
               : "memory");
}

// ------------------------------------------------------------------------------------------
// Workspace
// ------------------------------------------------------------------------------------------
constexpr int kMostChunk = 320;      // tokens of a chunk
constexpr int kMostList = 2560;      // choices of a chunk
constexpr int kShortChoices = 512;   // of a batch that takes one launch, at most

// A choice of a token: its expert (E: none, with dz 0), and dz. Tokens have an even number of them.
struct Pick {
  int32_t expert;
  float dz;
};
// A choice in the lists.
struct Entry {
  int32_t token;
  float dz;
};

struct Layout {   // the status word comes first
  size_t queue;      // int32: the next item of the products' work
  size_t picks;      // Pick [T][kp]
  size_t counts;     // int32 [chunks][E]
  size_t starts;     // int32 [E + 1]: of the experts' lists
  size_t segments;   // int32 [E + 1]: the experts' first segments
  size_t list;       // Entry [T * k]
  size_t partial;    // fp32 [segments][d]: sums of the segments of experts with several
  size_t total;
  int chunk, chunks, kp;   // tokens of a chunk, chunks, choices of a token rounded up to even
  int segment;             // choices of a segment
  bool one_launch;
};

Layout layout(const moe_cfg& c) {
  const auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  Layout L;
  const size_t tk = (size_t)c.T * c.k;
  // 64 chunks, of 64 tokens at least: 2048 tokens' counts and lists take 3.7 + 6.3 us in chunks of
  // 64,
  // 8.4 + 13 in chunks of 320, 3.7 + 8.2 in chunks of 32 (whose counts are more to add up)
  L.chunk = std::min({std::max((c.T + 63) / 64, 64), kMostList / c.k, kMostChunk}) / 8 * 8;
  L.chunks = (int)(((long long)c.T + L.chunk - 1) / L.chunk);
  L.kp = (c.k + 1) / 2 * 2;
  // a segment: a power of two from 32 to 128 that leaves each of the products' warps one to work on
  // (1500 tokens of 8 choices, 16 experts, 256 columns: 22 us, with segments of 128 30; 2048 tokens,
  // 256 experts, 7168 columns: 59 us in segments of 128, 64 of 32, which have to be joined); above, up
  // to 1024, the work of the SMs' warps some eight times over (16384 tokens of those: 280 us in
  // segments of 128, 297 of 256)
  const double work = (double)tk * ((c.d + 255) / 256), warps = kSms * 16;
  L.segment = 32;
  while (L.segment < 128 && work / (2 * L.segment) >= warps) L.segment *= 2;
  while (L.segment >= 128 && L.segment < 1024 && work / L.segment > 16 * warps) L.segment *= 2;
  L.one_launch = tk <= kShortChoices;
  size_t o = 256;
  L.queue = o;     o = up(o + sizeof(int32_t));
  if (!L.one_launch) {
    L.picks = o;     o = up(o + sizeof(Pick) * (size_t)c.T * L.kp);
    L.counts = o;    o = up(o + sizeof(int32_t) * (size_t)L.chunks * c.E);
    L.starts = o;    o = up(o + sizeof(int32_t) * (c.E + 1));
    L.segments = o;  o = up(o + sizeof(int32_t) * (c.E + 1));
    L.list = o;      o = up(o + sizeof(Entry) * tk);
    L.partial = o;   o = up(o + sizeof(float) * (tk / L.segment + c.E) * c.d);
  }
  L.total = o;
  return L;
}

__device__ __forceinline__ int checked(int e, int E, uint32_t* status) {
  if (e >= 0 && e < E) return e;
  if (e != -1) raise_status(status, MOE_DEV_BOUNDS);
  return -1;
}

// Lanes that take a token's choices, one each: a power of two, kp at least.
__host__ __device__ __forceinline__ int lanes_of(int kp) {
  int w = 2;
  while (w < kp) w *= 2;
  return w;
}
// A choice and its dz, from its lane's expert (-1: none), score and gradient of the weight; `in`:
// there is such a choice. A second choice of one expert is added to its first and becomes none
// itself. The lanes of a token are neighbours, `width` of them; all lanes of the warp take part.
__device__ __forceinline__ Pick pick_of(int e, float s, float g, bool in, int width, float scale,
                                        int E) {
  const auto sum_of_token = [&](float v) {
    for (int o = width / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  };
  // (a quotient: the reciprocal of a sum below 3e-39, of logits near -90, would be infinite)
  const float p = __fdiv_rn(s, sum_of_token(in ? s : 0.0f));
  const float dot = sum_of_token(in ? p * g : 0.0f);
  const bool live = in && e >= 0;
  if (!live) e = -1;
  const float z = live ? scale * p * (1.0f - s) * (g - dot) : 0.0f;
  float mine = z;
  bool second = false;
  const int lane = threadIdx.x & 31;
  for (int o = 1; o < width; ++o) {
    const int other = __shfl_xor_sync(0xffffffffu, e, o);
    const float add = __shfl_xor_sync(0xffffffffu, z, o);
    if (live && other == e) {
      if ((lane ^ o) < lane)
        second = true;
      else
        mine += add;
    }
  }
  return live && !second ? Pick{e, mine} : Pick{E, 0.0f};
}

// ------------------------------------------------------------------------------------------
// 1. dz, the tokens' picks, the chunk's counts
// ------------------------------------------------------------------------------------------
constexpr int kListThreads = 512, kListWarps = kListThreads / 32;
// (a token has at most twice as many lanes as choices)
constexpr int kPasses = 2 * kMostList / kListThreads;

__global__ void __launch_bounds__(kListThreads) route_grad_count_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ score, const float* __restrict__ dw,
    int T, int k, int kp, int E, float scale, int chunk, Pick* __restrict__ picks,
    int32_t* __restrict__ counts, int32_t* queue, uint32_t* status) {
  __shared__ int hist[1024];
  const int t0 = blockIdx.x * chunk, nt = min(chunk, T - t0);
  const int width = lanes_of(kp), j = threadIdx.x & (width - 1), per = kListThreads / width;
  for (int e = threadIdx.x; e < E; e += kListThreads) hist[e] = 0;
  if (blockIdx.x == 0 && threadIdx.x == 0) *queue = 0;
  __syncthreads();
  pdl_trigger();
  // a chunk takes kPasses rounds at most: all their loads first
  int e[kPasses];
  float s[kPasses], g[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * per + threadIdx.x / width;
    e[i] = -1, s[i] = g[i] = 0.0f;
    if (t < nt && j < k) {
      const size_t at = (size_t)(t0 + t) * k + j;
      e[i] = checked(idx[at], E, status), s[i] = score[at], g[i] = dw[at];
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    if (i * per >= nt) break;   // whole warps
    const int t = i * per + threadIdx.x / width;
    const Pick p = pick_of(e[i], s[i], g[i], t < nt && j < k, width, scale, E);
    if (t >= nt || j >= kp) continue;
    if (p.expert < E) atomicAdd(&hist[p.expert], 1);
    picks[(size_t)(t0 + t) * kp + j] = p;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kListThreads) counts[(size_t)blockIdx.x * E + e] = hist[e];
}

// ------------------------------------------------------------------------------------------
// 2. The lists. A choice's place: its expert's start, the choices of the chunks before, and those
// of its own chunk's tokens before, counted in a bit mask of the expert's tokens (set by atomic
// ORs, whose order does not matter). Every CTA adds up all counts for itself; the first one writes
// the starts.
// ------------------------------------------------------------------------------------------
constexpr int kOwn = (kMostList + kMostChunk) / kListThreads + 1;   // picks of a thread, at most
constexpr int kMaskWords = kMostChunk / 32, kMaskStride = kMaskWords + 1;   // (odd: bank conflicts)

// Exclusive sums of two numbers over the CTA's threads.
__device__ __forceinline__ int2 cta_scan(int2 own, int2* warp_sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int2 incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, o);
    const int y = __shfl_up_sync(0xffffffffu, incl.y, o);
    if (lane >= o) incl.x += x, incl.y += y;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  int2 at = make_int2(incl.x - own.x, incl.y - own.y);
  for (int w = 0; w < warp; ++w) at.x += warp_sum[w].x, at.y += warp_sum[w].y;
  return at;
}

__global__ void __launch_bounds__(kListThreads) route_grad_list_kernel(
    const Pick* __restrict__ picks, const int32_t* __restrict__ counts, int T, int kp, int E,
    int chunk, int chunks, int segment, int32_t* __restrict__ starts,
    int32_t* __restrict__ segments, Entry* __restrict__ list) {
  extern __shared__ __align__(16) char raw[];
  __shared__ int2 warp_sum[kListWarps];
  int* first = reinterpret_cast<int*>(raw);                              // [E]: in the list
  uint32_t* mask = reinterpret_cast<uint32_t*>(first + E);               // [E][kMaskStride]
  uint16_t* before = reinterpret_cast<uint16_t*>(mask + E * kMaskStride);   // [E][kMaskStride]
  const int t0 = blockIdx.x * chunk, nt = min(chunk, T - t0);
  for (int i = threadIdx.x; i < E * kMaskStride; i += kListThreads) mask[i] = 0;
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  const Pick* from = picks + (size_t)t0 * kp;
  Pick mine[kOwn];   // this thread's
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int at = threadIdx.x + i * kListThreads;
    mine[i] = at < nt * kp ? from[at] : Pick{E, 0.0f};
  }
  // Thread i: experts 2i, 2i + 1
  int total[2] = {0, 0}, ahead[2] = {0, 0};
  const int e0 = threadIdx.x * 2;
  if (e0 < E) {
    constexpr int kAtOnce = 16;   // chunks (2048 tokens: 55 -> 52 us; 8 at once as a plain loop)
    for (int c0 = 0; c0 < chunks; c0 += kAtOnce) {
      int n[kAtOnce][2];
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          n[c][q] = c0 + c < chunks && e0 + q < E ? counts[(size_t)(c0 + c) * E + e0 + q] : 0;
#pragma unroll
      for (int c = 0; c < kAtOnce; ++c)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          total[q] += n[c][q];
          ahead[q] += c0 + c < (int)blockIdx.x ? n[c][q] : 0;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int t = (threadIdx.x + i * kListThreads) / kp;
    if (mine[i].expert < E)
      atomicOr(&mask[mine[i].expert * kMaskStride + (t >> 5)], 1u << (t & 31));
  }
  const auto segs = [&](int n) { return (n + segment - 1) / segment; };
  int2 at = cta_scan(make_int2(total[0] + total[1], segs(total[0]) + segs(total[1])), warp_sum);
  for (int q = 0; q < 2; ++q) {
    const int e = e0 + q;
    if (e >= E) break;
    first[e] = at.x + ahead[q];
    if (blockIdx.x == 0) starts[e] = at.x, segments[e] = at.y;
    at.x += total[q];
    at.y += segs(total[q]);
    if (blockIdx.x == 0 && e == E - 1) starts[E] = at.x, segments[E] = at.y;
    int sum = 0;   // (the masks are complete: cta_scan had a barrier)
    for (int w = 0; w < kMaskWords; ++w) {
      before[e * kMaskStride + w] = static_cast<uint16_t>(sum);
      sum += __popc(mask[e * kMaskStride + w]);
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const Pick p = mine[i];
    if (p.expert >= E) continue;
    const int t = (threadIdx.x + i * kListThreads) / kp;
    const int w = p.expert * kMaskStride + (t >> 5);
    const int rank = before[w] + __popc(mask[w] & ((1u << (t & 31)) - 1u));
    list[first[p.expert] + rank] = Entry{t0 + t, p.dz};
  }
}

// ------------------------------------------------------------------------------------------
// 3. The products. A warp takes an item at a time: 256 columns of a token's dx or of a segment's sum;
// the segments from a queue (column blocks one after another: a block of x stays in L2 while it is
// used).
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ void add8(f32x2 (&acc)[4], float z, const uint4& u) {
  const f32x2 z2 = both(z);
  acc[0] = fma2(z2, pair_of_bf16(u.x), acc[0]);
  acc[1] = fma2(z2, pair_of_bf16(u.y), acc[1]);
  acc[2] = fma2(z2, pair_of_bf16(u.z), acc[2]);
  acc[3] = fma2(z2, pair_of_bf16(u.w), acc[3]);
}
__device__ __forceinline__ void add8(f32x2 (&acc)[4], float z, const ulonglong2& a,
                                     const ulonglong2& b) {
  const f32x2 z2 = both(z);
  acc[0] = fma2(z2, a.x, acc[0]);
  acc[1] = fma2(z2, a.y, acc[1]);
  acc[2] = fma2(z2, b.x, acc[2]);
  acc[3] = fma2(z2, b.y, acc[3]);
}
__device__ __forceinline__ uint4 bf16_of8(const f32x2* a) {
  return make_uint4(bf16_of_pair(a[0]), bf16_of_pair(a[1]), bf16_of_pair(a[2]), bf16_of_pair(a[3]));
}
// acc to 8 columns of an fp32 row, or added to them
__device__ __forceinline__ void store8(float* row, int v, const f32x2 (&acc)[4], bool add) {
  float4* o = reinterpret_cast<float4*>(row) + 2 * v;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 x = halves(acc[2 * i]), y = halves(acc[2 * i + 1]);
    float4 r = make_float4(x.x, x.y, y.x, y.y);
    if (add) {
      const float4 p = o[i];
      r.x += p.x, r.y += p.y, r.z += p.z, r.w += p.w;
    }
    o[i] = r;
  }
}

struct Args {
  const uint4* x;
  const float* w_gate;
  const uint4* dx_in;
  uint4* dx;
  float* dw_gate;
  const Pick* picks;
  const int32_t *starts, *segments;
  const Entry* list;
  float* partial;
  int32_t* queue;
  int T, kp, E, d, segment;
  bool accumulate;
  long long per_cta;   // slab: (slab, token) pairs of a CTA
};

// A lane's 8 of 256 columns of a token's dx: 4 of the first half and 4 of the second (which the last
// block may lack), so that neighbouring lanes read neighbouring 16 bytes of the gate weights.
struct DxColumns {
  size_t at;      // of the row's first columns
  int c0, c1;     // the same as c0 where there is no second half
  f32x2 acc[4];

  __device__ __forceinline__ DxColumns(const Args& a, int t, int block)
      : at((size_t)t * a.d), c0(block * 256 + (threadIdx.x & 31) * 4) {
    c1 = block * 256 + 128 < a.d ? c0 + 128 : c0;
    uint2 u = make_uint2(0, 0), v = u;
    if (a.dx_in) {
      const __nv_bfloat16* row = reinterpret_cast<const __nv_bfloat16*>(a.dx_in) + at;
      u = *reinterpret_cast<const uint2*>(row + c0);
      v = *reinterpret_cast<const uint2*>(row + c1);
    }
    acc[0] = pair_of_bf16(u.x), acc[1] = pair_of_bf16(u.y);
    acc[2] = pair_of_bf16(v.x), acc[3] = pair_of_bf16(v.y);
  }
  __device__ __forceinline__ void add(const Args& a, int e, float dz) {
    const float* w = a.w_gate + (size_t)e * a.d;
    add8(acc, dz, *reinterpret_cast<const ulonglong2*>(w + c0),
         *reinterpret_cast<const ulonglong2*>(w + c1));
  }
  __device__ __forceinline__ void store(const Args& a) const {
    __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(a.dx) + at;
    const uint4 o = bf16_of8(acc);
    *reinterpret_cast<uint2*>(row + c0) = make_uint2(o.x, o.y);
    if (c1 != c0) *reinterpret_cast<uint2*>(row + c1) = make_uint2(o.z, o.w);
  }
};

__device__ __forceinline__ void dx_item(const Args& a, int t, int block) {
  DxColumns c(a, t, block);
  const int4* two = reinterpret_cast<const int4*>(a.picks + (size_t)t * a.kp);
#pragma unroll 2
  for (int i = 0; i < a.kp / 2; ++i) {
    const int4 p = two[i];   // expert, dz, expert, dz
    if (p.x != a.E) c.add(a, p.x, __int_as_float(p.y));
    if (p.z != a.E) c.add(a, p.z, __int_as_float(p.w));
  }
  c.store(a);
}

// 32 choices of a warp's segment.
struct Staged {
  int4 token[8];
  float4 dz[8];
};
template <int kAtOnce>   // rows of x in flight
__device__ __forceinline__ void dw_item(const Args& a, Staged& staged, int segment, int v) {
  int lo = 0, hi = a.E - 1;   // the expert: the last whose first segment is at or before this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.segments[mid] <= segment)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int vecs = a.d / 8, s0 = a.segments[lo];
  const int from = a.starts[lo] + (segment - s0) * a.segment;
  const int to = min(from + a.segment, a.starts[lo + 1]);
  const int lane = threadIdx.x & 31;
  const uint4* x = a.x + min(v, vecs - 1);
  f32x2 acc[4] = {};
  // 32 choices at a time go through shared memory, the next 32 on their way.
  const auto fetch = [&](int i) { return i < to ? a.list[i] : Entry{0, 0.0f}; };
  const int* tokens = reinterpret_cast<const int*>(staged.token);
  const float* dzs = reinterpret_cast<const float*>(staged.dz);
  Entry next = fetch(from + lane);
  for (int i = from; i < to; i += 32) {
    __syncwarp();
    reinterpret_cast<int*>(staged.token)[lane] = next.token;
    reinterpret_cast<float*>(staged.dz)[lane] = next.dz;
    __syncwarp();
    next = fetch(i + 32 + lane);
    const int n = min(32, to - i);
    int j = 0;
    for (; j + kAtOnce <= n; j += kAtOnce) {
      uint4 u[kAtOnce];
#pragma unroll
      for (int c = 0; c < kAtOnce; c += 4) {
        const int4 t = staged.token[(j + c) / 4];
        u[c] = x[(size_t)t.x * vecs];
        u[c + 1] = x[(size_t)t.y * vecs];
        u[c + 2] = x[(size_t)t.z * vecs];
        u[c + 3] = x[(size_t)t.w * vecs];
      }
#pragma unroll
      for (int c = 0; c < kAtOnce; c += 4) {
        const float4 z = staged.dz[(j + c) / 4];
        add8(acc, z.x, u[c]);
        add8(acc, z.y, u[c + 1]);
        add8(acc, z.z, u[c + 2]);
        add8(acc, z.w, u[c + 3]);
      }
    }
    for (; j < n; ++j) add8(acc, dzs[j], x[(size_t)tokens[j] * vecs]);
  }
  if (v >= vecs) return;
  if (a.segments[lo + 1] - s0 == 1)
    store8(a.dw_gate + (size_t)lo * a.d, v, acc, a.accumulate);
  else
    store8(a.partial + (size_t)segment * a.d, v, acc, false);
}

// Long batches: half of a CTA's warps keep C columns of all gate weights in shared memory, and a
// row of zeros for picks that are none. The (slab of columns, token) pairs, slab by slab, are dealt
// to the CTAs in equal runs, so that a CTA loads one slab or two. C / 16 lanes take a token, 16
// columns a lane, so that the picks, which all of a token's lanes read, cost little beside the
// weights.
constexpr int kDxThreads = 512;
__device__ __forceinline__ void dx_barrier() {
  asm volatile("bar.sync 1, %0;" ::"n"(kDxThreads) : "memory");
}
template <int C>
__device__ __forceinline__ void dx_slabs(const Args& a, char* slab) {
  // A lane's columns are 8 of the slab's first half and 8 of its second, neighbours taking neighbouring
  // 16 bytes of a token's row. A row of the slab: the lanes' first 4 columns one after another, then
  // their other quarters. With 64 columns two of these quarters share a line of the 32 banks: their
  // order in it differs from expert to expert, so that the tokens of a warp meet less (512 experts,
  // 16384 tokens: 368 -> 323 us).
  constexpr int kLanes = C / 16, kAtOnce = kDxThreads / kLanes, kRow = C * 4, kQuarter = C;
  constexpr int kTurn = 128 / C - 1;
  const long long work = (long long)(a.d / C) * a.T;
  long long at = blockIdx.x * a.per_cta;
  const long long end = min(at + a.per_cta, work);
  const int l = threadIdx.x % kLanes, mine = threadIdx.x / kLanes;
  for (int i = threadIdx.x; i < C; i += kDxThreads)
    reinterpret_cast<float*>(slab + (size_t)a.E * kRow)[i] = 0.0f;
  while (at < end) {
    const int s = static_cast<int>(at / a.T), t0 = static_cast<int>(at - (long long)s * a.T);
    const int t1 = static_cast<int>(min((long long)a.T, t0 + (end - at)));
    dx_barrier();   // the slab before this one has been read
    for (int i = threadIdx.x; i < a.E * (C / 4); i += kDxThreads) {
      const int e = i / (C / 4), v = i % (C / 4);
      const int lane = (v >> 1) % kLanes, quarter = (v >> 1) / kLanes * 2 + (v & 1);
      copy16(slab + (size_t)e * kRow + (quarter ^ (e & kTurn)) * kQuarter + lane * 16,
             a.w_gate + (size_t)e * a.d + s * C + v * 4);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    pdl_wait();   // (the first slab comes while the lists are made)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    dx_barrier();
    const char* w = slab + l * 16;
    const unsigned vecs = a.d / 8, col = s * (C / 8) + l;
    // a token's dx_in is loaded while the one before it is worked on
    uint4 next[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    const auto fetch = [&](int t) {
      if (!a.dx_in || t >= t1) return;
      const uint4* from = a.dx_in + (size_t)t * vecs + col;
      next[0] = from[0];
      next[1] = from[kLanes];
    };
    fetch(t0 + mine);
    for (int t = t0 + mine; t < t1; t += kAtOnce) {
      f32x2 acc[8];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        acc[4 * i] = pair_of_bf16(next[i].x), acc[4 * i + 1] = pair_of_bf16(next[i].y);
        acc[4 * i + 2] = pair_of_bf16(next[i].z), acc[4 * i + 3] = pair_of_bf16(next[i].w);
      }
      const int4* two = reinterpret_cast<const int4*>(a.picks + (size_t)t * a.kp);
      const auto add = [&](int e, float z) {
        const char* row = w + e * kRow;
        const f32x2 z2 = both(z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const ulonglong2 u =
              *reinterpret_cast<const ulonglong2*>(row + (i ^ (e & kTurn)) * kQuarter);
          acc[2 * i] = fma2(z2, u.x, acc[2 * i]);
          acc[2 * i + 1] = fma2(z2, u.y, acc[2 * i + 1]);
        }
      };
      int4 p = two[0];
      fetch(t + kAtOnce);
#pragma unroll 2
      for (int i = 0; i < a.kp / 2; ++i) {
        const int4 q = p;
        if (i + 1 < a.kp / 2) p = two[i + 1];
        add(q.x, __int_as_float(q.y));
        add(q.z, __int_as_float(q.w));
      }
      uint4* o = a.dx + (size_t)t * vecs + col;
      o[0] = bf16_of8(acc);
      o[kLanes] = bf16_of8(acc + 4);
    }
    at += t1 - t0;
  }
}

// C: columns of a slab; 0: all warps first take tokens, an equal number each (from the queue they would
// wait for its atomics, a nanosecond an item), and five CTAs an SM, since there is no slab, keep more
// loads in flight.
constexpr int product_threads(int C) { return C ? 1024 : 256; }
constexpr int product_ctas(int C) { return C ? 1 : 5; }   // an SM
constexpr int staged_bytes(int C) { return product_threads(C) / 32 * (int)sizeof(Staged); }
template <int C>
__global__ void __launch_bounds__(product_threads(C), product_ctas(C))
    route_grad_products_kernel(const Args a) {
  extern __shared__ __align__(16) char raw[];
  Staged* staged = reinterpret_cast<Staged*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (C > 0 && warp < kDxThreads / 32) dx_slabs<C ? C : 128>(a, raw + staged_bytes(C));
  pdl_wait();
  const int blocks = (a.d / 8 + 31) / 32, segments = a.segments[a.E];
  const long long items = (long long)segments * blocks;
  // the warps that begin with segments have their first ones by number, the queue those after
  constexpr int kFirst = C > 0 ? kDxThreads / 32 : 0;
  const int beginners = product_threads(C) / 32 - kFirst, known = gridDim.x * beginners;
  const auto take = [&]() {
    int i = 0;
    if (lane == 0 && items > known) i = atomicAdd(a.queue, 1);
    return known + __shfl_sync(0xffffffffu, i, 0);
  };
  int item = warp >= kFirst ? blockIdx.x * beginners + warp - kFirst : take();
  if (C == 0) {
    const long long dx_items = (long long)a.T * blocks;
    for (long long i = item; i < dx_items; i += known) {
      const int t = static_cast<int>(i / blocks);
      dx_item(a, t, static_cast<int>(i - (long long)t * blocks));
    }
  }
  while (item < items) {
    const int next = take(), block = item / segments;
    dw_item<C ? 8 : 4>(a, staged[warp], item - block * segments, block * 32 + lane);
    item = next;
  }
}

// ------------------------------------------------------------------------------------------
// 4. Experts with several segments, or none: their sums, in order, eight segments at once, since an
// expert that every token chose has hundreds. PARTS of a CTA's threads take every PARTS-th segment:
// 4 while all CTAs run at the same time (16384 tokens of 4 unequal choices, 32 experts, 1024 columns:
// 49 us, with one part 59), else 1 (256 experts, 7168 columns: 263 us, with 4 parts 270, since most of
// the 7168 CTAs have one segment and nothing to do).
// ------------------------------------------------------------------------------------------
constexpr int kJoinThreads = 256;
template <int PARTS>
__global__ void __launch_bounds__(kJoinThreads) route_grad_join_kernel(
    const float4* __restrict__ partial, const int32_t* __restrict__ segments,
    float4* __restrict__ dw_gate, int quads, bool accumulate) {
  constexpr int kQuads = kJoinThreads / PARTS;
  __shared__ float4 sums[PARTS][kQuads];
  const int e = blockIdx.y, column = threadIdx.x % kQuads, part = threadIdx.x / kQuads;
  const int v = blockIdx.x * kQuads + column;
  pdl_wait();
  const int s0 = segments[e], s1 = segments[e + 1];
  if (s1 - s0 == 1 || (s0 == s1 && accumulate)) return;   // whole CTAs
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const auto add = [&](const float4& p) { s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w; };
  constexpr int kAtOnce = 8;
  for (int i = s0 + part; v < quads && i < s1; i += kAtOnce * PARTS) {
    float4 p[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j * PARTS < s1) p[j] = partial[(size_t)(i + j * PARTS) * quads + v];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j)
      if (i + j * PARTS < s1) add(p[j]);
  }
  if (PARTS > 1) {
    sums[part][column] = s;
    __syncthreads();
  }
  if (part > 0 || v >= quads) return;
#pragma unroll
  for (int i = 1; i < PARTS; ++i) add(sums[i][column]);
  float4* o = dw_gate + (size_t)e * quads + v;
  if (accumulate) add(*o);
  *o = s;
}

// ------------------------------------------------------------------------------------------
// A short batch, of 512 choices at most: every CTA works out all choices' dz for itself, then its
// warps take items: 256 columns of a token's dx, or of an expert's dw_gate, whose choices are found
// by looking through all of them. (7168 columns, 256 experts, 8 choices, from cold caches: 64 tokens 15
// us, and 23 through the lists, 25 and 22 with choices as uneven as 1/rank^1.2, since a warp adds up
// all of an expert's; 128 tokens 21 and 25, uneven 40 and 23.)
// ------------------------------------------------------------------------------------------
constexpr int kShortThreads = 1024, kShortWarps = kShortThreads / 32;
__global__ void __launch_bounds__(kShortThreads) route_grad_short_kernel(
    const int32_t* __restrict__ idx, const float* __restrict__ score, const float* __restrict__ dw,
    const Args a, int k, float scale, uint32_t* status) {
  __shared__ int expert[2 * kShortChoices];   // [T][kp]
  __shared__ float dz[2 * kShortChoices];
  __shared__ int found[kShortWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, kp = a.kp;
  {
    const int width = lanes_of(kp), j = threadIdx.x & (width - 1), per = kShortThreads / width;
    for (int b = 0; b < a.T; b += per) {   // whole warps
      const int t = b + threadIdx.x / width;
      const bool in = t < a.T && j < k;
      int e = -1;
      float s = 0.0f, g = 0.0f;
      if (in) e = checked(idx[t * k + j], a.E, status), s = score[t * k + j], g = dw[t * k + j];
      const Pick p = pick_of(e, s, g, in, width, scale, a.E);
      if (t < a.T && j < kp) expert[t * kp + j] = p.expert, dz[t * kp + j] = p.dz;
    }
  }
  __syncthreads();
  const int vecs = a.d / 8, blocks = (vecs + 31) / 32, dx_items = a.T * blocks;
  const int items = dx_items + a.E * blocks, step = gridDim.x * kShortWarps;
  for (int item = blockIdx.x * kShortWarps + warp; item < items; item += step) {
    if (item < dx_items) {
      const int t = item / blocks;
      DxColumns c(a, t, item - t * blocks);
#pragma unroll 4
      for (int i = t * kp; i < t * kp + kp; ++i)
        if (expert[i] != a.E) c.add(a, expert[i], dz[i]);
      c.store(a);
      continue;
    }
    const int i = item - dx_items, e = i / blocks, v = (i - e * blocks) * 32 + lane;
    f32x2 acc[4] = {};
    int n = 0;   // choices found, 32 at most before they are added
    bool any = false;
    const auto flush = [&]() {
      __syncwarp();
      if (v < vecs)
#pragma unroll 8
        for (int q = 0; q < n; ++q) {
          const int c = found[warp][q];
          add8(acc, dz[c], a.x[(size_t)(c / kp) * vecs + v]);
        }
      any |= n > 0;
      n = 0;
      __syncwarp();
    };
    for (int b = 0; b < a.T * kp; b += 32) {
      const bool hit = b + lane < a.T * kp && expert[b + lane] == e;
      const uint32_t hits = __ballot_sync(0xffffffffu, hit);
      if (!hits) continue;
      if (n + __popc(hits) > 32) flush();
      if (hit) found[warp][n + __popc(hits & ((1u << lane) - 1u))] = b + lane;
      n += __popc(hits);
    }
    flush();
    if (v < vecs && (any || !a.accumulate))
      store8(a.dw_gate + (size_t)e * a.d, v, acc, a.accumulate);
  }
}

template <int C>
cudaError_t run_products(Args a, cudaStream_t st) {
  auto kern = route_grad_products_kernel<C>;
  const size_t smem = staged_bytes(C) + (size_t)(a.E + 1) * C * 4;
  const cudaError_t e = ensure_smem_limit(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  if (C > 0) a.per_cta = ((long long)(a.d / std::max(C, 1)) * a.T + kSms - 1) / kSms;
  return launch_kernel(kern, dim3(kSms * product_ctas(C)), dim3(product_threads(C)), smem, st, true,
                       a);
}

}  // namespace

size_t route_grad_ws_bytes(const moe_cfg& c) { return layout(c).total; }

cudaError_t launch_route_grad(const moe_cfg& c, const void* x, const float* w_gate,
                              const int32_t* topk_idx, const float* topk_s, const float* dtopk_w,
                              const void* dx_in, void* dx, float* dw_gate, bool accumulate,
                              void* ws, cudaStream_t st) {
  const Layout L = layout(c);
  char* w = static_cast<char*>(ws);
  uint32_t* status = static_cast<uint32_t*>(ws);
  Args a{};
  a.x = static_cast<const uint4*>(x);
  a.w_gate = w_gate;
  a.dx_in = static_cast<const uint4*>(dx_in);
  a.dx = static_cast<uint4*>(dx);
  a.dw_gate = dw_gate;
  a.T = c.T, a.kp = L.kp, a.E = c.E, a.d = c.d, a.segment = L.segment;
  a.accumulate = accumulate;
  const long long blocks = (c.d / 8 + 31) / 32;
  if (L.one_launch) {
    const long long items = (c.T + c.E) * blocks;
    const long long full = (items + kShortWarps - 1) / kShortWarps;
    const unsigned ctas = (unsigned)std::min(full, (long long)kSms);
    return launch_kernel(route_grad_short_kernel, dim3(ctas), dim3(kShortThreads), 0, st, false,
                         topk_idx, topk_s, dtopk_w, a, c.k, c.route_scale, status);
  }
  Pick* picks = reinterpret_cast<Pick*>(w + L.picks);
  int32_t* counts = reinterpret_cast<int32_t*>(w + L.counts);
  int32_t* starts = reinterpret_cast<int32_t*>(w + L.starts);
  int32_t* segments = reinterpret_cast<int32_t*>(w + L.segments);
  Entry* list = reinterpret_cast<Entry*>(w + L.list);
  a.queue = reinterpret_cast<int32_t*>(w + L.queue);
  a.partial = reinterpret_cast<float*>(w + L.partial);
  a.picks = picks, a.starts = starts, a.segments = segments, a.list = list;
  cudaError_t e = launch_kernel(route_grad_count_kernel, dim3(L.chunks), dim3(kListThreads), 0, st,
                                false, topk_idx, topk_s, dtopk_w, c.T, c.k, L.kp, c.E,
                                c.route_scale, L.chunk, picks, counts, a.queue, status);
  if (e != cudaSuccess) return e;
  const size_t smem = (size_t)c.E * (4 + kMaskStride * (4 + 2));
  e = ensure_smem_limit(reinterpret_cast<const void*>(route_grad_list_kernel),
                        smem + 1024);   // (the static array counts, too)
  if (e != cudaSuccess) return e;
  e = launch_kernel(route_grad_list_kernel, dim3(L.chunks), dim3(kListThreads), smem, st, true,
                    static_cast<const Pick*>(picks), static_cast<const int32_t*>(counts), c.T, L.kp,
                    c.E, L.chunk, L.chunks, L.segment, starts, segments, list);
  if (e != cudaSuccess) return e;
  // Slabs of 128 columns up to 437 experts, of 64 up to 875, where the tokens are many. 8 choices, 7168
  // columns, with and without: 256 experts, 16384 tokens 245 and 362 us, 1024 tokens 41 and 44; 800
  // experts, 16384 tokens 352 and 383, 1024 tokens 59 and 56. (Slabs of 32 columns, for more experts,
  // share banks: 1024 experts, 16384 tokens 427 us, without slabs 381.)
  const size_t row = 4 * (size_t)(c.E + 1), most = 227 * 1024 - staged_bytes(128);
  e = c.T < 1024          ? run_products<0>(a, st)
      : row * 128 <= most ? run_products<128>(a, st)
      : row * 64 <= most  ? run_products<64>(a, st)
                          : run_products<0>(a, st);
  if (e != cudaSuccess) return e;
  const int quads = c.d / 4;
  const auto join = [&](auto kern, int parts) {
    const int columns = kJoinThreads / parts;
    return launch_kernel(kern, dim3((quads + columns - 1) / columns, c.E), dim3(kJoinThreads), 0, st,
                         true, reinterpret_cast<const float4*>(a.partial),
                         static_cast<const int32_t*>(segments), reinterpret_cast<float4*>(dw_gate),
                         quads, accumulate);
  };
  return (long long)c.E * quads * 4 <= 8ll * kSms * kJoinThreads
             ? join(route_grad_join_kernel<4>, 4)
             : join(route_grad_join_kernel<1>, 1);
}

}  // namespace moe
