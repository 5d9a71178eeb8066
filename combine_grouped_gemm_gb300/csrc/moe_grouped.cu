// Matrix products grouped by expert over ragged row counts: forward, gradient of the rows and
// gradient of the weights. Group e owns rows [s_e, s_e + c_e) of the row tensors:
//   fwd: y[r][i]    = sum_j x[r][j] W_e[i][j]
//   dx : dx[r][j]   = sum_i dy[r][i] W_e[i][j]
//   dw : dW_e[i][j] = sum_r dy[r][i] x[r][j]   (r over the group's rows)
// bf16 operands, fp32 sums, each result rounded once where it is stored in bf16.
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;

// First rows of the groups, off[0..E], from counts, in shared memory: warp 0 scans, each lane
// over ceil(E / 32) consecutive groups. A negative count is 0 and the offsets stop at `rows`;
// either is reported. Ends with a block barrier.
__device__ __forceinline__ void group_offsets(const int32_t* counts, int E, int rows, int* off,
                                              uint32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) off[e + 1] = counts[e];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (E + 31) / 32;
    const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
    bool bad = false;
    long long sum = 0;
    for (int e = e0; e < e1; ++e) {
      const int c = off[e + 1];
      bad |= c < 0;
      sum += max(c, 0);
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    bad |= incl > rows;
    long long at = incl - sum;
    for (int e = e0; e < e1; ++e) {
      at += max(off[e + 1], 0);
      off[e + 1] = static_cast<int>(at < rows ? at : rows);
    }
    if (lane == 0) off[0] = 0;
    if (bad && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0)
      raise_status(status, MOE_DEV_BOUNDS);
  }
  __syncthreads();
}

constexpr int kTile = 64, kStep = 16;

// 64x64 output tile, 256 threads, 4x4 outputs each, operands staged in shared memory as floats.
// fwd/dx: blockIdx.y numbers the 64-row tiles of all groups; dw: blockIdx.z is the group.
template <int DIR>
__global__ void __launch_bounds__(256) grouped_kernel(
    const __nv_bfloat16* __restrict__ in0, const __nv_bfloat16* __restrict__ in1,
    const int32_t* __restrict__ counts, void* out, int rows, int E, int n, int k, int out_f32,
    int accumulate, uint32_t* status) {
  __shared__ int off[kMaxGroups + 1];
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  group_offsets(counts, E, rows, off, status);
  int g = 0, r0 = 0, r1 = 0;
  if (DIR == kGroupedDw) {
    g = blockIdx.z;
    r0 = off[g];
    r1 = off[g + 1];
  } else {
    int t = blockIdx.y;
    for (; g < E; ++g) {
      const int nt = (off[g + 1] - off[g] + kTile - 1) / kTile;
      if (t < nt) break;
      t -= nt;
    }
    if (g == E) return;
    r0 = off[g] + t * kTile;
    r1 = off[g + 1];
  }
  // output rows m0.., columns c0.., the reduction's length
  const int m0 = DIR == kGroupedDw ? blockIdx.y * kTile : r0, c0 = blockIdx.x * kTile;
  const int m_end = DIR == kGroupedDw ? n : r1;
  const int cols = DIR == kGroupedFwd ? n : k;
  const int red = DIR == kGroupedFwd ? k : DIR == kGroupedDx ? n : r1 - r0;
  const size_t wbase = (size_t)g * n * k;
  float acc[4][4] = {};
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  for (int p0 = 0; p0 < red; p0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      int p, m;
      float va = 0.0f, vb = 0.0f;
      if (DIR == kGroupedDw) {
        p = i / kTile, m = i % kTile;
        if (p0 + p < red) {
          const size_t r = (size_t)r0 + p0 + p;
          if (m0 + m < n) va = __bfloat162float(in0[r * n + m0 + m]);
          if (c0 + m < k) vb = __bfloat162float(in1[r * k + c0 + m]);
        }
      } else {
        p = i % kStep, m = i / kStep;
        if (p0 + p < red && m0 + m < m_end)
          va = __bfloat162float(in0[(size_t)(m0 + m) * red + p0 + p]);
        if (p0 + p < red && c0 + m < cols)
          vb = __bfloat162float(DIR == kGroupedFwd
                                    ? in1[wbase + (size_t)(c0 + m) * k + p0 + p]
                                    : in1[wbase + (size_t)(p0 + p) * k + c0 + m]);
      }
      sa[p][m] = va;
      sb[p][m] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int p = 0; p < kStep; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += sa[p][ty * 4 + i] * sb[p][tx + 16 * j];
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty * 4 + i, c = c0 + tx + 16 * j;
      if (m >= m_end || c >= cols) continue;
      const size_t o = (DIR == kGroupedDw ? wbase : 0) + (size_t)m * cols + c;
      if (out_f32) {
        float* f = static_cast<float*>(out) + o;
        *f = accumulate ? *f + acc[i][j] : acc[i][j];
      } else {
        static_cast<__nv_bfloat16*>(out)[o] = __float2bfloat16_rn(acc[i][j]);
      }
    }
}

}  // namespace

size_t grouped_ws_bytes(const moe_group_cfg&) { return 256; }

cudaError_t launch_grouped(const moe_group_cfg& c, GroupedDir dir, const void* in0, const void* in1,
                           const int32_t* counts, void* out, bool out_f32, bool accumulate,
                           void* ws, cudaStream_t st) {
  auto t = [](int v) { return static_cast<unsigned>((v + kTile - 1) / kTile); };
  const unsigned row_tiles = t(c.rows) + c.E;
  const dim3 grid = dir == kGroupedFwd  ? dim3(t(c.n), row_tiles)
                    : dir == kGroupedDx ? dim3(t(c.k), row_tiles)
                                        : dim3(t(c.k), t(c.n), c.E);
  auto kern = dir == kGroupedFwd  ? grouped_kernel<kGroupedFwd>
              : dir == kGroupedDx ? grouped_kernel<kGroupedDx>
                                  : grouped_kernel<kGroupedDw>;
  return launch_kernel(kern, grid, dim3(256), 0, st, false,
                       static_cast<const __nv_bfloat16*>(in0),
                       static_cast<const __nv_bfloat16*>(in1), counts, out, c.rows, c.E, c.n, c.k,
                       out_f32 ? 1 : 0, accumulate ? 1 : 0, static_cast<uint32_t*>(ws));
}

}  // namespace moe
