// RMS norms before and after a block, fused with the block's gate, the residual's scale and the next
// block's norm, and their gradients. Each reads its inputs from HBM once and writes its outputs once.
//
// A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and a thread the same columns of each: 8
// a vector, VPT vectors. The weights of a thread's columns stay in its registers for all rows, and so
// do the gradients' column sums. Rows come through a ring of stages in shared memory that holds the
// next rows' copies in flight; a thread reads only what its own cp.async brought, so the ring needs
// no barrier. The one barrier of a reduction over a row is the one between its warps' partial sums.
#include "moe_device.cuh"

namespace moe {
namespace {

constexpr int kGpuSms = 152;       // grids are sized for GB300
constexpr int kMaxThreads = 1024;  // a CTA; also the threads that a grid puts on one SM
constexpr int kWsHead = 256;       // the status word's place at the head of the scratch

struct Shape {
  int rows, d, vecs;   // vecs = d / 8
  float eps, res, out;
  int gate;
};

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x), f[1] = bf16_hi(v.x), f[2] = bf16_lo(v.y), f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z), f[5] = bf16_hi(v.z), f[6] = bf16_lo(v.w), f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// 8 consecutive values of the residual stream: 16 bytes of bf16 or 32 of fp32.
template <bool F32>
__device__ __forceinline__ void read8(const char* at, float (&f)[8]) {
  if (F32) {
    const float4 a = *reinterpret_cast<const float4*>(at);
    const float4 b = *reinterpret_cast<const float4*>(at + 16);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    unpack8(*reinterpret_cast<const uint4*>(at), f);
  }
}
template <bool F32>
__device__ __forceinline__ void write8(char* at, const float (&f)[8]) {
  if (F32) {
    *reinterpret_cast<float4*>(at) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(at + 16) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<uint4*>(at) = pack8(f);
  }
}
__device__ __forceinline__ void load_weights(const float* w, int vec, bool in, float (&f)[8],
                                             float none) {
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = none;
  if (w && in) read8<true>(reinterpret_cast<const char*>(w) + (size_t)vec * 32, f);
}

__device__ __forceinline__ void copy16(char* smem, const char* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// K sums over the CTA, every thread gets them, in a fixed order. buf: 2 x 32 x K floats, the halves
// used in turn (flip), so that one barrier a reduction is enough.
template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K], float* buf, int& flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* b = buf + flip * 32 * K;
  flip ^= 1;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) b[i * 32 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = lane < warps ? b[i * 32 + lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

__device__ __forceinline__ float inv_root(float sum, const Shape& s) {
  return 1.0f / sqrtf(sum / static_cast<float>(s.d) + s.eps);
}

// The arrays of a row in the ring: slot(array, vec) of a stage. Sizes in bytes a vector.
struct Arrays {
  const char* p[5];
  int bytes[5];   // 16 or 32; 0: not there
};

// Starts the copies of one row (this thread's vectors) into a stage.
template <int N, int VPT>
__device__ __forceinline__ void fetch_row(const Arrays& a, char* stage, long long row, int vecs) {
  char* dst = stage;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int b = a.bytes[i];
    if (b == 0) continue;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v < vecs) {
        const char* src = a.p[i] + ((size_t)row * vecs + v) * b;
        copy16(dst + (size_t)v * b, src);
        if (b == 32) copy16(dst + (size_t)v * b + 16, src + 16);
      }
    }
    dst += (size_t)vecs * b;
  }
}

template <bool F32, int VPT, int STAGES>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(Shape s, NormFwd a, int stage_bytes) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float sums[2 * 32];
  constexpr int kSt = F32 ? 32 : 16;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, next = a.w_next != nullptr;
  const bool elem = s.gate == MOE_GATE_ELEMENT;
  Arrays in;
  in.p[0] = static_cast<const char*>(a.x), in.bytes[0] = kSt;
  in.p[1] = static_cast<const char*>(a.y), in.bytes[1] = has_y ? 16 : 0;
  in.p[2] = static_cast<const char*>(a.gate), in.bytes[2] = elem ? 16 : 0;
  const int off_y = s.vecs * kSt, off_g = off_y + (has_y ? s.vecs * 16 : 0);

  // what a column's normed output is multiplied by: out, the channel gate and the weight; and the
  // next norm's weight
  float gw[VPT][8], wn[VPT][8];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    const bool col = v < s.vecs;
    float g[8];
    load_weights(a.w_post, v, col, gw[k], 1.0f);
    load_weights(s.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, v, col, g,
                 1.0f);
    load_weights(a.w_next, v, col, wn[k], 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[k][j] *= s.out * g[j];
  }
  const int step = gridDim.x;
  int flip = 0, slot = 0;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    const long long r = blockIdx.x + (long long)i * step;
    if (r < s.rows) fetch_row<3, VPT>(in, ring + (size_t)i * stage_bytes, r, s.vecs);
    copies_commit();
  }
  for (long long row = blockIdx.x; row < s.rows; row += step) {
    {
      const long long ahead = row + (long long)(STAGES - 1) * step;
      const int to = slot == 0 ? STAGES - 1 : slot - 1;
      if (ahead < s.rows) fetch_row<3, VPT>(in, ring + (size_t)to * stage_bytes, ahead, s.vecs);
      copies_commit();
    }
    copies_wait<STAGES - 1>();
    const char* st = ring + (size_t)slot * stage_bytes;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    float h[VPT][8];
    float factor = 1.0f;   // of this row's y
    if (post) {
      float q[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = threadIdx.x + k * blockDim.x;
        if (v >= s.vecs) continue;
        float y[8];
        read8<false>(st + off_y + (size_t)v * 16, y);
#pragma unroll
        for (int j = 0; j < 8; ++j) q[0] = __fmaf_rn(y[j], y[j], q[0]);
      }
      cta_sum<1>(q, sums, flip);
      factor = inv_root(q[0], s);
      if (threadIdx.x == 0 && a.rstd_y) a.rstd_y[row] = factor;
    }
    if (s.gate == MOE_GATE_TOKEN) factor *= static_cast<const float*>(a.gate)[row];
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      read8<F32>(st + (size_t)v * kSt, h[k]);
      if (has_y) {
        float y[8], g[8];
        read8<false>(st + off_y + (size_t)v * 16, y);
        if (elem) {
          read8<false>(st + off_g + (size_t)v * 16, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] *= g[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) h[k][j] = __fmaf_rn(y[j] * factor, gw[k][j], s.res * h[k][j]);
        write8<F32>(static_cast<char*>(a.h) + ((size_t)row * s.vecs + v) * kSt, h[k]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) q[0] = __fmaf_rn(h[k][j], h[k][j], q[0]);
    }
    if (!next) continue;
    cta_sum<1>(q, sums, flip);
    const float r = inv_root(q[0], s);
    if (threadIdx.x == 0 && a.rstd_h) a.rstd_h[row] = r;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = h[k][j] * r * wn[k][j];
      write8<false>(static_cast<char*>(a.n) + ((size_t)row * s.vecs + v) * 16, o);
    }
  }
}

// The gradient. A row's three sums come from one pass, since the mean that the norm behind the block
// needs is linear in G: with u = out gate w_post yh, and a = dn w_next,
//   sum u G = sum u (dh + r_h a) - r_h mean(a hh) sum u hh.
// The second pass reads the row again from the ring. Column sums: acc_y = sum out G gate yh (without
// a channel gate, which like w_post is the same in all rows: dw_post = gate acc_y, dgate = w_post
// acc_y) and acc_n = sum dn hh.
template <bool F32, int VPT, int STAGES>
__global__ void __launch_bounds__(kMaxThreads, 1)
    norm_grad_kernel(Shape s, NormGrad a, int stage_bytes, float* partial) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float sums[2 * 32 * 3];
  constexpr int kSt = F32 ? 32 : 16;
  const bool post = a.w_post != nullptr, next = a.w_next != nullptr, has_dh = a.dh != nullptr;
  const bool elem = s.gate == MOE_GATE_ELEMENT, token = s.gate == MOE_GATE_TOKEN;
  const bool has_y = post || s.gate != MOE_GATE_NONE;   // y itself is needed
  const bool is_out = a.dy != nullptr;                  // the norm before a block has no y side
  const bool dot_y = post || token;
  Arrays in;
  in.p[0] = static_cast<const char*>(a.dh), in.bytes[0] = has_dh ? kSt : 0;
  in.p[1] = static_cast<const char*>(a.h), in.bytes[1] = next ? kSt : 0;
  in.p[2] = static_cast<const char*>(a.dn), in.bytes[2] = next ? 16 : 0;
  in.p[3] = static_cast<const char*>(a.y), in.bytes[3] = has_y ? 16 : 0;
  in.p[4] = static_cast<const char*>(a.gate), in.bytes[4] = elem ? 16 : 0;
  const int off_h = has_dh ? s.vecs * kSt : 0;
  const int off_n = off_h + (next ? s.vecs * kSt : 0);
  const int off_y = off_n + (next ? s.vecs * 16 : 0);
  const int off_g = off_y + (has_y ? s.vecs * 16 : 0);

  float gw[VPT][8], wn[VPT][8], acc_y[VPT][8], acc_n[VPT][8];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    const bool col = v < s.vecs;
    float g[8];
    load_weights(a.w_post, v, col, gw[k], 1.0f);
    load_weights(s.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr, v, col, g,
                 1.0f);
    load_weights(a.w_next, v, col, wn[k], 0.0f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      gw[k][j] *= g[j];
      acc_y[k][j] = acc_n[k][j] = 0.0f;
    }
  }
  const int step = gridDim.x;
  const float inv_d = 1.0f / static_cast<float>(s.d);
  int flip = 0, slot = 0;
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    const long long r = blockIdx.x + (long long)i * step;
    if (r < s.rows) fetch_row<5, VPT>(in, ring + (size_t)i * stage_bytes, r, s.vecs);
    copies_commit();
  }
  for (long long row = blockIdx.x; row < s.rows; row += step) {
    {
      const long long ahead = row + (long long)(STAGES - 1) * step;
      const int to = slot == 0 ? STAGES - 1 : slot - 1;
      if (ahead < s.rows) fetch_row<5, VPT>(in, ring + (size_t)to * stage_bytes, ahead, s.vecs);
      copies_commit();
    }
    const float rh = next ? a.rstd_h[row] : 0.0f, ry = post ? a.rstd_y[row] : 1.0f;
    const float gt = token ? static_cast<const float*>(a.gate)[row] : 1.0f;
    copies_wait<STAGES - 1>();
    const char* st = ring + (size_t)slot * stage_bytes;
    slot = slot + 1 == STAGES ? 0 : slot + 1;

    float q[3] = {0.0f, 0.0f, 0.0f};   // sum a hh, sum u (dh + rh a), sum u hh
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      float dh[8] = {}, h[8] = {}, dn[8] = {};
      if (has_dh) read8<F32>(st + (size_t)v * kSt, dh);
      if (next) {
        read8<F32>(st + off_h + (size_t)v * kSt, h);
        read8<false>(st + off_n + (size_t)v * 16, dn);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          h[j] *= rh;
          dn[j] *= wn[k][j];
          q[0] = __fmaf_rn(dn[j], h[j], q[0]);
          dh[j] = __fmaf_rn(rh, dn[j], dh[j]);
        }
      }
      if (dot_y) {
        float y[8], g[8];
        read8<false>(st + off_y + (size_t)v * 16, y);
        if (elem) read8<false>(st + off_g + (size_t)v * 16, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float u = y[j] * gw[k][j];
          if (elem) u *= g[j];
          q[1] = __fmaf_rn(u, dh[j], q[1]);
          q[2] = __fmaf_rn(u, h[j], q[2]);
        }
      }
    }
    if (next || dot_y) cta_sum<3>(q, sums, flip);
    const float c1 = q[0] * inv_d;
    const float along = s.out * ry * (q[1] - rh * c1 * q[2]);   // sum out G s (no token gate)
    const float mean = gt * along * inv_d;
    if (token && a.dgate && threadIdx.x == 0) static_cast<float*>(a.dgate)[row] = along;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      const size_t at = (size_t)row * s.vecs + v;
      float G[8] = {};
      if (has_dh) read8<F32>(st + (size_t)v * kSt, G);
      if (next) {
        float h[8], dn[8];
        read8<F32>(st + off_h + (size_t)v * kSt, h);
        read8<false>(st + off_n + (size_t)v * 16, dn);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float hh = h[j] * rh;
          G[j] = __fmaf_rn(rh, __fmaf_rn(dn[j], wn[k][j], -hh * c1), G[j]);
          acc_n[k][j] = __fmaf_rn(dn[j], hh, acc_n[k][j]);
        }
      }
      if (a.dx) {
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = s.res * G[j];
        write8<F32>(static_cast<char*>(a.dx) + at * kSt, o);
      }
      if (!is_out) continue;
      float y[8] = {}, g[8], o[8];
      if (has_y) read8<false>(st + off_y + (size_t)v * 16, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) G[j] *= s.out;
      if (elem) {
        read8<false>(st + off_g + (size_t)v * 16, g);
        if (a.dgate) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = G[j] * y[j] * ry * gw[k][j];
          write8<false>(static_cast<char*>(a.dgate) + at * 16, o);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) G[j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float yh = y[j] * ry, u = gt * G[j];
        acc_y[k][j] = __fmaf_rn(u, yh, acc_y[k][j]);
        o[j] = post ? ry * __fmaf_rn(u, gw[k][j], -yh * mean) : u * gw[k][j];
      }
      write8<false>(static_cast<char*>(a.dy) + at * 16, o);
    }
  }
  if (!partial) return;
  // partial sums of this CTA: [0][cta][d] acc_y, [1][cta][d] acc_n
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = threadIdx.x + k * blockDim.x;
    if (v >= s.vecs) continue;
    char* p = reinterpret_cast<char*>(partial) + ((size_t)blockIdx.x * s.vecs + v) * 32;
    write8<true>(p, acc_y[k]);
    write8<true>(p + (size_t)gridDim.x * s.vecs * 32, acc_n[k]);
  }
}

// Column sums over the CTAs' partial sums: a warp's lanes are 32 columns, a CTA's warps take parts of
// the CTAs one after another, joined in order. blockIdx.y: 0 the sums over yh, 1 those over hh.
struct ColSums {
  const float* partial;
  int ctas, d;
  const float *w_post, *gate;        // gate: a channel gate, else NULL
  float *dw_post, *dgate, *dw_next;  // NULL: not wanted
  int accumulate;
};
constexpr int kColThreads = 512;
__global__ void __launch_bounds__(kColThreads) norm_columns_kernel(ColSums a) {
  __shared__ float part[kColThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const bool y_side = blockIdx.y == 0;
  if (y_side ? !a.dw_post && !a.dgate : !a.dw_next) return;
  const float* p = a.partial + (size_t)blockIdx.y * a.ctas * a.d;
  float sum = 0.0f;
  if (c < a.d)
#pragma unroll 4
    for (int i = warp; i < a.ctas; i += kColThreads / 32) sum += p[(size_t)i * a.d + c];
  part[warp][lane] = sum;
  __syncthreads();
  if (warp != 0 || c >= a.d) return;
  sum = 0.0f;
  for (int i = 0; i < kColThreads / 32; ++i) sum += part[i][lane];
  const auto put = [&](float* to, float v) {
    if (to) to[c] = a.accumulate ? to[c] + v : v;
  };
  if (y_side) {
    const float g = a.gate ? a.gate[c] : 1.0f, w = a.w_post ? a.w_post[c] : 1.0f;
    put(a.dw_post, g * sum);
    if (a.gate) put(a.dgate, w * sum);
  } else {
    put(a.dw_next, sum);
  }
}

// Threads of a CTA, vectors a thread and the CTAs that an SM takes at once.
struct Plan {
  int vpt, threads, per_sm;
};
Plan plan_of(int d) {
  const int vecs = d / 8;
  Plan p;
  p.vpt = vecs > kMaxThreads ? 2 : 1;
  p.threads = ((vecs + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  p.per_sm = kMaxThreads / p.threads;
  return p;
}
unsigned grid_of(int rows, const Plan& p) {
  const int most = kGpuSms * p.per_sm;
  return rows < most ? rows : most;
}

constexpr int kFwdStages = 4, kGradStages = 3;

template <typename K>
cudaError_t set_smem(K kern, size_t bytes) {
  return ensure_smem_limit(reinterpret_cast<const void*>(kern), bytes);
}

template <bool F32, int VPT, int STAGES>
cudaError_t run_fwd(const Shape& s, const NormFwd& a, const Plan& p, int stage, cudaStream_t st) {
  auto kern = norm_kernel<F32, VPT, STAGES>;
  const size_t smem = (size_t)STAGES * stage;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid_of(s.rows, p)), dim3(p.threads), smem, st, false, s, a,
                       stage);
}

template <bool F32, int VPT, int STAGES>
cudaError_t run_grad(const Shape& s, const NormGrad& a, const Plan& p, int stage, float* partial,
                     cudaStream_t st) {
  auto kern = norm_grad_kernel<F32, VPT, STAGES>;
  const size_t smem = (size_t)STAGES * stage;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid_of(s.rows, p)), dim3(p.threads), smem, st, false, s, a, stage,
                       partial);
}

Shape shape_of(const moe_norm_cfg& c) {
  return Shape{c.rows, c.d, c.d / 8, c.eps, c.res_scale, c.out_scale, c.gate};
}

}  // namespace

size_t norm_ws_bytes(int rows, int d) {
  return kWsHead + (size_t)grid_of(rows, plan_of(d)) * d * 2 * sizeof(float);
}

cudaError_t launch_norm(const moe_norm_cfg& c, const NormFwd& a, cudaStream_t st) {
  const Shape s = shape_of(c);
  const Plan p = plan_of(c.d);
  const bool f32 = c.stream_dtype == MOE_F32;
  const int stage = s.vecs * ((f32 ? 32 : 16) + (a.y ? 16 : 0) +
                              (c.gate == MOE_GATE_ELEMENT ? 16 : 0));
  // widest row: 16384 columns of fp32 stream, y and an element gate are 128 KB a stage: one stage
  const bool deep = (size_t)stage * kFwdStages * p.per_sm <= 200 * 1024;
  if (p.vpt == 1) {
    if (f32) return deep ? run_fwd<true, 1, kFwdStages>(s, a, p, stage, st)
                         : run_fwd<true, 1, 2>(s, a, p, stage, st);
    return deep ? run_fwd<false, 1, kFwdStages>(s, a, p, stage, st)
                : run_fwd<false, 1, 2>(s, a, p, stage, st);
  }
  const bool two = (size_t)stage * 2 <= 220 * 1024;
  if (f32) return two ? run_fwd<true, 2, 2>(s, a, p, stage, st)
                      : run_fwd<true, 2, 1>(s, a, p, stage, st);
  return run_fwd<false, 2, 2>(s, a, p, stage, st);
}

cudaError_t launch_norm_grad(const moe_norm_cfg& c, const NormGrad& a, bool accumulate, void* ws,
                             cudaStream_t st) {
  const Shape s = shape_of(c);
  const Plan p = plan_of(c.d);
  const bool f32 = c.stream_dtype == MOE_F32, next = a.w_next != nullptr;
  const bool channel = c.gate == MOE_GATE_CHANNEL;
  const bool has_y = a.w_post || c.gate != MOE_GATE_NONE;
  const int b = f32 ? 32 : 16;
  const int stage = s.vecs * ((a.dh ? b : 0) + (next ? b + 16 : 0) + (has_y ? 16 : 0) +
                              (c.gate == MOE_GATE_ELEMENT ? 16 : 0));
  const bool sums = a.dw_post || a.dw_next || (channel && a.dgate);
  float* partial =
      sums ? reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHead) : nullptr;
  cudaError_t e;
  if (s.rows > 0) {
    const size_t per_sm = (size_t)stage * p.per_sm;
    const int stages = per_sm * kGradStages <= 220 * 1024 ? kGradStages
                       : per_sm * 2 <= 220 * 1024         ? 2
                                                          : 1;
#define MOE_GRAD_CASE(F, V, S) \
  if (f32 == F && p.vpt == V && stages == S) e = run_grad<F, V, S>(s, a, p, stage, partial, st)
    e = cudaErrorInvalidValue;
    MOE_GRAD_CASE(false, 1, 3);
    MOE_GRAD_CASE(false, 1, 2);
    MOE_GRAD_CASE(false, 1, 1);
    MOE_GRAD_CASE(true, 1, 3);
    MOE_GRAD_CASE(true, 1, 2);
    MOE_GRAD_CASE(true, 1, 1);
    MOE_GRAD_CASE(false, 2, 3);
    MOE_GRAD_CASE(false, 2, 2);
    MOE_GRAD_CASE(false, 2, 1);
    MOE_GRAD_CASE(true, 2, 3);
    MOE_GRAD_CASE(true, 2, 2);
    MOE_GRAD_CASE(true, 2, 1);
#undef MOE_GRAD_CASE
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  ColSums cs{partial, s.rows > 0 ? (int)grid_of(s.rows, p) : 0, s.d, a.w_post,
             channel ? static_cast<const float*>(a.gate) : nullptr, a.dw_post,
             channel ? static_cast<float*>(a.dgate) : nullptr, a.dw_next, accumulate};
  return launch_kernel(norm_columns_kernel, dim3((s.d + 31) / 32, 2), dim3(kColThreads), 0, st,
                       false, cs);
}

}  // namespace moe
