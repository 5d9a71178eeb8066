// RMS norms before and after a block, fused with the block's gate, the residual's scale and the
// next block's norm, and their gradients (the formulas stand at the kernels). Each reads its inputs
// from HBM once and writes its outputs once.
//
// A CTA takes rows blockIdx.x, blockIdx.x + gridDim.x, ... and a thread the same columns of each: 8
// a vector, VPT vectors. The weights of a thread's columns stay in its registers for all rows, and
// so do the gradients' column sums. Rows come through a ring of stages in shared memory that holds
// the next rows' copies in flight; a thread reads only what its own cp.async brought, so the ring
// needs no barrier. A reduction over a row has one barrier, between its warps' partial sums.
//
// Measured, 16384 rows of 7168, bf16 stream, channel gate, both norms: forward 143 us, 6.6 TB/s,
// bound by memory (195 with one vector a thread and single fp32 operations); gradient 244 us, 5.8
// TB/s, where the instructions of its two passes and the wait for a row's sums share the SM's one
// CTA with the copies (486 in its first form). 2048 rows, fp32 stream: norm_in's gradient 37.5 us,
// 5.5 TB/s. A row alone: 2.7 us.
#include "moe_device.cuh"
#include "moe_f32x2.cuh"

namespace moe {
namespace {

constexpr int kGpuSms = 152;   // grids are sized for GB300
constexpr int kWsHead = 256;   // the status word's place at the head of the scratch

struct Shape {
  int rows, d;
  unsigned vecs;   // d / 8
  float eps, res, out;
  int gate;
};

// 8 columns as fp32 pairs.
struct F8 {
  f32x2 p[4];
};
__device__ __forceinline__ F8 all(f32x2 v) { return F8{{v, v, v, v}}; }
__device__ __forceinline__ F8 mul(const F8& a, const F8& b) {
  return F8{{mul2(a.p[0], b.p[0]), mul2(a.p[1], b.p[1]), mul2(a.p[2], b.p[2]),
             mul2(a.p[3], b.p[3])}};
}
__device__ __forceinline__ F8 mul(const F8& a, f32x2 b) { return mul(a, all(b)); }
__device__ __forceinline__ F8 fma(const F8& a, const F8& b, const F8& c) {
  return F8{{fma2(a.p[0], b.p[0], c.p[0]), fma2(a.p[1], b.p[1], c.p[1]),
             fma2(a.p[2], b.p[2], c.p[2]), fma2(a.p[3], b.p[3], c.p[3])}};
}
__device__ __forceinline__ F8 fma(const F8& a, f32x2 b, const F8& c) { return fma(a, all(b), c); }
// adds the products of the columns to a pair of sums
__device__ __forceinline__ void dot(const F8& a, const F8& b, f32x2& sum) {
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma2(a.p[i], b.p[i], sum);
}

// Vector v of a row in an array of fp32 (WIDE) or bf16, each access 16 bytes a thread where it can
// be. With a bf16 stream a vector is 8 consecutive columns. With an fp32 stream (SPLIT) it is 4
// columns of the row's first half and 4 of its second, so that neighbouring threads take
// neighbouring 16 bytes of the fp32 arrays and 8 of the bf16 ones; 8 consecutive columns would
// leave every second 16 bytes to the other access of the thread (norm_in's gradient, 2048 x 7168:
// 55 -> 48 us).
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ F8 read8(const char* row, unsigned v, unsigned vecs) {
  if (WIDE) {
    const ulonglong2* at = reinterpret_cast<const ulonglong2*>(row);
    const ulonglong2 a = at[SPLIT ? v : 2 * v], b = at[SPLIT ? vecs + v : 2 * v + 1];
    return F8{{a.x, a.y, b.x, b.y}};
  }
  uint2 a, b;
  if (SPLIT) {
    a = reinterpret_cast<const uint2*>(row)[v], b = reinterpret_cast<const uint2*>(row)[vecs + v];
  } else {
    const uint4 u = reinterpret_cast<const uint4*>(row)[v];
    a = make_uint2(u.x, u.y), b = make_uint2(u.z, u.w);
  }
  return F8{{pair_of_bf16(a.x), pair_of_bf16(a.y), pair_of_bf16(b.x), pair_of_bf16(b.y)}};
}
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ void write8(char* row, unsigned v, unsigned vecs, const F8& f) {
  if (WIDE) {
    ulonglong2* at = reinterpret_cast<ulonglong2*>(row);
    at[SPLIT ? v : 2 * v] = make_ulonglong2(f.p[0], f.p[1]);
    at[SPLIT ? vecs + v : 2 * v + 1] = make_ulonglong2(f.p[2], f.p[3]);
    return;
  }
  const uint2 a = make_uint2(bf16_of_pair(f.p[0]), bf16_of_pair(f.p[1]));
  const uint2 b = make_uint2(bf16_of_pair(f.p[2]), bf16_of_pair(f.p[3]));
  if (SPLIT) {
    reinterpret_cast<uint2*>(row)[v] = a;
    reinterpret_cast<uint2*>(row)[vecs + v] = b;
  } else {
    reinterpret_cast<uint4*>(row)[v] = make_uint4(a.x, a.y, b.x, b.y);
  }
}
// A vector of a weight, `none` where there is no weight or no column.
template <bool SPLIT>
__device__ __forceinline__ F8 weights(const float* w, unsigned v, unsigned vecs, float none) {
  if (!w || v >= vecs) return all(both(none));
  return read8<true, SPLIT>(reinterpret_cast<const char*>(w), v, vecs);
}

__device__ __forceinline__ void copy16(char* smem, const char* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(smem)), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void copy8(char* smem, const char* gmem) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_addr(smem)), "l"(gmem)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sums over the CTA that every thread gets, in a fixed order. buf: two halves of 32 floats a sum,
// used in turn (flip), so that one barrier a reduction is enough.
__device__ __forceinline__ float lanes_xor(float v, int o) {
  return __shfl_xor_sync(0xffffffffu, v, o);
}
__device__ __forceinline__ void cta_sum(float& v, float* buf, int& flip) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += lanes_xor(v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* b = buf + flip * 32;
  flip ^= 1;
  if (lane == 0) b[warp] = v;
  __syncthreads();
  v = lane < warps ? b[lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += lanes_xor(v, o);
}
// Three sums over a warp in six shuffles: lanes that have handed on one go on with another. Lane 0
// ends with the first, lane 16 with the second, lane 8 with the third.
__device__ __forceinline__ float lanes_sum3(const float (&v)[3]) {
  const bool up = threadIdx.x & 16, third = threadIdx.x & 8;
  float a = (up ? v[1] : v[0]) + lanes_xor(up ? v[0] : v[1], 16);
  const float c = v[2] + lanes_xor(v[2], 16);
  a = (third ? c : a) + lanes_xor(third ? a : c, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) a += lanes_xor(a, o);
  return a;
}
__device__ __forceinline__ void cta_sum3(float (&v)[3], float* buf, int& flip) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float a = lanes_sum3(v);
  if (warps > 1) {
    float* b = buf + flip * 96;
    flip ^= 1;
    if (lane == 0) b[warp] = a;
    if (lane == 16) b[32 + warp] = a;
    if (lane == 8) b[64 + warp] = a;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) v[i] = lane < warps ? b[32 * i + lane] : 0.0f;
    a = lanes_sum3(v);
  }
  v[0] = __shfl_sync(0xffffffffu, a, 0);
  v[1] = __shfl_sync(0xffffffffu, a, 16);
  v[2] = __shfl_sync(0xffffffffu, a, 8);
}

// 1/sqrt(mean + eps). (rsqrtf is off by 2 ulp at most, less than the sum of a row of squares.)
__device__ __forceinline__ float inv_root(float sum, float inv_d, float eps) {
  return rsqrtf(__fmaf_rn(sum, inv_d, eps));
}

// A row of an array. (Its address is the same in all threads and the offset in it has 32 bits: that
// is one addressing mode, where a 64-bit offset of each thread costs several instructions an
// access.)
template <bool WIDE>
__device__ __forceinline__ const char* row_of(const void* array, size_t row, unsigned vecs) {
  return static_cast<const char*>(array) + row * vecs * (WIDE ? 32u : 16u);
}
template <bool WIDE>
__device__ __forceinline__ char* row_of(void* array, size_t row, unsigned vecs) {
  return static_cast<char*>(array) + row * vecs * (WIDE ? 32u : 16u);
}
// Starts the copy of vector v of a row to its place in a stage.
template <bool WIDE, bool SPLIT>
__device__ __forceinline__ void fetch8(char* to, const char* row, unsigned v, unsigned vecs) {
  if (WIDE) {
    copy16(to + v * 16, row + v * 16);
    copy16(to + (vecs + v) * 16, row + (vecs + v) * 16);
  } else if (SPLIT) {
    copy8(to + v * 8, row + v * 8);
    copy8(to + (vecs + v) * 8, row + (vecs + v) * 8);
  } else {
    copy16(to + v * 16, row + v * 16);
  }
}

// Most threads of a CTA that takes VPT vectors a thread, and the CTAs of that size an SM holds.
constexpr int most_threads(int vpt) { return vpt == 1 ? 128 : 512; }
constexpr int most_ctas(int vpt) { return vpt == 1 ? 6 : 1; }

template <bool F32, int VPT, int STAGES>
__global__ void __launch_bounds__(most_threads(VPT), most_ctas(VPT))
    norm_kernel(Shape s, NormFwd a, int stage_bytes) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float sums[2 * 32];
  constexpr unsigned kSt = F32 ? 32 : 16;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, next = a.w_next != nullptr;
  const bool elem = s.gate == MOE_GATE_ELEMENT;
  const int off_y = s.vecs * kSt, off_g = off_y + (has_y ? s.vecs * 16 : 0);
  const int step = gridDim.x;
  const float inv_d = 1.0f / static_cast<float>(s.d);
  int flip = 0, slot = 0;
  const auto fetch = [&](long long row, int to) {
    if (row < s.rows) {
      char* st = ring + to * stage_bytes;
      const char* x = row_of<F32>(a.x, row, s.vecs);
      const char* y = row_of<false>(a.y, row, s.vecs);
      const char* g = row_of<false>(a.gate, row, s.vecs);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const unsigned v = threadIdx.x + k * blockDim.x;
        if (v >= s.vecs) continue;
        fetch8<F32, F32>(st, x, v, s.vecs);
        if (has_y) fetch8<false, F32>(st + off_y, y, v, s.vecs);
        if (elem) fetch8<false, F32>(st + off_g, g, v, s.vecs);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(blockIdx.x + (long long)i * step, i);
  // what a column's normed output is multiplied by: out, the channel gate and the weight; and the
  // next norm's weight
  F8 gw[VPT], wn[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const unsigned v = threadIdx.x + k * blockDim.x;
    const float* g = s.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr;
    gw[k] = mul(weights<F32>(a.w_post, v, s.vecs, 1.0f), weights<F32>(g, v, s.vecs, 1.0f));
    gw[k] = mul(gw[k], both(s.out));
    wn[k] = weights<F32>(a.w_next, v, s.vecs, 0.0f);
  }
  for (long long row = blockIdx.x; row < s.rows; row += step) {
    const int free_slot = slot == 0 ? STAGES - 1 : slot - 1;
    if (STAGES == 1) fetch(row, 0);
    float factor = 1.0f;   // of this row's y
    if (s.gate == MOE_GATE_TOKEN) factor = static_cast<const float*>(a.gate)[row];
    copies_wait<(STAGES > 1 ? STAGES - 2 : 0)>();
    const char* st = ring + slot * stage_bytes;
    slot = slot + 1 == STAGES ? 0 : slot + 1;
    if (post) {
      f32x2 q = both(0.0f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const unsigned v = threadIdx.x + k * blockDim.x;
        if (v >= s.vecs) continue;
        const F8 y = read8<false, F32>(st + off_y, v, s.vecs);
        dot(y, y, q);
      }
      float sum = sum_of(q);
      cta_sum(sum, sums, flip);
      const float r = inv_root(sum, inv_d, s.eps);
      if (threadIdx.x == 0 && a.rstd_y) a.rstd_y[row] = r;
      factor *= r;
    }
    F8 h[VPT];
    f32x2 q = both(0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const unsigned v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      h[k] = read8<F32, F32>(st, v, s.vecs);
      if (has_y) {
        F8 y = read8<false, F32>(st + off_y, v, s.vecs);
        if (elem) y = mul(y, read8<false, F32>(st + off_g, v, s.vecs));
        h[k] = fma(mul(y, both(factor)), gw[k], mul(h[k], both(s.res)));
        write8<F32, F32>(row_of<F32>(a.h, row, s.vecs), v, s.vecs, h[k]);
      }
      dot(h[k], h[k], q);
    }
    if (STAGES > 1) fetch(row + (long long)(STAGES - 1) * step, free_slot);
    if (!next) continue;
    float sum = sum_of(q);
    cta_sum(sum, sums, flip);
    const float r = inv_root(sum, inv_d, s.eps);
    if (threadIdx.x == 0 && a.rstd_h) a.rstd_h[row] = r;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const unsigned v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      write8<false, F32>(row_of<false>(a.n, row, s.vecs), v, s.vecs,
                         mul(mul(h[k], both(r)), wn[k]));
    }
  }
}

// The gradient of the norm before a block, the residual's joined, has code of its own: 2048 rows of
// 7168 in fp32 37.5 us, 48 in the form for all cases. (For both norms behind a block such code has
// a quarter fewer instructions, too, but took 253 us against 244, 16384 rows of 7168.)
enum { kAnyForm, kInForm };

// The gradient. A row's three sums come from one pass, since the mean that the norm behind the
// block needs is linear in G: with u = out gate w_post yh, and a = dn w_next,
//   sum u G = sum u (dh + r_h a) - r_h mean(a hh) sum u hh.
// The second pass reads the row again from the ring; the next row's copies go out between the two,
// into the stage of the row before. Column sums: acc_y = sum out G gate yh (without a channel gate,
// which like w_post is the same in all rows: dw_post = gate acc_y, dgate = w_post acc_y) and acc_n
// = sum dn hh. With 4 vectors a thread the weights do not fit the registers beside those: they are
// read again for each row, from L2.
template <bool F32, int VPT, int STAGES, int FORM>
__global__ void __launch_bounds__(most_threads(VPT), most_ctas(VPT))
    norm_grad_kernel(Shape s, NormGrad a, int stage_bytes, float* partial) {
  extern __shared__ __align__(16) char ring[];
  __shared__ float sums[2 * 32 * 3];
  constexpr unsigned kSt = F32 ? 32 : 16;
  constexpr bool kKeep = VPT <= 2;
  constexpr bool kAny = FORM == kAnyForm;
  const bool post = kAny && a.w_post, next = !kAny || a.w_next, has_dh = !kAny || a.dh;
  const bool elem = kAny && s.gate == MOE_GATE_ELEMENT, token = kAny && s.gate == MOE_GATE_TOKEN;
  const bool has_y = kAny && (post || s.gate != MOE_GATE_NONE);   // y itself is needed
  const bool is_out = kAny && a.dy;   // the norm before a block has no y side
  const bool dot_y = post || token;
  const float* channel = s.gate == MOE_GATE_CHANNEL ? static_cast<const float*>(a.gate) : nullptr;
  const int off_h = has_dh ? s.vecs * kSt : 0;
  const int off_n = off_h + (next ? s.vecs * kSt : 0);
  const int off_y = off_n + (next ? s.vecs * 16 : 0);
  const int off_g = off_y + (has_y ? s.vecs * 16 : 0);
  const int step = gridDim.x;
  const float inv_d = 1.0f / static_cast<float>(s.d);
  int flip = 0, slot = 0;
  const auto fetch = [&](long long row, int to) {
    if (row < s.rows) {
      char* st = ring + to * stage_bytes;
      const char* dh = row_of<F32>(a.dh, row, s.vecs);
      const char* h = row_of<F32>(a.h, row, s.vecs);
      const char* dn = row_of<false>(a.dn, row, s.vecs);
      const char* y = row_of<false>(a.y, row, s.vecs);
      const char* g = row_of<false>(a.gate, row, s.vecs);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const unsigned v = threadIdx.x + k * blockDim.x;
        if (v >= s.vecs) continue;
        if (has_dh) fetch8<F32, F32>(st, dh, v, s.vecs);
        if (next) {
          fetch8<F32, F32>(st + off_h, h, v, s.vecs);
          fetch8<false, F32>(st + off_n, dn, v, s.vecs);
        }
        if (has_y) fetch8<false, F32>(st + off_y, y, v, s.vecs);
        if (elem) fetch8<false, F32>(st + off_g, g, v, s.vecs);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(blockIdx.x + (long long)i * step, i);
  const auto weight_y = [&](unsigned v) {
    F8 w = weights<F32>(a.w_post, v, s.vecs, 1.0f);
    return channel ? mul(w, weights<F32>(channel, v, s.vecs, 1.0f)) : w;
  };
  F8 keep_y[kKeep ? VPT : 1], keep_n[kKeep ? VPT : 1], acc_y[VPT], acc_n[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const unsigned v = threadIdx.x + k * blockDim.x;
    if (kKeep) {
      keep_y[k] = weight_y(v);
      keep_n[k] = weights<F32>(a.w_next, v, s.vecs, 0.0f);
    }
    acc_y[k] = acc_n[k] = all(0);
  }
  // a row's factors are loaded a row ahead
  const auto factors = [&](long long row, float& rh, float& ry, float& gt) {
    if (row >= s.rows) return;
    if (next) rh = a.rstd_h[row];
    if (post) ry = a.rstd_y[row];
    if (token) gt = static_cast<const float*>(a.gate)[row];
  };
  float rh_next = 0.0f, ry_next = 1.0f, gt_next = 1.0f;
  factors(blockIdx.x, rh_next, ry_next, gt_next);
  for (long long row = blockIdx.x; row < s.rows; row += step) {
    // the row that is STAGES - 1 ahead goes into the stage of the row before this one
    const int free_slot = slot == 0 ? STAGES - 1 : slot - 1;
    if (STAGES == 1) fetch(row, 0);
    const float rh = rh_next, ry = ry_next, gt = gt_next;
    factors(row + step, rh_next, ry_next, gt_next);
    copies_wait<(STAGES > 1 ? STAGES - 2 : 0)>();
    const char* st = ring + slot * stage_bytes;
    slot = slot + 1 == STAGES ? 0 : slot + 1;

    const f32x2 rh2 = both(rh);
    F8 G[VPT];   // dh + rh a, of which the next norm's mean is still to be taken
    f32x2 qa = 0, qg = 0, qh = 0;   // sums of a h, u (dh + rh a) and u h (h, u: without their r)
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const unsigned v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      F8 h = all(0);
      G[k] = h;
      if (has_dh) G[k] = read8<F32, F32>(st, v, s.vecs);
      if (next) {
        h = read8<F32, F32>(st + off_h, v, s.vecs);
        const F8 dn = read8<false, F32>(st + off_n, v, s.vecs);
        acc_n[k] = fma(dn, mul(h, rh2), acc_n[k]);
        const F8 d = mul(dn, kKeep ? keep_n[k] : weights<F32>(a.w_next, v, s.vecs, 0.0f));
        dot(d, h, qa);
        G[k] = fma(d, rh2, G[k]);
      }
      if (dot_y) {
        F8 u = mul(read8<false, F32>(st + off_y, v, s.vecs),
                   kKeep ? keep_y[k] : weight_y(v));
        if (elem) u = mul(u, read8<false, F32>(st + off_g, v, s.vecs));
        dot(u, G[k], qg);
        dot(u, h, qh);
      }
    }
    if (STAGES > 1) fetch(row + (long long)(STAGES - 1) * step, free_slot);
    float q[3] = {sum_of(qa), sum_of(qg), sum_of(qh)};
    if (next || dot_y) cta_sum3(q, sums, flip);
    const float c1 = rh * q[0] * inv_d;                                // mean a hh
    const float along = s.out * ry * (q[1] - rh * c1 * (rh * q[2]));   // sum out G s, no token gate
    const float mean = gt * along * inv_d;
    if (token && a.dgate && threadIdx.x == 0) static_cast<float*>(a.dgate)[row] = along;
    const f32x2 hc = both(-c1 * rh * rh), res = both(s.res);
    // dy = ry (u gw - yh mean), u = out gate G; acc_y adds u yh: both from u ry and y itself
    const f32x2 out = both(s.out * gt * ry), back = both(-ry * ry * mean);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const unsigned v = threadIdx.x + k * blockDim.x;
      if (v >= s.vecs) continue;
      if (next) G[k] = fma(read8<F32, F32>(st + off_h, v, s.vecs), hc, G[k]);
      if (a.dx) write8<F32, F32>(row_of<F32>(a.dx, row, s.vecs), v, s.vecs, mul(G[k], res));
      if (!is_out) continue;
      F8 u = mul(G[k], out), y = all(0);
      const F8 gw = kKeep ? keep_y[k] : weight_y(v);
      if (has_y) y = read8<false, F32>(st + off_y, v, s.vecs);
      if (elem) {
        if (a.dgate)
          write8<false, F32>(row_of<false>(a.dgate, row, s.vecs), v, s.vecs, mul(mul(u, y), gw));
        u = mul(u, read8<false, F32>(st + off_g, v, s.vecs));
      }
      acc_y[k] = fma(u, y, acc_y[k]);
      u = mul(u, gw);
      write8<false, F32>(row_of<false>(a.dy, row, s.vecs), v, s.vecs, post ? fma(y, back, u) : u);
    }
  }
  pdl_trigger();
  if (!partial) return;
  // partial sums of this CTA: [cta][d] acc_y if there is a y side, [cta][d] acc_n if there is a
  // next
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const unsigned v = threadIdx.x + k * blockDim.x;
    if (v >= s.vecs) continue;
    if (has_y) write8<true, F32>(row_of<true>(partial, blockIdx.x, s.vecs), v, s.vecs, acc_y[k]);
    if (next)
      write8<true, F32>(row_of<true>(partial, blockIdx.x + (has_y ? gridDim.x : 0), s.vecs), v,
                        s.vecs, acc_n[k]);
  }
}

// Column sums over the CTAs' partial sums: a warp's lanes are 32 columns, a CTA's warps take parts
// of the CTAs one after another, joined in order. The grid's first half (or all of it) takes the
// sums over yh, if there are any, the other one those over hh.
struct ColSums {
  const float* partial;
  int ctas, d;
  int sides;                         // 1: yh, 2: hh, 3: both
  const float *w_post, *gate;        // gate: a channel gate, else NULL (and NULL without rows)
  float *dw_post, *dgate, *dw_next;  // NULL: not wanted; dgate: a channel gate's
  int accumulate;
};
constexpr int kColThreads = 512;
__global__ void __launch_bounds__(kColThreads) norm_columns_kernel(ColSums a) {
  __shared__ float part[kColThreads / 32][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  const bool y_side = blockIdx.y == 0 && (a.sides & 1);
  pdl_wait();
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
    put(a.dgate, w * sum);
  } else {
    put(a.dw_next, sum);
  }
}

// Vectors a thread, threads of a CTA and the CTAs that an SM takes at once. Two vectors where they
// fit a CTA of 512 threads, whose registers then hold weights and sums of 16 columns each: 16384
// rows of 7168 forward 144 us, with one vector and 896 threads 195; gradient of 32768 rows of 1504
// 108 us, with one 130. Up to 1024 columns one vector: 65536 rows of 520 forward 66 us, gradient
// 126, with two 73 and 132. Above 8192 columns four, whose sums leave no registers for the weights.
struct Plan {
  int vpt, threads, per_sm;
};
Plan plan_of(int d) {
  const int vecs = d / 8;
  Plan p;
  p.vpt = vecs <= 128 ? 1 : vecs <= 1024 ? 2 : 4;
  p.threads = ((vecs + p.vpt - 1) / p.vpt + 31) / 32 * 32;
  p.per_sm = most_threads(p.vpt) * most_ctas(p.vpt) / p.threads;
  return p;
}
unsigned grid_of(int rows, const Plan& p) {
  const int most = kGpuSms * p.per_sm;
  return rows < most ? rows : most;
}

// Stages of the ring: as many as the SM's CTAs can have, 4 at most. (The widest row of a gradient,
// 16384 columns with an fp32 stream and an element gate, is 224 KB: one stage.)
int stages_of(size_t stage, const Plan& p) {
  const size_t all = stage * p.per_sm;
  return all * 4 <= 220 * 1024 ? 4 : all * 3 <= 220 * 1024 ? 3 : all * 2 <= 224 * 1024 ? 2 : 1;
}

template <typename K>
cudaError_t set_smem(K kern, size_t bytes) {   // (1 KB more: the static arrays count, too)
  return ensure_smem_limit(reinterpret_cast<const void*>(kern), bytes + 1024);
}

template <bool F32, int VPT, int STAGES>
cudaError_t run(const Shape& s, const NormFwd& a, const Plan& p, int stage, float*,
                cudaStream_t st) {
  auto kern = norm_kernel<F32, VPT, STAGES>;
  const size_t smem = (size_t)STAGES * stage;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid_of(s.rows, p)), dim3(p.threads), smem, st, false, s, a,
                       stage);
}
template <bool F32, int VPT, int STAGES>
cudaError_t run(const Shape& s, const NormGrad& a, const Plan& p, int stage, float* partial,
                cudaStream_t st) {
  auto kern = a.dh && !a.dy ? norm_grad_kernel<F32, VPT, STAGES, kInForm>
                            : norm_grad_kernel<F32, VPT, STAGES, kAnyForm>;
  const size_t smem = (size_t)STAGES * stage;
  const cudaError_t e = set_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3(grid_of(s.rows, p)), dim3(p.threads), smem, st, false, s, a, stage,
                       partial);
}
template <bool F32, int VPT, typename A>
cudaError_t run_stages(const Shape& s, const A& a, const Plan& p, int stage, float* partial,
                       cudaStream_t st) {
  switch (stages_of(stage, p)) {
    case 4: return run<F32, VPT, 4>(s, a, p, stage, partial, st);
    case 3: return run<F32, VPT, 3>(s, a, p, stage, partial, st);
    case 2: return run<F32, VPT, 2>(s, a, p, stage, partial, st);
    default: return run<F32, VPT, 1>(s, a, p, stage, partial, st);
  }
}
template <bool F32, typename A>
cudaError_t run_any(const Shape& s, const A& a, const Plan& p, int stage, float* partial,
                    cudaStream_t st) {
  return p.vpt == 1   ? run_stages<F32, 1>(s, a, p, stage, partial, st)
         : p.vpt == 2 ? run_stages<F32, 2>(s, a, p, stage, partial, st)
                      : run_stages<F32, 4>(s, a, p, stage, partial, st);
}

Shape shape_of(const moe_norm_cfg& c) {
  return Shape{c.rows, c.d, (unsigned)(c.d / 8), c.eps, c.res_scale, c.out_scale, c.gate};
}

}  // namespace

size_t norm_ws_bytes(int rows, int d) {
  return kWsHead + (size_t)grid_of(rows, plan_of(d)) * d * 2 * sizeof(float);
}

cudaError_t launch_norm(const moe_norm_cfg& c, const NormFwd& a, cudaStream_t st) {
  const Shape s = shape_of(c);
  const Plan p = plan_of(c.d);
  const bool f32 = c.stream_dtype == MOE_F32;
  const int stage = (int)s.vecs * ((f32 ? 32 : 16) + (a.y ? 16 : 0) +
                              (c.gate == MOE_GATE_ELEMENT ? 16 : 0));
  return f32 ? run_any<true>(s, a, p, stage, nullptr, st)
             : run_any<false>(s, a, p, stage, nullptr, st);
}

cudaError_t launch_norm_grad(const moe_norm_cfg& c, const NormGrad& a, bool accumulate, void* ws,
                             cudaStream_t st) {
  const Shape s = shape_of(c);
  const Plan p = plan_of(c.d);
  const bool f32 = c.stream_dtype == MOE_F32, next = a.w_next != nullptr;
  const bool channel = c.gate == MOE_GATE_CHANNEL;
  const bool has_y = a.w_post || c.gate != MOE_GATE_NONE;
  const int b = f32 ? 32 : 16;
  const int stage = (int)s.vecs * ((a.dh ? b : 0) + (next ? b + 16 : 0) + (has_y ? 16 : 0) +
                              (c.gate == MOE_GATE_ELEMENT ? 16 : 0));
  const bool sums = a.dw_post || a.dw_next || (channel && a.dgate);
  float* partial =
      sums ? reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHead) : nullptr;
  if (s.rows > 0) {
    const cudaError_t e = f32 ? run_any<true>(s, a, p, stage, partial, st)
                              : run_any<false>(s, a, p, stage, partial, st);
    if (e != cudaSuccess) return e;
  }
  if (!sums) return cudaSuccess;
  const int sides = (has_y ? 1 : 0) | (next ? 2 : 0);
  ColSums cs{partial, s.rows > 0 ? (int)grid_of(s.rows, p) : 0, s.d, sides, a.w_post,
             channel ? static_cast<const float*>(a.gate) : nullptr, a.dw_post,
             channel ? static_cast<float*>(a.dgate) : nullptr, a.dw_next, accumulate};
  return launch_kernel(norm_columns_kernel, dim3((s.d + 31) / 32, sides == 3 ? 2 : 1),
                       dim3(kColThreads), 0, st, s.rows > 0, cs);
}

}  // namespace moe
