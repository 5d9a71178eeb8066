// Matrix products grouped by expert over ragged row counts: forward, gradient of the rows and
// gradient of the weights. Group e owns rows [s_e, s_e + c_e) of the row tensors:
//   fwd: y[r][i]    = sum_j x[r][j] W_e[i][j]
//   dx : dx[r][j]   = sum_i dy[r][i] W_e[i][j]
//   dw : dW_e[i][j] = sum_r dy[r][i] x[r][j]   (r over the group's rows)
// bf16 operands, fp32 sums, each result rounded once where it is stored in bf16.
//
// One kernel for the three, on the 5th-generation tensor cores with CTA pairs (cta_group::2,
// M = 256). M is always the output's contiguous dimension, so an accumulator row (one tensor-
// memory lane, one thread of the epilogue) is an output column and a warp stores 32 consecutive
// columns at a time; N is the output's row:
//        M (256)        N (up to TN)            reduction    A                  B
//   fwd  columns of y   rows of the group       k            W_e, K-major       x, K-major
//   dx   columns of dx  rows of the group       n            W_e, MN-major      dy, K-major
//   dw   columns of dW  rows of dW              the rows     x, MN-major        dy, MN-major
// Weights come through 3-D tensor maps, so what a tile reads past a group's own matrix is zero.
// In fwd and dx, rows past a group's end only feed accumulator columns that are not stored. In
// dw they would be summed: the last k-step of a group zeroes what follows its rows in shared
// memory before the MMA reads it (0 x NaN is not 0, so both operands are).
//
// Each pair walks the units (group, 256 output columns, N tile) from its number in steps of the
// pairs; a group's units are weight-tile-major, so pairs that run side by side share a weight
// tile through L2. The tables of the units are built by every CTA from the counts itself: one
// launch, no schedule kernel.
//
// Roles in a CTA (one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer (leader CTA), warp 2
// zeroes dw's tails, the others the epilogue. Loads of both CTAs count on
// the leader's full barriers, its commits free the stages of both. Accumulators are double
// buffered. Every wait is bounded.
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

// Warps 0, 1 and 2 load, issue the MMAs and zero tails; the others are the epilogue: two warps per
// tensor-memory quarter, or four where the sums of a tile are held in registers (fp32 weight
// gradients: 64 columns a thread).
template <bool F32>
struct GroupedThreads {
  static constexpr int kEpi = F32 ? 16 : 8;
  static constexpr int kAll = (3 + kEpi) * 32;
};
// fp32 weight gradients: k-steps per tensor-core sum. The tensor core truncates as it adds, an
// error that grows with the number of additions (2.1e-6 of the result after 2048 products,
// 4.4e-6 after 4096, against 4e-7 for rounded fp32 sums); sums of 512 rows are therefore read
// out and added in registers, rounded.
constexpr int kSumSteps = 8;
// bf16 epilogue: a warp turns 32 output rows x 32 columns around in shared memory, rows 80 bytes
// apart (64 used), which keeps the eight 16-byte rows of a matrix store in different banks.
constexpr int kTurnPitch = 80, kTurnBytes = 32 * kTurnPitch;

struct GroupedArgs {
  const int32_t* counts;
  void* out;
  uint32_t* status;
  int rows, E, n, k;
  int cols;       // output columns (M)
  int red;        // fwd, dx: length of the reduction
  int mt;         // ceil(cols / 256)
  int accumulate;
};

template <int TN, int STAGES, bool F32>
struct GroupedShape {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = TN / 2 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * TN;
  static constexpr int TURN = F32 ? 0 : GroupedThreads<F32>::kEpi * kTurnBytes;
  static constexpr int SMEM = STAGES * STAGE_BYTES + TURN + 1024 + 512;
  static_assert(B_BYTES % 1024 == 0 && TMEM_COLS <= 512 && TMEM_COLS >= 32, "");
};

// The groups with work, in shared memory: fwd and dx list those that have rows.
struct GroupedTables {
  int off[kMaxGroups + 1];   // first row of each group
  int live[kMaxGroups];      // fwd, dx: the groups with rows
  int n_live;
};

// One unit of work: 256 output columns (the pair's) x one N tile of one group.
struct GroupedUnit {
  int g;      // group
  int f0;     // first output column of the pair
  int n0;     // fwd, dx: first row; dw: first row of dW_g
  int nlen;   // rows of the tile
  int r0;     // dw: the group's first row
  int red;    // length of the reduction
  int nt;     // N tiles that read this unit's weight tile
};

// Walks a pair's units: numbers pair, pair + pairs, ... of the groups' units one group after the
// other, weight-tile-major (unit m * nt + j of a group: N tile j of its 256 columns number m).
// fwd, dx: a group of c rows has nt = ceil(c / TN) N tiles of equal size (to 32 rows, the step of
// an MMA's N) rather than full ones and a rest, which would cost a whole pass over the weight
// tile for a few rows (16384 rows over 32 experts, about half of them just over 512: forward
// 796 -> 680 us).
template <int DIR, int TN>
struct GroupedWalk {
  const GroupedArgs& a;
  const GroupedTables& tab;
  int i, local, step, nt, w, base, len;

  __device__ __forceinline__ GroupedWalk(const GroupedArgs& a_, const GroupedTables& t_, int pair,
                                         int pairs)
      : a(a_), tab(t_), i(0), local(pair), step(pairs) {
    load();
    settle();
  }
  __device__ __forceinline__ int groups() const {
    return DIR == kGroupedDw ? a.E : tab.n_live;
  }
  __device__ __forceinline__ bool more() const { return i < groups(); }
  __device__ __forceinline__ void load() {   // the group at position i
    if (DIR == kGroupedDw) {
      nt = (a.n + TN - 1) / TN;
      w = TN;
    } else if (i < tab.n_live) {
      const int g = tab.live[i];
      base = tab.off[g];
      len = tab.off[g + 1] - base;
      nt = (len + TN - 1) / TN;
      w = nt == 1 ? TN : ((len + nt - 1) / nt + 31) & ~31;
    }
  }
  __device__ __forceinline__ void settle() {
    while (more() && local >= nt * a.mt) {
      local -= nt * a.mt;
      ++i;
      load();
    }
  }
  __device__ __forceinline__ void next() {
    local += step;
    settle();
  }
  __device__ __forceinline__ GroupedUnit unit() const {
    GroupedUnit r;
    const int m = nt == 1 ? local : local / nt;
    const int j = local - m * nt;
    r.f0 = m * 256;
    r.nt = nt;
    if (DIR == kGroupedDw) {
      r.g = i;
      r.n0 = j * TN;
      r.nlen = min(TN, a.n - r.n0);
      r.r0 = tab.off[i];
      r.red = tab.off[i + 1] - r.r0;
    } else {
      r.g = tab.live[i];
      r.n0 = base + j * w;
      r.nlen = min(w, len - j * w);
      r.r0 = 0;
      r.red = a.red;
    }
    return r;
  }
};

// A whole warp's wait: every lane gets the same answer, so the warp leaves its loop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status, uint64_t limit_ns = kWaitLimitNs) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status, limit_ns));
}

// Zeroes the reduction rows [from, to) of a stage's MN-major boxes (128-byte rows; the swizzle
// permutes bytes inside a row only) and orders the writes before the tensor core's reads.
__device__ __forceinline__ void zero_rows(uint8_t* stage, int boxes, int from, int to, int lane) {
  for (int b = lane >> 3; b < boxes; b += 4)   // eight lanes a row
    for (int p = from; p < to; ++p)
      *reinterpret_cast<uint4*>(stage + b * 8192 + p * 128 + (lane & 7) * 16) =
          make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

template <int DIR, int TN, int STAGES, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GroupedThreads<F32>::kAll, 1)
    grouped_kernel(const GroupedArgs a, const __grid_constant__ CUtensorMap mapA,
                   const __grid_constant__ CUtensorMap mapB) {
  using S = GroupedShape<TN, STAGES, F32>;
  constexpr bool kDw = DIR == kGroupedDw;
  constexpr int kEpiWarps = GroupedThreads<F32>::kEpi;
  constexpr int kBoxesB = kDw ? TN / 128 : 0;
  static_assert(!kDw || TN >= 128, "dw: whole 64-column boxes");
  extern __shared__ uint8_t smem_raw[];
  __shared__ GroupedTables tab;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* turn = smem + STAGES * S::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + S::TURN);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  // dw, steps whose tail is zeroed: each CTA's loads count on its own tail barrier; the leader's
  // ptail says that the peer has zeroed its part
  uint64_t* tail = tempty + 2;
  uint64_t* ptail = tail + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ptail + STAGES);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
      mbar_init(&tail[i], 1);
      mbar_init(&ptail[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch_map(&mapA);
    tma_prefetch_map(&mapB);
  }
  group_offsets(a.counts, a.E, a.rows, tab.off, a.status);
  if (!kDw && warp == 0) {
    int at = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const bool has = e < a.E && tab.off[e + 1] > tab.off[e];
      const uint32_t m = __ballot_sync(0xffffffffu, has);
      if (has) tab.live[at + __popc(m & ((1u << lane) - 1u))] = e;
      at += __popc(m);
    }
    if (lane == 0) tab.n_live = at;
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, S::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the peer's barriers and tensor memory are ready
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  GroupedWalk<DIR, TN> walk(a, tab, blockIdx.x >> 1, gridDim.x >> 1);
  constexpr int kNever = 1 << 30;
  constexpr int kSum = F32 ? kSumSteps : kNever;   // k-steps per tensor-core sum

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (elect_one()) {
      const uint64_t pol_once = l2_policy_evict_first(), pol_keep = l2_policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (; walk.more() && ok; walk.next()) {
        const GroupedUnit t = walk.unit();
        // each CTA's half of the N tile, a multiple of 16 rows (an MMA takes N in steps of 32)
        const int half = ((t.nlen + 31) & ~31) >> 1;
        const int steps = (t.red + 63) >> 6;
        const uint64_t pol_a = kDw || t.nt > 1 ? pol_keep : pol_once;
        const int f = t.f0 + static_cast<int>(rank) * 128;
        const int nb = t.n0 + static_cast<int>(rank) * half;
        for (int ks = 0; ks < steps; ++ks) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * S::STAGE_BYTES;
          uint8_t* sb = sa + S::A_BYTES;
          const bool cut = kDw && (t.red - ks * 64 < 64) && (t.red & 15);
          uint32_t bar;
          if (cut) {
            mbar_arrive_expect_tx(&tail[stage], S::STAGE_BYTES);
            bar = cluster_addr(&tail[stage], rank);
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], 2 * S::STAGE_BYTES);
            bar = cluster_addr(&full[stage], 0);
          }
          if (DIR == kGroupedFwd) {
            tma_load_3d_pair(sa, &mapA, bar, ks * 64, f, t.g, pol_a);
          } else if (DIR == kGroupedDx) {
            tma_load_3d_pair(sa, &mapA, bar, f, ks * 64, t.g, pol_a);
            tma_load_3d_pair(sa + 8192, &mapA, bar, f + 64, ks * 64, t.g, pol_a);
          } else {
            tma_load_2d_pair(sa, &mapA, bar, f, t.r0 + ks * 64, pol_a);
            tma_load_2d_pair(sa + 8192, &mapA, bar, f + 64, t.r0 + ks * 64, pol_a);
          }
          if (kDw) {
#pragma unroll
            for (int j = 0; j < kBoxesB; ++j)
              tma_load_2d_pair(sb + j * 8192, &mapB, bar, nb + 64 * j, t.r0 + ks * 64, pol_keep);
          } else {
            tma_load_2d_pair(sb, &mapB, bar, ks * 64, nb, pol_keep);
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (leader) ------------------------------
    // The next stage's barrier is tested before the last MMA of a stage is issued, so that the
    // tensor pipe has work while this thread moves on.
    if (leader && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true, ready = false;
      int it = 0;
      for (; walk.more() && ok; walk.next()) {
        const GroupedUnit t = walk.unit();
        const uint32_t n_mma = static_cast<uint32_t>((t.nlen + 31) & ~31);
        const uint32_t idesc = idesc_bf16(256, n_mma) | (DIR != kGroupedFwd ? kIdescAmn : 0u) |
                               (kDw ? kIdescBmn : 0u);
        const int steps = (t.red + 63) >> 6;
        for (int k0 = 0; k0 < steps && ok; k0 += kSum) {
          const int k1 = min(steps, k0 + kSum);
          const int b = it & 1;
          if (!mbar_wait_cluster(&tempty[b], ((it >> 1) & 1) ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + b * TN;
          for (int ks = k0; ks < k1; ++ks) {
            if (!ready && !mbar_wait_cluster(&full[stage], phase, abort_flag, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_addr(smem + stage * S::STAGE_BYTES);
            const uint32_t sb = sa + S::A_BYTES;
            auto issue = [&](int kk) {
              const uint64_t da = DIR == kGroupedFwd ? smem_desc_sw128(sa + kk * 32)
                                                     : smem_desc_sw128_mn(sa + kk * 2048);
              const uint64_t db = kDw ? smem_desc_sw128_mn(sb + kk * 2048)
                                      : smem_desc_sw128(sb + kk * 32);
              mma_f16_pair(d, da, db, idesc, (ks != k0 || kk != 0) ? 1u : 0u);
            };
            uint64_t* done = &empty[stage];
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
            const int left = t.red - ks * 64;
            if (left >= 64) {
              issue(0);
              issue(1);
              issue(2);
              ready = mbar_peek_cluster(&full[stage], phase);
              issue(3);
            } else {
              ready = false;
              for (int kk = 0; kk < (left + 15) >> 4; ++kk) issue(kk);
            }
            mma_commit_pair(done);
          }
          if (ok) mma_commit_pair(&tfull[b]);
          ++it;
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------ dw: tails ------------------------------
    // For a step that ends inside a 16-row slice: wait for this CTA's own loads, zero what follows
    // the group's rows, tell the leader; the leader then completes the stage's full barrier.
    if (kDw) {
      uint32_t phases = 0;   // bit s: parity of the next use of tail[s] (and ptail[s])
      int stage = 0;
      for (; walk.more(); walk.next()) {
        const GroupedUnit t = walk.unit();
        const int steps = (t.red + 63) >> 6;
        stage = (stage + steps) % STAGES;
        if ((t.red & 15) == 0) continue;
        const int last = (stage + STAGES - 1) % STAGES;   // stage of the unit's last step
        // (many units may pass between two tails; an abort of another role ends the wait)
        const uint32_t parity = (phases >> last) & 1u;
        if (!warp_wait(&tail[last], parity, abort_flag, a.status, 30 * kWaitLimitNs)) break;
        phases ^= 1u << last;
        const int left = t.red - (steps - 1) * 64;
        zero_rows(smem + last * S::STAGE_BYTES, 2 + kBoxesB, left, (left + 15) & ~15, lane);
        bool ok = true;
        if (lane == 0) {
          if (!leader) {
            mbar_arrive_cluster(cluster_addr(&ptail[last], 0));
          } else {
            ok = mbar_wait_cluster(&ptail[last], parity, abort_flag, a.status);
            if (ok) mbar_arrive_cluster(cluster_addr(&full[last], 0));
          }
        }
        if (!__all_sync(0xffffffffu, ok)) break;
      }
    }
  } else {
    // ------------------------------ epilogue ------------------------------
    // Warp w reads lanes 32 (w % 4) .. +31 (output columns) of its part of the tile's N columns.
    const int quarter = warp & 3, part = (warp - 3) >> 2;
    int it = 0;
    bool ok = true;
    for (; walk.more() && ok; walk.next()) {
      const GroupedUnit t = walk.unit();
      const int steps = (t.red + 63) >> 6;
      const int fw = t.f0 + static_cast<int>(rank) * 128 + quarter * 32;   // the warp's columns
      const size_t row0 = (kDw ? (size_t)t.g * a.n : 0) + t.n0;
      if constexpr (F32) {
        constexpr int kCols = TN / (kEpiWarps / 4);   // of this warp, in registers
        float acc[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
        for (int k0 = 0; k0 < steps; k0 += kSum) {
          const int b = it & 1;
          if (!warp_wait(&tfull[b], (it >> 1) & 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tb =
              tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * TN + part * kCols;
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            uint32_t v[16];
            tmem_ld16(tb + c, v);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += __uint_as_float(v[j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[b], 0));
          ++it;
        }
        if (!ok) break;
        if (fw + lane >= a.cols || (a.accumulate && steps == 0)) continue;
        float* out = static_cast<float*>(a.out) + (row0 + part * kCols) * a.cols + fw + lane;
        const int mine = t.nlen - part * kCols;   // rows of this warp's part that exist
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
          float* o = out + (size_t)c * a.cols;
          if (a.accumulate) {
            float old[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              old[j] = c + j < mine ? o[(size_t)j * a.cols] : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += old[j];
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            if (c + j < mine) o[(size_t)j * a.cols] = acc[c + j];
        }
      } else {
        // 32 rows x 32 columns at a time: accumulator fragments to bf16, turned around through
        // shared memory, stored as 16-byte pieces (four lanes a row)
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
        uint8_t* mine = turn + (warp - 3) * kTurnBytes;
        const uint32_t put = smem_addr(mine) + (lane & 7) * kTurnPitch + (lane >> 3) * 16;
        const uint8_t* get = mine + (lane >> 2) * kTurnPitch + (lane & 3) * 16;
        const int fl = fw + (lane & 3) * 8;   // this lane's first column when it stores
        const bool in = fl < a.cols;          // (cols is a multiple of 8)
        const int b = it & 1;
        if (steps > 0) {
          if (!warp_wait(&tfull[b], (it >> 1) & 1, abort_flag, a.status)) break;
          tc_fence_after();
        }
        const uint32_t tb = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * TN;
        for (int c = part * 32; c < t.nlen; c += kEpiWarps * 8) {
          uint4 v[4];
          if (steps > 0) {
            uint32_t lo[16], hi[16];   // lanes 0-15 and 16-31
            tmem_ld_16x256_x4(tb + c, lo);
            tmem_ld_16x256_x4(tb + (16u << 16) + c, hi);
            tmem_ld_wait();
            auto pack = [](uint32_t x, uint32_t y) {
              return pack_bf16x2(__uint_as_float(x), __uint_as_float(y));
            };
            __syncwarp();   // the previous rows have been read
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t m[4] = {
                  pack(lo[4 * i], lo[4 * i + 1]), pack(lo[4 * i + 2], lo[4 * i + 3]),
                  pack(hi[4 * i], hi[4 * i + 1]), pack(hi[4 * i + 2], hi[4 * i + 3])};
              stmatrix_x4_trans(put + i * 8 * kTurnPitch, m);
            }
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = *reinterpret_cast<const uint4*>(get + q * 8 * kTurnPitch);
          } else {   // dw of an empty group
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = make_uint4(0, 0, 0, 0);
          }
          const int p = c + (lane >> 2);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (in && p + 8 * q < t.nlen)
              *reinterpret_cast<uint4*>(out + (row0 + p + 8 * q) * a.cols + fl) = v[q];
        }
        if (steps > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[b], 0));
          ++it;
        }
      }
    }
  }

  // an aborted role leaves copies in flight: they land long before this ends
  if (*abort_flag) __nanosleep(1000000);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the other still reads or signals it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::TMEM_COLS);
  }
}

template <int DIR, int TN, int STAGES, bool F32>
cudaError_t run_grouped_kernel(const GroupedArgs& a, const CUtensorMap& mA, const CUtensorMap& mB,
                               cudaStream_t st) {
  using S = GroupedShape<TN, STAGES, F32>;
  auto kern = grouped_kernel<DIR, TN, STAGES, F32>;
  const cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kern), S::SMEM);
  if (err != cudaSuccess) return err;
  return launch_kernel(kern, dim3(sm_count() & ~1), dim3(GroupedThreads<F32>::kAll), S::SMEM, st, false, a,
                       mA, mB);
}

// N tile of fwd and dx: the smallest that takes a group's mean rows, so that a batch of few rows
// spends its shared memory on weight stages.
int row_tile(const moe_group_cfg& c) {
  const int live = c.E < c.rows ? c.E : c.rows;
  const long long mean = (c.rows + live - 1) / live;
  return mean <= 32 ? 32 : mean <= 64 ? 64 : mean <= 128 ? 128 : 256;
}

template <int DIR>
cudaError_t run_rows(int tn, const GroupedArgs& a, const CUtensorMap& mA, const CUtensorMap& mB,
                     cudaStream_t st) {
  switch (tn) {
    case 32: return run_grouped_kernel<DIR, 32, 10, false>(a, mA, mB, st);
    case 64: return run_grouped_kernel<DIR, 64, 9, false>(a, mA, mB, st);
    case 128: return run_grouped_kernel<DIR, 128, 8, false>(a, mA, mB, st);
    default: return run_grouped_kernel<DIR, 256, 6, false>(a, mA, mB, st);
  }
}

}  // namespace

size_t grouped_ws_bytes(const moe_group_cfg&) { return 256; }

cudaError_t launch_grouped(const moe_group_cfg& c, GroupedDir dir, const void* in0, const void* in1,
                           const int32_t* counts, void* out, bool out_f32, bool accumulate,
                           void* ws, cudaStream_t st) {
  if (c.rows == 0) {   // dw without rows: zeros, or nothing to add
    if (accumulate) return cudaSuccess;
    return cudaMemsetAsync(out, 0, (size_t)c.E * c.n * c.k * (out_f32 ? 4 : 2), st);
  }
  GroupedArgs a{};
  a.counts = counts;
  a.out = out;
  a.status = static_cast<uint32_t*>(ws);
  a.rows = c.rows;
  a.E = c.E;
  a.n = c.n;
  a.k = c.k;
  a.cols = dir == kGroupedFwd ? c.n : c.k;
  a.red = dir == kGroupedFwd ? c.k : c.n;
  a.mt = (a.cols + 255) / 256;
  a.accumulate = accumulate ? 1 : 0;
  CUtensorMap mA, mB;
  bool ok;
  const int tn = dir == kGroupedDw ? 256 : row_tile(c);
  if (dir == kGroupedDw) {
    ok = make_tensor_map_2d(&mA, in1, 2, c.k, c.rows, 64) &&
         make_tensor_map_2d(&mB, in0, 2, c.n, c.rows, 64);
  } else {
    ok = make_tensor_map_3d_bf16(&mA, in1, c.k, c.n, c.E, dir == kGroupedFwd ? 128 : 64) &&
         make_tensor_map_2d(&mB, in0, 2, a.red, c.rows, tn / 2);
  }
  if (!ok) return cudaErrorInvalidValue;
  switch (dir) {
    case kGroupedFwd: return run_rows<kGroupedFwd>(tn, a, mA, mB, st);
    case kGroupedDx: return run_rows<kGroupedDx>(tn, a, mA, mB, st);
    default:
      return out_f32 ? run_grouped_kernel<kGroupedDw, 256, 6, true>(a, mA, mB, st)
                     : run_grouped_kernel<kGroupedDw, 256, 6, false>(a, mA, mB, st);
  }
}

}  // namespace moe
