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
// dw they would be summed, and 0 x NaN is not 0, so both operands have to end with the group: a
// first small kernel writes for every group the two tensor maps whose extent ends at its last
// row, and the loads fill the rest of the last k-step with zeros. (Zeroing the stage in shared
// memory after the load cost a round trip between the two CTAs in every unit: 32 groups of 520
// rows, 7168 x 2048, 456 us that way, 322 us so.)
//
// The units (group, 256 output columns, N tile) are numbered group after group; a pair starts with
// its own number and takes further ones from a counter in the workspace as it gets free, since
// the groups' units differ in size (16384 rows dealt over 32 groups, forward 4096 x 7168: 620 us
// with fixed shares, 588 us so). Which pair computes a unit does not change its result. The tables
// are built by every CTA from the counts itself, without a schedule kernel.
//
// Where there are far fewer units than pairs, the reduction of each is split: every part leaves its
// fp32 sums in the workspace, and a second kernel over the whole GPU adds them up in the order of
// the parts and stores the results. (Joining in whichever part came last instead, by a counter,
// took 29 us for ten parts of a 256 x 256 tile: one pair cannot keep enough loads in flight.)
//
// Roles in a CTA (one CTA per SM): warp 0 TMA producer, warp 1 MMA issuer (leader CTA), warp 2
// scheduler (leader CTA: hands decoded units to the roles of both CTAs through a small ring), the
// others the epilogue. Loads of both CTAs count on the leader's full barriers, its commits free the
// stages of both. Accumulators are double buffered. Every wait is bounded.
//
// What bounds it. (us of ten calls after a pause, then of calls for a second or more, where the
// power cap sets the clock.) Full tiles keep the tensor pipe busy for 512 of 523 cycles a k-step
// (clock counters in the MMA thread): 8 groups of 2048 rows, 4096 x 7168, forward 500 (1.92
// PFLOP/s) and 579. A k-step brings 32 KB into each SM, 64 bytes a cycle, which is why narrower
// tiles (a group's rows spread over its tiles, 160 to 256 each) fall below that rate: 32 groups of
// 512 rows 543 and 630, of about 512 rows 582 and 687; row gradient of unevenly loaded ones,
// 7168 x 2048, 319 and 362; their bf16 weight gradient 318 and 366. Few rows a group: HBM, 64
// tokens through 256 experts 1840 (7.2 TB/s of weights). fp32 weight gradients of few rows a group:
// the stores, 4096 rows 577 (6.7 TB/s). Added to what is there 1612 (4.7 TB/s both ways): 64 sums
// and 16 old values a thread are more than its 96 registers hold, and the old values are asked for
// 16 at a time.
#include "moe_pair.cuh"

namespace moe {
namespace {

constexpr int kMaxGroups = 1024;

// The groups in shared memory, at most LIVE of them with rows.
template <int LIVE>
struct GroupedTables {
  int off[kMaxGroups + 1];   // first row of each group
  int live[LIVE];            // fwd, dx: the groups with rows
  int first[LIVE];           // and the N tiles before each of them
  int n_live;
  int n_tiles;
};

// The tables from the counts: warp 0, each lane over ceil(E / 32) consecutive groups. A negative
// count is 0 and the offsets stop at `rows` (sums saturate there, so none overflows); either is
// reported. TN: the N tile, or 0: offsets only. Ends with a block barrier.
template <int TN, int LIVE>
__device__ __forceinline__ void group_tables(const int32_t* counts, int E, int rows,
                                             GroupedTables<LIVE>& tab, uint32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) tab.off[e + 1] = counts[e];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (E + 31) / 32;
    const int e0 = min(E, lane * per), e1 = min(E, e0 + per);
    const uint32_t most = static_cast<uint32_t>(rows);
    bool bad = false;
    auto add = [&](uint32_t x, uint32_t y) {
      const uint32_t s = x + y;   // (both below 2^31)
      bad |= s > most;
      return min(s, most);
    };
    uint32_t incl = 0;
    for (int e = e0; e < e1; ++e) {
      const int c = tab.off[e + 1];
      bad |= c < 0;
      incl = add(incl, static_cast<uint32_t>(max(c, 0)));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = add(incl, v);
    }
    const uint32_t before = __shfl_up_sync(0xffffffffu, incl, 1);
    const uint32_t start = lane == 0 ? 0u : before;
    int live = 0, tiles = 0;   // of this lane's groups
    uint32_t at = start;
    for (int e = e0; e < e1; ++e) {
      const uint32_t end = min(at + static_cast<uint32_t>(max(tab.off[e + 1], 0)), most);
      tab.off[e + 1] = static_cast<int>(end);
      if (TN > 0) {
        live += end > at;
        tiles += static_cast<int>((end - at + TN - 1) / (TN > 0 ? TN : 1));
      }
      at = end;
    }
    if (lane == 0) tab.off[0] = 0;
    if (TN > 0) {
      int live_incl = live, tiles_incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, live_incl, o);
        const int w = __shfl_up_sync(0xffffffffu, tiles_incl, o);
        if (lane >= o) {
          live_incl += v;
          tiles_incl += w;
        }
      }
      int i = live_incl - live, t = tiles_incl - tiles;
      at = start;
      for (int e = e0; e < e1; ++e) {
        const uint32_t end = static_cast<uint32_t>(tab.off[e + 1]);
        if (end > at) {
          tab.live[i] = e;
          tab.first[i++] = t;
          t += static_cast<int>((end - at + TN - 1) / (TN > 0 ? TN : 1));
        }
        at = end;
      }
      if (lane == 31) {
        tab.n_live = live_incl;
        tab.n_tiles = tiles_incl;
      }
    }
    if (bad && blockIdx.x == 0) raise_status(status, MOE_DEV_BOUNDS);
  }
  __syncthreads();
}

// Warps 0, 1 and 2 load, issue the MMAs and schedule; the others are the epilogue: two warps per
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
// bf16 epilogue: two warps turn 32 output rows x 64 columns around in shared memory, rows 144 bytes
// apart (128 used), which keeps the eight 16-byte rows of a matrix store in different banks.
// Together they store whole 128-byte lines: the store path takes about one segment every four
// cycles, of 64 bytes or of 128.
constexpr int kTurnPitch = 144, kTurnBytes = 32 * kTurnPitch;

// (Results in bf16, and the row products, keep one tensor-core sum: at 1.1e-9 of the result a product
// its error reaches their own rounding after some two million.)

// Units on their way from the scheduler to the roles. A role frees its slot once it has read it:
// one slot ahead of the producer, which is itself a unit or two ahead of the epilogue.
constexpr int kRing = 3;

// Split reductions: at most kPairs parts in all, of at least kMinSteps k-steps each.
constexpr int kPairs = 76, kMinSteps = 8;

struct GroupedArgs {
  const int32_t* counts;
  void* out;
  uint32_t* status;
  uint32_t* counter;   // units taken, 0 before and after a launch
  int rows, E, n, k;
  int cols;       // output columns (M)
  int red;        // fwd, dx: length of the reduction
  int mt;         // ceil(cols / 256)
  int splits;     // parts of a unit's reduction, at most
  float* parts;   // [units][splits][TN][256]: their sums
};

template <int TN, int STAGES, bool F32>
struct GroupedShape {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = TN / 2 * 128;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int TMEM_COLS = 2 * TN;
  static constexpr int TURN = F32 ? 0 : GroupedThreads<F32>::kEpi / 2 * kTurnBytes;
  static constexpr int SMEM = STAGES * STAGE_BYTES + TURN + 1024 + 512;
  static_assert(B_BYTES % 1024 == 0 && TMEM_COLS <= 512 && TMEM_COLS >= 32, "");
};

// One unit of work: 256 output columns (the pair's) x one N tile of one group.
struct alignas(16) GroupedUnit {
  int g;      // group, or -1: no more units
  int f0;     // first output column of the pair
  int n0;     // fwd, dx: first row; dw: first row of dW_g
  int nlen;   // rows of the tile
  int r0;     // where the reduction starts: a column, dw: a row
  int red;    // its length
  int nt;     // N tiles that read this unit's weight tile
  int split;  // unit | part << 8 | parts << 16 where the reduction is split, else 0
};

// Units of all groups, in parts.
template <int DIR, int TN, typename Tables>
__device__ __forceinline__ int unit_count(const GroupedArgs& a, const Tables& tab) {
  const int tiles = DIR == kGroupedDw ? a.E * ((a.n + TN - 1) / TN) : tab.n_tiles;
  return tiles * a.mt * a.splits;
}

// Unit number u. fwd, dx: weight-tile-major (unit m * nt + j of a group: N tile j of its 256
// columns number m), so that pairs at work on neighbouring units share a weight tile through L2.
// dw: by rows of the output (unit j * mt + m), so that they write adjacent columns (fp32, 32 groups
// of 128 rows, 4096 x 7168: 680 us the other way, 644 us so with streaming stores).
// fwd, dx: a group of c rows has nt = ceil(c / TN) N tiles of equal size (to 32 rows, the step of
// an MMA's N) rather than full ones and a rest, which would cost a whole pass over the weight
// tile for a few rows. The group is found by binary search over the tiles before each: walking
// there from the unit before took several thousand cycles where groups are many and small.
template <int DIR, int TN, typename Tables>
__device__ __forceinline__ GroupedUnit grouped_unit(const GroupedArgs& a, const Tables& tab, int u) {
  GroupedUnit r{};
  if (u >= unit_count<DIR, TN>(a, tab)) {
    r.g = -1;
    return r;
  }
  int part = 0, number = 0;
  if (a.splits > 1) {
    number = u / a.splits;
    part = u - number * a.splits;
    u = number;
  }
  if (DIR == kGroupedDw) {
    const int row = u / a.mt;   // of the N tiles of all groups
    r.nt = (a.n + TN - 1) / TN;
    r.f0 = (u - row * a.mt) * 256;
    r.g = row / r.nt;
    r.n0 = (row - r.g * r.nt) * TN;
    r.nlen = min(TN, a.n - r.n0);
    r.r0 = tab.off[r.g];
    r.red = tab.off[r.g + 1] - r.r0;
  } else {
    const int t = u / a.mt;
    int lo = 0, hi = tab.n_live - 1;   // last group whose first tile is <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.first[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    r.g = tab.live[lo];
    const int base = tab.off[r.g], len = tab.off[r.g + 1] - base;
    const int local = u - tab.first[lo] * a.mt;
    r.nt = (len + TN - 1) / TN;
    const int m = r.nt == 1 ? local : local / r.nt, j = local - m * r.nt;
    const int w = r.nt == 1 ? TN : ((len - 1) / r.nt + 32) & ~31;   // ceil(len / nt), to 32
    r.f0 = m * 256;
    r.n0 = base + j * w;
    r.nlen = min(w, len - j * w);
    r.red = a.red;
  }
  if (a.splits > 1) {   // parts of equal length, as many as have kMinSteps; red < 0: no such part
    const int steps = (r.red + 63) >> 6;
    const int want = max(1, min(a.splits, steps / kMinSteps));
    const int per = (steps + want - 1) / want;
    const int have = steps ? (steps + per - 1) / per : 1;
    if (part >= have) {
      r.red = -1;
    } else if (have > 1) {
      r.r0 += part * per * 64;
      r.red = min(r.red - part * per * 64, per * 64);
      r.split = number | part << 8 | have << 16;
    }
  }
  return r;
}

// Where a part of a split unit leaves its sums.
template <int TN>
__device__ __forceinline__ float* part_sums(const GroupedArgs& a, const GroupedUnit& t) {
  return a.parts + ((size_t)(t.split & 255) * a.splits + ((t.split >> 8) & 255)) * (TN * 256);
}

// Barrier of the 64 threads of two warps, and whether both said yes.
__device__ __forceinline__ void pair_sync(int id) {
  asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool pair_agree(int id, bool yes) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %2, 0;\n\t"
      "barrier.cta.red.and.pred p, %1, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(all)
      : "r"(id), "r"(static_cast<uint32_t>(yes))
      : "memory");
  return all != 0;
}

// A role's end of the ring. next(): waits for the next unit and frees its slot; false at the end
// or after an abort. One thread (kWarp false) or a whole warp calls it.
// The scheduler, perhaps of the other CTA, writes the slot again once it is freed, so the arrival
// must not overtake the loads from it. It is conditional on every field that every lane loaded: the
// branch cannot be taken before those loads have returned their values. (Releasing arrivals order
// them too, but wait for all that the thread has in flight: in the two single-thread roles alone
// they cost the fp32 weight gradient of 4096 rows 583 -> 610 us, the bf16 one of 16384 365 -> 398.)
template <bool kWarp>
struct UnitReader {
  const GroupedUnit* ring;
  uint64_t* full;
  uint64_t* empty;   // of the leader
  volatile int* abort;
  uint32_t* status;
  int slot = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ bool next(GroupedUnit* u) {
    bool ok = mbar_wait_cluster(&full[slot], phase, abort, status);
    if (kWarp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    *u = ring[slot];
    if (u->g < 0) return false;
    // (no field of a unit is negative)
    bool held = (u->g | u->f0 | u->n0 | u->nlen | u->r0 | u->red | u->nt | u->split) >= 0;
    if (kWarp) held = __all_sync(0xffffffffu, held) && (threadIdx.x & 31) == 0;
    if (held) mbar_arrive_cluster_relaxed(cluster_addr(&empty[slot], 0));
    if (++slot == kRing) {
      slot = 0;
      phase ^= 1u;
    }
    return true;
  }
};

// A whole warp's wait: every lane gets the same answer, so the warp leaves its loop together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// dw: the tensor maps of x and dy for every group, ending at the group's last row; one warp a
// group. map_a, map_b: the whole tensors' maps.
constexpr int kMapWarps = 4;
__global__ void __launch_bounds__(kMapWarps * 32)
    group_maps_kernel(const int32_t* __restrict__ counts, CUtensorMap* maps, int rows, int E,
                      uint32_t* status, const __grid_constant__ CUtensorMap map_a,
                      const __grid_constant__ CUtensorMap map_b) {
  __shared__ GroupedTables<1> tab;
  __shared__ alignas(128) uint32_t copy[kMapWarps][2][32];
  pdl_trigger();
  group_tables<0>(counts, E, rows, tab, status);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x * kMapWarps + warp;
  if (g >= E) return;
  copy[warp][0][lane] = reinterpret_cast<const uint32_t*>(&map_a)[lane];
  copy[warp][1][lane] = reinterpret_cast<const uint32_t*>(&map_b)[lane];
  __syncwarp();
  const uint32_t sa = smem_addr(copy[warp][0]), sb = smem_addr(copy[warp][1]);
  if (lane == 0) {
    const uint32_t end = static_cast<uint32_t>(max(1, tab.off[g + 1]));   // (an extent is at least 1)
    tensor_map_set_rows(sa, end);
    tensor_map_set_rows(sb, end);
  }
  __syncwarp();
  tensor_map_publish(maps + 2 * g, sa);
  tensor_map_publish(maps + 2 * g + 1, sb);
}

template <int DIR, int TN, int STAGES, bool F32, bool ACC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GroupedThreads<F32>::kAll, 1)
    grouped_kernel(const GroupedArgs a, const CUtensorMap* __restrict__ maps,
                   const __grid_constant__ CUtensorMap mapA,
                   const __grid_constant__ CUtensorMap mapB) {
  using S = GroupedShape<TN, STAGES, F32>;
  constexpr bool kDw = DIR == kGroupedDw;
  constexpr int kEpiWarps = GroupedThreads<F32>::kEpi;
  constexpr int kBoxesB = kDw ? TN / 128 : 0;
  static_assert(!kDw || TN >= 128, "dw: whole 64-column boxes");
  extern __shared__ uint8_t smem_raw[];
  __shared__ GroupedTables<kDw ? 1 : kMaxGroups> tab;
  __shared__ GroupedUnit ring[kRing];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* turn = smem + STAGES * S::STAGE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + S::TURN);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* rfull = tempty + 2;
  uint64_t* rempty = rfull + kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rempty + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);   // uniform
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], 2 * kEpiWarps);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&rfull[i], 1);
      mbar_init(&rempty[i], 2 * kEpiWarps + 3);   // both epilogues and producers, the MMA thread
    }
    *abort_flag = 0;
    mbar_fence_init();
    if (!kDw) {
      tma_prefetch_map(&mapA);
      tma_prefetch_map(&mapB);
    }
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, S::TMEM_COLS);
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  group_tables<kDw ? 0 : TN>(a.counts, a.E, a.rows, tab, a.status);
  cluster_wait();   // the peer's barriers and tensor memory are ready
  tc_fence_after();
  if (kDw) pdl_wait();   // the groups' tensor maps are written
  if (a.splits > 1) pdl_trigger();   // the joining kernel may come up and wait
  const uint32_t tmem = *tmem_slot;

  // every role finds the pair's first unit itself (a microsecond sooner than through the ring); the
  // further ones come through the ring
  const int first = blockIdx.x >> 1;
  const int n_units = unit_count<DIR, TN>(a, tab);
  const bool any = first < n_units;
  constexpr int kNever = 1 << 30;
  constexpr int kSum = F32 ? kSumSteps : kNever;   // k-steps per tensor-core sum

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (elect_one()) {
      const uint64_t pol_once = l2_policy_evict_first(), pol_keep = l2_policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      int acquired = -1;   // dw: the group whose maps this thread has acquired
      UnitReader<false> units{ring, rfull, rempty, abort_flag, a.status};
      GroupedUnit t = grouped_unit<DIR, TN>(a, tab, first);
      for (bool more = any && (t.red >= 0 || units.next(&t)); more; more = ok && units.next(&t)) {
        const CUtensorMap *ma = &mapA, *mb = &mapB;
        if (kDw) {
          ma = maps + 2 * t.g;
          mb = ma + 1;
          if (t.g != acquired) {
            tensor_map_acquire(ma);
            tensor_map_acquire(mb);
            acquired = t.g;
          }
        }
        // each CTA's half of the N tile, a multiple of 16 rows (an MMA takes N in steps of 32)
        const int half = ((t.nlen + 31) & ~31) >> 1;
        const int steps = (t.red + 63) >> 6;
        // bytes of a step in both CTAs (dw: of B only the 64-column boxes that the tile has)
        const uint32_t bytes =
            2 * (S::A_BYTES + (kDw ? (half + 63) / 64 * 8192 : S::B_BYTES));
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
          if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
          const uint32_t bar = cluster_addr(&full[stage], 0);
          if (DIR == kGroupedFwd) {
            tma_load_3d_pair(sa, ma, bar, t.r0 + ks * 64, f, t.g, pol_a);
          } else if (DIR == kGroupedDx) {
            tma_load_3d_pair(sa, ma, bar, f, t.r0 + ks * 64, t.g, pol_a);
            tma_load_3d_pair(sa + 8192, ma, bar, f + 64, t.r0 + ks * 64, t.g, pol_a);
          } else {
            tma_load_2d_pair(sa, ma, bar, f, t.r0 + ks * 64, pol_a);
            tma_load_2d_pair(sa + 8192, ma, bar, f + 64, t.r0 + ks * 64, pol_a);
          }
          if (kDw) {
#pragma unroll
            for (int j = 0; j < kBoxesB; ++j)
              if (64 * j < half)
                tma_load_2d_pair(sb + j * 8192, mb, bar, nb + 64 * j, t.r0 + ks * 64, pol_keep);
          } else {
            tma_load_2d_pair(sb, mb, bar, t.r0 + ks * 64, nb, pol_keep);
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
      UnitReader<false> units{ring, rfull, rempty, abort_flag, a.status};
      GroupedUnit t = grouped_unit<DIR, TN>(a, tab, first);
      for (bool more = any && (t.red >= 0 || units.next(&t)); more; more = ok && units.next(&t)) {
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
    // ------------------------------ scheduler (leader) ------------------------------
    if (leader && elect_one()) {
      const uint32_t pairs = gridDim.x >> 1;
      int slot = 0;
      uint32_t phase = 0;
      // One number is taken for every unit, that of a unit while the one before is handed over;
      // whoever takes the last leaves the counter as it was.
      auto take = [&]() { return atomicAdd(a.counter, 1u); };
      uint32_t taken = any ? take() : 0;
      for (bool more = any; more;) {
        const uint32_t last = taken;
        const GroupedUnit u = grouped_unit<DIR, TN>(a, tab, static_cast<int>(pairs + taken));
        more = u.g >= 0;
        if (more) taken = take();
        if (u.red >= 0) {   // (below 0: a part that its unit does not have)
          if (!mbar_wait_cluster(&rempty[slot], phase ^ 1u, abort_flag, a.status)) break;
          const int4* v = reinterpret_cast<const int4*>(&u);
          for (uint32_t cta = 0; cta < 2; ++cta) {
            const uint32_t to = cluster_addr(&ring[slot], cta);
            st_cluster16(to, v[0]);
            st_cluster16(to + 16, v[1]);
          }
          fence_release_cluster();
          mbar_arrive_cluster_relaxed(cluster_addr(&rfull[slot], 0));
          mbar_arrive_cluster_relaxed(cluster_addr(&rfull[slot], 1));
          if (++slot == kRing) {
            slot = 0;
            phase ^= 1u;
          }
        }
        if (last + 1 == static_cast<uint32_t>(n_units)) *a.counter = 0;
      }
    }
    __syncwarp();
  } else {
    // ------------------------------ epilogue ------------------------------
    // Warp w reads lanes 32 (w % 4) .. +31 (output columns) of its part of the tile's N columns.
    const int quarter = warp & 3, part = (warp - 3) >> 2;
    int it = 0;
    bool ok = true;
    UnitReader<true> units{ring, rfull, rempty, abort_flag, a.status};
    GroupedUnit t = grouped_unit<DIR, TN>(a, tab, first);
    for (bool have = t.red >= 0; any && ok; have = false) {
      ok = have || units.next(&t);
      if (F32 && !ok) break;   // (bf16: the two warps of a pair leave together, below)
      const int steps = (t.red + 63) >> 6;
      const int fw = t.f0 + static_cast<int>(rank) * 128 + quarter * 32;   // the warp's columns
      if constexpr (F32) {
        // All sums but the last are added up in registers; the last goes straight to memory with
        // them, 128 bytes of a row per warp store. (Tile stores through shared memory were no
        // faster: 654 us for 32 groups of 128 rows, 4096 x 7168.)
        constexpr int kCols = TN / (kEpiWarps / 4);   // of this warp
        float acc[kCols];
#pragma unroll
        for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
        int k0 = 0;
        for (; k0 + kSum < steps; k0 += kSum) {
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
        if (ACC && steps == 0) continue;
        if (steps > 0) {
          const int b = it & 1;
          if (!warp_wait(&tfull[b], (it >> 1) & 1, abort_flag, a.status)) break;
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
        if (t.split) {
          float* sums = part_sums<TN>(a, t) + part * kCols * 256 + rank * 128 + quarter * 32 + lane;
#pragma unroll
          for (int j = 0; j < kCols; ++j) sums[j * 256] = acc[j];
          continue;
        }
        if (fw + lane >= a.cols) continue;
        const int first = t.n0 + part * kCols;   // this warp's first row of dW_g
        float* o = static_cast<float*>(a.out) + ((size_t)t.g * a.n + first) * a.cols + fw + lane;
        const int mine = a.n - first;            // rows from there to the last
        if constexpr (ACC) {
          const float* old = o;
#pragma unroll
          for (int c = 0; c < kCols; c += 16) {
            float was[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) was[j] = c + j < mine ? old[(size_t)j * a.cols] : 0.0f;
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[c + j] += was[j];
            old += 16 * (size_t)a.cols;
          }
        }
        if (mine >= kCols) {   // (the test in every store costs 5 %)
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            __stcs(o, acc[j]);
            o += a.cols;
          }
        } else {
#pragma unroll
          for (int j = 0; j < kCols; ++j) {
            if (j < mine) __stcs(o, acc[j]);
            o += a.cols;
          }
        }
      } else {
        // 32 rows x 64 columns of two warps at a time: accumulator fragments to bf16, turned around
        // through shared memory, stored as 16-byte pieces, eight lanes a row
        const int b = it & 1, duo = quarter >> 1;
        const int id = 1 + 2 * part + duo;
        if (ok && steps > 0) ok = warp_wait(&tfull[b], (it >> 1) & 1, abort_flag, a.status);
        if (!pair_agree(id, ok)) break;
        tc_fence_after();
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
        const size_t row0 = (kDw ? (size_t)t.g * a.n : 0) + t.n0;
        uint8_t* mine = turn + (2 * part + duo) * kTurnBytes;
        const uint32_t put = smem_addr(mine) + (lane & 7) * kTurnPitch + (quarter & 1) * 64 +
                             (lane >> 3) * 16;
        const int first = (quarter & 1) * 16 + (lane >> 3);   // of the rows this lane stores
        const uint8_t* get = mine + first * kTurnPitch + (lane & 7) * 16;
        const int fl = fw - (quarter & 1) * 32 + (lane & 7) * 8;   // and their columns
        const bool in = fl < a.cols;                               // (cols is a multiple of 8)
        const uint32_t tb = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + b * TN;
        if (t.split) {
          float* sums = part_sums<TN>(a, t) + rank * 128 + quarter * 32 + lane;
          for (int c = part * 16; c < t.nlen; c += kEpiWarps * 4) {
            uint32_t x[16];
            tmem_ld16(tb + c, x);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sums[(c + j) * 256] = __uint_as_float(x[j]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(cluster_addr(&tempty[b], 0));
          ++it;
          continue;
        }
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
            pair_sync(id);   // the previous rows have been read
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t m[4] = {
                  pack(lo[4 * i], lo[4 * i + 1]), pack(lo[4 * i + 2], lo[4 * i + 3]),
                  pack(hi[4 * i], hi[4 * i + 1]), pack(hi[4 * i + 2], hi[4 * i + 3])};
              stmatrix_x4_trans(put + i * 8 * kTurnPitch, m);
            }
            pair_sync(id);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              v[q] = *reinterpret_cast<const uint4*>(get + q * 4 * kTurnPitch);
          } else {   // dw of an empty group
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = make_uint4(0, 0, 0, 0);
          }
          const int p = c + first;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (in && p + 4 * q < t.nlen)
              *reinterpret_cast<uint4*>(out + (row0 + p + 4 * q) * a.cols + fl) = v[q];
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
  cluster_arrive();   // neither CTA leaves while the other still reads or signals it
  cluster_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, S::TMEM_COLS);
  }
}

// Adds the parts of split units. CTA: kJoinRows rows of one unit's tile, a thread a column.
constexpr int kJoinRows = 8;
template <int DIR, int TN>
__global__ void __launch_bounds__(256)
    join_kernel(const GroupedArgs a, int out_f32, int accumulate) {
  __shared__ GroupedTables<DIR == kGroupedDw ? 1 : kMaxGroups> tab;
  // counts are those that the products read: nothing before this has changed them
  group_tables<DIR == kGroupedDw ? 0 : TN>(a.counts, a.E, a.rows, tab, nullptr);
  constexpr int kSets = TN / kJoinRows;
  const int unit = blockIdx.x / kSets, j0 = (blockIdx.x - unit * kSets) * kJoinRows;
  const GroupedUnit t = grouped_unit<DIR, TN>(a, tab, unit * a.splits);   // its first part
  pdl_wait();
  const int f = t.f0 + threadIdx.x;
  if (t.g < 0 || !t.split || j0 >= t.nlen || f >= a.cols) return;
  const int have = t.split >> 16;
  const float* sums = part_sums<TN>(a, t) + j0 * 256 + threadIdx.x;
  float x[kJoinRows] = {};
#pragma unroll 4
  for (int s = 0; s < have; ++s)
#pragma unroll
    for (int j = 0; j < kJoinRows; ++j) x[j] += sums[((size_t)s * TN + j) * 256];
  const size_t row0 = (DIR == kGroupedDw ? (size_t)t.g * a.n : 0) + t.n0 + j0;
#pragma unroll
  for (int j = 0; j < kJoinRows; ++j) {
    if (j0 + j >= t.nlen) break;
    const size_t o = (row0 + j) * a.cols + f;
    if (out_f32) {
      float* out = static_cast<float*>(a.out) + o;
      *out = accumulate ? *out + x[j] : x[j];
    } else {
      static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x[j]);
    }
  }
}

template <int DIR, int TN, int STAGES, bool F32 = false, bool ACC = false>
cudaError_t run_grouped_kernel(const GroupedArgs& a, const CUtensorMap& mA, const CUtensorMap& mB,
                               long long units, cudaStream_t st,
                               const CUtensorMap* maps = nullptr) {
  using S = GroupedShape<TN, STAGES, F32>;
  auto kern = grouped_kernel<DIR, TN, STAGES, F32, ACC>;
  cudaError_t err = ensure_smem_limit(reinterpret_cast<const void*>(kern), S::SMEM);
  if (err != cudaSuccess) return err;
  // one pair for every two SMs, or for every part of a unit there can be
  const long long pairs = sm_count() / 2, parts = units * a.splits;
  err = launch_kernel(kern, dim3(2 * (unsigned)(parts < pairs ? parts : pairs)),
                      dim3(GroupedThreads<F32>::kAll), S::SMEM, st, maps != nullptr, a, maps, mA,
                      mB);
  if (err != cudaSuccess || a.splits == 1) return err;
  return launch_kernel(join_kernel<DIR, TN>, dim3((unsigned)(units * (TN / kJoinRows))), dim3(256),
                       0, st, true, a, F32 ? 1 : 0, ACC ? 1 : 0);
}

// The launch plan of a shape and direction, from host sizes alone.
struct GroupedPlan {
  int tn;            // N tile
  long long units;   // the most there can be
  int splits;
};
GroupedPlan grouped_plan(const moe_group_cfg& c, GroupedDir dir) {
  GroupedPlan p{};
  const long long live = c.E < c.rows ? c.E : c.rows;   // groups that can have rows
  const long long mt = ((dir == kGroupedFwd ? c.n : c.k) + 255ll) / 256;
  long long steps;
  if (dir == kGroupedDw) {
    p.tn = 256;
    p.units = c.E * mt * ((c.n + 255ll) / 256);
    steps = (c.rows + 63ll) / 64;   // of a group that has all the rows
  } else {
    // ceil(c / tn) tiles of a group of c rows are at most (c - 1) / tn + 1
    auto units = [&](int tn) { return ((c.rows - live) / tn + live) * mt; };
    // The mean is over all groups, of which the host knows no more: one crowded group among many
    // small ones takes their tile. Tiles of 128 rows up to that mean (64 groups, 2048 x 2048: of
    // 100 rows 90 us, with tiles of 256 95 us; of 200 rows 117 and 107 us); of 64 for a few rows,
    // whose smaller stages leave room for more weights in flight (4096 x 7168: 8 groups of a row 76
    // us, with 128 85 us; 32 uneven groups of 25 rows on average 288 and 279 us), and while they
    // leave half of the pairs idle (one group of 512 rows, 4096 x 7168: 29 us, with 256 34 us).
    const long long mean = live ? (c.rows + live - 1) / live : 0;
    p.tn = mean <= 16 ? 64 : mean <= 128 ? 128 : 256;
    while (p.tn > 64 && units(p.tn) < kPairs / 2) p.tn /= 2;
    p.units = units(p.tn);
    steps = ((dir == kGroupedFwd ? c.k : c.n) + 63ll) / 64;
  }
  long long splits = p.units ? kPairs / p.units : 1;
  if (splits > steps / kMinSteps) splits = steps / kMinSteps;
  // A part saves the k-steps of the others, about a quarter of a microsecond each, and the second
  // kernel takes about four: split from 24 saved steps on. Weight gradient, 512 x 512: 30000 rows
  // 134 us unsplit and 37 split, 2000 rows 20 and 17; forward of 64 rows, 4096 x 7168: 29 and 18.
  // A weight gradient's groups all count as units, whatever their rows: the 30000 rows in one of 9
  // groups take 76 us, in one of 10 or more, unsplit, 133 to 139.
  if (splits > 1 && steps - steps / splits < 24) splits = 1;
  p.splits = splits > 1 ? static_cast<int>(splits) : 1;
  return p;
}

// Workspace: status word; at byte 128 the unit counter; from the next 128-byte boundary after 256
// bytes on dw's tensor maps; then the split reductions' sums.
struct GroupedWs {
  size_t maps, parts, total;
};
GroupedWs grouped_ws(const moe_group_cfg& c) {
  GroupedWs w{};
  w.maps = 256;
  w.parts = w.maps + 2 * sizeof(CUtensorMap) * (size_t)c.E;
  size_t floats = 0;
  for (int d = 0; d < 3; ++d) {
    const GroupedPlan p = grouped_plan(c, static_cast<GroupedDir>(d));
    const size_t f = p.splits > 1 ? (size_t)p.units * p.splits * p.tn * 256 : 0;
    if (f > floats) floats = f;
  }
  w.total = w.parts + sizeof(float) * floats + 128;   // (128: ws is 16-byte aligned only)
  return w;
}

// 3-D bf16 tensor map [depth][rows][cols], box of one plane, box_rows x 64 columns, 128-byte
// swizzle. What a box reads outside its own plane's rows and columns is zero.
bool make_tensor_map_3d_bf16(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows,
                             uint64_t depth, uint32_t box_rows) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {cols, rows, depth};
  const cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

template <int DIR>
cudaError_t run_rows(const GroupedPlan& p, const GroupedArgs& a, const CUtensorMap& mA,
                     const CUtensorMap& mB, cudaStream_t st) {
  const long long units = p.units;
  switch (p.tn) {
    case 64: return run_grouped_kernel<DIR, 64, 9>(a, mA, mB, units, st);
    case 128: return run_grouped_kernel<DIR, 128, 8>(a, mA, mB, units, st);
    default: return run_grouped_kernel<DIR, 256, 6>(a, mA, mB, units, st);
  }
}

}  // namespace

size_t grouped_ws_bytes(const moe_group_cfg& c) { return grouped_ws(c).total; }

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
  a.counter = static_cast<uint32_t*>(ws) + 32;
  const GroupedPlan plan = grouped_plan(c, dir);
  const GroupedWs L = grouped_ws(c);
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 127) &
                                       ~static_cast<uintptr_t>(127));
  a.splits = plan.splits;
  a.parts = reinterpret_cast<float*>(base + L.parts);
  a.rows = c.rows;
  a.E = c.E;
  a.n = c.n;
  a.k = c.k;
  a.cols = dir == kGroupedFwd ? c.n : c.k;
  a.red = dir == kGroupedFwd ? c.k : c.n;
  a.mt = (a.cols + 255) / 256;
  CUtensorMap mA, mB;
  bool ok;
  if (dir == kGroupedDw) {
    ok = make_tensor_map_2d(&mA, in1, 2, c.k, c.rows, 64) &&
         make_tensor_map_2d(&mB, in0, 2, c.n, c.rows, 64);
  } else {
    ok = make_tensor_map_3d_bf16(&mA, in1, c.k, c.n, c.E, dir == kGroupedFwd ? 128 : 64) &&
         make_tensor_map_2d(&mB, in0, 2, a.red, c.rows, plan.tn / 2);
  }
  if (!ok) return cudaErrorInvalidValue;
  switch (dir) {
    case kGroupedFwd: return run_rows<kGroupedFwd>(plan, a, mA, mB, st);
    case kGroupedDx: return run_rows<kGroupedDx>(plan, a, mA, mB, st);
    default: break;
  }
  auto* maps = reinterpret_cast<CUtensorMap*>(base + L.maps);
  const cudaError_t err = launch_kernel(
      group_maps_kernel, dim3((c.E + kMapWarps - 1) / kMapWarps), dim3(kMapWarps * 32), 0, st,
      false, counts, maps, c.rows, c.E, static_cast<uint32_t*>(ws), mA, mB);
  if (err != cudaSuccess) return err;
  const long long units = plan.units;
  if (!out_f32) return run_grouped_kernel<kGroupedDw, 256, 6>(a, mA, mB, units, st, maps);
  return accumulate
             ? run_grouped_kernel<kGroupedDw, 256, 6, true, true>(a, mA, mB, units, st, maps)
             : run_grouped_kernel<kGroupedDw, 256, 6, true>(a, mA, mB, units, st, maps);
}

}  // namespace moe
