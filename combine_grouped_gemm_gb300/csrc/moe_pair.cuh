// Device-side helpers of the grouped products (moe_grouped.cu), beside moe_device.cuh: one-thread
// roles, tensor maps edited on the device, matrix loads and stores of an epilogue, and the CTA-pair
// forms of barriers, tile loads and MMAs. A file of its own, so that work on it does not touch
// the sources that the layer's own kernels are compiled from and measured with.
#pragma once

#include "moe_device.cuh"

namespace moe {

// True in one lane of a converged warp. A role of one thread is entered through this rather than
// by lane number: the compiler then knows that one thread runs it and keeps the operands of MMA
// and TMA instructions in uniform registers (by lane number each MMA took about 70 cycles to
// issue in the grouped products).
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// Tensor maps edited on the device: a 128-byte copy in shared memory whose extent in dimension 1
// is replaced (one thread), then written to global memory by the whole warp for loads of any later
// kernel or thread that acquires it.
__device__ __forceinline__ void tensor_map_set_rows(uint32_t smem_map, uint32_t rows) {
  asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(smem_map),
               "r"(rows)
               : "memory");
}
__device__ __forceinline__ void tensor_map_publish(void* global_map, uint32_t smem_map) {
  asm volatile(
      "tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned "
      "[%0], [%1], 128;" ::"l"(reinterpret_cast<uint64_t>(global_map)),
      "r"(smem_map)
      : "memory");
}
__device__ __forceinline__ void tensor_map_acquire(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(
                   reinterpret_cast<uint64_t>(map))
               : "memory");
}

// 16 lanes x 32 columns as four 16x8 accumulator fragments: of columns 8i..8i+7, thread t gets in
// r[4i], r[4i+1] columns 2(t%4), 2(t%4)+1 of lane t/4, and in r[4i+2], r[4i+3] those of lane t/4+8.
__device__ __forceinline__ void tmem_ld_16x256_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Four 8x8 matrices of 16-bit elements, stored transposed: lane l gives the address of row l%8 of
// matrix l/8; of matrix m, thread t's v[m] holds rows 2(t%4), 2(t%4)+1 of column t/4.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t saddr, const uint32_t (&v)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// ------------------------------------------------------------------------------------------
// CTA pairs (cluster of two, cta_group::2): one MMA over both SMs, M = 256. Each CTA's shared
// memory holds its 128 rows of A and half of B's rows at the same offsets; the leader (cluster
// rank 0) issues for both. The accumulator's rows 0-127 are in the leader's tensor memory, rows
// 128-255 in the peer's.
// ------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Address in the cluster's shared-memory window of p's counterpart in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}

// Makes this thread's earlier accesses visible in the cluster before its later relaxed arrivals.
__device__ __forceinline__ void fence_release_cluster() {
  asm volatile("fence.acq_rel.cluster;" ::: "memory");
}

// 16 bytes to an address of the cluster's shared-memory window (cluster_addr).
__device__ __forceinline__ void st_cluster16(uint32_t addr, const int4& v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

// Arrival on a barrier of either CTA, by itself not ordered after earlier memory accesses: after
// fence_release_cluster for what it publishes, alone where it hands over tensor memory
// (tcgen05.wait::ld and tcgen05.fence::before_thread_sync come before it), or conditional on the
// values of loads that have to come first. A releasing arrival would wait for the thread's
// outstanding global stores, about 1600 cycles in an epilogue.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

__device__ __forceinline__ bool mbar_test_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_peek_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait for a barrier that the other CTA of the pair arrives on.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort, uint32_t* status) {
  if (mbar_test_cluster(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
    if (mbar_test_cluster(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > kWaitLimitNs) {
      *abort = 1;
      raise_status(status, MOE_DEV_TIMEOUT);
      return false;
    }
  }
}

// Tile loads whose bytes count on a barrier of either CTA of the pair (bar: cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t x, int32_t y, int32_t z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst_smem)),
               "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive once on the barrier at this offset in both CTAs when every MMA this thread issued
// before has completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
      "[%0], %1;" ::"r"(smem_addr(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Descriptor of an operand whose M (or N) dimension is contiguous ("MN-major"), 128-byte swizzle:
// boxes of 64 columns x 64 reduction rows, a row of 128 bytes per reduction index, 8-row atoms
// 1024 bytes apart (stride byte offset), the next 64 columns one box (8192 bytes) further
// (leading byte offset). The next 16 reduction indices start 2048 bytes further.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (512ull << 16) | (64ull << 32) |
         (1ull << 46) | (2ull << 61);
}

// Instruction-descriptor bits for an MN-major A / B operand.
constexpr uint32_t kIdescAmn = 1u << 15, kIdescBmn = 1u << 16;

}  // namespace moe
