// ra_tensor.cuh -- the tensor cores' building blocks (sm_103a): copies of
// matrix tiles by tensor map, products issued by one thread with operands in
// shared memory and sums in tensor memory, and bounded waits for both.
//
// Operand tiles lie in shared memory as the copies' 128-byte swizzle leaves
// them: units of 8 rows of 128 bytes (64 16-bit elements), 1024 bytes each.
#pragma once

#include <cuda.h>

#include "ra_device.cuh"
#include "ra_ffn.h"

namespace ra {

// A matrix operand's descriptor: 128-byte swizzle; `rows8` bytes from one 8
// rows to the next, `across` from one 64 elements of a row to the next (used
// where the rows run along the terms of the sum).
__device__ __forceinline__ uint64_t operand_desc(uint32_t smem, uint32_t across, uint32_t rows8) {
  return (uint64_t)((smem & 0x3FFFFu) >> 4) | (uint64_t)(across >> 4) << 16 | (uint64_t)(rows8 >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// The instruction's descriptor: binary32 sums of products of 16-bit operands,
// M x N; `a_mn`, `b_mn`: the operand's rows run along M or N, not along the terms.
__host__ __device__ constexpr uint32_t product_desc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// The address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t smem, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
  return r;
}

// Relaxed: for who has only read (its loads have returned); a releasing arrival would
// first wait for the thread's stores to global memory.
__device__ __forceinline__ void mbar_arrive_cluster_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// One box at (x, y) of a matrix, x along its rows.  Pair: the bytes may be
// counted on a barrier of the pair's other CTA.
template <int Ctas>
__device__ __forceinline__ void load_box(uint32_t smem, const CUtensorMap* m, int x, int y, uint32_t bar) {
  if constexpr (Ctas == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem),
        "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem), "l"(m), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

template <int Ctas> __device__ __forceinline__ void tmem_alloc(uint32_t* to, uint32_t columns) {
  if constexpr (Ctas == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(to)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}

template <int Ctas> __device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  if constexpr (Ctas == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}

// tmem (+)= A B, 16 terms, by one thread.
template <int Ctas>
__device__ __forceinline__ void multiply(uint32_t tmem, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  if constexpr (Ctas == 2)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(desc), "r"((uint32_t)add)
        : "memory");
}

// Arrive on a barrier (of a pair: on both CTAs') once this thread's products so far are done.
template <int Ctas> __device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (Ctas == 2)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tensor_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tensor_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// 32 columns of a warp's 32 lanes.
__device__ __forceinline__ void tmem_load32(uint32_t tmem, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(tmem)
      : "memory");
}

// 8 columns.
__device__ __forceinline__ void tmem_load8(uint32_t tmem, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(tmem)
               : "memory");
}

// ------------------------------------------------------------ bounded waits
// Every wait for a barrier ends after about two seconds of SM cycles, or at
// once when another wait of the CTA has given up.  The roles then leave their
// loops; what is in flight is given time to land before the CTA ends.
constexpr long long kWaitCycles = 4000000000ll;

__device__ __forceinline__ void record_give_up(WaitRecord* record, int what, int job, uint32_t parity) {
  record_wait_error(&record->first, 2u, what, job, (int)blockIdx.x, -1, 0u, parity);
  if (RA_ACCESS_OK(&record->count, sizeof(record->count), 2u)) atomicAdd(&record->count, 1u);
}

struct Waits {
  volatile int* gave_up;   // in shared memory
  WaitRecord* record;
  int job;

  // For one thread that acts alone.
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity, int what) const {
    if (mbar_try_wait(bar, parity)) return true;
    return slow(bar, parity, what);
  }
  // For all lanes of a warp, and the same for each: lanes poll by themselves, and
  // where one gives up while the barrier completes for another, none goes on
  // to what the warp does together.
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity, int what) const {
    return __all_sync(0xFFFFFFFFu, (*this)(bar, parity, what));
  }
  __device__ __noinline__ bool slow(uint64_t* bar, uint32_t parity, int what) const {
    const uint64_t c0 = sm_cycles();
    while (!mbar_try_wait(bar, parity)) {
      if (*gave_up) return false;
      if ((long long)(sm_cycles() - c0) > kWaitCycles) {
        *gave_up = 1;
        record_give_up(record, what, job, parity);
        return false;
      }
    }
    return true;
  }
};

// Time for copies and products in flight to land, after a wait gave up.
__device__ __forceinline__ void let_land() {
  const uint64_t c0 = sm_cycles();
  while (sm_cycles() - c0 < 4000000ull) {
  }
}

}  // namespace ra
