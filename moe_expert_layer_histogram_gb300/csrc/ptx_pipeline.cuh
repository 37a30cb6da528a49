// ptx_pipeline.cuh -- more sm_103a primitives, those of the operators' pipelines: waits
// and arrives of whole warps, three-dimensional TMA loads, wide TMEM reads, and the
// fence between threads' reads of a stage and the copy that fills it again.
#pragma once

#include "ptx.cuh"

namespace moe {

// Order this thread's earlier generic-proxy accesses of shared memory before later
// async-proxy ones (of whoever learns of it): what has been read from a stage of a ring
// was read before the copy that fills it again.  An arrive alone does not see to that.
__device__ __forceinline__ void fence_proxy_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// mbar_wait by a whole warp, with its branches on votes: the lanes stay
// together without the compiler's reconvergence points, which made a wait on
// a phase that had completed cost 62 cycles instead of 36 in eight warps (and
// 176 when one lane waited for the others).
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity,
                                               volatile int* abort) {
  uint32_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    if ((i & 127u) == 0) {
      // (the low half of the timer: its differences are good for 4 s)
      uint32_t now;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      if (i == 0) t0 = now;
      if (__any_sync(0xFFFFFFFFu, *abort != 0 || now - t0 > static_cast<uint32_t>(kWaitTimeoutNs))) {
        *abort = 1;
        return false;
      }
    }
  }
}

// One thread of a whole warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map,
                                                 uint32_t bar_cluster, int32_t x, int32_t y,
                                                 int32_t z, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".cta_group::2.L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d_hint(void* dst, const CUtensorMap* map, uint64_t* bar,
                                                 int32_t x, int32_t y, int32_t z,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z),
      "l"(policy)
      : "memory");
}

// 32 consecutive 32-bit columns of the thread's TMEM lane; not valid before
// tmem_ld_wait() and reg_fence32().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19,"
      " %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
#pragma unroll
  for (int i = 0; i < 32; i += 8)
    asm volatile(""
                 : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]),
                   "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7]));
}

// Arrive, where `on`, on a barrier at a shared::cluster address (an address
// of this CTA's own shared memory is one; see also mbar_arrive_cluster): a
// predicated instruction, no branch.
__device__ __forceinline__ void mbar_arrive_if(bool on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar),
      "r"(static_cast<uint32_t>(on))
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(mapa_shared(saddr, rank))
               : "memory");
  return v;
}

// mbar_wait by a whole warp, without a look at the timer before the wait has
// lasted for many tries: reading it takes longer than most waits here.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
  uint32_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    if ((i & 127u) == 127u) {
      // (the low half of the timer: its differences are good for 4 s)
      uint32_t now;
      asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
      if (i == 127u) t0 = now;
      if (__any_sync(0xFFFFFFFFu, *abort != 0 || now - t0 > static_cast<uint32_t>(kWaitTimeoutNs))) {
        *abort = 1;
        return false;
      }
    }
  }
}

}  // namespace moe
