// What the tcgen05 kernels share: bounded mbarrier waits, elected TMA copies and
// commits, shared-memory descriptors, tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tl_launch.cuh"

namespace tl {

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // a bounded wait gives up after 2 s

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Bounded wait for the phase with the given parity to complete: false after
// limit_ns of global time.
__device__ __forceinline__ bool mbar_try(uint32_t addr, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(addr), "r"(parity)
      : "memory");
  return done != 0;
}

// Bounded wait for the phase with the given parity to complete: false after
// limit_ns of global time.  The clock is read only once the first try fails.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity,
                                          uint64_t limit_ns = kWaitLimitNs) {
  const uint32_t addr = smem_u32(bar);
  if (mbar_try(addr, parity)) return true;
  const uint64_t start = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try(addr, parity)) return true;
    if ((i & 63) == 0 && globaltimer_ns() - start > limit_ns) return false;
  }
}

// The producer and MMA warps run their loops with all 32 lanes converged and
// issue each TMA copy, MMA and commit from one lane chosen by elect.sync: a
// lone active lane issues far more slowly while the dequantisation warps on
// the same SM sub-partition keep its issue slots busy.
__device__ __forceinline__ void tma_issue_elect(uint64_t* bar, uint32_t bytes, void* dst,
                                                const CUtensorMap* map, int x, int y) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n"
      " @e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%2], [%3, "
      "{%4, %5}], [%0];\n}\n" ::"r"(smem_u32(bar)),
      "r"(bytes), "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y)
      : "memory");
}

__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t addr) {
  // K-major, 128-byte swizzle: rows of 128 bytes, 8-row groups 1024 bytes apart
  uint64_t d = 0;
  d |= (uint64_t)((addr >> 4) & 0x3FFF);
  d |= (uint64_t)1 << 16;                 // leading byte offset (unused for this layout)
  d |= (uint64_t)(1024 >> 4) << 32;       // stride byte offset
  d |= (uint64_t)1 << 46;                 // descriptor version for sm_100
  d |= (uint64_t)2 << 61;                 // SWIZZLE_128B
  return d;
}

__device__ __forceinline__ void mma_commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          smem_u32(bar))
      : "memory");
}

// Bounded wait (when needed) by lane 0 with the outcome (and the CTA's abort flag) broadcast
// to the warp, so the warp stays converged.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const int* abort_flag,
                                          bool needed, uint64_t limit_ns = kWaitLimitNs) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0)
    ok = (!needed || mbar_wait(bar, parity, limit_ns)) && !*(volatile const int*)abort_flag;
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// The elected lane arrives once on a barrier for the whole warp.
__device__ __forceinline__ void mbar_arrive_elect(uint64_t* bar) {
  asm volatile(
      "{\n .reg .pred e;\n elect.sync _|e, 0xffffffff;\n"
      " @e mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(smem_u32(bar))
      : "memory");
}

// 2D tensor map of a row-major matrix (gemm_tc.cu).
tl_status encode_2d(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner,
                    uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                    CUtensorMapSwizzle swz);

}  // namespace tl
