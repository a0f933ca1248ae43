// Inline-PTX building blocks for the 5th-generation tensor cores (sm_103a):
// tensor memory (TMEM) allocation, matrix and instruction descriptors,
// tcgen05.mma, its completion on an mbarrier, and TMEM loads and stores.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace pagedattn {

// ---------------------------------------------------------------- tensor memory

// One warp, converged: allocates `columns` (a power of two from 32 to 512)
// columns of 128 lanes and writes their address to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_addr(dst)),
               "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns)
               : "memory");
}

// Orders tcgen05 operations across a thread synchronisation (mbarrier, bar.sync).
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

#define PA_O4(a, i) "=r"((a)[i]), "=r"((a)[(i) + 1]), "=r"((a)[(i) + 2]), "=r"((a)[(i) + 3])
#define PA_O16(a, i) PA_O4(a, i), PA_O4(a, (i) + 4), PA_O4(a, (i) + 8), PA_O4(a, (i) + 12)
#define PA_O64(a, i) PA_O16(a, i), PA_O16(a, (i) + 16), PA_O16(a, (i) + 32), PA_O16(a, (i) + 48)
#define PA_I4(a, i) "r"((a)[i]), "r"((a)[(i) + 1]), "r"((a)[(i) + 2]), "r"((a)[(i) + 3])
#define PA_I16(a, i) PA_I4(a, i), PA_I4(a, (i) + 4), PA_I4(a, (i) + 8), PA_I4(a, (i) + 12)

#define PA_R16A "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
#define PA_R16B "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
#define PA_R16C "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47"
#define PA_R16D "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"

// Lane l of the warp receives `N` consecutive 32-bit columns of TMEM lane
// 32 (warp % 4) + l; returns when they have arrived (the wait sits in the same
// statement, so no use can be scheduled ahead of it).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {" PA_R16A ", " PA_R16B "}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PA_O16(r, 0), PA_O16(r, 16)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {" PA_R16A ", " PA_R16B ", " PA_R16C ", " PA_R16D
      "}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : PA_O64(r, 0)
      : "r"(addr)
      : "memory");
}

// The store of 32 consecutive columns; tmem_st_wait before anyone reads them.
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" PA_R16A ", " PA_R16B "};" ::PA_I16(
                   r, 0),
               PA_I16(r, 16), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- matrix products

// Shared-memory operand in the 128-byte swizzle: rows of 128 bytes in groups of
// eight (1024 bytes, 1024-byte aligned).  K-major (the contraction runs along
// the 128 bytes): `stride` bytes between groups, `lead` unused.  MN-major (the
// contraction runs over the rows): `stride` bytes between groups of eight rows,
// `lead` bytes between 128-byte blocks of the other dimension.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead, uint32_t stride) {
  return (uint64_t)((addr >> 4) & 0x3fff) | (uint64_t)((lead >> 4) & 0x3fff) << 16 |
         (uint64_t)((stride >> 4) & 0x3fff) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor: bf16 A and B, fp32 accumulators, M x N; `b_mn`: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int M, int N, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}

// One thread: D (TMEM) = A B (+ D when acc), K = 16.  A in shared memory or in TMEM.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc ? 1u : 0u)
      : "memory");
}

// Arrives on `bar` once every tcgen05.mma this thread has issued has completed.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}

}  // namespace pagedattn
