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

#define PA_F4(a, i) "=f"((a)[i]), "=f"((a)[(i) + 1]), "=f"((a)[(i) + 2]), "=f"((a)[(i) + 3])
#define PA_F16(a, i) PA_F4(a, i), PA_F4(a, (i) + 4), PA_F4(a, (i) + 8), PA_F4(a, (i) + 12)
#define PA_F64(a, i) PA_F16(a, i), PA_F16(a, (i) + 16), PA_F16(a, (i) + 32), PA_F16(a, (i) + 48)
#define PA_FU4(a, i) "+f"((a)[i]), "+f"((a)[(i) + 1]), "+f"((a)[(i) + 2]), "+f"((a)[(i) + 3])
#define PA_FU16(a, i) PA_FU4(a, i), PA_FU4(a, (i) + 4), PA_FU4(a, (i) + 8), PA_FU4(a, (i) + 12)
#define PA_FU64(a, i) \
  PA_FU16(a, i), PA_FU16(a, (i) + 16), PA_FU16(a, (i) + 32), PA_FU16(a, (i) + 48)
#define PA_I4(a, i) "r"((a)[i]), "r"((a)[(i) + 1]), "r"((a)[(i) + 2]), "r"((a)[(i) + 3])
#define PA_I16(a, i) PA_I4(a, i), PA_I4(a, (i) + 4), PA_I4(a, (i) + 8), PA_I4(a, (i) + 12)

#define PA_FI4(a, i) "f"((a)[i]), "f"((a)[(i) + 1]), "f"((a)[(i) + 2]), "f"((a)[(i) + 3])
#define PA_FI16(a, i) PA_FI4(a, i), PA_FI4(a, (i) + 4), PA_FI4(a, (i) + 8), PA_FI4(a, (i) + 12)
#define PA_R16A "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
#define PA_R16B "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
#define PA_R16C "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47"
#define PA_R16D "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63"

// Lane l of the warp receives 64 or 32 consecutive 32-bit columns of TMEM lane
// 32 (warp % 4) + l, in two halves: the load, and the wait for every load of the
// thread so far.  The wait names the registers, so their uses come after it.
__device__ __forceinline__ void tmem_ld_begin(uint32_t addr, float (&r)[64]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x64.b32 {" PA_R16A ", " PA_R16B ", " PA_R16C
               ", " PA_R16D "}, [%64];"
               : PA_F64(r, 0)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_begin(uint32_t addr, float (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {" PA_R16A ", " PA_R16B "}, [%32];"
               : PA_F16(r, 0), PA_F16(r, 16)
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_ld_end(float (&r)[64]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : PA_FU64(r, 0)::"memory");
}
__device__ __forceinline__ void tmem_ld_end(float (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : PA_FU16(r, 0), PA_FU16(r, 16)::"memory");
}

// The store of 32 or 16 consecutive columns; tmem_st_wait before anyone reads them.
__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&r)[32]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {" PA_R16A ", " PA_R16B "};" ::PA_FI16(
                   r, 0),
               PA_FI16(r, 16), "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {" PA_R16A "};" ::PA_I16(r, 0),
               "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// mbar_wait whose first looks may each suspend the warp for that long, so that a
// waiting warp leaves the issue slots to the working ones (plain prompt chunks 409 ->
// 401 us).  In all at most kTileWaits of them, then mbar_wait's own limit.
constexpr uint32_t kTileWaitNs = 16384;
constexpr int kTileWaits = 64;
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity) {
  for (int i = 0; i < kTileWaits; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity), "r"(kTileWaitNs)
        : "memory");
    if (done) return true;
  }
  return mbar_wait(bar, parity);
}

// ---------------------------------------------------------------- pairs of floats

// Two fp32 operations in one instruction (each rounded as its scalar form).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---------------------------------------------------------------- matrix products

// Shared-memory operand in the 128-byte swizzle: rows of 128 bytes in groups of
// eight (1024 bytes, 1024-byte aligned).  K-major (the contraction runs along
// the 128 bytes): 1024 bytes between groups, `lead` unused.  MN-major (the
// contraction runs over the rows): 1024 bytes between groups of eight rows,
// `lead` bytes between 128-byte blocks of the other dimension.  The low word
// holds the address in 16-byte units, so an operand a few bytes further on is
// the low word plus that many units: one addition per product for the issuing
// thread, whose instructions set its pace.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lead) {
  return addr >> 4 | (lead >> 4) << 16;
}

// Instruction descriptor: bf16 A and B, fp32 accumulators, M x N; `b_mn`: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int M, int N, bool b_mn) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn ? 1u << 16 : 0u) | (uint32_t)(N >> 3) << 17 |
         (uint32_t)(M >> 4) << 24;
}

// The warp in step, one lane of it (`lead`) issuing: D (TMEM) = A B (+ D when acc),
// K = 16.  A in shared memory or in TMEM; shared operands by the low words of
// their descriptors.  The predicate sits on the instruction itself, so the
// operands are computed in warp-uniform code and reach it in uniform registers.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "setp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d, uint32_t a, uint32_t b_lo,
                                       uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %5, 0;\n\t"
      "setp.ne.u32 q, %6, 0;\n\t"
      "mov.b64 b, {%2, %4};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(kDescHi), "r"(acc ? 1u : 0u), "r"(lead)
      : "memory");
}

// True in one lane of a converged warp (always the same one).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(r));
  return r;
}

// Arrives on `bar` once every tcgen05.mma the leading lane has issued has completed.
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_addr(bar)),
      "r"(lead)
      : "memory");
}

}  // namespace pagedattn
