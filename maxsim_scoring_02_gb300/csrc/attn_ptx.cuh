// attn_ptx.cuh -- inline-PTX wrappers that only the packed-attention kernels
// use: products with A in tensor memory, operands whose N dimension is the
// contiguous one, tensor-memory loads and stores of 16 and 32 columns, and a
// whole warp's bounded wait.
#pragma once

#include "ptx.cuh"

namespace msim {

// Bounded wait of a whole warp, every lane active: one vote a poll, so that the
// compiler keeps the warp's control flow and operands uniform around it.
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, volatile int* abort_flag,
                                               unsigned* status) {
#pragma unroll 1
  for (uint32_t it = 0; it < kFastSpins; ++it)
    if (__all_sync(0xffffffffu, mbar_try_wait_a(bar, parity))) return true;
  const uint64_t t0 = globaltimer_ns(), lim = wait_limit_ns(status);
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait_a(bar, parity))) return true;
    if ((it & 63u) == 0) {
      const bool late = globaltimer_ns() - t0 > lim;
      if (late) {
        atomicOr(status, kDevErrTimeout);
        *abort_flag = 1;
      }
      if (__any_sync(0xffffffffu, late || *abort_flag)) return false;
    }
  }
}

// D[tmem] (+)= A * B^T, kind::f16, with A in tensor memory (16-bit values, two along K in each
// 32-bit column, one row a lane); whole-warp form with one elected lane.
__device__ __forceinline__ void umma_f16_ts_el(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an operand whose M or N dimension is the contiguous one, stored
// by TMA with 128-byte swizzling as panels of 64 elements (128 B) a row of K:
// 8 rows of K make a 1024-byte atom, the next 8 rows follow it (stride offset),
// the next 64 elements of M or N lie panel_bytes further (leading offset).
// Stepping K by 16 adds 2048 bytes to the start address.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t panel_bytes) {
  uint64_t desc = 0;
  desc |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  desc |= static_cast<uint64_t>(panel_bytes >> 4) << 16;
  desc |= static_cast<uint64_t>(1024 >> 4) << 32;
  desc |= static_cast<uint64_t>(1) << 46;
  desc |= static_cast<uint64_t>(2) << 61;
  return desc;
}
// Flag of the instruction descriptor: B has its N dimension contiguous.
constexpr uint32_t kIdescBMnMajor = 1u << 16;

// 16 columns, load and wait in one.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// Issue-only stores of 16 columns, and the wait for all stores of this thread.
__device__ __forceinline__ void tmem_st_32x32b_x16_issue(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32_issue(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

}  // namespace msim
