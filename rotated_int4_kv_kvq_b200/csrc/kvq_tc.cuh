// kvq_tc.cuh -- tcgen05 (5th-generation tensor core) building blocks: tensor
// memory, matrix descriptors, MMA issue, and bulk copies.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

// ---------------------------------------------------------- tensor memory ---

// Allocation and release by one whole warp; `cols` a power of two >= 32.
__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols));
}

// N consecutive columns of this warp's 32 lanes (lane field of `addr` set to
// 32 * (warp % 4)) into registers; complete after tmem_wait_ld().
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]);
#define KVQ_R4(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define KVQ_R16(i) KVQ_R4(i), KVQ_R4(i + 4), KVQ_R4(i + 8), KVQ_R4(i + 12)
template <>
__device__ __forceinline__ void tmem_ld<8>(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : KVQ_R4(0), KVQ_R4(4)
               : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_ld<16>(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : KVQ_R16(0)
      : "r"(addr));
}
template <>
__device__ __forceinline__ void tmem_ld<32>(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
      "%30, %31}, [%32];"
      : KVQ_R16(0), KVQ_R16(16)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ------------------------------------------------------------ descriptors ---

constexpr uint32_t kSw128 = 2, kSw64 = 4, kSw32 = 6;  // swizzle field

// Shared-memory operand tile: start address, and the two strides in bytes.
// K-major, 128-byte swizzle: rows of 128 bytes in groups of 8 rows (1024
// bytes), sbo between groups, lbo unused.  MN-major with a swizzle of b bytes:
// b contiguous bytes along M or N, 8 such lines (along K) in a group, sbo
// between groups, lbo between blocks of b bytes along M or N.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo,
                                              uint32_t swizzle) {
  return uint64_t((addr >> 4) & 0x3FFF) | (uint64_t(lbo >> 4) << 16) | (uint64_t(sbo >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(swizzle) << 61);
}

constexpr uint32_t kFmtU8 = 0, kFmtS8 = 1, kAccS32 = 2;  // kind::i8
constexpr uint32_t kFmtF16 = 0, kAccF32 = 1;             // kind::f16

constexpr uint32_t instr_desc(uint32_t acc, uint32_t a_fmt, uint32_t b_fmt, bool a_mn, bool b_mn,
                              int m, int n) {
  return (acc << 4) | (a_fmt << 7) | (b_fmt << 10) | (uint32_t(a_mn) << 15) |
         (uint32_t(b_mn) << 16) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// D (+)= A B, 32 bytes of K; issued by one thread.
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                        bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(accumulate))
      : "memory");
}
// Arrives on the barrier when all MMAs issued by this thread have completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

}  // namespace kvq
