// Inline PTX of the fifth-generation tensor cores: tensor memory, tcgen05.mma
// on shared-memory descriptors, and the waits around them.
#pragma once
#include <stdint.h>

#include "lk_device.cuh"

namespace lk {

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// `count` arrivals at once.
__device__ __forceinline__ void mbar_arrive_many(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// ------------------------------------------------------------ tensor memory
// All of an SM's tensor memory (128 lanes x 512 columns of 32 bits); the
// address lands in shared memory.  One whole warp allocates and frees.
__device__ __forceinline__ void tmem_alloc_all(uint32_t smem_dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_dst) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_all(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(addr));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// Makes this thread's shared-memory writes visible to TMA and the tensor core.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 consecutive columns of the warp's 32 lanes: register c of lane r is
// column c of tensor-memory lane r of the warp's quarter.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
// Waits for this thread's tensor-memory loads; the values of r[0 .. n) may be
// used from here on (naming them keeps the compiler from using them earlier).
template <int n>
__device__ __forceinline__ void tmem_loaded(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// -------------------------------------------------------------- descriptors
// Shared-memory operand, a 64-bit word: in the lower half the address and
// `leading`, in the upper one `stride` (the byte strides between core-matrix
// groups) and the swizzle (2: 128-byte rows, 4: 64-byte rows).
//   K-major   rows of the operand are runs of K; `stride` between groups of 8
//             rows, `leading` unused.
//   MN-major  64-element runs of M or N; `leading` between those runs,
//             `stride` between groups of 8 K.
// Within one operand only the address moves: it is kept in units of 16 bytes
// in the lower half, and the upper half is a constant.
constexpr uint32_t kSwizzle128 = 2, kSwizzle64 = 4;
__host__ __device__ constexpr uint32_t desc_lo(uint32_t leading) { return (leading >> 4) << 16; }
__host__ __device__ constexpr uint32_t desc_hi(uint32_t stride, uint32_t swizzle) {
  return stride >> 4 | 1u << 14 | swizzle << 29;
}
// Instruction descriptor: bf16 x bf16 or f16 x f16 -> fp32, M x N, B K-major or
// MN-major.
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool b_mn_major, bool f16 = false) {
  return 1u << 4 | (f16 ? 0u : 1u << 7 | 1u << 10) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n / 8) << 17 |
         (uint32_t)(m / 16) << 24;
}

// D (tensor memory) = A B (+ D): A from shared memory, or from tensor memory
// (bf16 pairs packed two to a column).  One thread issues; the operations of
// a thread run in the order it issues them.
template <uint32_t kHi, bool kAccumulate>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t desc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(desc), "n"(kAccumulate ? 1 : 0), "n"(kHi)
      : "memory");
}
// The same with the descriptors' upper half and what to do with D known at run time.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t hi, uint32_t a_lo, uint32_t b_lo, uint32_t desc,
                                       bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(desc), "r"((uint32_t)accumulate), "r"(hi)
      : "memory");
}
template <uint32_t kHi>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t desc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.u32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(desc), "r"((uint32_t)accumulate), "n"(kHi)
      : "memory");
}
// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}
// The barrier gets one arrival once everything this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace lk
