// pkv_tcgen05.cuh -- the fifth-generation tensor core's instructions: tensor-memory
// allocation, loads and stores, matrix products of shared-memory and tensor-memory operands,
// and the operand descriptors, for one-CTA 16-bit products with fp32 accumulators.
#pragma once

#include <stdint.h>

#include "pkv_device.cuh"

namespace pkv {

// Columns of tensor memory (a power of two, 32 to 512) for this CTA; the whole warp calls, and
// the address lands in *at (shared memory).
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// Order tensor-memory accesses against a barrier: before arriving, and after waiting.
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrive on `bar` once all of this thread's matrix products so far are complete.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}

// Shared-memory operand in the 128-byte swizzle: rows (K-major: of the non-contracted index,
// 64 contracted 16-bit values each) of 128 bytes, in groups of 8 rows (1024 bytes).  `sbo`:
// bytes from one group of 8 rows to the next.  `lbo`: for an operand whose contiguous index is
// not the contracted one (MN-major), bytes from one 64-value span of that index to the next;
// unused for K-major.
// The descriptor is in two words: the low one holds address and lbo (add a byte offset / 16 to it
// to move the operand), the high one is the same for every operand of one sbo.
__device__ __forceinline__ uint32_t smem_operand(uint32_t addr, uint32_t lbo) {
  return (addr & 0x3ffffu) >> 4 | ((lbo & 0x3ffffu) >> 4) << 16;
}
constexpr uint32_t smem_operand_hi(uint32_t sbo) { return (sbo & 0x3ffffu) >> 4 | 1u << 14 | 2u << 29; }

// Instruction descriptor: bf16 operands, fp32 accumulator, M x N; A K-major, B K-major or MN-major.
constexpr uint32_t mma_bf16_desc(int m, int n, bool b_mn_major) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | uint32_t(n >> 3) << 17 | uint32_t(m >> 4) << 24;
}
// The same with fp16 operands.
constexpr uint32_t mma_f16_desc(int m, int n, bool b_mn_major) { return mma_bf16_desc(m, n, b_mn_major) & ~(1u << 7 | 1u << 10); }

// D (+)= A B^T over 16 contracted values; A and B in shared memory (low descriptor words).
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(uint32_t(accumulate)), "r"(hi)
      : "memory");
}
// The same with A in tensor memory (a lane to a row, two 16-bit values to a column).
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc),
      "r"(uint32_t(accumulate)), "r"(hi)
      : "memory");
}

// 32 or 16 columns of this warp's 32 lanes (a lane to a thread).  Loads are complete after
// tmem_wait_ld, stores after tmem_wait_st.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15]), "=f"(r[16]),
        "=f"(r[17]), "=f"(r[18]), "=f"(r[19]), "=f"(r[20]), "=f"(r[21]), "=f"(r[22]), "=f"(r[23]), "=f"(r[24]),
        "=f"(r[25]), "=f"(r[26]), "=f"(r[27]), "=f"(r[28]), "=f"(r[29]), "=f"(r[30]), "=f"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, float* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const float* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
      "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7]), "f"(r[8]), "f"(r[9]),
      "f"(r[10]), "f"(r[11]), "f"(r[12]), "f"(r[13]), "f"(r[14]), "f"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Pairs of fp32 values in one 64-bit register.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f32x2_parts(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Two codes with their sign bits flipped, u = x + 128, below 0x43 in each half of `y` -> two bf16, exactly: y
// stands for 256 + 2 x where x >= 0 and for 256 + x where it is not, so x = (y - 256) - max(0, (y - 256) / 2).  The
// products' pipe does this; with masks instead the codes' conversion kept the one of the integer instructions, half as
// wide, busy (prompt attention, 256 rows, cycles a tile: 4870 against 5490; the shared-prefix pass takes the same time
// with either: 256 sequences behind 16384 INT8 tokens 148.8 us against 148.6).
__device__ __forceinline__ uint32_t bf16x2_from_i8(uint32_t y) {
  const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&y);
  const __nv_bfloat162 half = __float2bfloat162_rn(0.5f), k128 = __float2bfloat162_rn(-128.0f), k256 = __float2bfloat162_rn(-256.0f);
  const __nv_bfloat162 r = __hsub2(__hadd2(v, k256), __hfma2_relu(v, half, k128));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Four codes of a word -> four bf16 in two words.
template <KvType KV>
__device__ __forceinline__ void bf16x4_from_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == KvType::kFp8) {
    uint32_t a, b;
    f16x2x2_from_e4m3x4(w, a, b);
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    lo = pack_bf16x2(x.x, x.y);
    hi = pack_bf16x2(y.x, y.y);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    lo = bf16x2_from_i8(__byte_perm(u, 0x43434343u, 0x4140u));
    hi = bf16x2_from_i8(__byte_perm(u, 0x43434343u, 0x4342u));
  }
}

// Four codes of a word -> four fp16 in two words, exactly.
template <KvType KV>
__device__ __forceinline__ void f16x4_from_codes(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (KV == KvType::kFp8) {
    f16x2x2_from_e4m3x4(w, lo, hi);
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 offset = __float2half2_rn(1152.0f);
    const uint32_t a = f16x2_biased(u, 0x4140u), b = f16x2_biased(u, 0x4342u);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), offset), y = __hsub2(*reinterpret_cast<const __half2*>(&b), offset);
    lo = *reinterpret_cast<const uint32_t*>(&x);
    hi = *reinterpret_cast<const uint32_t*>(&y);
  }
}

}  // namespace pkv
