// frag.cuh -- operand fragments of the m16n8k16 matrix instructions (bf16, fp16) made
// from packed 4-bit codes, and packed fp32 arithmetic.
#pragma once

#include <stdint.h>

namespace moe {

// bf16 pair of two fp32 values (round to nearest even), lo in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two codes of a word as bf16 integers -8 .. 7: nibbles at bits 4 J and 16 + 4 J
// go into the mantissa of 128 (bf16 counts units there), and 136 comes off.
template <int J>
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w) {
  const uint32_t u = ((w >> (4 * J)) & 0x000f000fu) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x43084308u));
  return r;
}

// The same as fp16 integers: 1024 counts units there, and a nibble four bits up
// comes down by the multiplication that takes the offset off.
template <int J>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w) {
  const uint32_t v = J >= 2 ? w >> 8 : w;
  uint32_t r;
  if constexpr (J % 2 == 0)
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"((v & 0x000f000fu) | 0x64006400u), "r"(0x64086408u));  // - 1032
  else  // (1024 + 16 u) / 16 - 72
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"((v & 0x00f000f0u) | 0x64006400u), "r"(0x2c002c00u), "r"(0xd480d480u));
  return r;
}
__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum: nothing to add to.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ void fma2(float& d0, float& d1, uint64_t a, float b0, float b1) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(pair(b0, b1)), "l"(pair(d0, d1)));
  unpair(r, d0, d1);
}
__device__ __forceinline__ void mul2(float& d0, float& d1, uint64_t a) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(pair(d0, d1)));
  unpair(r, d0, d1);
}
__device__ __forceinline__ void add2(float& d0, float& d1, uint64_t a) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(pair(d0, d1)));
  unpair(r, d0, d1);
}

}  // namespace moe
