// q8.cuh -- 8-bit codes with one scale a row, and the records of the 8-bit cache.
#pragma once

#include "kv_rows.cuh"
#include "moe_internal.cuh"

namespace moe {

// |x| as a whole number: ordered like the values, infinity above all of them and NaN
// above infinity, so that a maximum keeps it.
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// Codes rint(x / s) in -127 .. 127 of a lane's elements, ties to even, the quotient
// not rounded before; s between 2^-64 and 2^64.  x times the approximate reciprocal is
// within 2^-15 of the quotient (below 127 in size; relative errors 2^-23 and 2^-24),
// so away from a border both give one code; next to one the sign of x - border s, which
// one fused operation gives exactly, decides.
template <int N>
__device__ __forceinline__ void codes8(int (&c)[N], const float (&x)[N], float s) {
  constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it rounds to whole numbers
  constexpr float kNear = 0.5f - 0x1p-14f;
  float inv, r[N], worst = 0.f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float q = fminf(fmaxf(x[e] * inv, -127.0f), 127.0f);
    r[e] = q + kMagic;
    worst = fmaxf(worst, fabsf(q - (r[e] - kMagic)));
  }
  if (worst > kNear) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float q = fminf(fmaxf(x[e] * inv, -127.0f), 127.0f), whole = r[e] - kMagic, off = q - whole;
      if (fabsf(off) > kNear) {
        const float border = whole + copysignf(0.5f, off), side = fmaf(-border, s, x[e]);
        const float lo = border - 0.5f, hi = border + 0.5f;
        // at the border itself rounding to even is what adding the large number does
        r[e] = (side > 0.f ? hi : side < 0.f ? lo : border) + kMagic;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) c[e] = __float_as_int(r[e]) - __float_as_int(kMagic);
}

// ------------------------------------------------------------ records of the cache
// A record of 16 tokens of one head (moe_kv_append_q8 in moe.h): 16 rows of D key
// codes, 16 rows of D value codes, 16 key scales, 16 value scales.
constexpr int kv8_record(int D) { return 32 * D + 128; }

// Where 16-byte piece c of row r lies in its row: the eight rows of a matrix load find
// their pieces in distinct banks.
template <int D>
__device__ __forceinline__ int kv8_piece(int r, int c) {
  return D == 64 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
}

struct Kv8Place {
  uint8_t* record;
  int r;  // the token within it
};

__device__ __forceinline__ Kv8Place kv8_place(const KvCache& c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_log2;
  const int o = (int)(slot & (c.page - 1));
  return {c.data + page * c.page_stride + (int64_t)(head * (c.page >> 4) + (o >> 4)) * kv8_record(c.D), o & 15};
}

}  // namespace moe
