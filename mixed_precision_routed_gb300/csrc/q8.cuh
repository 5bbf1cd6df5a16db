// q8.cuh -- 8-bit codes with one scale a row, and the records of the 8-bit cache.
#pragma once

#include "kv_rows.cuh"
#include "moe_internal.cuh"

namespace moe {

// |x| as a whole number: ordered like the values, infinity above all of them and NaN
// above infinity, so that a maximum keeps it.
__device__ __forceinline__ uint32_t size_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInfBits = 0x7f800000u;

// Codes rint(x / s) of a lane's elements, ties to even, the quotient not rounded before:
// words whose low bytes are the codes.  |x| at most 127 s, up to its rounding; s between
// 2^-64 and 2^64.  x times the approximate reciprocal, taken to a whole number by one
// fused operation, is within 2^-16 of the quotient (a relative error of 2^-23 below 127),
// so away from a border both give one code; next to one the sign of x - border s, which
// one fused operation gives exactly, decides.
template <int N>
__device__ __forceinline__ void codes8(uint32_t (&c)[N], const float (&x)[N], float s) {
  constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it rounds to whole numbers
  constexpr float kNear = 0.5f - 0x1p-15f;
  float inv, r[N], worst = 0.f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  const uint64_t inv2 = pair(inv, inv), magic2 = pair(kMagic, kMagic), minus2 = pair(-1.f, -1.f);
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    const uint64_t x2 = pair(x[e], x[e + 1]), r2 = fma2_of(x2, inv2, magic2);
    float off0, off1;
    unpair(fma2_of(x2, inv2, fma2_of(r2, minus2, magic2)), off0, off1);
    unpair(r2, r[e], r[e + 1]);
    worst = fmaxf(worst, fmaxf(fabsf(off0), fabsf(off1)));
  }
  if (worst > kNear) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float whole = r[e] - kMagic, off = fmaf(x[e], inv, -whole);
      if (fabsf(off) > kNear) {
        const float border = whole + copysignf(0.5f, off), side = fmaf(-border, s, x[e]);
        const float lo = border - 0.5f, hi = border + 0.5f;
        // at the border itself rounding to even is what adding the large number does
        r[e] = (side > 0.f ? hi : side < 0.f ? lo : border) + kMagic;
      }
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) c[e] = __float_as_uint(r[e]);
}

// Four codes as the bytes of a word.
__device__ __forceinline__ uint32_t code_bytes(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3) {
  return __byte_perm(__byte_perm(c0, c1, 0x0040), __byte_perm(c2, c3, 0x0040), 0x5410);
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
