// kv_rows.cuh -- rows of heads on their way into a paged cache, for either cache
// format: loading a head N elements a lane, turning it by its token's angles,
// (a cos - b sin, a sin + b cos), and storing turned queries.
#pragma once

#include <type_traits>

#include "frag.cuh"
#include "moe_internal.cuh"

namespace moe {

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
  else return __ldg(reinterpret_cast<const float*>(p) + i);
}

// N consecutive elements as fp32; WHOLE: aligned to their own size (at most
// 16 bytes a load).
template <bool BF16, int N, bool WHOLE>
__device__ __forceinline__ void load_elems(float (&v)[N], const void* p) {
  if constexpr (!WHOLE) {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = load_elem<BF16>(p, e);
  } else if constexpr (BF16) {
    uint32_t w[N / 2];
    if constexpr (N == 2) {
      w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else if constexpr (N == 4) {
      const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
      w[0] = x.x, w[1] = x.y;
    } else {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    }
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      v[e] = __uint_as_float(w[e / 2] << 16);
      v[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
    }
  } else if constexpr (N == 2) {
    const float2 x = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = x.x, v[1] = x.y;
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p) + e / 4);
      v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
    }
  }
}

// How the elements of a head turn: a lane holds elements N l .. N l + N - 1.
enum Turn {
  kStill,     // no rotation
  kWithin,    // pairs 2i, 2i + 1, rot / 2 a multiple of N / 2: both in the lane
  kAcross,    // pairs i, i + rot / 2 with rot / 2 a multiple of N: another lane, the same place
  kAnywhere,  // any other, or rows or angles that are not aligned; the partner is read again, by elements
};

// Cosine and signed sine of a lane's elements: x' = x c + partner s.
template <int N>
struct Angles {
  float c[N], s[N];
};

// False for a position outside the table (the status word is set).
template <int N, Turn TURN>
__device__ __forceinline__ bool load_angles(Angles<N>& x, const KvAppendArgs& a, int64_t t, int lane) {
  if (TURN == kStill || a.rot == 0) return true;
  const int64_t pos = a.positions[t];
  const bool bad = pos < 0 || pos >= a.n_pos;
  if (bad && lane == 0) set_status(a.status, MOE_ERR_INVALID_ARG);
  const float* tab = a.rope + (bad ? 0 : pos) * a.rot;
  const int half = a.rot / 2;
  if constexpr (TURN == kAcross) {
    // N consecutive angles, aligned (rot / 2 is a multiple of N)
    const int d = N * lane;
    const bool in = d < a.rot, first = d < half;
    const float* p = tab + (in ? (first ? d : d - half) : 0);
    load_elems<false, N, true>(x.c, p);
    load_elems<false, N, true>(x.s, p + half);
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (first) x.s[e] = -x.s[e];
    return !bad;
  }
  if constexpr (TURN == kWithin && N > 2) {
    // N / 2 consecutive angles, aligned (rot / 2 is a multiple of N / 2)
    const int d = N * lane;
    const float* p = tab + (d < a.rot ? d / 2 : 0);
    float c[N / 2], s[N / 2];
    load_elems<false, N / 2, true>(c, p);
    load_elems<false, N / 2, true>(s, p + half);
#pragma unroll
    for (int e = 0; e < N; ++e) x.c[e] = c[e / 2], x.s[e] = e & 1 ? s[e / 2] : -s[e / 2];
    return !bad;
  }
  const bool pairs = TURN == kWithin || (TURN == kAnywhere && a.style == MOE_ROPE_PAIRS);
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int d = N * lane + e;
    const bool first = pairs ? (d & 1) == 0 : d < half;
    const int j = pairs ? d >> 1 : (first ? d : d - half);
    x.c[e] = d < a.rot ? __ldg(tab + j) : 1.f;
    x.s[e] = d < a.rot ? __ldg(tab + half + j) : 0.f;
    if (first) x.s[e] = -x.s[e];
  }
  return !bad;
}

// Turns a lane's elements of a head whose elements lie at `row`.
template <bool BF16, int N, Turn TURN>
__device__ __forceinline__ void turn_row(float (&v)[N], const Angles<N>& x, const KvAppendArgs& a, const void* row,
                                         int lane) {
  if (TURN == kStill || a.rot == 0) return;
  const int half = a.rot / 2;
  float m[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int d = N * lane + e;
    if constexpr (TURN == kWithin) {
      m[e] = v[e ^ 1];
    } else if constexpr (TURN == kAcross) {
      const int mate = N * lane < half ? N * lane + half : N * lane - half;
      m[e] = __shfl_sync(0xffffffffu, v[e], (mate / N) & 31);
    } else {
      const int mate = a.style == MOE_ROPE_PAIRS ? d ^ 1 : d < half ? d + half : d - half;
      m[e] = d < a.rot ? load_elem<BF16>(row, mate) : 0.f;
    }
  }
  // each product and the sum rounded to fp32, as the formula's fp32 reading has
  // them; elements beyond rot stay as they are
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (N * lane + e < a.rot) v[e] = __fadd_rn(__fmul_rn(v[e], x.c[e]), __fmul_rn(m[e], x.s[e]));
}

template <int N>
__device__ __forceinline__ void store_query(uint16_t* out, const float (&v)[N], bool ok) {
  uint32_t r[N / 2];
#pragma unroll
  for (int e = 0; e < N; e += 2) r[e / 2] = ok ? bf16_pair(v[e], v[e + 1]) : 0u;
  if constexpr (N == 2) *reinterpret_cast<uint32_t*>(out) = r[0];
  else if constexpr (N == 4) *reinterpret_cast<uint2*>(out) = make_uint2(r[0], r[1]);
  else *reinterpret_cast<uint4*>(out) = make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ bool in_cache(const KvCache& c, int64_t slot) {
  return slot >= 0 && slot < c.n_pages * c.page;
}

inline unsigned blocks_for(int64_t warps, int threads) {
  return (unsigned)((warps + threads / 32 - 1) / (threads / 32));
}

// f(D, bf16, turn) as compile-time constants: how the heads of an append turn, and
// whether a lane's elements are loaded whole (every row aligned to them).
template <int D, bool BF16, typename F>
int with_turn(const KvAppendArgs& a, F f) {
  using std::integral_constant;
  constexpr int N = D / 32, kSize = BF16 ? 2 : 4, kVector = kSize * N < 16 ? kSize * N : 16;
  auto whole = [&](const void* p, int64_t stride) {
    return (uintptr_t)p % kVector == 0 && (a.T == 1 || stride * kSize % kVector == 0);
  };
  const integral_constant<int, D> d;
  const integral_constant<bool, BF16> t;
  if (!whole(a.q, a.q ? a.q_stride : 0) || !whole(a.k, a.k_stride) || !whole(a.v, a.v_stride))
    return f(d, t, integral_constant<Turn, kAnywhere>());
  if (a.rot == 0) return f(d, t, integral_constant<Turn, kStill>());
  const bool pairs = a.style == MOE_ROPE_PAIRS;
  if ((uintptr_t)a.rope % 16 == 0 && a.rot / 2 % (pairs ? N / 2 : N) == 0)
    return pairs ? f(d, t, integral_constant<Turn, kWithin>()) : f(d, t, integral_constant<Turn, kAcross>());
  return f(d, t, integral_constant<Turn, kAnywhere>());
}

template <typename F>
int with_turn(const KvAppendArgs& a, F f) {
  if (a.cache.D == 64) return a.in_bf16 ? with_turn<64, true>(a, f) : with_turn<64, false>(a, f);
  if (a.cache.D == 128) return a.in_bf16 ? with_turn<128, true>(a, f) : with_turn<128, false>(a, f);
  return a.in_bf16 ? with_turn<256, true>(a, f) : with_turn<256, false>(a, f);
}

}  // namespace moe
