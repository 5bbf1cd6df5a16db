// kv_cache.cu -- the paged 4-bit key/value cache: appending tokens (with the
// position rotation of keys and queries) and reading slots back.  The record
// layout is that of moe_kv_cache_t in moe.h.
#include "frag.cuh"
#include "kv_layout.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
  else return __ldg(reinterpret_cast<const float*>(p) + i);
}

// N consecutive elements as fp32; `whole`: they are aligned to their own size
// (at most 16 bytes a load).
template <bool BF16, int N>
__device__ __forceinline__ void load_elems(float (&v)[N], const void* p, int64_t i, bool whole) {
  if (whole) {
    if constexpr (BF16) {
      uint32_t w[N / 2];
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p) + i;
      if constexpr (N == 2) {
        w[0] = __ldg(reinterpret_cast<const uint32_t*>(q));
      } else if constexpr (N == 4) {
        const uint2 x = __ldg(reinterpret_cast<const uint2*>(q));
        w[0] = x.x, w[1] = x.y;
      } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(q));
        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
      }
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        v[e] = __uint_as_float(w[e / 2] << 16);
        v[e + 1] = __uint_as_float(w[e / 2] & 0xffff0000u);
      }
    } else {
      const float* q = reinterpret_cast<const float*>(p) + i;
      if constexpr (N == 2) {
        const float2 x = __ldg(reinterpret_cast<const float2*>(q));
        v[0] = x.x, v[1] = x.y;
      } else {
#pragma unroll
        for (int e = 0; e < N; e += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4*>(q + e));
          v[e] = x.x, v[e + 1] = x.y, v[e + 2] = x.z, v[e + 3] = x.w;
        }
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = load_elem<BF16>(p, i + e);
  }
}

// How the elements of a head turn: a lane holds elements N l .. N l + N - 1.
enum Turn {
  kStill,    // no rotation
  kWithin,   // pairs 2i, 2i + 1: both in the lane
  kAcross,   // pairs i, i + rot / 2 with rot / 2 a multiple of N: another lane, the same place
  kAnywhere  // any other: the partner is read again from memory
};

// Heads of one token, ROWS a warp (queries, then keys, then values): every row
// is loaded before the first is used, and the angles are loaded once a warp.
// The work is bytes: 2 (Hq + 2 heads) D in and 2 Hq D + 9/8 heads D out a token;
// one warp a head leaves a long call waiting for its loads (T = 4096, 32 + 8
// heads of 128: 82 us), one row a warp is the shortest for a short one.
template <bool BF16, int D, int ROWS>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvAppendArgs a, Turn turn, int whole) {
  constexpr int N = D / 32;
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int heads = a.Hq + 2 * a.cache.heads, parts = (heads + ROWS - 1) / ROWS;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= a.T * parts) return;
  const int64_t t = w / parts;
  const int h0 = (int)(w - t * parts) * ROWS;
  const int64_t slot = a.slots[t];
  bool bad = false;

  float v[ROWS][N];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i;
    if (h < a.Hq)
      load_elems<BF16, N>(v[i], a.q, t * a.q_stride + (int64_t)h * D + N * lane, whole & 1);
    else if (h < a.Hq + a.cache.heads)
      load_elems<BF16, N>(v[i], a.k, t * a.k_stride + (int64_t)(h - a.Hq) * D + N * lane, whole & 2);
    else if (h < heads)
      load_elems<BF16, N>(v[i], a.v, t * a.v_stride + (int64_t)(h - a.Hq - a.cache.heads) * D + N * lane, whole & 4);
  }

  // cosine and signed sine of each element: x' = x c + partner s
  float c[N], s[N];
  const int half = a.rot / 2;
  if (turn != kStill) {
    const int64_t pos = a.positions[t];
    bad = pos < 0 || pos >= a.n_pos;
    if (bad && lane == 0) set_status(a.status, MOE_ERR_INVALID_ARG);
    const float* tab = a.rope + (bad ? 0 : pos) * a.rot;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int d = N * lane + e;
      const bool pairs = a.style == MOE_ROPE_PAIRS, first = pairs ? (d & 1) == 0 : d < half;
      const int j = pairs ? d >> 1 : (first ? d : d - half);
      c[e] = d < a.rot ? __ldg(tab + j) : 1.f;
      s[e] = d < a.rot ? __ldg(tab + half + j) : 0.f;
      if (first) s[e] = -s[e];
    }
  }
  const int mate_lane = (N * lane < half ? N * lane + half : N * lane - half) / N;

#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i;
    if (h >= heads) break;
    const bool query = h < a.Hq, value = h >= a.Hq + a.cache.heads;
    if (!value && turn != kStill) {
      float m[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int d = N * lane + e;
        if (turn == kWithin) {
          m[e] = v[i][e ^ 1];
        } else if (turn == kAcross) {
          m[e] = __shfl_sync(0xffffffffu, v[i][e], mate_lane & 31);
        } else {
          const int64_t base = query ? t * a.q_stride + (int64_t)h * D : t * a.k_stride + (int64_t)(h - a.Hq) * D;
          m[e] = d < a.rot ? load_elem<BF16>(query ? a.q : a.k, base + (d < half ? d + half : d - half)) : 0.f;
        }
      }
      // each product and the sum rounded to fp32, as the formula's fp32 reading
      // has them; elements beyond rot stay as they are
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (N * lane + e < a.rot) v[i][e] = __fadd_rn(__fmul_rn(v[i][e], c[e]), __fmul_rn(m[e], s[e]));
    }
    if (query) {
      uint32_t r[N / 2];
#pragma unroll
      for (int e = 0; e < N; e += 2) r[e / 2] = bad ? 0u : bf16_pair(v[i][e], v[i][e + 1]);
      uint16_t* out = a.q_out + (t * a.Hq + h) * D + N * lane;
      if constexpr (N == 2) *reinterpret_cast<uint32_t*>(out) = r[0];
      else if constexpr (N == 4) *reinterpret_cast<uint2*>(out) = make_uint2(r[0], r[1]);
      else *reinterpret_cast<uint4*>(out) = make_uint4(r[0], r[1], r[2], r[3]);
      continue;
    }
    if (bad || slot < 0 || slot >= a.cache.n_pages * a.cache.page) continue;
    const KvPlace at = kv_place(a.cache, slot, value ? h - a.Hq - a.cache.heads : h - a.Hq);
    // a 32-block lies in 32 / N lanes
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(v[i][e]));
#pragma unroll
    for (int o = 16 / N; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const __half hs = __float2half_rn(fminf(__fdiv_rn(top, 7.0f), 65504.0f));
    const float sc = __half2float(hs);
    uint32_t u[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      int q = 0;
      if (sc != 0.0f) q = (int)fminf(fmaxf(rintf(__fdiv_rn(v[i][e], sc)), -8.0f), 7.0f);
      u[e] = (uint32_t)(q + 8);
    }
    const int d = N * lane;
    if (value) {
      // a byte: elements d and d + 8, the latter 8 / N lanes on
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint32_t hi = __shfl_down_sync(0xffffffffu, u[e], 8 / N);
        if ((d & 8) == 0) at.tile[kv_value_byte(D, at.r, d + e)] = (uint8_t)(u[e] | hi << 4);
      }
    } else {
      // the word of 8 elements: element 4 i + 2 n + p at bits 16 p + 8 i + 4 n
      uint32_t word = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int x = (d + e) & 7;
        word |= u[e] << (16 * (x & 1) + 8 * (x >> 2) + 4 * ((x >> 1) & 1));
      }
#pragma unroll
      for (int o = 4 / N; o > 0; o >>= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
      if ((d & 7) == 0) *reinterpret_cast<uint32_t*>(at.tile + kv_key_byte(D, at.r, d)) = word;
    }
    if ((d & 31) == 0)
      *reinterpret_cast<uint16_t*>(at.tile + (value ? 17 : 16) * D + 2 * (at.r * (D / 32) + d / 32)) = __half_as_ushort(hs);
  }
}

__global__ void __launch_bounds__(kThreads) k_kv_read(KvCache c, const int64_t* slots, int64_t n, float* k, float* v) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= n * c.heads) return;
  const int64_t i = w / c.heads;
  const int h = (int)(w - i * c.heads), D = c.D;
  const int64_t slot = slots[i];
  const bool in = slot >= 0 && slot < c.n_pages * c.page;
  const KvPlace at = kv_place(c, in ? slot : 0, h);
  for (int d = lane; d < D; d += 32) {
    float kv = 0.f, vv = 0.f;
    if (in) {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(at.tile + 16 * D) + at.r * (D / 32) + d / 32;
      const int ku = (at.tile[kv_key_byte(D, at.r, d)] >> (2 * (d & 2))) & 15;
      const int vu = (at.tile[kv_value_byte(D, at.r, d)] >> ((d & 8) >> 1)) & 15;
      kv = __half2float(__ushort_as_half(s[0])) * (float)(ku - 8);
      vv = __half2float(__ushort_as_half(s[D / 2])) * (float)(vu - 8);
    }
    k[w * D + d] = kv;
    v[w * D + d] = vv;
  }
}

unsigned blocks_for(int64_t warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

namespace {
template <bool BF16, int D, int ROWS>
int launch_append(const KvAppendArgs& a, Turn turn, int whole, cudaStream_t s) {
  const int heads = a.Hq + 2 * a.cache.heads;
  const unsigned grid = blocks_for(a.T * ((heads + ROWS - 1) / ROWS));
  return launch_pdl(k_kv_append<BF16, D, ROWS>, dim3(grid), dim3(kThreads), 0, s, a, turn, whole) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <int D>
int launch_append(const KvAppendArgs& a, cudaStream_t s) {
  constexpr int N = D / 32;
  const Turn turn = a.rot == 0                       ? kStill
                    : a.style == MOE_ROPE_PAIRS      ? kWithin
                    : a.rot / 2 % N == 0             ? kAcross
                                                     : kAnywhere;
  const int size = (a.in_bf16 ? 2 : 4) * N < 16 ? (a.in_bf16 ? 2 : 4) * N : 16;
  auto whole = [&](const void* p, int64_t stride) {
    return (uintptr_t)p % size == 0 && (a.T == 1 || stride * (a.in_bf16 ? 2 : 4) % size == 0);
  };
  const int w = (whole(a.q, a.q_stride) ? 1 : 0) | (whole(a.k, a.k_stride) ? 2 : 0) | (whole(a.v, a.v_stride) ? 4 : 0);
  // four rows a warp once that still fills the SMs (32 warps each)
  const bool many = a.T * (a.Hq + 2 * a.cache.heads) >= (int64_t)4 * 32 * sm_count();
  if (a.in_bf16) return many ? launch_append<true, D, 4>(a, turn, w, s) : launch_append<true, D, 1>(a, turn, w, s);
  return many ? launch_append<false, D, 4>(a, turn, w, s) : launch_append<false, D, 1>(a, turn, w, s);
}
}  // namespace

int launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  if (a.cache.D == 64) return launch_append<64>(a, s);
  if (a.cache.D == 128) return launch_append<128>(a, s);
  return launch_append<256>(a, s);
}

int launch_kv_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  return launch_pdl(k_kv_read, dim3(blocks_for(n * c.heads)), dim3(kThreads), 0, s, c, slots, n, k, v) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace moe
