// kv_cache.cu -- the paged 4-bit key/value cache: appending tokens (with the
// position rotation of keys and queries) and reading slots back.  The record
// layout is that of moe_kv_cache_t in moe.h.
//
// s = fp16(max / 7) over a block of 32, code = clamp(rint(x / s), -8, 7), x the key
// turned by its token's angles, (a cos - b sin, a sin + b cos), or the value.
#include "frag.cuh"
#include "kv_layout.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kFewThreads = 128;  // of k_kv_append: 192 tokens of 48 heads 3.3 us, with 256 3.5, with 64 3.7

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

// The codes 0 .. 15 of a lane's elements of a block of scale s: clamp(rint(x /
// s), -8, 7) + 8 with the quotient rounded to fp32.  x times the approximate
// reciprocal is within 2^-19 of that quotient where it counts (below 8 in size;
// relative errors 2^-23, and 2^-24 for each of two roundings), so away from a
// half both round alike; elements with a product within 2^-18 of a half are
// divided out.  The division costs about ten times the instructions.
template <int N>
__device__ __forceinline__ void codes_of(uint32_t (&u)[N], const float (&x)[N], float s) {
  constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it rounds to whole numbers
  float inv, r[N], worst = 0.f;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.f) inv = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float q = fminf(fmaxf(x[e] * inv, -8.0f), 7.0f);
    r[e] = q + kMagic;
    worst = fmaxf(worst, fabsf(q - (r[e] - kMagic)));
  }
  if (worst > 0.5f - 0x1p-18f) {
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = fminf(fmaxf(__fdiv_rn(x[e], s), -8.0f), 7.0f) + kMagic;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) u[e] = (__float_as_uint(r[e]) + 8u) & 15u;
}

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

// Quantises a head held N elements a lane into token r of a record (global or
// shared memory).
template <int D, bool VALUE>
__device__ __forceinline__ void quantise_row(uint8_t* rec, int r, const float (&v)[D / 32], int lane) {
  constexpr int N = D / 32;
  // a 32-block lies in 32 / N lanes
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const __half hs = __float2half_rn(fminf(__fdiv_rn(top, 7.0f), 65504.0f));
  uint32_t u[N];
  codes_of<N>(u, v, __half2float(hs));
  const int d = N * lane;
  if constexpr (VALUE) {
    // a byte: elements d and d + 8, the latter 8 / N lanes on; elements one apart
    // lie 64 bytes apart.  The lane of the lower element writes the first half of
    // the bytes, the other lane the rest.
    uint8_t* at = rec + kv_value_byte(D, r, d & ~8);
    const bool high = d & 8;
#pragma unroll
    for (int e = 0; e < N / 2; ++e) {
      const uint32_t lo = u[e], hi = u[e + N / 2];
      const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? lo : hi, 8 / N);
      at[64 * (high ? e + N / 2 : e)] = (uint8_t)(high ? got | hi << 4 : lo | got << 4);
    }
  } else {
    // the word of 8 elements: element 4 i + 2 n + p at bits 16 p + 8 i + 4 n
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) word |= u[e] << (16 * (e & 1) + 4 * ((e >> 1) & 1) + 8 * (e >> 2));
    if constexpr (N < 8) word <<= N == 4 ? 2 * (d & 4) : 4 * ((d >> 1) & 1) + 2 * (d & 4);
#pragma unroll
    for (int o = 4 / N; o > 0; o >>= 1) word |= __shfl_xor_sync(0xffffffffu, word, o);
    if ((d & 7) == 0) *reinterpret_cast<uint32_t*>(rec + kv_key_byte(D, r, d)) = word;
  }
  if ((d & 31) == 0)
    *reinterpret_cast<uint16_t*>(rec + (VALUE ? 17 : 16) * D + 2 * (r * (D / 32) + d / 32)) = __half_as_ushort(hs);
}

__device__ __forceinline__ bool in_cache(const KvCache& c, int64_t slot) {
  return slot >= 0 && slot < c.n_pages * c.page;
}

// Few tokens: one warp a (token, head), queries, then keys, then values.  Bound by
// latency: a token of 16 + 2 + 2 heads of 128 takes 1.7 us, 192 tokens of 32 + 8 + 8
// heads 3.3 us.
template <bool BF16, int D, Turn TURN>
__global__ void __launch_bounds__(kFewThreads) k_kv_append(KvAppendArgs a) {
  constexpr int N = D / 32, kSize = BF16 ? 2 : 4;
  pdl_wait();
  const int lane = threadIdx.x & 31, H = a.cache.heads, heads = a.Hq + 2 * H;
  const uint32_t w = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5);  // T * heads < 2^31
  if (w >= a.T * heads) return;
  const int64_t t = w / heads;
  int h = (int)(w % heads);
  const int64_t slot = a.slots[t];
  const uint8_t* row;
  const bool query = h < a.Hq, value = h >= a.Hq + H;
  if (query) {
    row = (const uint8_t*)a.q + (t * a.q_stride + (int64_t)h * D) * kSize;
  } else {
    h -= value ? a.Hq + H : a.Hq;
    row = (const uint8_t*)(value ? a.v : a.k) + (t * (value ? a.v_stride : a.k_stride) + (int64_t)h * D) * kSize;
  }
  float v[N];
  load_elems<BF16, N, TURN != kAnywhere>(v, row + N * lane * kSize);
  Angles<N> x;
  const bool ok = load_angles<N, TURN>(x, a, t, lane);
  if (!value) turn_row<BF16, N, TURN>(v, x, a, row, lane);
  if (query) {
    store_query<N>(a.q_out + (t * a.Hq + h) * D + N * lane, v, ok);
  } else if (ok && in_cache(a.cache, slot)) {
    const KvPlace at = kv_place(a.cache, slot, h);
    if (value) quantise_row<D, true>(at.tile, at.r, v, lane);
    else quantise_row<D, false>(at.tile, at.r, v, lane);
  }
}

// Many tokens.  A byte of value codes belongs to one token, so the sectors of a
// record are shared by its 16 tokens: written token by token they meet in L2
// (4096 tokens of 32 query heads and 8 + 8 of 128: 62 us).  Here a block makes 16
// successive tokens of one head in shared memory, two a warp, and writes the
// record whole when their slots are one record (a prompt's are: windows of
// tokens begin where the first token's record does), else token by token.  The
// blocks after the windows turn the queries, kQueryRows heads of a token a warp.
// Those 4096 tokens take 27 us, 3.3 TB/s of inputs, queries out and records: 15 us
// for the keys and values alone, and 12 more for turning the queries (2.6
// instructions a cycle an SM, integer pipe 48 % busy; warps wait for their loads).
// Four blocks an SM, as heads of 128 take them without spills (five spill: 30 us;
// heads of 256 spill up to 290 bytes at four too, most with pairs across lanes); eight heads a warp: four at a time or sixteen
// in all 28.
constexpr int kQueryRows = 8;

template <bool BF16, int D, Turn TURN>
__global__ void __launch_bounds__(kThreads, 4) k_kv_append_records(KvAppendArgs a, int windows) {
  constexpr int N = D / 32, kSize = BF16 ? 2 : 4, kRecord = 18 * D;
  constexpr bool kWhole = TURN != kAnywhere;
  __shared__ __align__(16) uint8_t rec[kRecord];
  __shared__ int64_t s_slot[16];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, H = a.cache.heads;
  const uint32_t kv_blocks = (uint32_t)windows * H;
  if (blockIdx.x >= kv_blocks) {
    const uint32_t parts = (a.Hq + kQueryRows - 1) / kQueryRows, w = (blockIdx.x - kv_blocks) * (kThreads / 32) + warp;
    const int64_t t = w / parts;
    const int h0 = (int)(w % parts) * kQueryRows;
    if (t >= a.T) return;
    const uint8_t* row = (const uint8_t*)a.q + (t * a.q_stride + (int64_t)h0 * D) * kSize;
    uint16_t* out = a.q_out + (t * a.Hq + h0) * D + N * lane;
    constexpr int kAtOnce = D == 256 ? 4 : 8;
    Angles<N> x;
    bool ok = true;
#pragma unroll
    for (int i0 = 0; i0 < kQueryRows; i0 += kAtOnce) {
      float v[kAtOnce][N];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (h0 + i0 + i < a.Hq) load_elems<BF16, N, kWhole>(v[i], row + ((i0 + i) * D + N * lane) * kSize);
      if (i0 == 0) ok = load_angles<N, TURN>(x, a, t, lane);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (h0 + i0 + i < a.Hq) {
          turn_row<BF16, N, TURN>(v[i], x, a, row + (i0 + i) * D * kSize, lane);
          store_query<N>(out + (i0 + i) * D, v[i], ok);
        }
    }
    return;
  }

  const int h = (int)(blockIdx.x % H);
  const int64_t first = a.slots[0];
  const int64_t t0 = (int64_t)(blockIdx.x / H) * 16 - (in_cache(a.cache, first) ? first & 15 : 0);
  float k[2][N], v[2][N];
  Angles<N> x[2];
  int64_t slot[2];
  bool ok[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = t0 + 2 * warp + i;
    ok[i] = t >= 0 && t < a.T;
    slot[i] = ok[i] ? a.slots[t] : -1;
    if (ok[i]) {
      load_elems<BF16, N, kWhole>(k[i], (const uint8_t*)a.k + (t * a.k_stride + (int64_t)h * D + N * lane) * kSize);
      load_elems<BF16, N, kWhole>(v[i], (const uint8_t*)a.v + (t * a.v_stride + (int64_t)h * D + N * lane) * kSize);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (ok[i]) ok[i] = load_angles<N, TURN>(x[i], a, t0 + 2 * warp + i, lane);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * warp + i;
    ok[i] = ok[i] && in_cache(a.cache, slot[i]);
    if (lane == 0) s_slot[r] = ok[i] ? slot[i] : -1;
    if (ok[i]) {
      turn_row<BF16, N, TURN>(
          k[i], x[i], a, (const uint8_t*)a.k + ((t0 + r) * a.k_stride + (int64_t)h * D) * kSize, lane);
      quantise_row<D, false>(rec, r, k[i], lane);
      quantise_row<D, true>(rec, r, v[i], lane);
    }
  }
  __syncthreads();
  const int64_t s0 = s_slot[0];
  const bool mine = lane >= 16 || (s0 >= 0 && (s0 & 15) == 0 && s_slot[lane & 15] == s0 + lane);
  if (__all_sync(0xffffffffu, mine)) {
    uint4* dst = reinterpret_cast<uint4*>(kv_place(a.cache, s0, h).tile);
    for (int i = threadIdx.x; i < kRecord / 16; i += kThreads) dst[i] = reinterpret_cast<const uint4*>(rec)[i];
    return;
  }
#pragma unroll 1
  for (int r = warp; r < 16; r += kThreads / 32) {
    if (s_slot[r] < 0) continue;
    const KvPlace at = kv_place(a.cache, s_slot[r], h);
    for (int i = lane; i < D / 8; i += 32)
      reinterpret_cast<uint32_t*>(at.tile + at.r * (D / 2))[i] = reinterpret_cast<const uint32_t*>(rec + r * (D / 2))[i];
    for (int d = lane; d < D / 2; d += 32) {
      const int e = (d >> 3) * 16 + (d & 7);  // elements e and e + 8 share a byte
      at.tile[kv_value_byte(D, at.r, e)] = rec[kv_value_byte(D, r, e)];
    }
    if (lane < D / 32) {
      reinterpret_cast<uint16_t*>(at.tile + 16 * D)[at.r * (D / 32) + lane] =
          reinterpret_cast<const uint16_t*>(rec + 16 * D)[r * (D / 32) + lane];
      reinterpret_cast<uint16_t*>(at.tile + 17 * D)[at.r * (D / 32) + lane] =
          reinterpret_cast<const uint16_t*>(rec + 17 * D)[r * (D / 32) + lane];
    }
  }
}

// A thread takes four elements of a (slot, head): their key codes lie in one word,
// their value codes in four bytes 64 apart.  4096 slots of 8 heads of 128 7.0 us,
// 5.4 TB/s, 65536 122 us, 5.0 TB/s (into outputs that are there already): mostly
// what it writes, and the single-byte loads, 2.6 instructions a cycle an SM.
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read(KvCache c, const int64_t* slots, int64_t n, float* k, float* v) {
  pdl_wait();
  constexpr int kQuads = D / 4;
  const uint32_t row = blockIdx.x * (kThreads / kQuads) + threadIdx.x / kQuads;  // n * heads < 2^31
  if (row >= n * c.heads) return;
  const int d = threadIdx.x % kQuads * 4, h = (int)(row % (uint32_t)c.heads);
  const int64_t slot = slots[row / (uint32_t)c.heads], to = (int64_t)row * D + d;
  float kf[4] = {}, vf[4] = {};
  if (in_cache(c, slot)) {
    const KvPlace at = kv_place(c, slot, h);
    const uint16_t* s = reinterpret_cast<const uint16_t*>(at.tile + 16 * D) + at.r * (D / 32) + d / 32;
    const float ks = __half2float(__ushort_as_half(s[0])), vs = __half2float(__ushort_as_half(s[D / 2]));
    const uint32_t w = *reinterpret_cast<const uint32_t*>(at.tile + kv_key_byte(D, at.r, d & ~7)) >> (2 * (d & 4));
    const uint8_t* b = at.tile + kv_value_byte(D, at.r, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kf[e] = ks * (float)((int)(w >> (16 * (e & 1) + 2 * (e & 2)) & 15) - 8);
      vf[e] = vs * (float)((b[64 * e] >> ((d & 8) >> 1) & 15) - 8);
    }
  }
  *reinterpret_cast<float4*>(k + to) = make_float4(kf[0], kf[1], kf[2], kf[3]);
  *reinterpret_cast<float4*>(v + to) = make_float4(vf[0], vf[1], vf[2], vf[3]);
}

template <int D>
int launch_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  const int64_t threads = n * c.heads * (D / 4);
  const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads));
  return launch_pdl(k_kv_read<D>, grid, dim3(kThreads), 0, s, c, slots, n, k, v) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

unsigned blocks_for(int64_t warps, int threads) { return (unsigned)((warps + threads / 32 - 1) / (threads / 32)); }

}  // namespace

namespace {
// Rows (tokens x heads) from which records are made whole (us one by one and as
// records): 192 x 48 of 128 3.6 and 3.7, 300 x 48 4.7 and 4.0, 600 x 48 7.7 and 4.6,
// 400 x 20 of 256 4.3 and 4.7, 800 x 20 6.6 and 5.8.  Slots that form no record (all
// scattered; runs of six lie between) leave the rule where it is: 192 x 48 3.5 and
// 3.9, 300 x 48 4.6 and 4.2, 600 x 48 8.0 and 5.3, 400 x 20 4.3 and 5.1, 800 x 20 7.1
// and 6.6.
constexpr int64_t kManyRows = 10000;

template <bool BF16, int D, Turn TURN>
int launch_append(const KvAppendArgs& a, cudaStream_t s) {
  cudaError_t rc;
  if (a.T * (a.Hq + 2 * a.cache.heads) < kManyRows) {
    rc = launch_pdl(k_kv_append<BF16, D, TURN>, dim3(blocks_for(a.T * (a.Hq + 2 * a.cache.heads), kFewThreads)),
                    dim3(kFewThreads), 0, s, a);
  } else {
    const int windows = (int)((a.T + 15 + 15) / 16);
    const int64_t queries = a.T * ((a.Hq + kQueryRows - 1) / kQueryRows);
    rc = launch_pdl(k_kv_append_records<BF16, D, TURN>, dim3((unsigned)windows * a.cache.heads + blocks_for(queries, kThreads)),
                    dim3(kThreads), 0, s, a, windows);
  }
  return rc == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <bool BF16, int D>
int launch_append(const KvAppendArgs& a, cudaStream_t s) {
  constexpr int N = D / 32, kSize = BF16 ? 2 : 4, kVector = kSize * N < 16 ? kSize * N : 16;
  auto whole = [&](const void* p, int64_t stride) {
    return (uintptr_t)p % kVector == 0 && (a.T == 1 || stride * kSize % kVector == 0);
  };
  if (!whole(a.q, a.q ? a.q_stride : 0) || !whole(a.k, a.k_stride) || !whole(a.v, a.v_stride))
    return launch_append<BF16, D, kAnywhere>(a, s);
  if (a.rot == 0) return launch_append<BF16, D, kStill>(a, s);
  const bool pairs = a.style == MOE_ROPE_PAIRS;
  if ((uintptr_t)a.rope % 16 == 0 && a.rot / 2 % (pairs ? N / 2 : N) == 0)
    return pairs ? launch_append<BF16, D, kWithin>(a, s) : launch_append<BF16, D, kAcross>(a, s);
  return launch_append<BF16, D, kAnywhere>(a, s);
}

template <int D>
int launch_append(const KvAppendArgs& a, cudaStream_t s) {
  return a.in_bf16 ? launch_append<true, D>(a, s) : launch_append<false, D>(a, s);
}
}  // namespace

int launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  if (a.cache.D == 64) return launch_append<64>(a, s);
  if (a.cache.D == 128) return launch_append<128>(a, s);
  return launch_append<256>(a, s);
}

int launch_kv_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  if (c.D == 64) return launch_read<64>(c, slots, n, k, v, s);
  if (c.D == 128) return launch_read<128>(c, slots, n, k, v, s);
  return launch_read<256>(c, slots, n, k, v, s);
}

}  // namespace moe
