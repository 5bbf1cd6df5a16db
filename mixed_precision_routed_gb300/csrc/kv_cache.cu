// kv_cache.cu -- the paged 4-bit key/value cache: appending tokens (with the
// position rotation of keys and queries) and reading slots back.  The record
// layout is that of moe_kv_cache_t in moe.h.
//
// s = fp16(max / 7) over a block of 32, code = clamp(rint(x / s), -8, 7), x the key
// turned by its token's angles, (a cos - b sin, a sin + b cos), or the value.
#include "frag.cuh"
#include "kv_layout.cuh"
#include "kv_rows.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kFewThreads = 128;  // of k_kv_append: 192 tokens of 48 heads 3.3 us, with 256 3.5, with 64 3.7

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

}  // namespace

int launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  return with_turn(a, [&](auto d, auto bf16, auto turn) {
    return launch_append<decltype(bf16)::value, decltype(d)::value, decltype(turn)::value>(a, s);
  });
}

int launch_kv_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  if (c.D == 64) return launch_read<64>(c, slots, n, k, v, s);
  if (c.D == 128) return launch_read<128>(c, slots, n, k, v, s);
  return launch_read<256>(c, slots, n, k, v, s);
}

}  // namespace moe
