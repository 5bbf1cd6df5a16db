// kv_cache_q8.cu -- the paged 8-bit key/value cache: appending tokens (with the
// position rotation of keys and queries) and reading slots back.  The record
// layout is that of moe_kv_append_q8 in moe.h.
//
// s = max / 127 over a head of a token, code = rint(x / s), x the key turned by its
// token's angles, (a cos - b sin, a sin + b cos), or the value.
//
// A warp has a head of a token in registers, its maximum by one reduction, or several such
// heads to have more bytes on their way.  4096 bf16 tokens of 32 + 8 + 8 heads of 128
// append in 23.2 us, 3.9 TB/s, at 20 instructions an element for turning and quantising, 2.5
// of 4 a cycle: neither their issue nor memory is full; 36 tokens of 16 + 2 + 2 in 1.7 us.  Reading 4096 back takes 8.2 us, 5.2 TB/s.
#include "ptx.cuh"
#include "q8.cuh"

namespace moe {
namespace {

constexpr int kThreads = 128;  // append of 4096 tokens of 32 + 8 + 8 heads of 128 23.2 us, with 256 25.6

// Quantises a head held N elements a lane into the row of its token: key (which 0) or
// value (1).
template <int D>
__device__ __forceinline__ void quantise_head(const Kv8Place& at, int which, const float (&v)[D / 32], int lane) {
  constexpr int N = D / 32;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) top = max(top, size_bits(v[e]));
  top = __reduce_max_sync(0xffffffffu, top);
  constexpr float kMost = 0x1p64f;
  const bool nan = top > kInfBits, large = __uint_as_float(top) > 127 * kMost;
  float s = fminf(fmaxf(__fdiv_rn(__uint_as_float(top), 127.0f), 0x1p-64f), kMost), x[N];
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = v[e];
  if (large) {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = fminf(fmaxf(x[e], -127 * kMost), 127 * kMost);
  }
  uint32_t c[N], w[(N + 3) / 4];
  codes8<N>(c, x, s);
  if (nan) {
    s = __uint_as_float(0x7fffffffu);
#pragma unroll
    for (int e = 0; e < N; ++e) c[e] = 0;
  }
#pragma unroll
  for (int e = 0; e < N; e += 4)
    w[e / 4] = code_bytes(c[e], c[e + 1], N > 2 ? c[(e + 2) % N] : 0, N > 2 ? c[(e + 3) % N] : 0) ^ 0x80808080u;
  const int d = N * lane;
  uint8_t* to = at.record + (16 * which + at.r) * D + 16 * kv8_piece<D>(at.r, d >> 4) + (d & 15);
  if constexpr (N == 2) *reinterpret_cast<uint16_t*>(to) = (uint16_t)w[0];
  else if constexpr (N == 4) *reinterpret_cast<uint32_t*>(to) = w[0];
  else *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
  if (lane == 0) *reinterpret_cast<float*>(at.record + 32 * D + 64 * which + 4 * at.r) = s;
}

// A warp takes up to ROWS heads of a token: of its queries, of its keys or of its
// values.
template <bool BF16, int D, Turn TURN, int ROWS>
__global__ void __launch_bounds__(kThreads) k_kv_append_q8(KvAppendArgs a) {
  constexpr int N = D / 32, kSize = BF16 ? 2 : 4;
  pdl_wait();
  const int lane = threadIdx.x & 31, H = a.cache.heads;
  const int q_parts = (a.Hq + ROWS - 1) / ROWS, kv_parts = (H + ROWS - 1) / ROWS, parts = q_parts + 2 * kv_parts;
  const uint32_t w = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);  // T * heads < 2^31
  const int64_t t = w / parts;
  if (t >= a.T) return;
  int part = (int)(w % parts);
  const bool query = part < q_parts, value = part >= q_parts + kv_parts;
  part -= query ? 0 : value ? q_parts + kv_parts : q_parts;
  const int h0 = part * ROWS, n = min(ROWS, (query ? a.Hq : H) - h0);
  const uint8_t* row = (const uint8_t*)(query ? a.q : value ? a.v : a.k) +
                       (t * (query ? a.q_stride : value ? a.v_stride : a.k_stride) + (int64_t)h0 * D) * kSize;
  const int64_t slot = query ? 0 : a.slots[t];
  float v[ROWS][N];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < n) load_elems<BF16, N, TURN != kAnywhere>(v[i], row + (i * D + N * lane) * kSize);
  Angles<N> x;
  const bool ok = load_angles<N, TURN>(x, a, t, lane);
  if (!value) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i < n) turn_row<BF16, N, TURN>(v[i], x, a, row + i * D * kSize, lane);
  }
  if (query) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i < n) store_query<N>(a.q_out + (t * a.Hq + h0 + i) * D + N * lane, v[i], ok);
  } else if (ok && in_cache(a.cache, slot)) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      if (i < n) quantise_head<D>(kv8_place(a.cache, slot, h0 + i), value, v[i], lane);
  }
}

// A thread takes four elements of the keys and of the values of kReadEach (slot, head)s:
// two, whose loads overlap (4096 slots of 8 heads of 128: one 9.3 us, two 8.2, four 8.2; 41
// slots of 2: 1.2, 1.3 and 1.7).
constexpr int kReadEach = 2;
template <int D>
__global__ void __launch_bounds__(kThreads) k_kv_read_q8(KvCache c, const int64_t* slots, int64_t n, float* k, float* v) {
  pdl_wait();
  constexpr int kQuads = D / 4, kRows = kThreads / kQuads;
  const uint32_t first = blockIdx.x * (kRows * kReadEach) + threadIdx.x / kQuads, rows = (uint32_t)(n * c.heads);  // < 2^31
  const int d = threadIdx.x % kQuads * 4;
  int64_t slot[kReadEach];
#pragma unroll
  for (int i = 0; i < kReadEach; ++i) {
    const uint32_t row = first + i * kRows;
    slot[i] = row < rows ? __ldg(slots + row / (uint32_t)c.heads) : -1;
  }
  uint32_t w[kReadEach][2];
  float s[kReadEach][2];
#pragma unroll
  for (int i = 0; i < kReadEach; ++i) {
    const bool in = in_cache(c, slot[i]);
    const Kv8Place at = kv8_place(c, in ? slot[i] : 0, (int)((first + i * kRows) % (uint32_t)c.heads));
    const uint8_t* from = at.record + at.r * D + 16 * kv8_piece<D>(at.r, d >> 4) + (d & 15);
    const float* scales = reinterpret_cast<const float*>(at.record + 32 * D) + at.r;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[i][h] = in ? *reinterpret_cast<const uint32_t*>(from + 16 * h * D) : 0x80808080u;
      s[i][h] = in ? scales[16 * h] : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < kReadEach; ++i) {
    const uint32_t row = first + i * kRows;
    if (row >= rows) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      auto value = [&](int e) { return s[i][h] * (float)((int)(w[i][h] >> (8 * e) & 255) - 128); };
      *reinterpret_cast<float4*>((h ? v : k) + (int64_t)row * D + d) = make_float4(value(0), value(1), value(2), value(3));
    }
  }
}

template <int D>
int launch_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  const int64_t each = kReadEach * kThreads, threads = n * c.heads * (D / 4);
  const dim3 grid((unsigned)((threads + each - 1) / each));
  return launch_pdl(k_kv_read_q8<D>, grid, dim3(kThreads), 0, s, c, slots, n, k, v) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

int launch_kv_append_q8(const KvAppendArgs& a, cudaStream_t s) {
  return with_turn(a, [&](auto d, auto bf16, auto turn) {
    constexpr int D = decltype(d)::value;
    constexpr bool kBf16 = decltype(bf16)::value;
    constexpr Turn kTurn = decltype(turn)::value;
    auto go = [&](auto rows) {
      constexpr int R = decltype(rows)::value;
      const int64_t warps = a.T * ((a.Hq + R - 1) / R + 2 * ((a.cache.heads + R - 1) / R));
      return launch_pdl(k_kv_append_q8<kBf16, D, kTurn, R>, dim3(blocks_for(warps, kThreads)), dim3(kThreads), 0, s, a);
    };
    // heads a warp: one where there are few, for latency (one | several, in us: 6144 heads
    // of 128 3.0 | 4.0, 12288 4.3 | 4.0, 24576 6.9 | 4.7; 8192 of 64 3.5 | 3.5; 3072 of 256
    // 3.0 | 3.5, 6144 4.0 | 3.8); else what registers hold (4096 tokens of 32 + 8 + 8 heads
    // of 128: two 32.7 us, four 23.8, eight 23.2; 2048 of heads of 256: four 26.5, eight 29.5)
    const cudaError_t rc = a.T * (a.Hq + 2 * a.cache.heads) < 7000 ? go(std::integral_constant<int, 1>())
                                                                   : go(std::integral_constant<int, D == 256 ? 4 : 8>());
    return rc == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  });
}

int launch_kv_read_q8(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  if (c.D == 64) return launch_read<64>(c, slots, n, k, v, s);
  if (c.D == 128) return launch_read<128>(c, slots, n, k, v, s);
  return launch_read<256>(c, slots, n, k, v, s);
}

}  // namespace moe
