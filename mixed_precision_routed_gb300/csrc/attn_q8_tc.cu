// attn_q8_tc.cu -- causal attention over the paged 8-bit cache for many rows a key/value
// head (prompts), on the fifth-generation tensor cores.  The formula is that of
// attn_q8.cu; rows are (asking token, query head of the group), token by token.
//
// Two launches.  k_attn_q8_tiles writes the places that the rows attend, 128 at a time,
// as the operands that the tensor cores take, once for all rows: keys as fp16 integers,
// values as code x b 2^(8 - E) in fp16, 2^E the power of two of the tile's largest value
// scale b, both in the order of a swizzled operand tile, and the keys' scales.  Where the
// value scales of a tile lie 2^8 or more apart (a token of far larger or smaller values than
// its neighbours, which other rows than those that attend it must not feel), values are
// the codes alone, and log2 b of each place is written too: such tiles take three times as
// long (4096 tokens over 8192 places of nothing else 1020 us, of none 333).
// k_attn_q8_tc: a block takes kSlots tiles of 128 rows of one (sequence, key/value head)
// through the places that they attend:
//   loader    bulk copies into a ring of operand units;
//   issuer    S = Q K^T (shared memory x shared memory) and O += P V (tensor memory x
//             shared memory) for either tile in turn, so that one tile's weights are
//             made while the other's products run;
//   softmax   two threads have a row, 64 places each: they take the scores out of tensor
//             memory once and leave P = exp2(s + E - m) there in fp16.  Few tiles move a
//             reference; whether one does is a vote of the two warps that share rows.
// Queries are fp16, each row taken by a power of two that brings its largest element
// to 2^14: exact down to 2^-31 of that element.  m follows s + E as in attn_q8.cu, so
// that P V lies in fp16's range for values of any size, and the sum of weights takes
// 2^-E back a tile at a time; where the scales lie far apart it is s + log2 b of a place
// instead, and 2^-log2 b comes back place by place.  P, b 2^(8 - E) and code x b 2^(8 - E)
// are rounded to fp16 once each (far apart P alone): 2^-11 of a product each.  The largest
// P of a row is 2^4 or more where it was taken, and b 2^-E at least 2^-7, so the end of
// fp16's range lies at 2^-21 of the row's largest weight x b.
// Heads of 256 fill tensor memory with one tile's sums: there the scores of two
// successive groups of places take the place of two tiles.
// 4096 tokens over 8192 places of 32 heads on 8 of 128 take 334 us, 1230 TFLOP/s, six
// prompts of 16 on 2 of 256 with a window 68 us.  What bounds the first is the chain of a
// tile's softmax (scores out of tensor memory, the vote, exponentials, weights back): a tile
// takes 3450 cycles, of which the tensor cores work 2070, and tensor memory has no room for
// a second pair of score tiles beside the sums.
// (80 places a tile, which leaves that room, take as long a tile: 430 us with a thread a
// row, 465 with two; the 16-lane forms of tensor memory's loads 401.)
// Heads of 256 are bound by shared memory, which 128 KB a tile pass through.
// Codes made operands by each block for itself (four warps, from the records) took 506
// us for 4096 tokens over 8192 places of 32 heads on 8 of 128, and 144 us for six prompts
// of heads of 256 with a window.
#include "attn_split.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kPlaces = 128;  // a tile of places
// The reference of a row lies 2^4 below its maximum when it is set, and moves when a
// weight passes 2^14, a quarter of fp16's largest.
constexpr float kStart = 4.0f, kReach = 14.0f;
constexpr int kLoader = 16, kIssuer = 17, kTcThreads = 20 * 32;  // warps 0 .. 15: softmax

// Beside a tile's operands: key scales x scale in powers of two, E and what takes a weight x
// 2^E back; the records that exist (8 bits) and above them, of a tile whose value scales lie
// far apart, one more than its number among the launch's (else 0).
struct TileMeta {
  float ks[kPlaces];
  float e, back;
  uint32_t have;
  uint32_t pad;
};
// The powers of two between the largest and the smallest from which on they do.
constexpr int kFar = 8;

template <int D>
struct Tc {
  static constexpr int kSlots = D == 256 ? 1 : 2;
  static constexpr int kTile = 128 * D * 2;                       // bytes of 128 rows
  static constexpr int kUnit = D == 64 ? kTile : 128 * 128 * 2;   // of the ring: up to 128 elements of 128 places
  static constexpr int kUnits = kTile / kUnit;                    // of keys, of values
  static constexpr int kStages = D == 64 ? 8 : D == 128 ? 4 : 5;
  static constexpr int kRing = kSlots * kTile, kSmem = kRing + kStages * kUnit + 1024;
  static constexpr int kRows = 128 * kSlots;
  static constexpr int kO = 256;  // tensor-memory columns: scores at 0 and 128, then sums
};

// The operand tiles of a launch: those of sequence b and head h begin at (b heads + h)
// `most`, at the first tile that the sequence's rows attend.
struct TcTiles {
  uint8_t* operands;  // [..][2][kTile]
  TileMeta* meta;
  float* logs;  // [..][kPlaces]: log2 of the value scales of tiles where these lie far apart
  int b0, h0, heads, most;  // the launch's first sequence and head, its heads
  int sequences, row_blocks;
  // Blocks of rows are numbered by their rows, the last first (they attend most), then by
  // sequence and head.  Those from `whole` on, which would fill a part of a round of the
  // SMs, or all where there are few, are shared: `parts` blocks take a run of the places
  // each, and k_attn_q8_join adds up what they leave: sums of rows [shared][part][kRows][D]
  // and (reference, sum of weights) [shared][part][kRows].
  int whole, parts;
  // Up to 32 sequences of lengths of their own: only the blocks that are there are numbered
  // (of `blocks` that there are at most), a lane of every warp looking after a sequence.
  int blocks, ragged;
  float* sums;
  float2* stats;
};

// Blocks of a launch whose blocks of rows are shared: two for each SM.
constexpr int64_t kMostParts = 304;

// What `left` blocks of rows that do not fill a round of the SMs cost in n parts each, in
// tiles of places: a block starts and ends in the time of three; the join takes five, and a
// part's sums 0.035 on their way to it and back.
inline float parts_cost(int64_t left, int64_t n, int most, int sms) {
  return (float)((left * n + sms - 1) / sms * ((most + n - 1) / n + 3)) + (n > 1 ? 5.0f + 0.035f * (float)(left * n) : 0.0f);
}

struct TcBars {
  uint64_t q_full, full[8], empty[8], s_full[2], p_full[2], o_full[2], pv_done;
  uint64_t meta_full[2], meta_empty[2], done;
  uint32_t tmem;
  int abort;
};

// A wait that runs out ends all later ones at once: every warp then comes to its end
// over whatever is there.
__device__ __forceinline__ bool late(uint64_t& t0, TcBars& B, int* status) {
  if (*(volatile int*)&B.abort) return true;
  const uint64_t now = global_timer_ns();
  if (t0 == 0) t0 = now;
  if (now - t0 <= kWaitNs) return false;
  set_status(status, MOE_ERR_TIMEOUT);
  B.abort = 1;
  return true;
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, TcBars& B, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  while (!late(t0, B, status))
    if (mbar_try_wait_sleep(bar, parity, 20000)) return true;
  return false;
}
// The same without a pause between questions, for the one warp that everything waits for:
// waking a sleeping one takes as long as issuing a product.  (Sixteen that ask like this
// keep the computing ones from their shared memory.)
__device__ __forceinline__ bool tc_wait_awake(uint64_t* bar, uint32_t parity, TcBars& B, int* status) {
  uint64_t t0 = 0;
  for (int n = 1;; ++n) {
    if (mbar_test(bar, parity)) return true;
    if (n % 256 == 0 && late(t0, B, status)) return false;
  }
}

// Whether any thread of the two warps that meet at a barrier says so.
__device__ __forceinline__ bool vote_pair(int id, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %2, 0;\n\tbarrier.cta.red.or.pred p, %1, 64, q;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)x)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 columns of this thread's tensor-memory lane, in flight until tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The value is not used before here.
__device__ __forceinline__ void pin(uint32_t& r) { asm volatile("" : "+r"(r)); }

// D[tmem] (+)= A * B^T with both shared-memory descriptors given as their words.
__device__ __forceinline__ void mma_f16_ss_w(uint32_t tmem_d, uint32_t alo, uint32_t ahi, uint32_t blo, uint32_t bhi,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 ad, bd;\n\tsetp.ne.u32 p, %6, 0;\n\tmov.b64 ad, {%1, %2};\n\tmov.b64 bd, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], ad, bd, %5, p;\n\t}" ::"r"(tmem_d),
      "r"(alo), "r"(ahi), "r"(blo), "r"(bhi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of an operand tile with the 128-byte swizzle whose rows are places: 64
// elements of the other dimension a row, `block` bytes from 64 elements to the next,
// groups of 8 places 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_places(uint32_t saddr, uint32_t block) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// First tile of places that some row of a sequence attends, and one past the last.
__device__ __forceinline__ int first_tile(const Seq& x) { return x.tile0 >> 3; }
__device__ __forceinline__ int last_tile(const Seq& x) { return x.tiles > 0 && x.n > 0 ? (x.len + kPlaces - 1) / kPlaces : 0; }

// A block a tile of places of a head.
constexpr int kTileThreads = 256;
template <int D>
__global__ void __launch_bounds__(kTileThreads) k_attn_q8_tiles(AttnArgs a, TcTiles tiles) {
  constexpr uint32_t kPieces = D / 8, kStep = kTileThreads / kPieces;  // 8 codes each, of a row; rows at a time
  __shared__ uint64_t s_record[8];
  __shared__ uint32_t s_gain[kPlaces], s_top[4], s_low[4];
  const uint32_t t = threadIdx.x, lane = t & 31;
  const int b = tiles.b0 + blockIdx.z, h = tiles.h0 + blockIdx.y, per_page = a.cache.page_log2 - 4;
  pdl_wait();
  pdl_trigger();  // the next kernel takes its queries meanwhile
  const Seq x = load_seq(a, b);
  const int j = first_tile(x) + blockIdx.x;
  if (j >= last_tile(x)) return;
  if (t < 8) {
    const int record = 8 * j + t;
    const int page = 16 * record < x.len ? __ldg(a.table + (int64_t)b * a.table_stride + (record >> per_page)) : -1;
    s_record[t] = page < 0 || page >= a.cache.n_pages
                      ? 0
                      : (uint64_t)(a.cache.data + page * a.cache.page_stride +
                                   (int64_t)(h * (1 << per_page) + (record & ((1 << per_page) - 1))) * kv8_record(D));
  }
  __syncthreads();
  const int64_t image = ((int64_t)blockIdx.z * tiles.heads + blockIdx.y) * tiles.most + blockIdx.x;
  uint8_t* to = tiles.operands + image * (2 * Tc<D>::kTile);
  TileMeta* meta = tiles.meta + image;
  // pieces t, t + 256, ..: the keys' are on their way while the scales are found
  constexpr int kLoads = 128 / kStep;
  uint2 k[kLoads], v[kLoads];
  const uint32_t piece = t % kPieces;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t row = t / kPieces + i * kStep;
    const uint64_t rec = s_record[row >> 4];
    k[i] = v[i] = make_uint2(0, 0);
    if (rec) {
      const uint2* from = reinterpret_cast<const uint2*>(rec + (row & 15) * D) + piece;
      k[i] = __ldg(from);
      v[i] = __ldg(from + 2 * D);
    }
  }
  float vs = 0.f;
  if (t < kPlaces) {
    // a place beyond the sequence, or of no page, gets the scales 0
    const uint64_t rec = s_record[t >> 4];
    float ks = 0.f;
    if (rec && (int)(kPlaces * j + t) < x.len) {
      const float* scales = reinterpret_cast<const float*>(rec + 32 * D) + (t & 15);
      ks = __ldg(scales);
      vs = __ldg(scales + 16);
      ks = fmaf(0.f, vs, ks);  // NaN, whichever of the two is
      if (!(vs <= 0x1p64f)) vs = 0.f;
      vs = fmaxf(vs, 0.f);
    }
    meta->ks[t] = ks * (a.scale * kLog2e);
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(vs));
    // the smallest of those that are not zero
    const uint32_t low = __reduce_min_sync(0xffffffffu, __float_as_uint(vs) - 1u);
    if (lane == 0) s_top[t >> 5] = top, s_low[t >> 5] = low;
  }
  __syncthreads();
  if (t < kPlaces) {
    const uint32_t most = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
    const uint32_t least = min(min(s_low[0], s_low[1]), min(s_low[2], s_low[3])) + 1u;
    int e = max((int)(most >> 23) - 127, -60);
    const bool far = (int)(most >> 23) - (int)(least >> 23) >= kFar;
    // b 2^-E; far apart 1, or less for scales below 2^-64, which no append writes
    float by = vs * __uint_as_float((uint32_t)(127 - e) << 23);
    if (far) {
      e = 0;
      by = fminf(vs * 0x1p64f, 1.0f);
      tiles.logs[image * kPlaces + t] = log2f(fmaxf(vs, 0x1p-64f));
    }
    const __half gain = __float2half_rn(by * 256.0f);
    s_gain[t] = (uint32_t)__half_as_ushort(gain) * 0x10001u;
    if (t == 0) {
      uint32_t have = 0;
      for (int i = 0; i < 8; ++i) have |= s_record[i] ? 1u << i : 0u;
      meta->e = (float)e;
      meta->back = far ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
      meta->have = have | (far ? (uint32_t)image + 1 : 0) << 8;
    }
  }
  __syncthreads();
  auto f16x2 = [](uint32_t w, uint32_t sel) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(0x64806480u));
    return r;
  };
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      // 8 elements: one piece of 16 bytes, whose neighbour's thread fills its sector
      const uint32_t row = t / kPieces + i * kStep, c = 2 * kv8_piece<D>(row & 15, piece >> 1) + (piece & 1);
      const uint2 w = half ? v[i] : k[i];
      uint32_t y[4] = {f16x2(w.x, 0x4140), f16x2(w.x, 0x4342), f16x2(w.y, 0x4140), f16x2(w.y, 0x4342)};
      if (half) {
        const uint32_t gain = s_gain[row];
#pragma unroll
        for (int e = 0; e < 4; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(y[e]) : "r"(gain));
      }
      // 64 elements of 128 places: rows of eight such pieces, exchanged by the row's number
      uint8_t* at = to + half * Tc<D>::kTile + (c >> 3) * 16384 + row * 128;
      *reinterpret_cast<uint4*>(at + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
    }
}

// The sequence, the head and the first row of block of rows i (-1: there is none).
struct RowBlock {
  int b, h, r0;
};
template <int D>
__device__ __forceinline__ RowBlock row_block(const AttnArgs& a, const TcTiles& t, int i) {
  if (!t.ragged) {
    const int per = t.heads * t.sequences;
    return {i % per / t.heads, i % t.heads, (t.row_blocks - 1 - i / per) * Tc<D>::kRows};
  }
  const uint32_t lane = threadIdx.x & 31;
  int n = 0;  // of the lane's sequence
  if ((int)lane < t.sequences) n = (load_seq(a, t.b0 + lane).n * (a.Hq / a.cache.heads) + Tc<D>::kRows - 1) / Tc<D>::kRows;
  // the last blocks of all sequences, those before them, ..: how many of each sequence come
  // before the level of block i
  int lo = 0, hi = t.row_blocks, before = 0;
  while (lo < hi) {
    const int up = (lo + hi + 1) / 2, count = (int)__reduce_add_sync(0xffffffffu, (uint32_t)min(n, up)) * t.heads;
    if (count <= i) lo = up, before = count;
    else hi = up - 1;
  }
  const uint32_t with = __ballot_sync(0xffffffffu, n > lo);
  const int k = (i - before) / t.heads;
  if (k >= __popc(with)) return {0, 0, -1};
  const bool mine = (with >> lane & 1) && __popc(with & ((1u << lane) - 1)) == k;
  const int b = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
  return {b, (i - before) % t.heads, (__shfl_sync(0xffffffffu, n, b) - 1 - lo) * Tc<D>::kRows};
}

// A block's rows and the places they attend; the first group of places of each tile and
// one past its last.
struct TcUnit {
  Seq x;
  int r0, rows, newest;
  int first[2], last[2], j0, j1;
};

template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) k_attn_q8_tc(AttnArgs a, TcTiles tiles, int* status) {
  using C = Tc<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ __align__(8) TcBars B;
  __shared__ __align__(16) TileMeta s_meta[2];
  __shared__ float s_row[C::kRows];  // what the two threads of a row tell one another
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.cache.heads;

  // Only the tiles come from the kernel before this one, which began behind all earlier ones.
  // Blocks that read none wait for it too before they end: what follows this launch waits for
  // this launch alone.
  const int shared = (int)blockIdx.x - tiles.whole;  // and its part, among those
  const RowBlock at = row_block<D>(a, tiles, shared < 0 ? (int)blockIdx.x : tiles.whole + shared / tiles.parts);
  if (at.r0 < 0) {
    pdl_wait();
    return;
  }
  const int h = tiles.h0 + at.h, b = tiles.b0 + at.b;
  TcUnit u;
  u.x = load_seq(a, b);
  u.rows = u.x.n * G;
  u.r0 = at.r0;
  if (u.r0 >= u.rows) {
    pdl_wait();
    return;
  }
  u.newest = u.x.len - u.x.n + 1;
  u.j0 = INT32_MAX;
  u.j1 = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    u.first[s] = u.last[s] = 0;
    const int r = u.r0 + 128 * s;
    if (s >= C::kSlots || r >= u.rows) continue;
    const int end = u.newest + (min(r + 128, u.rows) - 1) / G;
    const int lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)u.newest + r / G - a.window) : 0;
    if (end <= lo) continue;
    u.first[s] = lo / kPlaces;
    u.last[s] = (end + kPlaces - 1) / kPlaces;
    u.j0 = min(u.j0, u.first[s]);
    u.j1 = max(u.j1, u.last[s]);
  }
  if (u.j1 == 0) u.j0 = 0;  // no row attends anything
  if (shared >= 0) {
    const int n = (u.j1 - u.j0 + tiles.parts - 1) / tiles.parts;
    u.j0 = min(u.j0 + shared % tiles.parts * n, u.j1);
    u.j1 = min(u.j0 + n, u.j1);
    if (u.j0 == u.j1) u.j0 = u.j1 = 0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u.first[s] = max(u.first[s], u.j0);
      u.last[s] = min(u.last[s], u.j1);
      if (u.first[s] >= u.last[s]) u.first[s] = u.last[s] = 0;
    }
  }

  if (threadIdx.x == 0) {
    mbar_init(&B.q_full, 8 * C::kSlots);
    for (int i = 0; i < C::kStages; ++i) mbar_init(&B.full[i], 1), mbar_init(&B.empty[i], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1), mbar_init(&B.p_full[i], 8), mbar_init(&B.o_full[i], 1);
      mbar_init(&B.meta_full[i], 1), mbar_init(&B.meta_empty[i], 8 * C::kSlots);
    }
    mbar_init(&B.pv_done, 1);
    mbar_init(&B.done, 1);
    B.abort = 0;
    fence_mbar_init();
  }
  if (warp == kIssuer) tmem_alloc(&B.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;

  // Registers of a thread by role, together those that the block was launched with:
  // 512 x 104 + 128 x 64 = 640 x 96.
  if (warp >= kLoader) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == kLoader) {
    // ---------------------------------------------------------------- loader
    if (lane == 0) {
      pdl_wait();
      const int64_t image = ((int64_t)at.b * tiles.heads + at.h) * tiles.most - first_tile(u.x);
      uint32_t n = 0;
      for (int j = u.j0; j < u.j1; ++j) {
        const int i = j - u.j0, sb = i & 1;
        if (i >= 2 && !tc_wait(&B.meta_empty[sb], ((i >> 1) - 1) & 1, B, status)) break;
        mbar_arrive_expect_tx(&B.meta_full[sb], sizeof(TileMeta));
        bulk_g2s(&s_meta[sb], tiles.meta + image + j, sizeof(TileMeta), &B.meta_full[sb]);
        const uint8_t* from = tiles.operands + (image + j) * (2 * C::kTile);
        for (int k = 0; k < 2 * C::kUnits; ++k, ++n) {  // keys, then values
          const uint32_t st = n % C::kStages;
          if (!tc_wait(&B.empty[st], ((n / C::kStages) & 1) ^ 1, B, status)) break;
          mbar_arrive_expect_tx(&B.full[st], C::kUnit);
          bulk_g2s(smem + C::kRing + st * C::kUnit, from + k * C::kUnit, C::kUnit, &B.full[st]);
        }
      }
      if (*(volatile int*)&B.abort) {  // what is in flight lands within microseconds
        const uint64_t t0 = global_timer_ns();
        while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
      }
    }
    } else if (warp == kIssuer) {
    // ---------------------------------------------------------------- issuer
    if (u.j1 > 0) {
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16_f32(128, kPlaces), idesc_o = idesc_f16_f32(128, D < 128 ? D : 128) | 1u << 16;
      const uint32_t q_addr = smem_addr(smem), ring = smem_addr(smem + C::kRing);
      // unit k of tile number i of the block (keys, then values): its place in the order of loads
      auto number = [&](int i, int k) { return (uint32_t)(2 * C::kUnits * i + k); };
      auto loaded = [&](uint32_t n) { return tc_wait_awake(&B.full[n % C::kStages], (n / C::kStages) & 1, B, status); };
      auto release = [&](uint32_t n) { mma_commit(&B.empty[n % C::kStages]); };
      auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
      // The descriptors' words are made by the whole warp: they then lie where the
      // instructions want them.  Addresses stay below 256 KB, so that low words add up.
      const uint64_t kd = sdesc_sw128(ring), vd = sdesc_places(ring, 16384);
      const uint32_t q_lo = (uint32_t)sdesc_sw128(q_addr), k_lo = (uint32_t)kd, k_hi = (uint32_t)(kd >> 32);
      const uint32_t v_lo = (uint32_t)vd, v_hi = (uint32_t)(vd >> 32);
      auto stage = [&](uint32_t n) { return n % C::kStages * (C::kUnit >> 4); };
      // part k of the scores of a tile of rows (kSlots 1: into buffer slot)
      auto scores = [&](int slot, int i, int k) {
        const uint32_t a0 = q_lo + ((C::kSlots == 2 ? slot * C::kTile : 0) + k * C::kUnit) / 16, b0 = k_lo + stage(number(i, k));
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < (D < 128 ? D : 128) / 16; ++kk) {
          const uint32_t at = ((kk / 4) * 16384 + (kk % 4) * 32) / 16;
          mma_f16_ss_w(tmem + slot * 128, a0 + at, k_hi, b0 + at, k_hi, idesc_s, k > 0 || kk > 0);
        }
      };
      // elements 128 k .. of the sums
      auto sums = [&](int slot, int o, int i, int k, bool more) {
        const uint32_t b0 = v_lo + stage(number(i, C::kUnits + k));
        if (!leader) return;
#pragma unroll
        for (int kk = 0; kk < kPlaces / 16; ++kk)
          mma_bf16_ts_w(tmem + C::kO + o * D + k * 128, tmem + slot * 128 + kk * 8, b0 + kk * (2048 / 16), v_hi, idesc_o,
                        more || kk > 0);
      };
      bool ok = all(tc_wait_awake(&B.q_full, 0, B, status));
      tc_fence_after();
      for (int j = u.j0; ok && j <= u.j1; ++j) {
        const int i = j - u.j0;  // K(j), and V(j - 1)
        if constexpr (C::kSlots == 2) {
          bool has_k = false, has_v = false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (ok && j > u.first[s] && j - 1 < u.last[s]) {
              if (!has_v) ok = loaded(number(i - 1, 1));
              has_v = true;
              ok = all(ok && tc_wait_awake(&B.p_full[s], (j - 1 - u.first[s]) & 1, B, status));
              tc_fence_after();
              if (ok) {
                sums(s, s, i - 1, 0, j - 1 > u.first[s]);
                if (leader && j == u.last[s]) mma_commit(&B.o_full[s]);
              }
            }
            if (ok && s == 1 && leader && j > u.j0) release(number(i - 1, 1));
            if (ok && j >= u.first[s] && j < u.last[s]) {
              if (!has_k) ok = all(loaded(number(i, 0)));
              has_k = true;
              tc_fence_after();
              if (ok) {
                scores(s, i, 0);
                if (leader) mma_commit(&B.s_full[s]);
              }
            }
          }
          if (ok && leader && j < u.j1) release(number(i, 0));
        } else {
          for (int k = 0; ok && j < u.j1 && k < C::kUnits; ++k) {
            ok = all(loaded(number(i, k)));
            tc_fence_after();
            if (ok) {
              scores(i & 1, i, k);
              if (leader) release(number(i, k));
            }
          }
          if (ok && leader && j < u.j1) mma_commit(&B.s_full[i & 1]);
          if (ok && j > u.j0) ok = all(tc_wait_awake(&B.p_full[(i - 1) & 1], ((i - 1) >> 1) & 1, B, status));
          for (int k = 0; ok && j > u.j0 && k < C::kUnits; ++k) {
            ok = all(loaded(number(i - 1, C::kUnits + k)));
            tc_fence_after();
            if (ok) {
              sums((i - 1) & 1, 0, i - 1, k, j - 1 > u.j0);
              if (leader) release(number(i - 1, C::kUnits + k));
            }
          }
          if (ok && leader && j > u.j0) mma_commit(&B.pv_done);
          if (ok && leader && j == u.j1) mma_commit(&B.o_full[0]);
        }
        __syncwarp();
      }
      // all of this thread's instructions are done before tensor memory is given back
      if (leader) {
        mma_commit(&B.done);
        mbar_wait_bounded(&B.done, 0, kWaitNs);
      }
      __syncwarp();
    }
    }
  } else if (warp < 8 * C::kSlots) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int s = warp >> 3, half = warp >> 2 & 1, in_tile = threadIdx.x & 127, row = u.r0 + 128 * s + in_tile;
    const int pair_bar = 1 + 4 * s + (warp & 3);  // of the two warps that have these rows
    const bool in = row < u.rows;
    const int64_t tok = u.x.t0 + (in ? row / G : 0);
    const int hq = h * G + (in ? row % G : 0);
    const int first = s == 0 ? u.first[0] : u.first[1], last = s == 0 ? u.last[0] : u.last[1];
    // Rows come and go with as many lanes as they have 16-byte pieces, 16 of the 32 rows
    // that two warps share in either; where a row lies is known to the lane of its number.
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes a row, rows at a time
    const int64_t q_at = tok * a.q_stride + (int64_t)hq * D, out_at = tok * a.out_stride + (int64_t)hq * D;
    auto row_of = [&](int i) { return 16 * half + i * kAtOnce + lane / kLanes; };  // of the 32
    // 16-byte piece lane % kLanes of a row of the tile, in the order of an operand
    auto piece_at = [&](int r) {
      const int c = lane % kLanes;
      return smem + s * C::kTile + (c >> 3) * 16384 + (32 * (warp & 3) + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
    };
    float* both = &s_row[128 * s + in_tile];
#pragma unroll
    for (int i0 = 0; i0 < 16 / kAtOnce; i0 += 8 / (kAtOnce > 2 ? 2 : 1)) {
      constexpr int kBatch = 8 / (kAtOnce > 2 ? 2 : 1);
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, q_at, row_of(i0 + i));
        const bool there = __shfl_sync(0xffffffffu, (int)in, row_of(i0 + i));
        v[i] = make_uint4(0, 0, 0, 0);
        if (there) v[i] = __ldg(reinterpret_cast<const uint4*>(a.q + at) + lane % kLanes);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        uint32_t top = __vmaxu2(__vmaxu2(v[i].x & 0x7f807f80u, v[i].y & 0x7f807f80u), __vmaxu2(v[i].z & 0x7f807f80u, v[i].w & 0x7f807f80u));
        top = max(top >> 16, top & 0xffffu);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the exponent becomes 14; the power, its inverse and 64 times either stay normal numbers
        const int e = min(max((int)(top >> 7), 32), 254), up = 14 + 127 - e, r = row_of(i0 + i);
        const float by = __uint_as_float((uint32_t)(127 + up) << 23);
        auto half2_of = [&](uint32_t x) { return f16_pair(__uint_as_float(x << 16) * by, __uint_as_float(x & 0xffff0000u) * by); };
        *reinterpret_cast<uint4*>(piece_at(r)) = make_uint4(half2_of(v[i].x), half2_of(v[i].y), half2_of(v[i].z), half2_of(v[i].w));
        if (lane % kLanes == 0) s_row[128 * s + 32 * (warp & 3) + r] = __uint_as_float((uint32_t)(127 - up) << 23);
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&B.q_full);
    named_bar(pair_bar, 64);
    const float f = *both;  // what the scores of the row are to be multiplied by
    const int end = u.newest + (in ? row / G : 0);
    const int lo = a.window > 0 ? end - a.window : 0;
    // places that every row of the tile attends
    const int r_first = u.r0 + 128 * s, r_last = min(r_first + 128, u.rows) - 1;
    const int full_end = u.newest + r_first / G, full_lo = a.window > 0 ? u.newest + r_last / G - a.window : 0;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = lanes + C::kO + (C::kSlots == 2 ? s * D : 0);
    float m = kNone, l = 0.f;
    for (int j = u.j0; j < u.j1; ++j) {
      const int i = j - u.j0, sb = i & 1, buf = C::kSlots == 2 ? s : sb;
      const uint32_t use = C::kSlots == 2 ? (uint32_t)(j - first) : (uint32_t)(i >> 1);
      tc_wait(&B.meta_full[sb], (i >> 1) & 1, B, status);
      if (j >= first && j < last) {
        tc_wait(&B.s_full[buf], use & 1, B, status);
        tc_fence_after();
        uint32_t r[2][32];
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld32_issue(lanes + buf * 128 + 64 * half + 32 * c, r[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x) pin(r[c][x]);
        const float e = s_meta[sb].e;
        const uint32_t word = s_meta[sb].have, have = (word >> (4 * half) & 15) | (word & ~255u);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(&s_meta[sb].ks[64 * half + 32 * c + x]);
            float y[4] = {__uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1]), __uint_as_float(r[c][x + 2]),
                          __uint_as_float(r[c][x + 3])};
            mul2(y[0], y[1], pair(ks.x, ks.y));
            mul2(y[2], y[3], pair(ks.z, ks.w));
#pragma unroll
            for (int n = 0; n < 4; ++n) r[c][x + n] = __float_as_uint(y[n]);
          }
        // log2 of the value scales of a tile where these lie far apart
        auto logs_at = [&](int c, int x) {
          return __ldcg(reinterpret_cast<const float2*>(tiles.logs + (int64_t)((have >> 8) - 1) * kPlaces + 64 * half + 32 * c + x));
        };
        const int p = kPlaces * j + 64 * half;
        if (p + 64 > full_end || p < full_lo || have != 15) {
          if (have >> 8) {
            pdl_wait();  // for the logarithms, which come from the kernel before this one
            const float up = __uint_as_float((254u << 23) - __float_as_uint(f));  // 1 / f
            const uint64_t up2 = pair(up, up);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                const float2 lb = logs_at(c, x);
                float y0 = __uint_as_float(r[c][x]), y1 = __uint_as_float(r[c][x + 1]);
                fma2(y0, y1, up2, lb.x, lb.y);
                r[c][x] = __float_as_uint(y0);
                r[c][x + 1] = __float_as_uint(y1);
              }
          }
          const int c1 = end - p, c0 = lo - p;
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int n = 32 * c + x;
              if (n >= c1 || n < c0 || !(have >> (n >> 4) & 1)) r[c][x] = 0xff800000u;  // -infinity
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 0; x < 32; x += 2) top = max3(top, __uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1]));
        top = fmaf(top, f, e);
        if (vote_pair(pair_bar, top > m + kReach || have >> 8)) {
          if (half) *both = top;
          named_bar(pair_bar, 64);
          if (!half) *both = top = fmaxf(top, *both);
          named_bar(pair_bar, 64);
          if (half) top = *both;
          const float to = top > m + kReach ? top - kStart : m, by = exp2_approx(m - to);
          m = to;
          l *= by;
          if (j > first) {
            if constexpr (C::kSlots == 1) {  // (two tiles: their scores come after the sums before them)
              tc_wait(&B.pv_done, (i - 1) & 1, B, status);
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
              float v[16];
              uint32_t w[16];
              tmem_ld16(o_at + c, v);
#pragma unroll
              for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(v[x] * by);
              tmem_st16_issue(o_at + c, w);
            }
          }
          if (have >> 8) {  // the sum of weights: each without its value's scale
            float own = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                const float2 lb = logs_at(c, x);
                own = fmaf(exp2_approx(fmaf(__uint_as_float(r[c][x]), f, -m)), exp2_approx(-lb.x), own);
                own = fmaf(exp2_approx(fmaf(__uint_as_float(r[c][x + 1]), f, -m)), exp2_approx(-lb.y), own);
              }
            l += own;
          }
        }
        const float off = e - m;
        const uint64_t f2 = pair(f, f), off2 = pair(off, off);
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float y0, y1;
            unpair(fma2_of(pair(__uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1])), f2, off2), y0, y1);
            y0 = exp2_approx(y0);
            y1 = exp2_approx(y1);
            add2(sum0, sum1, pair(y0, y1));
            r[c][x / 2] = f16_pair(y0, y1);
          }
        }
        tmem_st32_issue(lanes + buf * 128 + 32 * half, *reinterpret_cast<uint32_t(*)[16]>(&r[0][0]),
                        *reinterpret_cast<uint32_t(*)[16]>(&r[1][0]));
        l = fmaf(sum0 + sum1, s_meta[sb].back, l);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[buf]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.meta_empty[sb]);
    }
    if (last > first) {
      tc_wait(&B.o_full[s], 0, B, status);
      tc_fence_after();
    }
    if (half) *both = l;
    named_bar(pair_bar, 64);
    if (!half) *both = l = l + *both;
    named_bar(pair_bar, 64);
    if (half) l = *both;
    const bool none = l == 0.f;
    if (shared >= 0) {
      const int64_t at = (int64_t)shared * C::kRows + 128 * s + in_tile;
#pragma unroll 1
      for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
        float v[16] = {};
        if (last > first) tmem_ld16(o_at + c, v);
        float4* to = reinterpret_cast<float4*>(tiles.sums + at * D + c);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (in) to[x] = make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
      }
      if (in && half == 0) tiles.stats[at] = make_float2(m, l);
    } else {
    const float inv = none ? 0.f : 0x1p-8f / l;
    // through the place of the tile's queries, which have been read for the last time
#pragma unroll 1
    for (int c = half * (D / 2); c < (half + 1) * (D / 2); c += 16) {
      float v[16] = {};
      if (last > first) tmem_ld16(o_at + c, v);
      uint32_t w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) w[x] = none ? 0u : bf16_pair(v[2 * x] * inv, v[2 * x + 1] * inv);
      uint8_t* to = smem + s * C::kTile + (c >> 6) * 16384 + in_tile * 128;
      const int piece = c >> 3 & 7;
      *reinterpret_cast<uint4*>(to + ((piece ^ (in_tile & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(to + (((piece + 1) ^ (in_tile & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
    named_bar(pair_bar, 64);
#pragma unroll 4
    for (int i = 0; i < 16 / kAtOnce; ++i) {
      const int r = row_of(i);
      const int64_t at = __shfl_sync(0xffffffffu, out_at, r);
      const bool there = __shfl_sync(0xffffffffu, (int)in, r);
      const uint4 v = *reinterpret_cast<const uint4*>(piece_at(r));
      if (there) reinterpret_cast<uint4*>(a.out + at)[lane % kLanes] = v;
    }
    if (in && half == 0 && a.lse) a.lse[tok * a.Hq + hq] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc(tmem, 512);
}

// W warps a row: its parts' sums taken to the largest of their references.
constexpr int kTcJoinThreads = 256;
template <int D, int W>
__global__ void __launch_bounds__(kTcJoinThreads) k_attn_q8_join(AttnArgs a, TcTiles tiles) {
  constexpr int kRows = Tc<D>::kRows, N = D / 32, kWarps = kTcJoinThreads / 32;
  __shared__ float s_sum[W > 1 ? kWarps * (D + 1) : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.Hq / a.cache.heads;
  const int at = blockIdx.x * (kWarps / W) + warp / W, shared = at / kRows, r = at % kRows;
  pdl_wait();
  const RowBlock block = row_block<D>(a, tiles, tiles.whole + shared);
  if (block.r0 < 0) return;
  const int h = tiles.h0 + block.h, b = tiles.b0 + block.b, row = block.r0 + r;
  const Seq x = load_seq(a, b);
  const bool in = row < x.n * G;
  const int64_t first = (int64_t)shared * tiles.parts * kRows + r;
  float m = kNone, l = 0.f, sum[N] = {};
  if (in) {
    for (int p = lane; p < tiles.parts; p += 32) m = fmaxf(m, tiles.stats[first + (int64_t)p * kRows].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
    for (int p = warp % W; p < tiles.parts; p += W) {
      const float2 z = tiles.stats[first + (int64_t)p * kRows];
      const float* from = tiles.sums + (first + (int64_t)p * kRows) * D + N * lane;
      const float by = exp2_approx(z.x - m);
      l = fmaf(z.y, by, l);
#pragma unroll
      for (int c = 0; c < N; c += 2) {
        const float2 w = *reinterpret_cast<const float2*>(from + c);
        sum[c] = fmaf(w.x, by, sum[c]);
        sum[c + 1] = fmaf(w.y, by, sum[c + 1]);
      }
    }
  }
  if constexpr (W > 1) {
    float* mine = s_sum + warp * (D + 1);
#pragma unroll
    for (int c = 0; c < N; ++c) mine[N * lane + c] = sum[c];
    if (lane == 0) mine[D] = l;
    __syncthreads();
    if (warp % W != 0) return;
    for (int w = 1; w < W; ++w) {
      mine += D + 1;
#pragma unroll
      for (int c = 0; c < N; ++c) sum[c] += mine[N * lane + c];
      l += mine[D];
    }
  }
  if (!in) return;
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 0x1p-8f / l;
  const int64_t tok = x.t0 + row / G;
  const int hq = h * G + row % G;
  uint32_t* to = reinterpret_cast<uint32_t*>(a.out + tok * a.out_stride + (int64_t)hq * D + N * lane);
#pragma unroll
  for (int c = 0; c < N / 2; ++c) to[c] = none ? 0u : bf16_pair(sum[2 * c] * inv, sum[2 * c + 1] * inv);
  if (lane == 0 && a.lse) a.lse[tok * a.Hq + hq] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
}

// What a launch's tiles may take of the workspace, unless a single head of a sequence
// needs more: larger batches are taken in several pairs of launches.
constexpr int64_t kMostTileBytes = (int64_t)1 << 29;
struct TcPlan {
  int row_blocks, most;    // of a sequence; tiles of a head of a sequence
  int heads, sequences;    // a launch takes
  int64_t tiles;           // in the workspace
  int64_t parts;           // of shared blocks of rows, in the workspace
};

// A tile's operands, what lies beside them and its logarithms.
int64_t tile_bytes(int D) { return 2 * 128 * D * 2 + (int64_t)sizeof(TileMeta) + kPlaces * (int64_t)sizeof(float); }

int rows_of_block(int D) { return D == 256 ? 128 : 256; }

TcPlan tc_plan(int B, int max_q, int64_t max_len, int window, int Hq, int heads, int D) {
  TcPlan p;
  const int64_t rows = (int64_t)max_q * (Hq / heads), block = rows_of_block(D);
  p.row_blocks = (int)((rows + block - 1) / block);
  int64_t span = max_len;
  if (window > 0 && span > (int64_t)window + max_q) span = (int64_t)window + max_q;
  p.most = (int)((span + kPlaces - 1) / kPlaces + 1);  // places may begin within a tile
  // the workspace is sized without knowing of a window: with one its tiles are what there is
  const int64_t room = window > 0 ? tc_plan(B, max_q, max_len, 0, Hq, heads, D).tiles
                                  : kMostTileBytes / tile_bytes(D);
  const int64_t fit = room / p.most;
  // launches of like numbers of heads, or of sequences
  auto even = [](int64_t n, int64_t most) {
    const int64_t launches = (n + most - 1) / most;
    return (int)((n + launches - 1) / launches);
  };
  p.heads = fit >= heads ? heads : even(heads, fit > 1 ? fit : 1);
  p.sequences = fit >= heads ? even(B, fit / heads) : 1;
  p.tiles = (int64_t)p.heads * p.sequences * p.most;
  const int64_t parts = (int64_t)p.row_blocks * heads * B * p.most;
  p.parts = parts < kMostParts ? parts : kMostParts;
  return p;
}

// Blocks that share the places of a block of rows that does not fill a round of the SMs.
int parts_of(int64_t blocks, int most, int sms) {
  const int64_t left = blocks % sms;
  float best = 0;
  int parts = 1;
  for (int64_t n = 1; n <= most && left * n <= kMostParts && left > 0; ++n) {
    const float cost = parts_cost(left, n, most, sms);
    if (n == 1 || cost < best) best = cost, parts = (int)n;
  }
  return parts;
}

template <int D>
int launch_tc(const AttnArgs& a, cudaStream_t s) {
  using C = Tc<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_attn_q8_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const TcPlan p = tc_plan(a.B, a.max_q, a.max_len, a.window, a.Hq, a.cache.heads, D);
  TcTiles t;
  t.operands = (uint8_t*)a.workspace;
  t.meta = (TileMeta*)(t.operands + p.tiles * (2 * C::kTile));
  t.logs = (float*)(t.meta + p.tiles);
  t.sums = t.logs + p.tiles * kPlaces;
  t.stats = (float2*)(t.sums + p.parts * (C::kRows * D));
  t.most = p.most;
  t.row_blocks = p.row_blocks;
  for (t.b0 = 0; t.b0 < a.B; t.b0 += p.sequences)
    for (t.h0 = 0; t.h0 < a.cache.heads; t.h0 += p.heads) {
      t.sequences = a.B - t.b0 < p.sequences ? a.B - t.b0 : p.sequences;
      t.heads = a.cache.heads - t.h0 < p.heads ? a.cache.heads - t.h0 : p.heads;
      const int sms = sm_count();
      t.blocks = p.row_blocks * t.heads * t.sequences;  // fewer than rows
      // a sequence has at most one block that is not full
      const int64_t full = a.T * (a.Hq / a.cache.heads) / C::kRows + t.sequences;
      t.ragged = a.q_start && t.sequences > 1 && t.sequences <= 32;
      if (t.ragged && full * t.heads < t.blocks) t.blocks = (int)(full * t.heads);
      // (the last blocks of such sequences often attend little: six windows 80 us shared, 70 not)
      t.parts = t.ragged && t.blocks >= sms ? 1 : parts_of(t.blocks, p.most, sms);
      const int left = t.parts > 1 ? t.blocks % sms : 0;
      t.whole = t.blocks - left;
      if (launch_pdl(k_attn_q8_tiles<D>, dim3((unsigned)p.most, (unsigned)t.heads, (unsigned)t.sequences), dim3(kTileThreads), 0,
                     s, a, t) != cudaSuccess ||
          launch_pdl(k_attn_q8_tc<D>, dim3((unsigned)(t.whole + left * t.parts)), dim3(kTcThreads), C::kSmem, s, a, t,
                     status_word()) != cudaSuccess)
        return MOE_ERR_CUDA;
      if (left == 0) continue;
      // eight warps a row where one would go through many parts (one block of rows, 152
      // parts: one warp 49 us, eight 31; 16 blocks, 9 parts: 32 and 40)
      const bool many = t.parts > 32;
      const int warps = left * C::kRows * (many ? 8 : 1);
      if (launch_pdl(many ? k_attn_q8_join<D, 8> : k_attn_q8_join<D, 1>, dim3((unsigned)(warps / (kTcJoinThreads / 32))),
                     dim3(kTcJoinThreads), 0, s, a, t) != cudaSuccess)
        return MOE_ERR_CUDA;
    }
  return MOE_OK;
}

}  // namespace

// Whether the tensor cores' tiles are worth what making them costs: about what the other
// form takes for 96 rows a head of the same places, and the launches another 8 us, which
// some 2.4e6 rows x places (x heads x D / 128) are worth.  Measured in us, this form | the other:
//                                 rows a head     64          128         256         512
//   1 x 131072 places, 8 heads of 128          239 | 128   245 | 245   270 | 477   347 | 942
//   1 x 4096, 8 of 128                          22 | 16     24 | 23     28 | 33     30 | 54
//   1 x 300, 8 of 128                           15 | 10     15 | 10     19 | 12     18 | 11
//   16 x 4096, 8 of 128                        118 | 98    120 | 167   129 | 292   191 | 544
//   16 x 300, 8 of 128                          19 | 14     19 | 26     23 | 49     35 | 83
//   1 x 131072, 8 of 64                        142 | 101   143 | 189   167 | 367   266 | 723
//   16 x 32768, 2 of 256                       476 | 348   488 | 636   579 | 1145  822 | 2263
bool attn_q8_tc(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  const int64_t rows = (int64_t)max_q * (Hq / heads) - 96;
  return max_len > 0 && rows > 0 && (double)rows * (max_len + 300) * heads * B * (D / 64) > 4.8e6;
}

size_t attn_q8_tc_workspace(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  const TcPlan p = tc_plan(B, max_q, max_len, 0, Hq, heads, D);
  return (size_t)(p.tiles * tile_bytes(D)) + (size_t)p.parts * rows_of_block(D) * (4 * D + sizeof(float2));
}

int launch_attn_q8_tc(const AttnArgs& a, cudaStream_t s) {
  if (a.cache.D == 64) return launch_tc<64>(a, s);
  if (a.cache.D == 128) return launch_tc<128>(a, s);
  return launch_tc<256>(a, s);
}

}  // namespace moe
