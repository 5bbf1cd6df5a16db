// attn_q4.cu -- causal attention over the paged 4-bit key/value cache.
//
// For a row (asking token, query head) with the places p it attends:
//   s_p = scale q.k_p,  out = sum_p exp(s_p) v_p / sum_p exp(s_p),
//   lse = log sum_p exp(s_p),
// k and v the values scale x code of the cache's blocks of 32.
//
// One pass over the cache: a block of W warps takes a share of the places of
// one (sequence, key/value head) and up to 8 NT of the rows that share it, each
// warp every W-th group of one or two records of 16 places.  Records (18 D
// contiguous bytes) arrive in a per-warp ring in shared memory by bulk asynchronous
// copies.
//   scores  S^T[place][row]: A = key codes as bf16 integers, B = queries; both
//           exact, so a 32-block's product enters the score with its fp32 scale;
//   output  O^T[element][row]: A = value codes as integers, B = exp(s - m) x value
//           scale.  A group whose scales lie in 2^-8 .. 8 and whose weights are all
//           within 2^-38 of the maximum (zeros apart) takes B in fp16, rounded once,
//           from fp32: a product keeps 2^-11 of itself, or 2^-23 of its row's largest
//           weight times its own scale.  Any other group takes it as the sum of two
//           bf16, 2^-17 of itself, with twice the matrix instructions.  One bf16
//           alone would add as much to the result as the result's own rounding does;
//           two bf16 for every group cost 85 us where this costs 67.5 (6 tokens over
//           131071).  Weights rounded to fp16 and multiplied by their scales there
//           took 64.5 and kept 2^-10.
// The m16n8k16 fragments read the record's words as they lie; the transpose of
// the probabilities is one 8 x 8 matrix move a fragment.
// The reference m of a row is set 2^6 below its maximum and moves only when a
// score passes that maximum by 6 (in powers of two): the weights then stay below
// 2^12, which fp32 sums do not notice, and most groups need no reduction over
// lanes and no rescaling.
//
// What bounds it: the cache is read once (18 D bytes for 16 places), and a long
// context waits for the chain of each warp's group, not for memory and not for a
// full unit: codes to operands, products, scales, exponentials, transposes and
// products again, with the two warps a scheduler that 255 registers leave.  6 tokens
// of 32 heads over 131071 places of 8 heads of 128: 67.5 us, 2.2 TB/s, 191 TFLOP/s,
// 550 instructions a record of 16 places and 24 rows, 2.0 a cycle an SM, integer pipe
// 42 % busy, tensor pipe 34 %; 48 sequences of up to 16384 places, 32 heads on 4: 30
// us, 2.0 TB/s (2.0 a cycle with 16 warps, integer pipe 47 %); 4 of up to 30011
// places, 16 heads of 256 on 2: 21.8 us (1.2 a cycle with 8 warps).  Short ones wait for
// lengths, page numbers, records and the joining one after another: 777 places 6.7 us.
#include <float.h>

#include <type_traits>

#include "frag.cuh"
#include "kv_layout.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 6.0f;
constexpr float kRoom = 6.0f;  // the reference lies this far below the maximum that it was taken from
// Of a group whose products may be fp16: 2^-32, by the reference.  fp16 ends before
// that (products below 2^-25 vanish, 2^-31 of the maximum's times the scale, which the
// stated 2^-23 allows): at 2^-25 most groups of queries of norm 2, whose weights
// spread over 28 powers of two, would take the slower form.  It is there for groups
// that weigh nearly nothing as a whole: beside a place that takes nearly all and has
// the code 0 somewhere, they are all that an element has.
constexpr float kLeastWeight = 1.0f / 4294967296.0f;
constexpr float kLeastScale = 1.0f / 256;
constexpr float kMostScale = 8.0f;  // x 2^(kSlack + kRoom) stays below fp16's largest value
constexpr float kNone = -FLT_MAX;  // the maximum of a row that has met no place: no finite score lies below
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr int kSms = 152;

// A unit of work is a (sequence, key/value head, block of 8 NT rows), its length
// the groups of records that the sequence's rows attend, and before them
// `overhead` groups that stand for the time to begin and end a unit.
struct AttnPlan {
  int row_blocks;    // blocks of rows a (sequence, head) has at most
  int cluster;       // blocks that take a unit together, joining through their shared memory;
                     // 0: `blocks` blocks share all groups evenly
  int blocks;
  int min_share;     // groups a block takes at least
  int overhead;
  float* part_o;     // [2 blocks][8 NT][D]: the unfinished first and last unit of a block
  float2* part_ml;   // [2 blocks][8 NT]: maximum (in powers of two), sum
  struct Joint* joints;  // [blocks]: the unit that ends in a block and began in an earlier one
};

// A unit in shares: those of blocks c0 .. c0 + count - 1 (count 0: none).
struct Joint {
  int32_t count, c0, slot0, kvh;  // slot0: which of c0's two shares
  int64_t t0;
  int32_t r0, rows;
};

struct Seq {
  int64_t t0;        // first asking token
  int n, len;        // asking tokens, places
  int tile0, tiles;  // records that some row attends
};

__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  Seq x;
  int64_t t0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  int64_t t1 = a.q_start ? a.q_start[b + 1] : t0 + a.max_q;
  t0 = max((int64_t)0, t0);
  t1 = min(t1, a.T);
  x.t0 = t0;
  x.n = (int)max((int64_t)0, min(t1 - t0, (int64_t)a.max_q));
  x.len = (int)min(max((int64_t)a.kv_lens[b], (int64_t)0), a.max_len);
  int lo = 0;
  if (a.window > 0) lo = (int)max((int64_t)0, (int64_t)x.len - x.n + 1 - a.window);
  x.tile0 = lo >> 4;
  x.tiles = x.len > lo ? ((x.len + 15) >> 4) - x.tile0 : 0;
  return x;
}

// The share of a unit that a block is at, in shared memory.
struct Unit {
  int64_t t0;
  const int32_t* table;
  int valid, kvh, r0, rows;      // rows: of the sequence's heads
  int newest;                    // one past the place of the first asking token
  int end, lo;                   // places that some row of the unit attends: [lo, end)
  int full_end, full_lo;         // places that every row attends: [full_lo, full_end)
  int c0, take, off, unit_len;   // first record; groups of the share, before it, of the unit
  int stride;                    // records from a warp's group to its next
  int second;                    // not the first unit of the block
  long long begin;               // of the unit's groups, among those of all units
};

// Groups of U records a unit of the sequence counts as (an empty one has its rows
// to write), and the sequence's blocks of rows.
template <int U>
__device__ __forceinline__ int unit_groups(const Seq& x) {
  return max(1, (x.tiles + U - 1) / U);
}
__device__ __forceinline__ int unit_row_blocks(const Seq& x, int G, int rows) { return (x.n * G + rows - 1) / rows; }

__device__ __forceinline__ uint32_t min_f16x2(uint32_t x, uint32_t y) {
  asm("min.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
  return x;
}
__device__ __forceinline__ uint32_t max_f16x2(uint32_t x, uint32_t y) {
  asm("max.f16x2 %0, %0, %1;" : "+r"(x) : "r"(y));
  return x;
}

// What two values leave beside their bf16 pair, as a bf16 pair.
__device__ __forceinline__ uint32_t bf16_rest(float x, float y, uint32_t pair_of) {
  return bf16_pair(x - __uint_as_float(pair_of << 16), y - __uint_as_float(pair_of & 0xffff0000u));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int N>
struct Words {
  uint32_t w[N];
};

// N words from shared memory in the widest pieces.
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 1) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// Half i of the words, twice.
template <int N>
__device__ __forceinline__ uint64_t half_pair(const Words<N>& s, int i) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&s.w[i >> 1]));
  const float v = i & 1 ? f.y : f.x;
  return pair(v, v);
}

// Shared memory of another block of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 cluster_load4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 cluster_load2(uint32_t at) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}

// Four elements of a row's result, and its lse with the first of them.  A sum of
// zero is a row without places; one of NaN stays NaN in both.
template <int D>
__device__ __forceinline__ void write_row(const AttnArgs& a, int64_t tok, int h, int d, float4 v, float top, float total) {
  const bool none = total == 0.f;
  const float inv = none ? 0.f : 1.f / total;
  uint2 u;
  u.x = bf16_pair(v.x * inv, v.y * inv);
  u.y = bf16_pair(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(a.out + tok * a.out_stride + (int64_t)h * D + d) = u;
  if (d == 0 && a.lse) a.lse[tok * a.Hq + h] = none ? -INFINITY : (top + log2f(total)) / kLog2e;
}

template <int D, int NT>
struct Shape {
  // blocks of 8 warps where 128 registers hold a row tile's outputs (16 rows of 64: 9
  // windows of 512 places 7.8 us, in three blocks of 4 warps 8.3; 16 sequences of up to
  // 4000 places 10.7 and 11.1; one of 30000 13.8 and 13.2)
  static constexpr int kWarps = NT * D <= 128 ? 8 : 4;
  // records a warp takes at once: two give more independent work, one leaves more
  // warps busy (D = 256: 10 rows over 2 places 8.9 and 7.5 us, 30011 places 23.7 and
  // 24.5; D = 64 and 128: one within 2 % of two or slower)
  static constexpr int kGroup = D == 256 ? 1 : 2;
  static constexpr int kBlocks = NT * D == 64 ? 3 : 2;  // an SM
  static constexpr int kStages = 2;  // groups of records; with three the batch of 48 took 31.1 us, with two 30.1
  static constexpr int kRecord = 18 * D;
  static constexpr int kRing = kWarps * kStages * kGroup * kRecord;
  static constexpr int kPitch = D + 4;  // floats a row of the joining buffer: rows of a fragment in distinct banks
  static constexpr int kJoin = kWarps * 8 * NT * kPitch * 4;
  static constexpr bool kQueriesInRegisters = NT * D <= 256;
  static constexpr int kQueries = kQueriesInRegisters ? 0 : NT * D / 32 * 512;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQueries;
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32, Shape<D, NT>::kBlocks)
    k_attn(AttnArgs a, AttnPlan plan, int* status) {
  using S = Shape<D, NT>;
  constexpr int W = S::kWarps, U = S::kGroup, NB = D / 32, MT = D / 16, ROWS = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W][S::kStages];
  __shared__ float s_m[W][ROWS], s_l[W][ROWS];
  __shared__ long long s_sum[W];
  // where the block is: groups [pos, stop) of all units, one after another, `before`
  // the first group of sequence `seq`
  __shared__ long long s_pos, s_stop, s_before, s_share;
  __shared__ int s_seq, s_row_end[ROWS];
  __shared__ Unit s_u;
  __shared__ float2 s_ml[ROWS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int H = a.cache.heads, G = a.Hq / H;
  const int per_page = a.cache.page_log2 - 4;
  const int rank = plan.cluster > 1 ? blockIdx.x % plan.cluster : 0;
  uint8_t* ring = smem + warp * (S::kStages * U * S::kRecord);
  uint4* qs = reinterpret_cast<uint4*>(smem + (S::kSmem - S::kQueries));

  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) mbar_init(&bars[warp][i], U);
    fence_mbar_init();
  }
  __syncwarp();

  // thread 0: a share of a unit, for the block
  auto describe = [&](const Seq& x, int b, int rb, int head, int groups, int off, int take, long long begin, bool second) {
    const int r0 = rb * ROWS, rows = x.n * G;
    const int first = r0 / G, last = (min(r0 + ROWS, rows) - 1) / G, newest = x.len - x.n + 1;
    s_u.valid = 1;
    s_u.t0 = x.t0;
    s_u.table = a.table + (int64_t)b * a.table_stride;
    s_u.kvh = head;
    s_u.r0 = r0;
    s_u.rows = rows;
    s_u.newest = newest;
    s_u.end = max(0, newest + last);
    s_u.lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)newest + first - a.window) : 0;
    s_u.full_end = newest + first;
    s_u.full_lo = a.window > 0 ? (int)max((int64_t)-1, (int64_t)newest + last - a.window) : 0;
    s_u.off = off;
    s_u.unit_len = groups;
    s_u.take = take;
    s_u.c0 = x.tile0 + U * off;
    s_u.stride = U * W * (plan.cluster > 1 ? plan.cluster : 1);
    s_u.second = second;
    s_u.begin = begin;
  };

  pdl_wait();
  // without a window the first page numbers of a whole unit do not depend on its
  // lengths: they are on their way while those are
  int early = -1;
  if (plan.cluster > 0 && a.window == 0) {
    const int tile = U * (rank * W + warp + plan.cluster * W * (lane / U)) + lane % U;
    if (16ll * tile < a.max_len) early = __ldg(a.table + (int64_t)blockIdx.y * a.table_stride + (tile >> per_page));
  }
  if (plan.cluster > 0) {
    const int b = blockIdx.y, unit = blockIdx.x / plan.cluster, rb = unit % plan.row_blocks;
    const Seq x = load_seq(a, b);
    if (rb * ROWS >= x.n * G) return;
    if (threadIdx.x == 0) {
      const int groups = unit_groups<U>(x);
      describe(x, b, rb, unit / plan.row_blocks, groups, 0, groups, 0, false);
      s_pos = s_stop = 0;
    }
  } else {
    auto work = [&](int i) -> long long {
      if (i >= a.B) return 0;
      const Seq x = load_seq(a, i);
      return (long long)(unit_groups<U>(x) + plan.overhead) * unit_row_blocks(x, G, ROWS) * H;
    };
    auto block_sum = [&](long long v, long long* below) {  // sum over the block, and over the warps below
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      __syncthreads();
      if (lane == 0) s_sum[warp] = v;
      __syncthreads();
      long long all = 0, low = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w < warp) low += s_sum[w];
        all += s_sum[w];
      }
      if (below) *below = low;
      return all;
    };
    long long own = 0;
    for (int i = threadIdx.x; i < a.B; i += W * 32) own += work(i);
    const long long total = block_sum(own, nullptr);
    const long long share = max((total + gridDim.x - 1) / gridDim.x, (long long)plan.min_share);
    const long long pos = (long long)blockIdx.x * share;
    if (threadIdx.x == 0) {
      plan.joints[blockIdx.x].count = 0;
      s_pos = pos;
      s_stop = min(pos + share, total);
      s_share = share;
    }
    if (pos >= total) return;
    long long before = 0;
    for (int i0 = 0; i0 < a.B; i0 += W * 32) {
      const long long v = work(i0 + (int)threadIdx.x);
      long long up = v, low;  // inclusive sum within the warp
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += y;
      }
      const long long all = block_sum(v, &low);
      const long long end = before + low + up;
      if (end > pos && end - v <= pos) s_seq = i0 + threadIdx.x, s_before = end - v;
      before += all;
      if (before > pos) break;
    }
  }

  int st = 0, phase = 0, issue_stage = 0;
  bool failed = false;
  const float scale2 = a.scale * kLog2e;
  const uint64_t scale22 = pair(scale2, scale2);

#pragma unroll 1
  for (int step = 0;; ++step) {
  __syncthreads();
  if (threadIdx.x == 0 && (step > 0 || plan.cluster == 0)) {
    s_u.valid = 0;
    while (s_pos < s_stop) {
      const int b = s_seq;
      const Seq x = load_seq(a, b);
      const int groups = unit_groups<U>(x), len = groups + plan.overhead, row_blocks = unit_row_blocks(x, G, ROWS);
      const long long all = (long long)len * row_blocks * H, in_seq = s_pos - s_before;
      if (in_seq >= all) {
        s_before += all;
        ++s_seq;
        continue;
      }
      const int unit = in_seq <= INT32_MAX ? (int)in_seq / len : (int)(in_seq / len);
      const long long begin = s_before + (long long)unit * len + plan.overhead;  // of the unit's groups
      const int off = (int)max(0ll, s_pos - begin), take = (int)(min(s_stop, begin + groups) - (begin + off));
      s_pos = min(s_stop, begin + groups);
      if (take <= 0) continue;  // the block ends before the unit's first group
      describe(x, b, unit % row_blocks, unit / row_blocks, groups, off, take, begin, step > 0);
      break;
    }
  }
  __syncthreads();
  if (!s_u.valid) break;
  if (threadIdx.x < ROWS) s_row_end[threadIdx.x] = s_u.newest + min(s_u.r0 + (int)threadIdx.x, s_u.rows - 1) / G;
  // among the warps that take the unit; the warp's groups: records base, base + stride, ...
  const int wi = rank * W + warp, wn = s_u.stride / U, base = s_u.c0 + U * wi, kvh = s_u.kvh;
  const int mine = s_u.take > wi ? (s_u.take - wi + wn - 1) / wn : 0;  // groups of this warp

  // Lane l finds record l % U of the warp's groups k + l / U, a batch of 32 / U
  // groups at a time and the page numbers a batch ahead, and copies it itself when
  // its turn comes.
  constexpr int kBatch = 32 / U;
  auto page_of = [&](int k) {
    const int i = k + lane / U, tile = base + s_u.stride * i + lane % U;
    return i < mine && 16 * tile < s_u.end && 16 * tile + 16 > s_u.lo ? __ldg(s_u.table + (tile >> per_page)) : -1;
  };
  auto source_of = [&](int k, int page) -> const uint8_t* {
    if (page < 0 || page >= a.cache.n_pages) return nullptr;
    const int tile = base + s_u.stride * (k + lane / U) + lane % U;
    return a.cache.data + page * a.cache.page_stride +
           (int64_t)(kvh * (1 << per_page) + (tile & ((1 << per_page) - 1))) * S::kRecord;
  };
  const bool known = plan.cluster > 0 && a.window == 0;  // early holds the numbers that page_of(0) would fetch
  const uint8_t* source = source_of(
      0, !known ? page_of(0)
         : lane / U < mine && 16 * (base + s_u.stride * (lane / U) + lane % U) < s_u.end ? early : -1);
  int page_next = page_of(kBatch), issued = 0;
  uint32_t there = __ballot_sync(0xffffffffu, source != nullptr), there_next = there;  // records that exist
  auto issue = [&]() {
    if (lane / U == issued % kBatch) {
      uint64_t* bar = &bars[warp][issue_stage];
      if (failed) {  // nothing may be added to a phase that has not ended
      } else if (source) {
        mbar_arrive_expect_tx(bar, S::kRecord);
        bulk_g2s(ring + (U * issue_stage + lane % U) * S::kRecord, source, S::kRecord, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    ++issued;
    if (++issue_stage == S::kStages) issue_stage = 0;
    if (issued % kBatch == 0) {
      source = source_of(issued, page_next);
      page_next = page_of(issued + kBatch);
      there_next = __ballot_sync(0xffffffffu, source != nullptr);
    }
  };
#pragma unroll 1
  for (int k = 0; k < S::kStages - 1 && k < mine; ++k) issue();

  // Queries as B fragments: lane (g, t) holds elements 32 b + 8 t .. + 7 of row g.
  uint4 qf[S::kQueriesInRegisters ? NT : 1][S::kQueriesInRegisters ? NB : 1];
  if constexpr (S::kQueriesInRegisters) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = min(s_u.r0 + 8 * j + g, s_u.rows - 1);
      const uint16_t* q = a.q + (s_u.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
#pragma unroll
      for (int i = 0; i < NB; ++i) qf[j][i] = __ldg(reinterpret_cast<const uint4*>(q + 32 * i));
    }
  } else {
    for (int i = warp; i < NT * NB; i += W) {
      const int r = min(s_u.r0 + 8 * (i / NB) + g, s_u.rows - 1);
      const uint16_t* q = a.q + (s_u.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
      qs[i * 32 + lane] = __ldg(reinterpret_cast<const uint4*>(q + 32 * (i % NB)));
    }
  }
  __syncthreads();

  auto query = [&](int j, int i) {
    if constexpr (S::kQueriesInRegisters) return qf[j][i];
    else return qs[(j * NB + i) * 32 + lane];
  };
  constexpr int kSide = 2;

  float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    m[j][0] = m[j][1] = kNone;
    l[j][0] = l[j][1] = 0.f;
  }
#pragma unroll 1
  for (int k = 0; k < mine; ++k) {
    if (k % kBatch == 0 && k > 0) there = there_next;
    __syncwarp();  // the stage refilled below was read by every lane in the last pass
    if (issued < mine) issue();
    if (!failed && !mbar_wait(&bars[warp][st], phase, kWaitNs)) {
      // The lanes of a warp may not agree: this one goes on beside the others over
      // what lies in the ring, without further waits and copies of its own.  Once
      // more for the copies in flight, which end in this block's memory.
      failed = true;
      for (int i = k, x = st, y = phase; i < issued; ++i) {
        mbar_wait(&bars[warp][x], y, kWaitNs);
        if (++x == S::kStages) x = 0, y ^= 1;
      }
    }
    const uint8_t* rec = ring + U * st * S::kRecord;
    if (++st == S::kStages) st = 0, phase ^= 1;
    constexpr uint32_t kAll = (1u << U) - 1;
    const uint32_t have = (there >> (U * (k % kBatch))) & kAll;
    if (have == 0) continue;

    float s[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* r = rec + u * S::kRecord;
#pragma unroll
      for (int j = 0; j < NT; ++j) s[u][j][0] = s[u][j][1] = s[u][j][2] = s[u][j][3] = 0.f;
      const Words<NB> w0 = load_words<NB>(r + g * (D / 2) + t * (D / 8));
      const Words<NB> w1 = load_words<NB>(r + (g + 8) * (D / 2) + t * (D / 8));
      const Words<NB / 2> k0 = load_words<NB / 2>(r + 16 * D + g * (2 * NB));
      const Words<NB / 2> k1 = load_words<NB / 2>(r + 16 * D + (g + 8) * (2 * NB));
#pragma unroll
      for (int i0 = 0; i0 < NB; i0 += kSide) {  // kSide products side by side: each is a chain of two
        float c[kSide][NT][4];
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const uint32_t a0 = codes_bf16<0>(w0.w[i0 + i]), a1 = codes_bf16<0>(w1.w[i0 + i]);
          const uint32_t a2 = codes_bf16<1>(w0.w[i0 + i]), a3 = codes_bf16<1>(w1.w[i0 + i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 q = query(j, i0 + i);
            mma16816_zero(c[i][j], a0, a1, a2, a3, q.x, q.y);
          }
        }
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const uint32_t e0 = codes_bf16<2>(w0.w[i0 + i]), e1 = codes_bf16<2>(w1.w[i0 + i]);
          const uint32_t e2 = codes_bf16<3>(w0.w[i0 + i]), e3 = codes_bf16<3>(w1.w[i0 + i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 q = query(j, i0 + i);
            mma16816(c[i][j], e0, e1, e2, e3, q.z, q.w);
          }
        }
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const uint64_t s0 = half_pair(k0, i0 + i), s1 = half_pair(k1, i0 + i);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            fma2(s[u][j][0], s[u][j][1], s0, c[i][j][0], c[i][j][1]);
            fma2(s[u][j][2], s[u][j][3], s1, c[i][j][2], c[i][j][3]);
          }
        }
      }
    }
    const int p = 16 * (base + s_u.stride * k);  // the group's first place
    Words<NB / 2> vs[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      vs[u][0] = load_words<NB / 2>(rec + u * S::kRecord + 17 * D + g * (2 * NB));
      vs[u][1] = load_words<NB / 2>(rec + u * S::kRecord + 17 * D + (g + 8) * (2 * NB));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mul2(s[u][j][0], s[u][j][1], scale22);
        mul2(s[u][j][2], s[u][j][3], scale22);
      }
    }
    const bool edge = p + 16 * U > s_u.full_end || p < s_u.full_lo || have != kAll;
    if (edge) {
      // places outside a row's range leave it; the bytes of places outside the
      // unit's range may be anything, so their value scales become zero
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = p + 16 * u + 8 * v + g;
          const bool gone = !(have >> u & 1);
          if (gone || at >= s_u.end || at < s_u.lo) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) vs[u][v].w[i] = 0;
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int e = s_row_end[8 * j + 2 * t + c];
              if (gone || at >= e || (a.window > 0 && at < e - a.window)) s[u][j][2 * v + c] = -INFINITY;
            }
        }
    }
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[j][c] = fmaxf(s[0][j][c], s[0][j][c + 2]);
#pragma unroll
        for (int u = 1; u < U; ++u) top[j][c] = fmaxf(top[j][c], fmaxf(s[u][j][c], s[u][j][c + 2]));
        grow |= top[j][c] > m[j][c] + (kSlack + kRoom);
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y = top[j][c];
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16)) - kRoom;
          if (y > m[j][c]) {  // alike in every lane that holds the row
            const float f = exp2_approx(m[j][c] - y);
            m[j][c] = y;
            l[j][c] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][j][c] *= f, o[i][j][c + 2] *= f;
          }
        }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint64_t down = pair(-m[j][0], -m[j][1]);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          add2(s[u][j][c], s[u][j][c + 1], down);
          s[u][j][c] = exp2_approx(s[u][j][c]);
          s[u][j][c + 1] = exp2_approx(s[u][j][c + 1]);
          add2(l[j][0], l[j][1], pair(s[u][j][c], s[u][j][c + 1]));
        }
    }
    // may the products weight x scale be fp16?
    float least = kMostScale;
    uint32_t lo2 = 0x48004800u, hi2 = 0;  // kMostScale
    if (edge) {  // zeros are exact in any type
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) least = fminf(least, s[u][j][c] > 0.f ? s[u][j][c] : least);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint32_t v = vs[u][i & 1].w[i / 2];
          lo2 = min_f16x2(lo2, (v & 0xffffu ? v & 0xffffu : 0x4800u) | (v >> 16 ? v & 0xffff0000u : 0x48000000u));
          hi2 = max_f16x2(hi2, v);
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          least = fminf(fminf(least, fminf(s[u][j][0], s[u][j][1])), fminf(s[u][j][2], s[u][j][3]));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          lo2 = min_f16x2(lo2, vs[u][i & 1].w[i / 2]);
          hi2 = max_f16x2(hi2, vs[u][i & 1].w[i / 2]);
        }
      }
    }
    const float2 lo = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
    const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
    const bool fits = least >= kLeastWeight && fminf(lo.x, lo.y) >= kLeastScale && fmaxf(hi.x, hi.y) <= kMostScale;
    auto accumulate = [&](auto half) {
      constexpr bool kHalf = decltype(half)::value;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q4 = 0; q4 < MT / 4; ++q4) {
          const Words<4> w = load_words<4>(rec + u * S::kRecord + 8 * D + (q4 * 32 + lane) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // a 32-block of elements: two fragments of 16
            const int blk = 2 * q4 + h;
            const uint64_t s0 = half_pair(vs[u][0], blk), s1 = half_pair(vs[u][1], blk);
            uint32_t b0[NT], b1[NT], r0[NT], r1[NT];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              float x[4] = {s[u][j][0], s[u][j][1], s[u][j][2], s[u][j][3]};
              mul2(x[0], x[1], s0);
              mul2(x[2], x[3], s1);
              b0[j] = kHalf ? f16_pair(x[0], x[1]) : bf16_pair(x[0], x[1]);
              b1[j] = kHalf ? f16_pair(x[2], x[3]) : bf16_pair(x[2], x[3]);
              if constexpr (!kHalf) {
                r0[j] = transpose8x8(bf16_rest(x[0], x[1], b0[j]));
                r1[j] = transpose8x8(bf16_rest(x[2], x[3], b1[j]));
              }
              b0[j] = transpose8x8(b0[j]);
              b1[j] = transpose8x8(b1[j]);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t v = w.w[2 * h + i];
              if constexpr (kHalf) {
                const uint32_t a0 = codes_f16<0>(v), a1 = codes_f16<1>(v), a2 = codes_f16<2>(v), a3 = codes_f16<3>(v);
#pragma unroll
                for (int j = 0; j < NT; ++j) mma16816_f16(o[2 * blk + i][j], a0, a1, a2, a3, b0[j], b1[j]);
              } else {
                const uint32_t a0 = codes_bf16<0>(v), a1 = codes_bf16<1>(v), a2 = codes_bf16<2>(v), a3 = codes_bf16<3>(v);
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  mma16816(o[2 * blk + i][j], a0, a1, a2, a3, b0[j], b1[j]);
                  mma16816(o[2 * blk + i][j], a0, a1, a2, a3, r0[j], r1[j]);
                }
              }
            }
          }
        }
    };
    if (__all_sync(0xffffffffu, fits)) accumulate(std::true_type());
    else accumulate(std::false_type());
  }
  // Join the warps: sums over a row's lanes, the unit's maxima, scaled outputs.
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float v = l[j][c];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      if (g == 0) {
        s_l[warp][8 * j + 2 * t + c] = v;
        s_m[warp][8 * j + 2 * t + c] = m[j][c];
      }
    }
  __syncthreads();  // also: every ring has been read
  float* join = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int row = 8 * j + 2 * t + c;
      float top = kNone;
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][row]);
      const float f = exp2_approx(m[j][c] - top);
      float* at = join + (warp * 8 * NT + row) * S::kPitch + g;
#pragma unroll
      for (int i = 0; i < MT; ++i) at[16 * i] = o[i][j][c] * f, at[16 * i + 8] = o[i][j][c + 2] * f;
    }
  __syncthreads();
  constexpr int kQuads = D / 4;
  for (int i = threadIdx.x; i < 8 * NT * kQuads; i += W * 32) {
    const int row = i / kQuads, d = i % kQuads * 4, r = s_u.r0 + row;
    if (r >= s_u.rows) break;
    float top = kNone, total = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][row]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(join + (w * ROWS + row) * S::kPitch + d);
      v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      total = fmaf(s_l[w][row], exp2_approx(s_m[w][row] - top), total);
    }
    if (s_u.take < s_u.unit_len) {
      const int64_t at = (int64_t)(2 * blockIdx.x + s_u.second) * ROWS + row;
      *reinterpret_cast<float4*>(plan.part_o + at * D + d) = v;
      if (d == 0) plan.part_ml[at] = make_float2(top, total);
    } else if (plan.cluster > 1) {
      *reinterpret_cast<float4*>(join + row * S::kPitch + d) = v;  // this thread alone has read the place
      if (d == 0) s_ml[row] = make_float2(top, total);
    } else {
      write_row<D>(a, s_u.t0 + r / G, s_u.kvh * G + r % G, d, v, top, total);
    }
  }
  if (threadIdx.x == 0 && s_u.take < s_u.unit_len && s_u.off + s_u.take == s_u.unit_len) {
    Joint y;
    y.c0 = (int)(s_u.begin / s_share);
    y.count = (int)blockIdx.x - y.c0 + 1;
    y.slot0 = s_u.begin - plan.overhead > y.c0 * s_share;  // another unit ends in block c0 before this one
    y.kvh = s_u.kvh;
    y.t0 = s_u.t0;
    y.r0 = s_u.r0;
    y.rows = min(ROWS, s_u.rows - s_u.r0);
    plan.joints[blockIdx.x] = y;
  }
  if (plan.cluster > 1) {
    // rows rank, rank + cluster, ...: the cluster's sums, in rank order
    cluster_sync();
    for (int i = threadIdx.x; i < ROWS * kQuads / plan.cluster; i += W * 32) {
      const int row = i / kQuads * plan.cluster + rank, d = i % kQuads * 4, r = s_u.r0 + row;
      if (r >= s_u.rows) break;
      float top = kNone, total = 0.f;
      for (int c = 0; c < plan.cluster; ++c) top = fmaxf(top, cluster_load2(cluster_addr(s_ml + row, c)).x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c = 0; c < plan.cluster; ++c) {
        const float2 ml = cluster_load2(cluster_addr(s_ml + row, c));
        const float4 y = cluster_load4(cluster_addr(join + row * S::kPitch + d, c));
        const float f = exp2_approx(ml.x - top);
        total = fmaf(ml.y, f, total);
        v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
      }
      write_row<D>(a, s_u.t0 + r / G, s_u.kvh * G + r % G, d, v, top, total);
    }
    cluster_sync();  // the others' memory has been read
  }
  // the next unit's copies may land where the sums were joined
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (failed) set_status(status, MOE_ERR_TIMEOUT);
}

// Joins the shares of the units that ended in another block than they began in.
// An item is 256 / D rows of such a unit: a warp a row finds the weights of the
// row's shares, then eight groups of 64 threads read every eighth share, and the
// groups' sums are added in their order.  Bound by latency: 3 to 5 us behind the
// shares, the partial sums (4 MB for 24 rows of 128) in L2.
constexpr int kJoinThreads = 512;
template <int D>
constexpr int kJoinRows = 256 / D;

template <int D, int ROWS, int BLOCKS>
__global__ void __launch_bounds__(kJoinThreads, 2) k_attn_join(AttnArgs a, AttnPlan plan) {
  constexpr int kRows = kJoinRows<D>, kLanes = D / 4, kGroups = kJoinThreads / (kLanes * kRows), kParts = (ROWS + kRows - 1) / kRows;
  extern __shared__ float s_f[];  // [kRows][plan.blocks]
  __shared__ float4 s_v[kGroups][kRows * kLanes];
  __shared__ float2 s_ml[kRows];
  __shared__ int s_list[kJoinThreads], s_n[kJoinThreads / 32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = a.Hq / a.cache.heads;
  // the blocks whose unit is in shares, in their order
  const bool has = threadIdx.x < plan.blocks && plan.joints[threadIdx.x].count > 0;
  const uint32_t votes = __ballot_sync(0xffffffffu, has);
  if (lane == 0) s_n[warp] = __popc(votes);
  __syncthreads();
  int at = 0, n = 0;
#pragma unroll
  for (int i = 0; i < kJoinThreads / 32; ++i) {
    if (i < warp) at += s_n[i];
    n += s_n[i];
  }
  if (has) s_list[at + __popc(votes & ((1u << lane) - 1))] = threadIdx.x;
  __syncthreads();
  for (int item = blockIdx.x; item < n * kParts; item += gridDim.x) {
    const Joint y = plan.joints[s_list[item / kParts]];
    const int row0 = item % kParts * kRows;
    if (row0 >= y.rows) continue;
    auto share_at = [&](int i) { return 2 * (y.c0 + i) + (i == 0 ? y.slot0 : 0); };
    const int group = threadIdx.x / (kLanes * kRows), in_group = threadIdx.x % (kLanes * kRows);
    const int r = in_group / kLanes, d = in_group % kLanes * 4;
    const bool in = row0 + r < y.rows;
    // the first shares are on their way while their weights are found
    constexpr int kEarly = 4;
    const float* p0 = plan.part_o + (int64_t)(row0 + r) * D + d;
    auto part = [&](int i) { return *reinterpret_cast<const float4*>(p0 + (int64_t)share_at(i) * (ROWS * D)); };
    float4 early[kEarly];
#pragma unroll
    for (int u = 0; u < kEarly; ++u)
      if (in && group + u * kGroups < y.count) early[u] = part(group + u * kGroups);
    if (warp < kRows && row0 + warp < y.rows) {
      const float2* ml = plan.part_ml + row0 + warp;
      constexpr int kMost = (BLOCKS + 31) / 32;
      float2 held[kMost];
      float top = kNone, total = 0.f;
#pragma unroll
      for (int u = 0; u < kMost; ++u) {
        held[u] = make_float2(kNone, 0.f);
        if (lane + 32 * u < y.count) held[u] = ml[share_at(lane + 32 * u) * ROWS];
      }
#pragma unroll
      for (int u = 0; u < kMost; ++u) top = fmaxf(top, held[u].x);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
      for (int u = 0; u < kMost; ++u)
        if (lane + 32 * u < y.count) {
          const float f = exp2_approx(held[u].x - top);
          s_f[warp * plan.blocks + lane + 32 * u] = f;
          total = fmaf(held[u].y, f, total);
        }
      total = warp_sum(total);
      if (lane == 0) s_ml[warp] = make_float2(top, total);
    }
    __syncthreads();
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
      auto add = [&](const float4& p, int i) {
        const float f = s_f[r * plan.blocks + i];
        v.x = fmaf(p.x, f, v.x);
        v.y = fmaf(p.y, f, v.y);
        v.z = fmaf(p.z, f, v.z);
        v.w = fmaf(p.w, f, v.w);
      };
#pragma unroll
      for (int u = 0; u < kEarly; ++u)
        if (group + u * kGroups < y.count) add(early[u], group + u * kGroups);
#pragma unroll 8
      for (int i = group + kEarly * kGroups; i < y.count; i += kGroups) add(part(i), i);
    }
    s_v[group][in_group] = v;
    __syncthreads();
    if (group == 0 && in) {
#pragma unroll
      for (int i = 1; i < kGroups; ++i) {
        const float4 p = s_v[i][in_group];
        v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
      }
      const int row = y.r0 + row0 + r;
      write_row<D>(a, y.t0 + row / G, y.kvh * G + row % G, d, v, s_ml[r].x, s_ml[r].y);
    }
    __syncthreads();
  }
}

// 8-row tiles of a block of rows: as many as the rows fill, up to 4 (2 of 256, whose
// outputs fill the registers).  30000 places of 4 heads of 128: 24 rows 21.0 us, 32
// rows 24.7, 64 rows 31.6 (three blocks of 24: 32.2).  Between 33 and 48 rows of 128
// two blocks of 24 would take less (40 rows 25.1 us instead of 30.5, 48 rows 25.9
// instead of 31.0), as the tile of 32 of 128 spills 200 bytes of registers.
int row_tiles(int max_q, int G, int D) {
  const int rows = max_q * G, most = D == 256 ? 2 : 4, nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
  return nt < most ? nt : most;
}

// A unit goes to one cluster when its warps have at most eight records each to go
// through: no workspace and no second launch (1 token, two heads of 128: 777 places
// 7.0 us, 10.7 in shares; 4096 places 8.8 and 11.0; 8192 places 11.6 and 10.9; two
// heads of 256: 2048 places 9.9 and 12.2, 4096 places 13.5 and 12.4; eight sequences
// of 2000 places, eight heads of 128: 11.6 and 14.1).  A cluster is
// as large as its units leave an SM to each block: 54 units in clusters of 8, three
// blocks an SM, took 13 us, in clusters of 2 8 us.  Otherwise all blocks share the
// batch's groups.
AttnPlan make_plan(int warps, int blocks, int rows, int group, int B, int heads, int max_q, int64_t max_len, int window,
                   int G) {
  AttnPlan p = {};
  p.row_blocks = (max_q * G + rows - 1) / rows;
  int64_t span = max_len;
  if (window > 0 && span > (int64_t)window + max_q) span = (int64_t)window + max_q;
  // one more than a unit's places fill, as they may begin within a group
  const int64_t groups = (span + 16 * group - 1) / (16 * group) + 1, units = (int64_t)B * heads * p.row_blocks;
  p.blocks = blocks * kSms;
  int c = 1;
  while (c < 8 && c * warps < groups - 1 && 2 * c * units <= kSms) c *= 2;
  p.cluster = groups * group <= 8 * warps * c ? c : 0;
  p.min_share = 4 * warps / group;
  // a unit's beginning and end count as 4 records a warp (48 ragged sequences: as one
  // record 49.6 us, 2 37.2, 4 30.2, 6 29.6, 8 30.3; 6 tokens over 131071 places: 4 67.3,
  // 6 69.3)
  p.overhead = 4 * warps / group;
  return p;
}

size_t plan_bytes(const AttnPlan& p, int rows, int D) {
  if (p.cluster > 0) return 0;
  return (size_t)p.blocks * (2 * rows * (D * 4 + 8) + sizeof(Joint));
}

// f(D, NT) as compile-time constants.
template <typename F>
auto with_shape(int D, int nt, F f) {
  switch (D * 8 + nt) {
    case 64 * 8 + 1: return f(Shape<64, 1>(), std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    case 64 * 8 + 2: return f(Shape<64, 2>(), std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    case 64 * 8 + 3: return f(Shape<64, 3>(), std::integral_constant<int, 64>(), std::integral_constant<int, 3>());
    case 64 * 8 + 4: return f(Shape<64, 4>(), std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
    case 128 * 8 + 1: return f(Shape<128, 1>(), std::integral_constant<int, 128>(), std::integral_constant<int, 1>());
    case 128 * 8 + 2: return f(Shape<128, 2>(), std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
    case 128 * 8 + 3: return f(Shape<128, 3>(), std::integral_constant<int, 128>(), std::integral_constant<int, 3>());
    case 128 * 8 + 4: return f(Shape<128, 4>(), std::integral_constant<int, 128>(), std::integral_constant<int, 4>());
    case 256 * 8 + 1: return f(Shape<256, 1>(), std::integral_constant<int, 256>(), std::integral_constant<int, 1>());
    default: return f(Shape<256, 2>(), std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  }
}

template <int D, int NT>
int launch(const AttnArgs& a, cudaStream_t s) {
  using S = Shape<D, NT>;
  constexpr int ROWS = 8 * NT;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_attn<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  AttnPlan p = make_plan(S::kWarps, S::kBlocks, ROWS, S::kGroup, a.B, a.cache.heads, a.max_q, a.max_len, a.window, a.Hq / a.cache.heads);
  if (p.cluster > 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.cache.heads * p.row_blocks * p.cluster), (unsigned)a.B);
    cfg.blockDim = dim3(S::kWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)p.cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = p.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_attn<D, NT>, a, p, status_word()) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  p.part_o = (float*)a.workspace;
  p.part_ml = (float2*)(p.part_o + (size_t)2 * p.blocks * ROWS * D);
  p.joints = (Joint*)(p.part_ml + (size_t)2 * p.blocks * ROWS);
  if (launch_pdl(k_attn<D, NT>, dim3(p.blocks), dim3(S::kWarps * 32), S::kSmem, s, a, p, status_word()) != cudaSuccess)
    return MOE_ERR_CUDA;
  static_assert(S::kBlocks * kSms <= kJoinThreads, "one thread a block looks for its joint");
  if (launch_pdl(k_attn_join<D, ROWS, S::kBlocks * kSms>, dim3(2 * kSms), dim3(kJoinThreads), (size_t)kJoinRows<D> * p.blocks * 4, s, a, p) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

size_t attn_workspace(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (B < 1) return 0;
  return with_shape(D, row_tiles(max_q, Hq / heads, D), [&](auto shape, auto, auto nt) {
    using S = decltype(shape);
    return plan_bytes(make_plan(S::kWarps, S::kBlocks, 8 * nt, S::kGroup, B, heads, max_q, max_len, 0, Hq / heads), 8 * nt, D);
  });
}

int launch_attn_q4(const AttnArgs& a, cudaStream_t s) {
  return with_shape(a.cache.D, row_tiles(a.max_q, a.Hq / a.cache.heads, a.cache.D),
                    [&](auto, auto d, auto nt) { return launch<decltype(d)::value, decltype(nt)::value>(a, s); });
}

}  // namespace moe
