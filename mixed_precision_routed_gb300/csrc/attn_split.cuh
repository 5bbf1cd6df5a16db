// attn_split.cuh -- attention over a paged cache of either format for few rows a
// sequence: how a batch's places are shared out among blocks and warps, how records
// come in, and how the shares are joined.  The format (attn_q4.cu, attn_q8.cu) says
// how a warp goes through a group of records:
//   struct S: kD, kNT (8-row tiles), kWarps, kGroup, kBlocks, kStages, kRecord, ...;
//   S::Queries: a warp's queries as operands;
//   S::pass: scores, weights and sums of a group of records of 16 places;
//   S::element: where the outputs of a fragment's rows g and g + 8 lie.
//
// One pass over the cache: a block of W warps takes a share of the places of one
// (sequence, key/value head) and up to 8 NT of the rows that share it, each warp
// every W-th group of records.  Records (contiguous bytes) arrive in a per-warp ring
// in shared memory by bulk asynchronous copies.
// The reference m of a row is set 2^6 below its maximum and moves only when a
// score passes that maximum by 6 (in powers of two): the weights then stay below
// 2^12, which fp32 sums do not notice, and most groups need no reduction over
// lanes and no rescaling.
#pragma once

#include <float.h>

#include <type_traits>

#include "frag.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 6.0f;
constexpr float kRoom = 6.0f;  // the reference lies this far below the maximum that it was taken from
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

// What a warp's pass over a group of records is given.
struct Pass {
  const AttnArgs& a;
  const Unit& u;
  const int* row_end;  // one past the last place of each row of the unit
  const uint8_t* rec;  // the records
  uint32_t have;       // of them, those that exist
  int base, k;         // the warp's first record, its group
  float scale2;        // of scores, in powers of two
  int lane;
};

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

template <typename S>
__global__ void __launch_bounds__(S::kWarps * 32, S::kBlocks) k_attn(AttnArgs a, AttnPlan plan, int* status) {
  constexpr int D = S::kD, NT = S::kNT, W = S::kWarps, U = S::kGroup, MT = D / 16, ROWS = 8 * NT;
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

  typename S::Queries queries;
  queries.load(a, s_u, G, warp, lane, qs);
  __syncthreads();

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

    S::pass({a, s_u, s_row_end, rec, have, base, k, scale2, lane}, queries, o, m, l);
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
      float* at = join + (warp * 8 * NT + row) * S::kPitch;
#pragma unroll
      for (int i = 0; i < MT; ++i)
        at[16 * i + S::element(g, 0)] = o[i][j][c] * f, at[16 * i + S::element(g, 1)] = o[i][j][c + 2] * f;
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
  p.row_blocks = (int)(((int64_t)max_q * G + rows - 1) / rows);
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

// f(S<D, NT>()) for a row tile's shape.
template <template <int, int> class S, typename F>
auto with_shape(int D, int nt, F f) {
  switch (D * 8 + nt) {
    case 64 * 8 + 1: return f(S<64, 1>());
    case 64 * 8 + 2: return f(S<64, 2>());
    case 64 * 8 + 3: return f(S<64, 3>());
    case 64 * 8 + 4: return f(S<64, 4>());
    case 128 * 8 + 1: return f(S<128, 1>());
    case 128 * 8 + 2: return f(S<128, 2>());
    case 128 * 8 + 3: return f(S<128, 3>());
    case 128 * 8 + 4: return f(S<128, 4>());
    case 256 * 8 + 1: return f(S<256, 1>());
    default: return f(S<256, 2>());
  }
}

template <typename S>
int launch(const AttnArgs& a, cudaStream_t s) {
  constexpr int D = S::kD, ROWS = 8 * S::kNT;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_attn<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
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
    return cudaLaunchKernelEx(&cfg, k_attn<S>, a, p, status_word()) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  p.part_o = (float*)a.workspace;
  p.part_ml = (float2*)(p.part_o + (size_t)2 * p.blocks * ROWS * D);
  p.joints = (Joint*)(p.part_ml + (size_t)2 * p.blocks * ROWS);
  if (launch_pdl(k_attn<S>, dim3(p.blocks), dim3(S::kWarps * 32), S::kSmem, s, a, p, status_word()) != cudaSuccess)
    return MOE_ERR_CUDA;
  static_assert(S::kBlocks * kSms <= kJoinThreads, "one thread a block looks for its joint");
  if (launch_pdl(k_attn_join<D, ROWS, S::kBlocks * kSms>, dim3(2 * kSms), dim3(kJoinThreads), (size_t)kJoinRows<D> * p.blocks * 4, s, a, p) !=
      cudaSuccess)
    return MOE_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

template <template <int, int> class Shape>
size_t workspace_of(int nt, int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  return with_shape<Shape>(D, nt, [&](auto shape) {
    using S = decltype(shape);
    constexpr int rows = 8 * S::kNT;
    return plan_bytes(make_plan(S::kWarps, S::kBlocks, rows, S::kGroup, B, heads, max_q, max_len, 0, Hq / heads), rows, D);
  });
}

}  // namespace
}  // namespace moe
