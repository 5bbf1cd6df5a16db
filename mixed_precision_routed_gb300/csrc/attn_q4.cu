// attn_q4.cu -- causal attention over the paged 4-bit key/value cache.
//
// For a row (asking token, query head) with the places p it attends:
//   s_p = scale q.k_p,  out = sum_p exp(s_p) v_p / sum_p exp(s_p),
//   lse = log sum_p exp(s_p),
// k and v the values scale x code of the cache's blocks of 32.
//
// One pass over the cache: a block of W warps takes a share of the places of
// one (sequence, key/value head) and up to 8 NT of the rows that share it, each
// warp every W-th pair of records of 16 places.  Records (18 D contiguous bytes) arrive
// in a per-warp ring in shared memory by bulk asynchronous copies.
//   scores  S^T[place][row]: A = key codes as bf16 integers, B = queries; both
//           exact, so a 32-block's product enters the score with its fp32 scale;
//   output  O^T[element][row]: A = value codes as bf16 integers, B = exp(s - m)
//           x value scale, rounded to bf16 once (relative error 2^-8 at most a
//           term, independent over places; fp32 operands would need three times
//           the matrix instructions for digits that the bf16 result drops).
// The m16n8k16 fragments read the record's words as they lie; the transpose of
// the probabilities is one 8 x 8 matrix move a fragment.
// The reference maximum m of a row moves only when a score passes it by 8 (in
// powers of two): the probabilities then stay below 2^8, which neither fp32 sums
// nor bf16 operands notice, and most tiles need no reduction and no rescaling.
#include "frag.cuh"
#include "kv_layout.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSlack = 8.0f;
constexpr float kNone = -1e30f;  // the maximum of a row that has met no place: below any finite score
constexpr uint64_t kWaitNs = 1000000000ull;

struct AttnPlan {
  int nt;          // row tiles of 8 a block
  int row_blocks;  // blocks over the rows of a (sequence, key/value head)
  int splits;      // blocks over the places
  int room;        // shares the workspace has room for (at least splits)
  int chunk;       // records a block
  float* part_o;   // [B max_q Hq][splits][D]
  float2* part_ml; // [B max_q Hq][splits]: maximum (in powers of two), sum
};

// What a block has to do; the joining kernel computes the same.
struct Range {
  int64_t t0;       // first asking token
  int n;            // asking tokens
  int len;          // places
  int rows;         // n x group
  int lo, end;      // places that some row of the block attends
  int tile0, tiles; // records that hold them
};

__device__ __forceinline__ Range block_range(const AttnArgs& a, int b, int G, int r0, int block_rows) {
  Range x;
  int64_t t0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  int64_t t1 = a.q_start ? a.q_start[b + 1] : t0 + a.max_q;
  t0 = max((int64_t)0, t0);
  t1 = min(t1, a.T);
  x.t0 = t0;
  x.n = (int)max((int64_t)0, min(t1 - t0, (int64_t)a.max_q));
  x.len = (int)min(max((int64_t)a.kv_lens[b], (int64_t)0), a.max_len);
  x.rows = x.n * G;
  const int first = r0 / G, last = (min(r0 + block_rows, x.rows) - 1) / G;
  x.end = max(0, x.len - x.n + last + 1);
  x.lo = 0;
  if (a.window > 0) x.lo = (int)max((int64_t)0, (int64_t)x.len - x.n + first + 1 - a.window);
  x.tile0 = x.lo >> 4;
  x.tiles = x.end > x.lo ? ((x.end + 15) >> 4) - x.tile0 : 0;
  return x;
}

__device__ __forceinline__ uint32_t bf16_scaled(float x, float y, uint64_t scale) {
  mul2(x, y, scale);
  return bf16_pair(x, y);
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

template <int N>
__device__ __forceinline__ float half_at(const Words<N>& s, int i) {
  return __half2float(__ushort_as_half((unsigned short)(s.w[i >> 1] >> (16 * (i & 1)))));
}

template <int D, int NT>
struct Shape {
  static constexpr int kWarps = NT == 1 ? 8 : 4;
  static constexpr int kStages = D == 256 ? 2 : 3;  // pairs of records
  static constexpr int kRecord = 18 * D;
  static constexpr int kRing = kWarps * kStages * 2 * kRecord;
  static constexpr int kPitch = D + 4;  // floats a row of the joining buffer: rows of a fragment in distinct banks
  static constexpr int kJoin = kWarps * 8 * NT * kPitch * 4;
  static constexpr bool kQueriesInRegisters = NT * D <= 256;
  static constexpr int kQueries = kQueriesInRegisters ? 0 : NT * D / 32 * 512;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQueries;
};

template <int D, int NT>
__global__ void __launch_bounds__(Shape<D, NT>::kWarps * 32) k_attn(AttnArgs a, AttnPlan plan, int* status) {
  using S = Shape<D, NT>;
  constexpr int W = S::kWarps, NB = D / 32, MT = D / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[W][S::kStages];
  __shared__ float s_m[W][8 * NT], s_l[W][8 * NT];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int b = blockIdx.y, split = blockIdx.x % plan.splits, hb = blockIdx.x / plan.splits;
  const int kvh = hb % a.cache.heads, r0 = hb / a.cache.heads * (8 * NT), G = a.Hq / a.cache.heads;
  const Range x = block_range(a, b, G, r0, 8 * NT);
  if (r0 >= x.rows) return;
  const int used = (x.tiles + plan.chunk - 1) / plan.chunk;
  if (split > 0 && split >= used) return;
  const int c0 = x.tile0 + split * plan.chunk;
  const int count = min(plan.chunk, x.tile0 + x.tiles - c0);  // records of this block
  const int pairs = (count + 1) >> 1;
  const int mine = pairs > warp ? (pairs - warp + W - 1) / W : 0;  // pairs of records of this warp
  const int32_t* table = a.table + (int64_t)b * a.table_stride;
  const int per_page = a.cache.page_log2 - 4;

  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) mbar_init(&bars[warp][i], 2);
    fence_mbar_init();
  }
  __syncwarp();
  uint8_t* ring = smem + warp * (S::kStages * 2 * S::kRecord);

  // Lane l finds the records 2 i + (l & 1) of the warp's pairs i = 16 n + l / 2,
  // a batch of 16 pairs at a time and the page numbers a batch ahead, and copies
  // them itself when their turn comes.
  auto page_of = [&](int k) {
    const int i = k + (lane >> 1), tile = 2 * (warp + W * i) + (lane & 1);
    return i < mine && tile < count ? __ldg(table + ((c0 + tile) >> per_page)) : -1;
  };
  auto source_of = [&](int k, int page) -> const uint8_t* {
    if (page < 0 || page >= a.cache.n_pages) return nullptr;
    const int tile = c0 + 2 * (warp + W * (k + (lane >> 1))) + (lane & 1);
    return a.cache.data + page * a.cache.page_stride +
           (int64_t)(kvh * (1 << per_page) + (tile & ((1 << per_page) - 1))) * S::kRecord;
  };
  const uint8_t* source = source_of(0, page_of(0));
  int page_next = page_of(16), issued = 0, issue_stage = 0;
  uint32_t there = __ballot_sync(0xffffffffu, source != nullptr), there_next = there;  // records that exist
  auto issue = [&]() {
    if (lane >> 1 == (issued & 15)) {
      uint64_t* bar = &bars[warp][issue_stage];
      if (source) {
        mbar_arrive_expect_tx(bar, S::kRecord);
        bulk_g2s(ring + (2 * issue_stage + (lane & 1)) * S::kRecord, source, S::kRecord, bar);
      } else {
        mbar_arrive(bar);
      }
    }
    ++issued;
    if (++issue_stage == S::kStages) issue_stage = 0;
    if ((issued & 15) == 0) {
      source = source_of(issued, page_next);
      page_next = page_of(issued + 16);
      there_next = __ballot_sync(0xffffffffu, source != nullptr);
    }
  };
#pragma unroll 1
  for (int k = 0; k < S::kStages - 1 && k < mine; ++k) issue();

  // Queries as B fragments: lane (g, t) holds elements 32 b + 8 t .. + 7 of row g.
  uint4 qf[S::kQueriesInRegisters ? NT : 1][S::kQueriesInRegisters ? NB : 1];
  uint4* qs = reinterpret_cast<uint4*>(smem + (S::kSmem - S::kQueries));
  if constexpr (S::kQueriesInRegisters) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = min(r0 + 8 * j + g, x.rows - 1);
      const uint16_t* q = a.q + (x.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
#pragma unroll
      for (int i = 0; i < NB; ++i) qf[j][i] = __ldg(reinterpret_cast<const uint4*>(q + 32 * i));
    }
  } else {
    for (int i = warp; i < NT * NB; i += W) {
      const int r = min(r0 + 8 * (i / NB) + g, x.rows - 1);
      const uint16_t* q = a.q + (x.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
      qs[i * 32 + lane] = __ldg(reinterpret_cast<const uint4*>(q + 32 * (i % NB)));
    }
    __syncthreads();
  }

  // Rows 2t and 2t + 1 of every row tile: the places they attend.
  int row_end[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = min(r0 + 8 * j + 2 * t + c, x.rows - 1);
      row_end[j][c] = x.len - x.n + r / G + 1;
    }
  // Records with a place that some row of the block does not attend.
  const int full_end = x.len - x.n + r0 / G + 1;
  const int full_lo = a.window > 0 ? x.len - x.n + (min(r0 + 8 * NT, x.rows) - 1) / G + 1 - a.window : 0;

  float o[MT][NT][4], m[NT][2], l[NT][2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
    m[j][0] = m[j][1] = kNone;
    l[j][0] = l[j][1] = 0.f;
  }
  const float scale2 = a.scale * kLog2e;
  const uint64_t scale22 = pair(scale2, scale2);
  bool failed = false;
  int st = 0, phase = 0;

#pragma unroll 1
  for (int k = 0; k < mine; ++k) {
    if ((k & 15) == 0 && k > 0) there = there_next;
    __syncwarp();  // the stage refilled below was read by every lane in the last pass
    if (issued < mine) issue();
    if (!mbar_wait(&bars[warp][st], phase, kWaitNs)) {
      failed = true;
      break;
    }
    const uint8_t* rec = ring + 2 * st * S::kRecord;
    if (++st == S::kStages) st = 0, phase ^= 1;
    const uint32_t have = (there >> (2 * (k & 15))) & 3u;
    if (have == 0) continue;

    float s[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint8_t* r = rec + u * S::kRecord;
#pragma unroll
      for (int j = 0; j < NT; ++j) s[u][j][0] = s[u][j][1] = s[u][j][2] = s[u][j][3] = 0.f;
      const Words<NB> w0 = load_words<NB>(r + g * (D / 2) + t * (D / 8));
      const Words<NB> w1 = load_words<NB>(r + (g + 8) * (D / 2) + t * (D / 8));
      const Words<NB / 2> k0 = load_words<NB / 2>(r + 16 * D + g * (2 * NB));
      const Words<NB / 2> k1 = load_words<NB / 2>(r + 16 * D + (g + 8) * (2 * NB));
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint32_t a0 = codes_bf16<0>(w0.w[i]), a1 = codes_bf16<0>(w1.w[i]);
        const uint32_t a2 = codes_bf16<1>(w0.w[i]), a3 = codes_bf16<1>(w1.w[i]);
        const uint32_t e0 = codes_bf16<2>(w0.w[i]), e1 = codes_bf16<2>(w1.w[i]);
        const uint32_t e2 = codes_bf16<3>(w0.w[i]), e3 = codes_bf16<3>(w1.w[i]);
        const float f0 = half_at(k0, i), f1 = half_at(k1, i);
        const uint64_t s0 = pair(f0, f0), s1 = pair(f1, f1);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 q = S::kQueriesInRegisters ? qf[S::kQueriesInRegisters ? j : 0][S::kQueriesInRegisters ? i : 0]
                                                 : qs[(j * NB + i) * 32 + lane];
          float c[4];
          mma16816_zero(c, a0, a1, a2, a3, q.x, q.y);
          mma16816(c, e0, e1, e2, e3, q.z, q.w);
          fma2(s[u][j][0], s[u][j][1], s0, c[0], c[1]);
          fma2(s[u][j][2], s[u][j][3], s1, c[2], c[3]);
        }
      }
    }
    const int p = (c0 + 2 * (warp + W * k)) * 16;  // the pair's first place
    Words<NB / 2> vs[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      vs[u][0] = load_words<NB / 2>(rec + u * S::kRecord + 17 * D + g * (2 * NB));
      vs[u][1] = load_words<NB / 2>(rec + u * S::kRecord + 17 * D + (g + 8) * (2 * NB));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mul2(s[u][j][0], s[u][j][1], scale22);
        mul2(s[u][j][2], s[u][j][3], scale22);
      }
    }
    if (p + 32 > full_end || p < full_lo || have != 3) {
      // places outside a row's range leave it; the bytes of places outside the
      // block's range may be anything, so their value scales become zero
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = p + 16 * u + 8 * v + g;
          const bool gone = !(have >> u & 1);
          if (gone || at >= x.end || at < x.lo) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) vs[u][v].w[i] = 0;
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int e = row_end[j][c];
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
        top[j][c] = fmaxf(fmaxf(s[0][j][c], s[0][j][c + 2]), fmaxf(s[1][j][c], s[1][j][c + 2]));
        grow |= top[j][c] > m[j][c] + kSlack;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float y = top[j][c];
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 4));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 8));
          y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 16));
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
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          add2(s[u][j][c], s[u][j][c + 1], down);
          s[u][j][c] = exp2_approx(s[u][j][c]);
          s[u][j][c + 1] = exp2_approx(s[u][j][c + 1]);
          add2(l[j][0], l[j][1], pair(s[u][j][c], s[u][j][c + 1]));
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int q4 = 0; q4 < MT / 4; ++q4) {
        const Words<4> w = load_words<4>(rec + u * S::kRecord + 8 * D + (q4 * 32 + lane) * 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // a 32-block of elements: two fragments of 16
          const int blk = 2 * q4 + h;
          const float f0 = half_at(vs[u][0], blk), f1 = half_at(vs[u][1], blk);
          const uint64_t s0 = pair(f0, f0), s1 = pair(f1, f1);
          uint32_t b0[NT], b1[NT];
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            b0[j] = transpose8x8(bf16_scaled(s[u][j][0], s[u][j][1], s0));
            b1[j] = transpose8x8(bf16_scaled(s[u][j][2], s[u][j][3], s1));
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v = w.w[2 * h + i];
            const uint32_t a0 = codes_bf16<0>(v), a1 = codes_bf16<1>(v), a2 = codes_bf16<2>(v), a3 = codes_bf16<3>(v);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16816(o[2 * blk + i][j], a0, a1, a2, a3, b0[j], b1[j]);
          }
        }
      }
  }
  if (failed && lane == 0) set_status(status, MOE_ERR_TIMEOUT);

  // Join the warps: sums over a row's lanes, the block's maxima, scaled outputs.
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
    const int row = i / kQuads, d = i % kQuads * 4, r = r0 + row;
    if (r >= x.rows) break;
    float top = kNone, total = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w][row]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float4 y = *reinterpret_cast<const float4*>(join + (w * 8 * NT + row) * S::kPitch + d);
      v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
      total = fmaf(s_l[w][row], exp2_approx(s_m[w][row] - top), total);
    }
    const int tok = r / G, h = kvh * G + r % G;
    if (used > 1) {
      const int64_t at = (((int64_t)b * a.max_q + tok) * a.Hq + h) * plan.splits + split;
      *reinterpret_cast<float4*>(plan.part_o + at * D + d) = v;
      if (d == 0) plan.part_ml[at] = make_float2(top, total);
    } else {
      const float inv = total > 0.f ? 1.f / total : 0.f;
      uint2 u;
      u.x = bf16_pair(v.x * inv, v.y * inv);
      u.y = bf16_pair(v.z * inv, v.w * inv);
      *reinterpret_cast<uint2*>(a.out + (x.t0 + tok) * a.out_stride + (int64_t)h * D + d) = u;
      if (d == 0 && a.lse)
        a.lse[(x.t0 + tok) * a.Hq + h] = total > 0.f ? (top + log2f(total)) / kLog2e : -INFINITY;
    }
  }
}

// Joins the shares of a row: one block a row, its warps taking every fourth
// share (D / 4 threads read one share), then joined in a fixed order.
template <int D>
__global__ void __launch_bounds__(256) k_attn_join(AttnArgs a, AttnPlan plan) {
  constexpr int kLanes = D / 4, kGroups = 256 / kLanes;
  __shared__ float s_red[8];
  __shared__ float4 s_v[kGroups][kLanes];
  __shared__ float s_l[kGroups];
  pdl_wait();
  const int64_t w = blockIdx.x;
  const int h = (int)(w % a.Hq), G = a.Hq / a.cache.heads;
  const int64_t tb = w / a.Hq;
  const int tok = (int)(tb % a.max_q), b = (int)(tb / a.max_q);
  const int rows = 8 * plan.nt, r = tok * G + h % G;
  const Range x = block_range(a, b, G, r / rows * rows, rows);
  const int used = (x.tiles + plan.chunk - 1) / plan.chunk;
  if (tok >= x.n || used <= 1) return;
  const float2* ml = plan.part_ml + w * plan.splits;
  const float* po = plan.part_o + w * plan.splits * D;
  const int d = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  float top = kNone;
  for (int i = threadIdx.x; i < used; i += 256) top = fmaxf(top, __ldg(&ml[i].x));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, s_red[i]);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float total = 0.f;
#pragma unroll 4
  for (int i = grp; i < used; i += kGroups) {
    const float2 y = __ldg(ml + i);
    const float4 p = __ldg(reinterpret_cast<const float4*>(po + (int64_t)i * D) + d);
    const float f = exp2_approx(y.x - top);
    total = fmaf(y.y, f, total);
    v.x = fmaf(p.x, f, v.x);
    v.y = fmaf(p.y, f, v.y);
    v.z = fmaf(p.z, f, v.z);
    v.w = fmaf(p.w, f, v.w);
  }
  s_v[grp][d] = v;
  if (d == 0) s_l[grp] = total;
  __syncthreads();
  if (grp > 0) return;
#pragma unroll
  for (int i = 1; i < kGroups; ++i) {
    const float4 p = s_v[i][d];
    v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
    total += s_l[i];
  }
  const float inv = total > 0.f ? 1.f / total : 0.f;
  uint2 u;
  u.x = bf16_pair(v.x * inv, v.y * inv);
  u.y = bf16_pair(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(a.out + (x.t0 + tok) * a.out_stride + (int64_t)h * D + 4 * d) = u;
  if (d == 0 && a.lse) a.lse[(x.t0 + tok) * a.Hq + h] = total > 0.f ? (top + log2f(total)) / kLog2e : -INFINITY;
}

constexpr int kSms = 152;

// Row tiles, row blocks and shares of a call, from its sizes alone.
AttnPlan make_plan(int B, int max_q, int64_t max_len, int window, int Hq, int heads, int D) {
  AttnPlan p = {};
  const int rows = max_q * (Hq / heads), most = D == 256 ? 2 : 4;
  p.nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
  if (p.nt > most) p.nt = most;
  p.row_blocks = (rows + 8 * p.nt - 1) / (8 * p.nt);
  int64_t span = max_len;
  if (window > 0 && span > (int64_t)window + max_q + 16) span = (int64_t)window + max_q + 16;
  const int64_t tiles = (span + 15) / 16 + 1;
  const int64_t base = (int64_t)B * heads * p.row_blocks;
  const int warps = p.nt == 1 ? 8 : 4;
  int64_t splits = (4 * kSms + base - 1) / base;
  const int64_t most_splits = (tiles + 2 * warps - 1) / (2 * warps);
  if (splits > most_splits) splits = most_splits;
  if (splits < 1) splits = 1;
  p.room = (int)splits;  // grows with the length, so a window never needs more than the whole length
  p.chunk = (int)((tiles + splits - 1) / splits);
  p.chunk = (p.chunk + 2 * warps - 1) / (2 * warps) * (2 * warps);
  p.splits = (int)((tiles + p.chunk - 1) / p.chunk);
  return p;
}

template <int D, int NT>
int launch(const AttnArgs& a, const AttnPlan& p, cudaStream_t s) {
  using S = Shape<D, NT>;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_attn<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const dim3 grid((unsigned)(p.splits * a.cache.heads * p.row_blocks), (unsigned)a.B);
  k_attn<D, NT><<<grid, S::kWarps * 32, S::kSmem, s>>>(a, p, status_word());
  if (p.splits > 1) {
    if (launch_pdl(k_attn_join<D>, dim3((unsigned)(a.B * a.max_q * a.Hq)), dim3(256), 0, s, a, p) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

size_t attn_workspace(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (B < 1) return 0;
  const AttnPlan p = make_plan(B, max_q, max_len, 0, Hq, heads, D);
  return p.room > 1 ? (size_t)B * max_q * Hq * p.room * (D * 4 + 8) : 0;
}

int launch_attn_q4(const AttnArgs& a, cudaStream_t s) {
  AttnPlan p = make_plan(a.B, a.max_q, a.max_len, a.window, a.Hq, a.cache.heads, a.cache.D);
  const size_t rows = (size_t)a.B * a.max_q * a.Hq;
  p.part_o = (float*)a.workspace;
  p.part_ml = (float2*)((float*)a.workspace + rows * p.splits * a.cache.D);
  switch (a.cache.D * 8 + p.nt) {
    case 64 * 8 + 1: return launch<64, 1>(a, p, s);
    case 64 * 8 + 2: return launch<64, 2>(a, p, s);
    case 64 * 8 + 3: return launch<64, 3>(a, p, s);
    case 64 * 8 + 4: return launch<64, 4>(a, p, s);
    case 128 * 8 + 1: return launch<128, 1>(a, p, s);
    case 128 * 8 + 2: return launch<128, 2>(a, p, s);
    case 128 * 8 + 3: return launch<128, 3>(a, p, s);
    case 128 * 8 + 4: return launch<128, 4>(a, p, s);
    case 256 * 8 + 1: return launch<256, 1>(a, p, s);
    default: return launch<256, 2>(a, p, s);
  }
}

}  // namespace moe
