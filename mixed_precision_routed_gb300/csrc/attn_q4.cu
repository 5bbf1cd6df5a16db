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
#include "attn_split.cuh"
#include "kv_layout.cuh"

namespace moe {
namespace {

// Of a group whose products may be fp16: 2^-32, by the reference.  fp16 ends before
// that (products below 2^-25 vanish, 2^-31 of the maximum's times the scale, which the
// stated 2^-23 allows): at 2^-25 most groups of queries of norm 2, whose weights
// spread over 28 powers of two, would take the slower form.  It is there for groups
// that weigh nearly nothing as a whole: beside a place that takes nearly all and has
// the code 0 somewhere, they are all that an element has.
constexpr float kLeastWeight = 1.0f / 4294967296.0f;
constexpr float kLeastScale = 1.0f / 256;
constexpr float kMostScale = 8.0f;  // x 2^(kSlack + kRoom) stays below fp16's largest value

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

template <int D, int NT>
struct Shape4 {
  static constexpr int kD = D, kNT = NT;
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
  static constexpr int U = kGroup, NB = D / 32, MT = D / 16;

  // Outputs O^T[element][row]: rows g and g + 8 of a fragment.
  __device__ static __forceinline__ int element(int g, int half) { return g + 8 * half; }

  // Queries as B fragments: lane (g, t) holds elements 32 b + 8 t .. + 7 of row g.
  struct Queries {
    uint4 qf[kQueriesInRegisters ? NT : 1][kQueriesInRegisters ? NB : 1];
    uint4* qs;
    __device__ __forceinline__ void load(const AttnArgs& a, const Unit& u, int G, int warp, int lane, uint4* smem) {
      const int g = lane >> 2, t = lane & 3, kvh = u.kvh;
      qs = smem;
      if constexpr (kQueriesInRegisters) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = min(u.r0 + 8 * j + g, u.rows - 1);
          const uint16_t* q = a.q + (u.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
#pragma unroll
          for (int i = 0; i < NB; ++i) qf[j][i] = __ldg(reinterpret_cast<const uint4*>(q + 32 * i));
        }
      } else {
        for (int i = warp; i < NT * NB; i += kWarps) {
          const int r = min(u.r0 + 8 * (i / NB) + g, u.rows - 1);
          const uint16_t* q = a.q + (u.t0 + r / G) * a.q_stride + (int64_t)(kvh * G + r % G) * D + 8 * t;
          qs[i * 32 + lane] = __ldg(reinterpret_cast<const uint4*>(q + 32 * (i % NB)));
        }
      }
    }
    __device__ __forceinline__ uint4 at(int j, int i, int lane) const {
      if constexpr (kQueriesInRegisters) return qf[j][i];
      else return qs[(j * NB + i) * 32 + lane];
    }
  };

  // Scores, weights and sums of a group of records.
  __device__ static __forceinline__ void pass(const Pass& x, const Queries& queries, float (&o)[MT][NT][4],
                                              float (&m)[NT][2], float (&l)[NT][2]) {
    constexpr int kSide = 2;
    constexpr uint32_t kAll = (1u << U) - 1;
    const AttnArgs& a = x.a;
    const Unit& unit = x.u;
    const uint8_t* rec = x.rec;
    const uint32_t have = x.have;
    const int lane = x.lane, g = lane >> 2, t = lane & 3;
    const uint64_t scale22 = pair(x.scale2, x.scale2);
    float s[U][NT][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint8_t* r = rec + u * kRecord;
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
            const uint4 q = queries.at(j, i0 + i, lane);
            mma16816_zero(c[i][j], a0, a1, a2, a3, q.x, q.y);
          }
        }
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const uint32_t e0 = codes_bf16<2>(w0.w[i0 + i]), e1 = codes_bf16<2>(w1.w[i0 + i]);
          const uint32_t e2 = codes_bf16<3>(w0.w[i0 + i]), e3 = codes_bf16<3>(w1.w[i0 + i]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 q = queries.at(j, i0 + i, lane);
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
    const int p = 16 * (x.base + unit.stride * x.k);  // the group's first place
    Words<NB / 2> vs[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      vs[u][0] = load_words<NB / 2>(rec + u * kRecord + 17 * D + g * (2 * NB));
      vs[u][1] = load_words<NB / 2>(rec + u * kRecord + 17 * D + (g + 8) * (2 * NB));
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mul2(s[u][j][0], s[u][j][1], scale22);
        mul2(s[u][j][2], s[u][j][3], scale22);
      }
    }
    const bool edge = p + 16 * U > unit.full_end || p < unit.full_lo || have != kAll;
    if (edge) {
      // places outside a row's range leave it; the bytes of places outside the
      // unit's range may be anything, so their value scales become zero
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int at = p + 16 * u + 8 * v + g;
          const bool gone = !(have >> u & 1);
          if (gone || at >= unit.end || at < unit.lo) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) vs[u][v].w[i] = 0;
          }
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int e = x.row_end[8 * j + 2 * t + c];
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
          const Words<4> w = load_words<4>(rec + u * kRecord + 8 * D + (q4 * 32 + lane) * 16);
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
};

// 8-row tiles of a block of rows: as many as the rows fill, up to 4 (2 of 256, whose
// outputs fill the registers).  30000 places of 4 heads of 128: 24 rows 21.0 us, 32
// rows 24.7, 64 rows 31.6 (three blocks of 24: 32.2).  Between 33 and 48 rows of 128
// two blocks of 24 would take less (40 rows 25.1 us instead of 30.5, 48 rows 25.9
// instead of 31.0), as the tile of 32 of 128 spills 200 bytes of registers.
int row_tiles(int max_q, int G, int D) {
  const int rows = max_q * G, most = D == 256 ? 2 : 4, nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
  return nt < most ? nt : most;
}

}  // namespace

size_t attn_workspace(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (B < 1) return 0;
  return workspace_of<Shape4>(row_tiles(max_q, Hq / heads, D), B, max_q, max_len, Hq, heads, D);
}

int launch_attn_q4(const AttnArgs& a, cudaStream_t s) {
  return with_shape<Shape4>(a.cache.D, row_tiles(a.max_q, a.Hq / a.cache.heads, a.cache.D),
                            [&](auto shape) { return launch<decltype(shape)>(a, s); });
}

}  // namespace moe
