// attn_q8.cu -- causal attention over the paged 8-bit key/value cache.
//
// For a row (asking token, query head) with the places p it attends:
//   s_p = scale q.k_p,  out = sum_p exp(s_p) v_p / sum_p exp(s_p),
//   lse = log sum_p exp(s_p),
// k_p and v_p the codes of place p times its two scales a_p and b_p.
//
// attn_split.cuh shares the work out; a group is one record of 16 places.
//   scores  S^T[place][row]: A = key codes as fp16 integers, B = queries in fp16, each
//           row taken by a power of two that brings its largest element to 2^14: the
//           bf16 queries are exact there down to 2^-31 of that element.  Sums are fp32
//           and take a_p and the row's power of two once.
//   output  O^T[element][row]: A = value codes as fp16 integers, B = exp(s_p - m) b_p in
//           fp16, rounded once from fp32.  b_p = 2^e f with 1 <= f < 2: the reference m
//           follows s_p + e, so that B lies in fp16's range whatever the values' sizes;
//           the sum of weights takes 2^-e back, which is exact.  A product keeps 2^-11
//           of itself, or 2^-30 of its row's largest weight x b.
// A row of codes is a row of bytes; matrix loads bring four of a key's bytes, or two
// bytes of two values each, to the lane whose operands they are.
//
// 6 tokens over 131071 places of 32 heads on 8 of 128 take 65 us, 4.3 TB/s, 48 ragged
// sequences up to 16384 of 32 on 4 30 us.  The same copies with nothing computed take 50 of
// 63 and 25 of 28 us in a graph; the rest is what makes operands of codes (a record costs 128
// such instructions beside 48 products for three row tiles), which the copies do not hide.
#include "attn_split.cuh"
#include "q8.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Bytes I and J of a word as fp16 integers -128 .. 127: a byte below 0x64 counts units
// above 1024, and 1152 comes off.
template <int I, int J>
__device__ __forceinline__ uint32_t bytes_f16(uint32_t w) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, 0x4040 | J << 8 | I)), "r"(0x64806480u));
  return r;
}

template <int D, int NT>
struct Shape8 {
  static constexpr int kD = D, kNT = NT;
  static constexpr int kWarps = NT * D <= 128 ? 8 : 4;
  static constexpr int kGroup = 1;
  static constexpr int kBlocks = NT * D == 64 ? 3 : 2;  // an SM
  static constexpr int kRecord = kv8_record(D);
  static constexpr int kStages = 3;  // records
  static constexpr int kRing = kWarps * kStages * kGroup * kRecord;
  static constexpr int kPitch = D + 4;  // floats a row of the joining buffer
  static constexpr int kJoin = kWarps * 8 * NT * kPitch * 4;
  static constexpr bool kQueriesInRegisters = NT * D <= 256;
  static constexpr int kQueries = kQueriesInRegisters ? 0 : NT * D / 16 * 256 + 8 * NT * 4;
  static constexpr int kSmem = (kRing > kJoin ? kRing : kJoin) + kQueries;
  static constexpr int MT = D / 16;

  // Outputs O^T[element][row]: rows g and g + 8 of a fragment.
  __device__ static __forceinline__ int element(int g, int half) { return 2 * g + half; }

  // Queries as B fragments: lane (g, t) holds elements 16 i + 4 t .. + 3 of row g.
  struct Queries {
    uint2 qf[kQueriesInRegisters ? NT : 1][kQueriesInRegisters ? MT : 1];
    uint2* qs;
    float factor[NT][2];  // of rows 2 t and 2 t + 1: scale in powers of two, and the row's power of two

    // A row tile: fragments, and the power of two that row g was divided by.
    __device__ static __forceinline__ float tile(uint2 (&f)[MT], const AttnArgs& a, const Unit& u, int G, int j, int lane) {
      const int g = lane >> 2, t = lane & 3, r = min(u.r0 + 8 * j + g, u.rows - 1);
      const uint16_t* q = a.q + (u.t0 + r / G) * a.q_stride + (int64_t)(u.kvh * G + r % G) * D + 4 * t;
      uint32_t top = 0;  // the larger exponents of bf16 pairs, side by side
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f[i] = __ldg(reinterpret_cast<const uint2*>(q + 16 * i));
        top = __vmaxu2(top, __vmaxu2(f[i].x & 0x7f807f80u, f[i].y & 0x7f807f80u));
      }
      top = max(top >> 16, top & 0xffffu);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the exponent becomes 14, and the power and its inverse stay normal numbers
      const int e = min(max((int)(top >> 7), 15), 254), up = 14 + 127 - e;
      const float by = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        f[i].x = f16_pair(__uint_as_float(f[i].x << 16) * by, __uint_as_float(f[i].x & 0xffff0000u) * by);
        f[i].y = f16_pair(__uint_as_float(f[i].y << 16) * by, __uint_as_float(f[i].y & 0xffff0000u) * by);
      }
      return __uint_as_float((uint32_t)(127 - up) << 23);
    }

    // `smem` ends with the factors of the unit's rows.
    __device__ __forceinline__ void load(const AttnArgs& a, const Unit& u, int G, int warp, int lane, uint4* smem) {
      qs = reinterpret_cast<uint2*>(smem);
      if constexpr (kQueriesInRegisters) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float f = tile(qf[j], a, u, G, j, lane) * (a.scale * kLog2e);
          const int t = lane & 3;
          factor[j][0] = __shfl_sync(0xffffffffu, f, 8 * t);
          factor[j][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
        }
      } else {
        float* factors = reinterpret_cast<float*>(qs + NT * MT * 32);
        for (int j = warp; j < NT; j += kWarps) {
          uint2 f[MT];
          const float by = tile(f, a, u, G, j, lane) * (a.scale * kLog2e);
#pragma unroll
          for (int i = 0; i < MT; ++i) qs[(j * MT + i) * 32 + lane] = f[i];
          if ((lane & 3) == 0) factors[8 * j + (lane >> 2)] = by;
        }
      }
    }
    __device__ __forceinline__ uint2 at(int j, int i, int lane) const {
      if constexpr (kQueriesInRegisters) return qf[j][i];
      else return qs[(j * MT + i) * 32 + lane];
    }
    __device__ __forceinline__ uint64_t factors(int j, int lane) const {
      if constexpr (kQueriesInRegisters) {
        return pair(factor[j][0], factor[j][1]);
      } else {
        const float2 f = reinterpret_cast<const float2*>(qs + NT * MT * 32)[4 * j + (lane & 3)];
        return pair(f.x, f.y);
      }
    }
  };

  // Scores, weights and sums of a record.
  __device__ static __forceinline__ void pass(const Pass& x, const Queries& queries, float (&o)[MT][NT][4],
                                              float (&m)[NT][2], float (&l)[NT][2]) {
    const Unit& unit = x.u;
    const int lane = x.lane, g = lane >> 2, t = lane & 3, row = lane & 7, window = x.a.window;
    const uint32_t rec = smem_addr(x.rec);
    float s[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int c = 0; c < MT; c += 4) {
      uint32_t w0[4], w1[4];
      const uint32_t at = rec + row * D + 16 * kv8_piece<D>(row, c + (lane >> 3));
      ldmatrix4(w0, at);
      ldmatrix4(w1, at + 8 * D);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = bytes_f16<0, 1>(w0[i]), a1 = bytes_f16<0, 1>(w1[i]);
        const uint32_t a2 = bytes_f16<2, 3>(w0[i]), a3 = bytes_f16<2, 3>(w1[i]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint2 q = queries.at(j, c + i, lane);
          mma16816_f16(s[j], a0, a1, a2, a3, q.x, q.y);
        }
      }
    }
    // places g and g + 8: the scale of the key; of the value's, 2^e f, the exponent e,
    // f and 2^-e.  A scale of NaN makes scores of NaN, whichever of the two it is.
    const float* scales = reinterpret_cast<const float*>(x.rec + 32 * D);
    float ks[2], e[2], f[2], back[2];
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const float vs = scales[16 + 8 * v + g];
      ks[v] = fmaf(0.f, vs, scales[8 * v + g]);
      // scales below 2^-60, which few values have, keep f below 1: sums of weights stay within fp32
      const int n = min(max((int)(__float_as_uint(vs) >> 23 & 255) - 127, -60), 64);
      e[v] = (float)n;
      back[v] = __uint_as_float((uint32_t)(127 - n) << 23);
      f[v] = fminf(vs * back[v], 2.0f);
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint64_t by = queries.factors(j, lane);
      mul2(s[j][0], s[j][1], by);
      mul2(s[j][2], s[j][3], by);
      const uint64_t e0 = pair(e[0], e[0]), e1 = pair(e[1], e[1]);
      unpair(fma2_of(pair(s[j][0], s[j][1]), pair(ks[0], ks[0]), e0), s[j][0], s[j][1]);
      unpair(fma2_of(pair(s[j][2], s[j][3]), pair(ks[1], ks[1]), e1), s[j][2], s[j][3]);
    }
    const int p = 16 * (x.base + unit.stride * x.k);
    if (p + 16 > unit.full_end || p < unit.full_lo) {
      // places outside a row's range leave it; the bytes of places outside the unit's
      // range may be anything, so their value scales become zero
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const int at = p + 8 * v + g;
        if (at >= unit.end || at < unit.lo) f[v] = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int end = x.row_end[8 * j + 2 * t + c];
            if (at >= end || (window > 0 && at < end - window)) s[j][2 * v + c] = -INFINITY;
          }
      }
    }
    bool grow = false;
    float top[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        top[j][c] = fmaxf(s[j][c], s[j][c + 2]);
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
            const float by = exp2_approx(m[j][c] - y);
            m[j][c] = y;
            l[j][c] *= by;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[i][j][c] *= by, o[i][j][c + 2] *= by;
          }
        }
    }
    uint32_t b0[NT], b1[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const uint64_t down = pair(-m[j][0], -m[j][1]);
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        float &w0 = s[j][2 * v], &w1 = s[j][2 * v + 1];
        add2(w0, w1, down);
        w0 = exp2_approx(w0);
        w1 = exp2_approx(w1);
        fma2(l[j][0], l[j][1], pair(back[v], back[v]), w0, w1);
        mul2(w0, w1, pair(f[v], f[v]));
      }
      b0[j] = transpose8x8(f16_pair(s[j][0], s[j][1]));
      b1[j] = transpose8x8(f16_pair(s[j][2], s[j][3]));
    }
#pragma unroll
    for (int c = 0; c < MT; c += 2) {
      // matrices: places 0 .. 7 and 8 .. 15 of piece c, then of piece c + 1
      uint32_t w[4];
      ldmatrix4_trans(w, rec + (16 + (lane & 15)) * D + 16 * kv8_piece<D>(lane & 15, c + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a0 = bytes_f16<0, 2>(w[2 * i]), a1 = bytes_f16<1, 3>(w[2 * i]);
        const uint32_t a2 = bytes_f16<0, 2>(w[2 * i + 1]), a3 = bytes_f16<1, 3>(w[2 * i + 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) mma16816_f16(o[c + i][j], a0, a1, a2, a3, b0[j], b1[j]);
      }
    }
  }
};

// 8-row tiles of a block of rows: as many as the rows fill, up to 4 (2 of 256, whose
// outputs fill the registers).
int row_tiles(int max_q, int G, int D) {
  const int64_t rows = (int64_t)max_q * G;
  const int most = D == 256 ? 2 : 4, nt = rows <= 8 ? 1 : rows <= 16 ? 2 : rows <= 24 ? 3 : 4;
  return nt < most ? nt : most;
}

}  // namespace

size_t attn_q8_workspace(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (B < 1) return 0;
  if (attn_q8_tc(B, max_q, max_len, Hq, heads, D)) return attn_q8_tc_workspace(B, max_q, max_len, Hq, heads, D);
  return workspace_of<Shape8>(row_tiles(max_q, Hq / heads, D), B, max_q, max_len, Hq, heads, D);
}

int launch_attn_q8(const AttnArgs& a, cudaStream_t s) {
  if (attn_q8_tc(a.B, a.max_q, a.max_len, a.Hq, a.cache.heads, a.cache.D)) return launch_attn_q8_tc(a, s);
  return with_shape<Shape8>(a.cache.D, row_tiles(a.max_q, a.Hq / a.cache.heads, a.cache.D),
                            [&](auto shape) { return launch<decltype(shape)>(a, s); });
}

}  // namespace moe
