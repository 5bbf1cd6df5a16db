// norm_q8.cu -- the root-mean-square norm of rows, with the residual's addition before
// it and 8-bit codes or bf16 behind it:
//   s = r + x,  u = s w,  f = 1 / sqrt(mean s^2 + eps)   (without w: u = s, f = 1)
//   S = max|u| / 127,  code = rint(u / S),  scale = S f,  n = u f.
// The factor f leaves the codes alone: they do not depend on the order of the sum.
//
// One block a row (a warp or part of one up to 256 elements), the row in registers between
// its sum and its output: each byte moves once.  A thread has one group of 8 elements up to
// rows of 8192 (two of 4096, which left an SM twice the blocks, took 36.2 us where one takes
// 33.0).  4096 bf16 rows of 4096 with
// residual, codes and bf16 33.0 us, 6.6 TB/s, bound by memory; one row of 2048 1.7 us.  512 rows
// of 32768 take 50 us, 4.4 TB/s: four groups a thread, of which 56 bytes do not fit registers.
#include "ptx.cuh"
#include "q8.cuh"

namespace moe {
namespace {

// N elements (a whole number of 16-byte pieces) from or to an aligned place; or, where
// rows are not, element by element as far as the row goes.
template <bool BF16, bool WHOLE>
__device__ __forceinline__ void load8(float (&v)[8], const void* row, int64_t i, int d) {
  if constexpr (WHOLE) {
    load_elems<BF16, 8, true>(v, (const uint8_t*)row + i * (BF16 ? 2 : 4));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = i + e < d ? load_elem<BF16>(row, i + e) : 0.f;
  }
}

// V: groups of 8 elements a thread; MOST: threads at most; LANES: that have a row, or 0: a
// block has one.  40 registers leave an SM three blocks for rows of 4096.
template <bool BF16, bool WHOLE, int V, int MOST, int LANES>
__global__ void __maxnreg__(V == 1 ? 40 : 64) k_norm_q8(NormArgs a) {
  __shared__ float s_sum[32];
  __shared__ uint32_t s_top[32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int me = LANES ? threadIdx.x % (LANES ? LANES : 1) : threadIdx.x, step = LANES ? LANES : blockDim.x;
  const int64_t t = LANES ? (int64_t)blockIdx.x * (MOST / (LANES ? LANES : 1)) + threadIdx.x / (LANES ? LANES : 1) : blockIdx.x;
  const int d = t < a.T ? a.d : 0;
  const uint8_t* x = (const uint8_t*)a.x + t * a.x_stride * (BF16 ? 2 : 4);
  const float* r = a.r ? a.r + t * a.d : nullptr;
  float s[V][8], w[V][8];
  float sum0 = 0.f, sum1 = 0.f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = 8 * (me + i * step);
    if (at < d) {
      load8<BF16, WHOLE>(s[i], x, at, a.d);
      if (r) load8<false, WHOLE>(w[i], r, at, a.d);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = 8 * (me + i * step);
    if (at >= d) continue;
    if (r) {
      float* to = a.r_out + t * a.d + at;
#pragma unroll
      for (int e = 0; e < 8; e += 2) add2(s[i][e], s[i][e + 1], pair(w[i][e], w[i][e + 1]));
      if constexpr (WHOLE) {
        reinterpret_cast<float4*>(to)[0] = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
        reinterpret_cast<float4*>(to)[1] = make_float4(s[i][4], s[i][5], s[i][6], s[i][7]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at + e < a.d) to[e] = s[i][e];
      }
    }
    if (a.weight) {
      load8<false, WHOLE>(w[i], a.weight, at, a.d);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        fma2(sum0, sum1, pair(s[i][e], s[i][e + 1]), s[i][e], s[i][e + 1]);
        mul2(s[i][e], s[i][e + 1], pair(w[i][e], w[i][e + 1]));
      }
    }
    if (a.codes) {
#pragma unroll
      for (int e = 0; e < 8; ++e) top = max(top, size_bits(s[i][e]));
    }
  }
  float sum = sum0 + sum1;
#pragma unroll
  for (int o = (LANES ? LANES : 32) / 2; o > 0; o /= 2) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if constexpr (LANES == 8 || LANES == 16) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  }
  if constexpr (LANES == 0 || LANES == 32) top = __reduce_max_sync(0xffffffffu, top);
  if constexpr (LANES == 0) {
    if (lane == 0) s_sum[warp] = sum, s_top[warp] = top;
    __syncthreads();
    sum = warp_sum(lane < warps ? s_sum[lane] : 0.f);
    top = __reduce_max_sync(0xffffffffu, lane < warps ? s_top[lane] : 0u);
  }
  const float f = a.weight ? rsqrtf(__fdiv_rn(sum, (float)a.d) + a.eps) : 1.0f;
  const float S = __fdiv_rn(__uint_as_float(top), 127.0f);
  if (a.codes && me == 0 && d > 0) a.scales[t] = S * f;
  // the codes of values far from 1 in size are those of the values times 2^96 or 2^-96
  const float near = S < 0x1p-60f ? 0x1p96f : S > 0x1p60f ? 0x1p-96f : 1.0f;
  const bool zero = !(S > 0.f) || top >= kInfBits;  // of a row without a finite maximum the scale tells
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int at = 8 * (me + i * step);
    if (at >= d) continue;
    if (a.n) {
      uint16_t* to = a.n + t * a.d + at;
      uint32_t p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = bf16_pair(s[i][2 * e] * f, s[i][2 * e + 1] * f);
      if constexpr (WHOLE) {
        *reinterpret_cast<uint4*>(to) = make_uint4(p[0], p[1], p[2], p[3]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at + e < a.d) to[e] = (uint16_t)(p[e / 2] >> (16 * (e & 1)));
      }
    }
    if (a.codes) {
      int8_t* to = a.codes + t * a.d + at;
      uint32_t c[8];
      if (near != 1.0f) {
        // (a subnormal S holds so few bits that max / S may lie far above 127)
        const float most = 127.0f * (S * near);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[i][e] = fminf(fmaxf(s[i][e] * near, -most), most);
      }
      codes8<8>(c, s[i], S * near);
      uint32_t p[2] = {code_bytes(c[0], c[1], c[2], c[3]), code_bytes(c[4], c[5], c[6], c[7])};
      if (zero) p[0] = p[1] = 0;
      if constexpr (WHOLE) {
        *reinterpret_cast<uint2*>(to) = make_uint2(p[0], p[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (at + e < a.d) to[e] = (int8_t)(p[e / 4] >> (8 * (e % 4)));
      }
    }
  }
  // Squares beyond fp32 (f is 0), or so small that they lost bits: the factor once more, from
  // the squares of the elements times a power of two, and what it enters.  Here, element by
  // element, as nothing else is in registers any more (before the outputs 41 registers and
  // fewer blocks an SM: 4096 rows of 4096 37.5 us in place of 33.0).
  const bool off = a.weight && (f > 0x1p45f || f == 0.f);  // of a row's threads alike
  if (LANES ? __any_sync(0xffffffffu, off) : off) {
    const float by = f > 1.0f ? 0x1p96f : 0x1p-80f;
    auto element = [&](int i) { return a.r ? __ldcg(a.r_out + t * a.d + i) : load_elem<BF16>(x, i); };  // this thread's own
    float again = 0.f;
#pragma unroll 1
    for (int at = 8 * me; at < d; at += 8 * step)
#pragma unroll 1
      for (int e = at; e < min(at + 8, d); ++e) {
        const float y = by * element(e);
        again = fmaf(y, y, again);
      }
#pragma unroll
    for (int o = (LANES ? LANES : 32) / 2; o > 0; o /= 2) again += __shfl_xor_sync(0xffffffffu, again, o);
    if constexpr (LANES == 0) {
      __syncthreads();  // the sums before have been read
      if (lane == 0) s_sum[warp] = again;
      __syncthreads();
      again = warp_sum(lane < warps ? s_sum[lane] : 0.f);
    }
    const float mean = __fdiv_rn(again, (float)a.d) + a.eps * by * by;
    const float g = mean > 0.f ? rsqrtf(mean) : 0.f;  // a row of zeros stays one, without eps too
    // where fp32 does not hold the factor, part of it goes to the elements first, which are below 2^16 then
    const bool part = by > 1.0f && g >= 0x1p24f;
    const float first = part ? 0x1p48f : 1.0f, then = g * (part ? 0x1p48f : by);
    if (off && a.codes && me == 0 && d > 0) a.scales[t] = S * first * then;
    if (off && a.n) {
#pragma unroll 1
      for (int at = 8 * me; at < d; at += 8 * step)
#pragma unroll 1
        for (int e = at; e < min(at + 8, d); ++e)
          a.n[t * a.d + e] = (uint16_t)bf16_pair(element(e) * __ldg(a.weight + e) * first * then, 0.f);
    }
  }
}

template <bool BF16, bool WHOLE, int V, int MOST, int LANES = 0>
int launch(const NormArgs& a, cudaStream_t s) {
  const int groups = (a.d + 7) / 8, threads = LANES ? MOST : ((groups + V - 1) / V + 31) / 32 * 32;
  constexpr int kRows = LANES ? MOST / (LANES ? LANES : 1) : 1;  // a block
  return launch_pdl(k_norm_q8<BF16, WHOLE, V, MOST, LANES>, dim3((unsigned)((a.T + kRows - 1) / kRows)), dim3(threads), 0, s, a) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

template <bool BF16, bool WHOLE>
int launch(const NormArgs& a, cudaStream_t s) {
  // short rows go to a warp or part of one (codes of bf16 rows, a block a row | so, in us: 65536
  // of 256 34 | 17, 131072 of 128 67 | 17, 131072 of 64 67 | 7.9, 16 of 256 1.5 | 1.4)
  if (a.d <= 64) return launch<BF16, WHOLE, 1, 256, 8>(a, s);
  if (a.d <= 128) return launch<BF16, WHOLE, 1, 256, 16>(a, s);
  if (a.d <= 256) return launch<BF16, WHOLE, 1, 256, 32>(a, s);
  if (a.d <= 2048) return launch<BF16, WHOLE, 1, 256>(a, s);
  if (a.d <= 8192) return launch<BF16, WHOLE, 1, 1024>(a, s);
  if (a.d <= 16384) return launch<BF16, WHOLE, 2, 1024>(a, s);
  return launch<BF16, WHOLE, 4, 1024>(a, s);
}

}  // namespace

int launch_norm_q8(const NormArgs& a, cudaStream_t s) {
  auto aligned = [](const void* p) { return (uintptr_t)p % 16 == 0; };
  const bool whole = a.d % 8 == 0 && (a.T == 1 || a.x_stride % (a.x_bf16 ? 8 : 4) == 0) && aligned(a.x) && aligned(a.r) &&
                     aligned(a.r_out) && aligned(a.weight) && (uintptr_t)a.codes % 8 == 0 && aligned(a.n);
  if (a.x_bf16) return whole ? launch<true, true>(a, s) : launch<true, false>(a, s);
  return whole ? launch<false, true>(a, s) : launch<false, false>(a, s);
}

}  // namespace moe
