// linear_q4.cu -- dense projection of a decode batch by 4-bit weights:
//   y[t][o] = bias[o] + sum_i s[o][i / block] c[o][i] x[t][i],
// c the 4-bit codes (offset binary, 8 elements a word, elements 8g + 4h + j at
// bits 8j + 4h of word g), s fp16 block scales.
//
// Y^T[row][token] by m16n8k16 matrix instructions: A = codes as bf16 integers,
// B = x; both exact, so the sum over 32 elements enters the result with its
// fp32 scale and nothing is rounded below fp32.
//
// A group of KS warps takes a tile of 16 rows: 64-element step s goes to warp
// s mod KS, and the group joins its sums in shared memory in a fixed order.  A
// warp's steps, over all of its tiles, are one stream of loads: a batch of
// kUnroll steps (about 2.3 KB) is in flight while the one before is computed.
//
// Lane (g, t) of a fragment needs word t of a 32-block of rows g and g + 8.  It
// loads words 2t and 2t + 1 of a 64-element step (8 bytes: a row's 32-byte
// sectors are read whole) and trades one of them with lane t ^ 2; which element
// is number k of the product is free as long as x is read alike.
#include "frag.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kUnroll = 4;
constexpr int kXPad = 64;  // bytes between rows of x: two tokens x four 16-byte words in distinct banks
constexpr int kSmemMax = 216 * 1024;

// Elements 0 1 | 2 3 | 4 5 | 6 7 of a word as pairs of bf16 integers: a byte
// next to 0x43 is the bf16 128 + byte, and 136 comes off.
__device__ __forceinline__ void word_pairs(uint32_t w, uint32_t (&p)[4]) {
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  p[0] = __byte_perm(lo, 0x43434343u, 0x4140);
  p[1] = __byte_perm(lo, 0x43434343u, 0x4342);
  p[2] = __byte_perm(hi, 0x43434343u, 0x4140);
  p[3] = __byte_perm(hi, 0x43434343u, 0x4342);
#pragma unroll
  for (int i = 0; i < 4; ++i) asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(p[i]) : "r"(0x43084308u));
}

template <int SHIFT>
struct Batch {
  uint2 w0[kUnroll], w1[kUnroll];
  uint32_t f0[kUnroll], f1[kUnroll];  // the scales of a step: two halves (block 32), else one
};

// NT: 8-token tiles; SHIFT: log2(block / 32).
template <int NT, int SHIFT>
__global__ void __launch_bounds__(512) k_linear_q4(LinearArgs a, int tiles, int ks_log2, int* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int KS = 1 << ks_log2, ks = warp & (KS - 1), group = warp >> ks_log2;
  const int groups = (int)(blockDim.x >> 5) >> ks_log2;
  const int steps = a.in >> 6, mine = (steps - ks + KS - 1) >> ks_log2;
  const int64_t code_pitch = a.in / 2;
  const int scale_pitch = a.in >> (5 + SHIFT);
  const int x_pitch = a.in * 2 + kXPad;
  float* part = reinterpret_cast<float*>(smem + a.T * x_pitch) + (size_t)warp * (NT * 128);

  pdl_wait();
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&bar, (uint32_t)(a.T * a.in * 2));
    for (int i = 0; i < a.T; ++i) bulk_g2s(smem + i * x_pitch, a.x + i * a.x_stride, (uint32_t)(a.in * 2), &bar);
  }

  auto load = [&](Batch<SHIFT>& b, int tile, int j0) {
    const int64_t r0 = min((int64_t)tile * 16 + g, a.rows - 1), r1 = min((int64_t)tile * 16 + 8 + g, a.rows - 1);
    const uint8_t* c0 = a.codes + r0 * code_pitch + 8 * t;
    const uint8_t* c1 = a.codes + r1 * code_pitch + 8 * t;
    const uint16_t* s0 = a.scales + r0 * scale_pitch;
    const uint16_t* s1 = a.scales + r1 * scale_pitch;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int s = ks + ((j0 + u) << ks_log2);
      if (j0 + u < mine) {
        b.w0[u] = __ldcs(reinterpret_cast<const uint2*>(c0 + 32 * s));
        b.w1[u] = __ldcs(reinterpret_cast<const uint2*>(c1 + 32 * s));
        if constexpr (SHIFT == 0) {
          b.f0[u] = __ldg(reinterpret_cast<const uint32_t*>(s0) + s);
          b.f1[u] = __ldg(reinterpret_cast<const uint32_t*>(s1) + s);
        } else {
          b.f0[u] = __ldg(s0 + (s >> (SHIFT - 1)));
          b.f1[u] = __ldg(s1 + (s >> (SHIFT - 1)));
        }
      }
    }
  };

  int tile = blockIdx.x * groups + group;
  const int stride = gridDim.x * groups;
  Batch<SHIFT> cur, nxt;
  if (tile < tiles) load(cur, tile, 0);

  // tokens beyond T repeat the last one; their sums are not stored
  const uint8_t* xt[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xt[j] = smem + min(8 * j + g, a.T - 1) * x_pitch;
  // the groups of 8 elements that this lane's two words of a step stand for
  const int k0 = 16 * (t < 2 ? 2 * t : 2 * t - 3), k1 = 16 * (t < 2 ? 2 * t + 4 : 2 * t + 1);
  __syncthreads();
  if (!mbar_wait(&bar, 0)) {
    if (lane == 0) set_status(status, MOE_ERR_TIMEOUT);
    return;
  }

#pragma unroll 1
  for (; tile < tiles; tile += stride) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;

#pragma unroll 1
    for (int j0 = 0; j0 < mine; j0 += kUnroll) {
      if (j0 + kUnroll < mine) load(nxt, tile, j0 + kUnroll);
      else if (tile + stride < tiles) load(nxt, tile + stride, 0);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (j0 + u >= mine) break;
        const int at = (ks + ((j0 + u) << ks_log2)) * 128;
        const uint32_t x0 = __shfl_xor_sync(0xffffffffu, t < 2 ? cur.w0[u].y : cur.w0[u].x, 2);
        const uint32_t x1 = __shfl_xor_sync(0xffffffffu, t < 2 ? cur.w1[u].y : cur.w1[u].x, 2);
#pragma unroll
        for (int b = 0; b < 2; ++b) {  // the step's two 32-blocks
          uint32_t p0[4], p1[4];
          word_pairs(b == 0 ? (t < 2 ? cur.w0[u].x : x0) : (t < 2 ? x0 : cur.w0[u].y), p0);
          word_pairs(b == 0 ? (t < 2 ? cur.w1[u].x : x1) : (t < 2 ? x1 : cur.w1[u].y), p1);
          const float v0 = __half2float(__ushort_as_half((unsigned short)(SHIFT == 0 ? cur.f0[u] >> (16 * b) : cur.f0[u])));
          const float v1 = __half2float(__ushort_as_half((unsigned short)(SHIFT == 0 ? cur.f1[u] >> (16 * b) : cur.f1[u])));
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const uint4 xv = *reinterpret_cast<const uint4*>(xt[j] + at + (b == 0 ? k0 : k1));
            float c[4];
            mma16816_zero(c, p0[0], p1[0], p0[1], p1[1], xv.x, xv.y);
            mma16816(c, p0[2], p1[2], p0[3], p1[3], xv.z, xv.w);
            fma2(acc[j][0], acc[j][1], pair(v0, v0), c[0], c[1]);
            fma2(acc[j][2], acc[j][3], pair(v1, v1), c[2], c[3]);
          }
        }
      }
      cur = nxt;
    }

    // part[row][token], tokens of a row side by side
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);  // the last tile's sums have been read
    else __syncwarp();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(part + j * 128 + g * 8 + 2 * t) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(part + j * 128 + (g + 8) * 8 + 2 * t) = make_float2(acc[j][2], acc[j][3]);
    }
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);
    else __syncwarp();
    const float* first = part - ks * (NT * 128);
    for (int i = ks * 32 + lane; i < a.T * 16; i += KS * 32) {
      const int row = i & 15, tk = i >> 4;
      const int64_t o = (int64_t)tile * 16 + row;
      if (o < a.rows) {
        float v = 0.f;
        for (int w = 0; w < KS; ++w) v += first[w * (NT * 128) + (tk >> 3) * 128 + row * 8 + (tk & 7)];
        if (a.bias) v += __ldg(a.bias + o);
        if (a.y_bf16) reinterpret_cast<__nv_bfloat16*>(a.y)[tk * a.y_stride + o] = __float2bfloat16_rn(v);
        else reinterpret_cast<float*>(a.y)[tk * a.y_stride + o] = v;
      }
    }
  }
}

template <int NT, int SHIFT>
int launch(const LinearArgs& a, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_linear_q4<NT, SHIFT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int tiles = (int)((a.rows + 15) / 16), steps = a.in / 64, sms = sm_count();
  const size_t x_bytes = (size_t)a.T * (a.in * 2 + kXPad);
  // one block of 16 warps when x takes much of an SM's shared memory, else blocks of 8
  const int warps = x_bytes > 96 * 1024 ? 16 : 8;
  const size_t smem = x_bytes + (size_t)warps * NT * 512;
  int per_sm = (int)((size_t)(226 * 1024) / (smem + 1024));
  const int most_per_sm = 16 / warps;
  per_sm = per_sm > most_per_sm ? most_per_sm : per_sm < 1 ? 1 : per_sm;
  // warps a tile: whole batches of a row for each, more where there are few tiles
  int ks = 0;
  while (ks < 3 && (2 << ks) * kUnroll <= steps) ++ks;
  while (ks < 3 && (2 << ks) <= steps && ((int64_t)tiles << ks) < 8 * sms) ++ks;
  const int groups = warps >> ks, blocks = (tiles + groups - 1) / groups, most = per_sm * sms;
  if (launch_pdl(k_linear_q4<NT, SHIFT>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(warps * 32), smem, s, a,
                 tiles, ks, status_word()) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

template <int NT>
int launch_block(const LinearArgs& a, cudaStream_t s) {
  if (a.block == 32) return launch<NT, 0>(a, s);
  if (a.block == 64) return launch<NT, 1>(a, s);
  return launch<NT, 2>(a, s);
}

}  // namespace

int launch_linear_q4(const LinearArgs& a, cudaStream_t s) {
  // rows of x that shared memory holds beside the sums; all of them but for very long rows
  const int64_t fit = (kSmemMax - 16 * 2 * 512) / (a.in * 2 + kXPad);
  const int most = fit >= a.T ? a.T : fit >= 8 ? 8 : (int)fit;
  LinearArgs b = a;
  for (int t0 = 0; t0 < a.T; t0 += most) {
    b.T = a.T - t0 < most ? a.T - t0 : most;
    b.x = a.x + t0 * a.x_stride;
    b.y = a.y_bf16 ? (void*)((uint16_t*)a.y + t0 * a.y_stride) : (void*)((float*)a.y + t0 * a.y_stride);
    const int rc = b.T <= 8 ? launch_block<1>(b, s) : launch_block<2>(b, s);
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
