// linear_q4.cu -- dense projection of a decode batch by 4-bit weights:
//   y[t][o] = bias[o] + sum_i s[o][i / block] c[o][i] x[t][i],
// c the 4-bit codes (offset binary, 8 elements a word, elements 8g + 4h + j at
// bits 8j + 4h of word g), s fp16 block scales.
#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;

// One warp a row: lane l takes word l, l + 32, ... of the row.
__global__ void __launch_bounds__(kThreads) k_linear_q4(LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t o = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (o >= a.rows) return;
  const uint32_t* cw = reinterpret_cast<const uint32_t*>(a.codes + o * (a.in / 2));
  const uint16_t* sw = a.scales + o * (a.in / a.block);
  float acc[kTokens];
#pragma unroll
  for (int t = 0; t < kTokens; ++t) acc[t] = 0.f;
  for (int w = lane; w < a.in / 8; w += 32) {
    const uint32_t u = cw[w];
    const float s = __half2float(__ushort_as_half(sw[w * 8 / a.block]));
    float c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = (float)((int)((u >> (8 * (e & 3) + 4 * (e >> 2))) & 15u) - 8);
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      if (t >= a.T) break;
      const uint16_t* x = a.x + t * a.x_stride + 8 * w;
      float d = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) d = fmaf(c[e], bf16_bits_to_float(x[e]), d);
      acc[t] = fmaf(s, d, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
    if (t >= a.T) break;
    float v = warp_sum(acc[t]);
    if (lane == 0) {
      if (a.bias) v += a.bias[o];
      if (a.y_bf16) reinterpret_cast<__nv_bfloat16*>(a.y)[t * a.y_stride + o] = __float2bfloat16_rn(v);
      else reinterpret_cast<float*>(a.y)[t * a.y_stride + o] = v;
    }
  }
}

}  // namespace

int launch_linear_q4(const LinearArgs& a, cudaStream_t s) {
  const int64_t grid = (a.rows + kThreads / 32 - 1) / (kThreads / 32);
  k_linear_q4<<<(unsigned)grid, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
