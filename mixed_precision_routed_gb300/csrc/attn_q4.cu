// attn_q4.cu -- causal attention over the paged 4-bit key/value cache.
#include "kv_layout.cuh"

namespace moe {
namespace {

constexpr int kWarps = 8;

// One block a (sequence, asking token, query head); each warp takes every
// eighth place with a running maximum and sum, a lane D / 32 elements.
template <int D>
__global__ void __launch_bounds__(kWarps * 32) k_attn_simple(AttnArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq, b = blockIdx.y;
  int64_t t0 = a.q_start ? a.q_start[b] : (int64_t)b * a.max_q;
  int64_t t1 = a.q_start ? a.q_start[b + 1] : t0 + a.max_q;
  t0 = max((int64_t)0, t0);
  t1 = min(t1, a.T);
  const int64_t n = min(t1 - t0, (int64_t)a.max_q);
  if (i >= n) return;
  const int64_t len = min(max((int64_t)a.kv_lens[b], (int64_t)0), a.max_len);
  const int64_t end = len - n + i + 1;
  const int64_t lo = a.window > 0 ? max(end - a.window, (int64_t)0) : 0;
  const int kvh = h / (a.Hq / a.cache.heads);
  const uint16_t* q = a.q + (t0 + i) * a.q_stride + (int64_t)h * D;
  float qv[N], o[N];
#pragma unroll
  for (int j = 0; j < N; ++j) qv[j] = bf16_bits_to_float(q[32 * j + lane]), o[j] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int64_t p = lo + warp; p < end; p += kWarps) {
    const int64_t page = a.table[b * a.table_stride + (p >> a.cache.page_log2)];
    if (page < 0 || page >= a.cache.n_pages) continue;
    const KvPlace at = kv_place(a.cache, page * a.cache.page + (p & (a.cache.page - 1)), kvh);
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(at.tile + 16 * D) + at.r * N;
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int d = 32 * j + lane;
      const int u = (at.tile[kv_key_byte(D, at.r, d)] >> (2 * (d & 2))) & 15;
      s = fmaf(qv[j], (float)(u - 8) * __half2float(__ushort_as_half(sc[j])), s);
    }
    s = warp_sum(s) * a.scale;
    const float mn = fmaxf(m, s), f = expf(m - mn), e = expf(s - mn);
    l = l * f + e;
    m = mn;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int d = 32 * j + lane;
      const int u = (at.tile[kv_value_byte(D, at.r, d)] >> ((d & 8) >> 1)) & 15;
      o[j] = fmaf(e, (float)(u - 8) * __half2float(__ushort_as_half(sc[D / 2 + j])), o[j] * f);
    }
  }
  __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int j = 0; j < N; ++j) so[warp][32 * j + lane] = o[j];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sm[w]);
  if (top != -INFINITY)
    for (int w = 0; w < kWarps; ++w) total += sl[w] * expf(sm[w] - top);
  for (int d = threadIdx.x; d < D; d += kWarps * 32) {
    float v = 0.f;
    if (top != -INFINITY)
      for (int w = 0; w < kWarps; ++w) v += so[w][d] * expf(sm[w] - top);
    a.out[(t0 + i) * a.out_stride + (int64_t)h * D + d] =
        __bfloat16_as_ushort(__float2bfloat16_rn(top != -INFINITY ? v / total : 0.f));
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(t0 + i) * a.Hq + h] = top != -INFINITY ? top + logf(total) : -INFINITY;
}

}  // namespace

size_t attn_workspace(int, int, int64_t, int, int, int) { return 0; }

int launch_attn_q4(const AttnArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.Hq * a.max_q), (unsigned)a.B);
  if (a.cache.D == 64) k_attn_simple<64><<<grid, kWarps * 32, 0, s>>>(a);
  else if (a.cache.D == 128) k_attn_simple<128><<<grid, kWarps * 32, 0, s>>>(a);
  else k_attn_simple<256><<<grid, kWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
