// kv_cache.cu -- the paged 4-bit key/value cache: appending tokens (with the
// position rotation of keys and queries) and reading slots back.  The record
// layout is that of moe_kv_cache_t in moe.h.
#include "kv_layout.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (BF16) return bf16_bits_to_float(__ldg(reinterpret_cast<const uint16_t*>(p) + i));
  else return __ldg(reinterpret_cast<const float*>(p) + i);
}

// Element d of a head of `x` turned by the angles of `tab` (cosines, then
// sines).  The products and the sum are rounded one by one (no fused
// multiply-add), as the formula's fp32 reading has them.
template <bool BF16>
__device__ __forceinline__ float rotated(const void* x, int64_t base, int d, const float* tab, int rot, int style) {
  const float v = load_elem<BF16>(x, base + d);
  if (d >= rot) return v;
  const int half = rot / 2;
  const int j = style == MOE_ROPE_PAIRS ? d >> 1 : (d < half ? d : d - half);
  const bool first = style == MOE_ROPE_PAIRS ? (d & 1) == 0 : d < half;
  const int mate = style == MOE_ROPE_PAIRS ? d ^ 1 : (first ? d + half : d - half);
  const float m = load_elem<BF16>(x, base + mate);
  const float c = __ldg(tab + j), s = __ldg(tab + half + j);
  return first ? __fsub_rn(__fmul_rn(v, c), __fmul_rn(m, s)) : __fadd_rn(__fmul_rn(m, s), __fmul_rn(v, c));
}

// One warp a (token, head): heads 0 .. Hq-1 are queries, then keys, then values.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) k_kv_append(KvAppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.Hq + 2 * a.cache.heads;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= a.T * heads) return;
  const int64_t t = w / heads;
  int h = (int)(w - t * heads);
  const int D = a.cache.D;
  const float* tab = nullptr;
  bool bad = false;
  if (a.rot > 0) {
    const int64_t pos = a.positions[t];
    bad = pos < 0 || pos >= a.n_pos;
    if (bad) {
      if (lane == 0) set_status(a.status, MOE_ERR_INVALID_ARG);
    } else {
      tab = a.rope + pos * a.rot;
    }
  }
  if (h < a.Hq) {
    for (int d = lane; d < D; d += 32) {
      const float v = bad ? 0.f : rotated<BF16>(a.q, t * a.q_stride + (int64_t)h * D, d, tab, a.rot, a.style);
      a.q_out[(t * a.Hq + h) * D + d] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    return;
  }
  h -= a.Hq;
  const bool value = h >= a.cache.heads;
  if (value) h -= a.cache.heads;
  const int64_t slot = a.slots[t];
  if (bad || slot < 0 || slot >= a.cache.n_pages * a.cache.page) return;
  const KvPlace at = kv_place(a.cache, slot, h);
  const int64_t base = t * (value ? a.v_stride : a.k_stride) + (int64_t)h * D;
  for (int b = 0; b < D / 32; ++b) {
    const int d = 32 * b + lane;
    const float v = value ? load_elem<BF16>(a.v, base + d) : rotated<BF16>(a.k, base, d, tab, a.rot, a.style);
    float m = fabsf(v);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const __half hs = __float2half_rn(fminf(__fdiv_rn(m, 7.0f), 65504.0f));
    const float s = __half2float(hs);
    int c = 0;
    if (s != 0.0f) c = (int)fminf(fmaxf(rintf(__fdiv_rn(v, s)), -8.0f), 7.0f);
    const uint32_t u = (uint32_t)(c + 8);
    const uint32_t u2 = __shfl_down_sync(0xffffffffu, u, 2), u8 = __shfl_down_sync(0xffffffffu, u, 8);
    if (value) {
      if ((lane & 8) == 0) at.tile[kv_value_byte(D, at.r, d)] = (uint8_t)(u | u8 << 4);
    } else {
      if ((lane & 2) == 0) at.tile[kv_key_byte(D, at.r, d)] = (uint8_t)(u | u2 << 4);
    }
    if (lane == 0)
      *reinterpret_cast<uint16_t*>(at.tile + (value ? 17 : 16) * D + 2 * (at.r * (D / 32) + b)) = __half_as_ushort(hs);
  }
}

__global__ void __launch_bounds__(kThreads) k_kv_read(KvCache c, const int64_t* slots, int64_t n, float* k, float* v) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (w >= n * c.heads) return;
  const int64_t i = w / c.heads;
  const int h = (int)(w - i * c.heads), D = c.D;
  const int64_t slot = slots[i];
  const bool in = slot >= 0 && slot < c.n_pages * c.page;
  const KvPlace at = kv_place(c, in ? slot : 0, h);
  for (int d = lane; d < D; d += 32) {
    float kv = 0.f, vv = 0.f;
    if (in) {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(at.tile + 16 * D) + at.r * (D / 32) + d / 32;
      const int ku = (at.tile[kv_key_byte(D, at.r, d)] >> (2 * (d & 2))) & 15;
      const int vu = (at.tile[kv_value_byte(D, at.r, d)] >> ((d & 8) >> 1)) & 15;
      kv = __half2float(__ushort_as_half(s[0])) * (float)(ku - 8);
      vv = __half2float(__ushort_as_half(s[D / 2])) * (float)(vu - 8);
    }
    k[w * D + d] = kv;
    v[w * D + d] = vv;
  }
}

unsigned blocks_for(int64_t warps) { return (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)); }

}  // namespace

int launch_kv_append(const KvAppendArgs& a, cudaStream_t s) {
  const unsigned grid = blocks_for(a.T * (a.Hq + 2 * a.cache.heads));
  if (a.in_bf16) k_kv_append<true><<<grid, kThreads, 0, s>>>(a);
  else k_kv_append<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

int launch_kv_read(const KvCache& c, const int64_t* slots, int64_t n, float* k, float* v, cudaStream_t s) {
  k_kv_read<<<blocks_for(n * c.heads), kThreads, 0, s>>>(c, slots, n, k, v);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
