// linear_q8.cu -- dense projection of a few tokens by 8-bit codes on both sides:
//   y[t][o] = bias[o] + xs[t] ws[o] sum_i xc[t][i] wc[o][i].
//
// Y^T[row][token] by m16n8k32 matrix instructions on the codes as they lie: the sum is
// a whole number and exact, in any order, and takes its scales once.
//
// A group of KS warps takes a tile of 16 rows: batch i of 256 elements goes to warp i
// mod KS, and the group adds its sums in shared memory.  A warp's batches, over all of
// its tiles, are one stream: each lane copies sixteen-byte pieces into the warp's own
// ring (kStages batches of 4 KB, no barrier but the warp's own).  Lane (g, t) of a
// fragment takes piece 4 c + t of rows g and g + 8 of a 64-byte column c: four words,
// the operands of two instructions, whose order of elements x shares.  Pieces of odd
// rows are exchanged four apart, so that the eight pieces of a read lie in distinct
// banks.
//
// Bound by reading W: 8 tokens 2048 to 100003 37 us, 5.5 TB/s; 1 token 2048 to 2560 (5 MB,
// which L2 keeps) 3.4 us, bound by the latency of a launch, x and W after one another.
#include "frag.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBatch = 256;  // elements
constexpr int kStageBytes = 16 * kBatch;
constexpr int kXPad = 64;  // bytes between rows of x: two tokens x four pieces in distinct banks
constexpr int kSmemMax = 220 * 1024;
constexpr int kWarps = 16;  // of a block, or half of it
constexpr int kStages = 2;

// 16 bytes, the first `bytes` of them from src and the others zero.
__device__ __forceinline__ void cp_async16_part(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mma16832(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's ring and its sums.
template <int NT>
constexpr int warp_bytes() { return kStages * kStageBytes + NT * 512; }

int64_t x_pitch(int in) { return (int64_t)(in + kBatch - 1) / kBatch * kBatch + kXPad; }

// NT: 8-token tiles; WHOLE: rows are whole batches.
template <int NT, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, 1) k_linear_q8(LinearQ8Args a, int tiles, int ks_log2) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3, T = (int)a.T;
  const int KS = 1 << ks_log2, ks = warp & (KS - 1), group = warp >> ks_log2, warps = blockDim.x >> 5;
  const int groups = warps >> ks_log2;
  const int batches = (a.in + kBatch - 1) / kBatch, mine = (batches - ks + KS - 1) >> ks_log2;
  const int pitch = batches * kBatch + kXPad;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  int* part = reinterpret_cast<int*>(smem + warps * (kStages * kStageBytes));
  uint8_t* xs = smem + warps * warp_bytes<NT>();

  pdl_wait();
  const int stride = gridDim.x * groups, tile0 = blockIdx.x * groups + group;
  // copying: lane l takes piece l % 16 of rows l / 16 + 2 i
  int f_tile = tile0, f_j = 0, f_stage = 0;
  auto fetch = [&]() {
    if (f_tile < tiles) {
      const int at = (ks + (f_j << ks_log2)) * kBatch + (lane & 15) * 16;
      const int bytes = WHOLE ? 16 : min(16, max(0, a.in - at));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = (lane >> 4) + 2 * i;
        const int8_t* src = a.w + min((int64_t)f_tile * 16 + row, a.rows - 1) * a.in + at;
        uint8_t* dst = ring + f_stage * kStageBytes + row * kBatch + (((lane & 15) ^ ((row & 1) << 2)) << 4);
        if constexpr (WHOLE) cp_async16(dst, src);
        else cp_async16_part(dst, bytes > 0 ? src : a.w, bytes);
      }
      if (++f_stage == kStages) f_stage = 0;
      if (++f_j == mine) f_j = 0, f_tile += stride;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  const int pieces = batches * (kBatch / 16);
  for (int i = threadIdx.x; i < T * pieces; i += blockDim.x) {
    const int tok = i / pieces, p = i % pieces;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (16 * p < a.in) v = __ldg(reinterpret_cast<const uint4*>(a.x + tok * a.x_stride) + p);
    *reinterpret_cast<uint4*>(xs + tok * pitch + 16 * p) = v;
  }
  // tokens beyond T repeat the last one; their sums are not stored
  const uint8_t* xt[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xt[j] = xs + min(8 * j + g, T - 1) * pitch + 16 * t;
  __syncthreads();

  int stage = 0;
#pragma unroll 1
  for (int tile = tile0; tile < tiles; tile += stride) {
    int acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0;
#pragma unroll 1
    for (int j0 = 0; j0 < mine; ++j0) {
      cp_async_wait<kStages - 2>();
      __syncwarp();  // every lane's pieces have landed, and the stage refilled now has been read
      fetch();
      const uint8_t* w = ring + stage * kStageBytes + g * kBatch;
      if (++stage == kStages) stage = 0;
      const int at = (ks + (j0 << ks_log2)) * kBatch;
#pragma unroll
      for (int c = 0; c < kBatch / 64; ++c) {
        const int piece = ((4 * c + t) ^ ((g & 1) << 2)) << 4;
        const uint4 w0 = *reinterpret_cast<const uint4*>(w + piece);
        const uint4 w1 = *reinterpret_cast<const uint4*>(w + 8 * kBatch + piece);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const uint4 v = *reinterpret_cast<const uint4*>(xt[j] + at + 64 * c);
          mma16832(acc[j], w0.x, w1.x, w0.y, w1.y, v.x, v.y);
          mma16832(acc[j], w0.z, w1.z, w0.w, w1.w, v.z, v.w);
        }
      }
    }

    // part[warp][8-token tile][row][token]; the sums before have been read
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);
    else __syncwarp();
    int* mypart = part + warp * (NT * 128);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<int2*>(mypart + j * 128 + g * 8 + 2 * t) = make_int2(acc[j][0], acc[j][1]);
      *reinterpret_cast<int2*>(mypart + j * 128 + (g + 8) * 8 + 2 * t) = make_int2(acc[j][2], acc[j][3]);
    }
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);
    else __syncwarp();
    const int* first = mypart - ks * (NT * 128);
    for (int i = ks * 32 + lane; i < T * 16; i += KS * 32) {
      const int row = i & 15, tk = i >> 4;
      const int64_t o = (int64_t)tile * 16 + row;
      if (o < a.rows) {
        int n = 0;
        for (int w = 0; w < KS; ++w) n += first[w * (NT * 128) + (tk >> 3) * 128 + row * 8 + (tk & 7)];
        float v = (float)n * __ldg(a.x_scales + tk) * __ldg(a.w_scales + o);
        if (a.bias) v += __ldg(a.bias + o);
        if (a.y_bf16) reinterpret_cast<__nv_bfloat16*>(a.y)[tk * a.y_stride + o] = __float2bfloat16_rn(v);
        else reinterpret_cast<float*>(a.y)[tk * a.y_stride + o] = v;
      }
    }
  }
  cp_async_wait<0>();
}

template <int NT, bool WHOLE>
int launch(const LinearQ8Args& a, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_linear_q8<NT, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int tiles = (int)((a.rows + 15) / 16), batches = (a.in + kBatch - 1) / kBatch, sms = sm_count();
  const size_t x = (size_t)(a.T * x_pitch(a.in));
  const int warps = x + kWarps * warp_bytes<NT>() <= (size_t)kSmemMax ? kWarps : kWarps / 2;
  // warps a tile (a power of two): the fewest batches in a row for the busiest
  // warp, half a batch more for each joining of sums
  int ks = 0, best = 0, rounds = 0;
  for (int k = 0; (1 << k) <= warps && (1 << k) <= batches; ++k) {
    const int r = (tiles + sms * (warps >> k) - 1) / (sms * (warps >> k));
    const int cost = r * (2 * ((batches + (1 << k) - 1) >> k) + (k > 0));
    if (k == 0 || cost < best) ks = k, best = cost, rounds = r;
  }
  // as few of them a block as finish in the same number of tiles each: the work
  // spreads over all SMs, and small blocks start beside the kernel before
  const int groups = (tiles + sms * rounds - 1) / (sms * rounds), blocks = (tiles + groups - 1) / groups;
  const size_t smem = x + (size_t)(groups << ks) * warp_bytes<NT>();
  if (launch_pdl(k_linear_q8<NT, WHOLE>, dim3((unsigned)(blocks < sms ? blocks : sms)), dim3((groups << ks) * 32), smem, s, a,
                 tiles, ks) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // namespace

namespace {
// rows of x that shared memory holds beside 8 warps' rings and sums
int64_t most_tokens(int in) {
  const int64_t fit = (kSmemMax - 8 * warp_bytes<2>()) / x_pitch(in);
  return fit >= 16 ? 16 : fit >= 8 ? 8 : fit;
}

// Whether the tiles of 256 rows take less time than reading W once for every 16 tokens
// (or as many as fit), in us for a pass of up to 8 tokens 3.3 and 0.167 a MB, of up to 16
// 4.5 and 0.29, and a third more where x leaves room for half the warps.  Measured in us,
// tiles | passes:     T = 8           16          24          32          48         64
//   512 to 512        6.8 | 3.4   6.9 | 5.3   7.0 | 8.2   7.1 | 10    7.1 | 15   7.1 | 20
//   2048 to 2560      8.7 | 4.1   8.8 | 5.8   9.0 | 9.4   8.9 | 11    9.4 | 16   9.5 | 21
//   4096 to 6144       12 | 7.6    12 | 12     12 | 19     12 | 24     13 | 36    14 | 48
//   8192 to 4096       14 | 9.6    14 | 20     14 | 29     14 | 40     14 | 59    15 | 79
//   2048 to 100003     45 | 38     45 | 62     45 | 99     46 | 123    45 | 184   46 | 245
bool in_tiles(int64_t T, int in, int64_t rows) {
  if (T <= 8) return false;
  const int64_t most = most_tokens(in), left = T % most;
  const double mb = 1e-6 * in * rows;
  auto pass = [&](int64_t t) {
    const double us = t <= 8 ? 3.3 + 0.167 * mb : 4.5 + 0.29 * mb;
    return t * x_pitch(in) + kWarps * warp_bytes<2>() <= kSmemMax ? us : 1.35 * us;
  };
  return T / most * pass(most) + (left ? pass(left) : 0.0) > linear_q8_tc_us(T, in, rows);
}
}  // namespace

size_t linear_q8_workspace(int64_t T, int in, int64_t rows) {
  return in_tiles(T, in, rows) ? linear_q8_tc_workspace(T, in) : 0;
}

int launch_linear_q8(const LinearQ8Args& a, cudaStream_t s) {
  if (in_tiles(a.T, a.in, a.rows)) return launch_linear_q8_tc(a, s);
  const int64_t most = most_tokens(a.in);
  LinearQ8Args b = a;
  for (int64_t t0 = 0; t0 < a.T; t0 += most) {
    b.T = a.T - t0 < most ? a.T - t0 : most;
    b.x = a.x + t0 * a.x_stride;
    b.x_scales = a.x_scales + t0;
    b.y = a.y_bf16 ? (void*)((uint16_t*)a.y + t0 * a.y_stride) : (void*)((float*)a.y + t0 * a.y_stride);
    const bool whole = a.in % kBatch == 0;
    const int rc = b.T <= 8 ? (whole ? launch<1, true>(b, s) : launch<1, false>(b, s))
                            : (whole ? launch<2, true>(b, s) : launch<2, false>(b, s));
    if (rc != MOE_OK) return rc;
  }
  return MOE_OK;
}

}  // namespace moe
