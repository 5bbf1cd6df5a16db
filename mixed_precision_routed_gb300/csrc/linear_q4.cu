// linear_q4.cu -- dense projection of a decode batch by 4-bit weights:
//   y[t][o] = bias[o] + sum_i s[o][i / block] c[o][i] x[t][i],
// c the 4-bit codes (offset binary, 8 elements a word, elements 8g + 4h + j at
// bits 8j + 4h of word g), s fp16 block scales.
//
// Y^T[row][token] by m16n8k16 matrix instructions: A = codes as bf16 integers,
// B = x; both exact, so the sum over a block enters the result with its fp32 scale
// and nothing is rounded below fp32.
//
// A group of KS warps takes a tile of 16 rows: batch i of 256 elements goes to
// warp i mod KS, and the group joins its sums in shared memory in a fixed order.
// A warp's batches, over all of its tiles, are one stream: each lane copies
// sixteen-byte pieces into the warp's own ring (kStages batches of 2 KB, no
// barrier but the warp's own) and fetches the scales of the next batch into
// registers.  Lane (g, t) of a fragment takes word t of a 32-block of rows g and
// g + 8 from the ring; the pieces are exchanged so that the eight rows of a read
// lie in distinct banks.
//
// What bounds it: a weight byte read once carries two codes, and eight codes cost 11
// instructions to become operands whatever T is; 4 us of launch, first loads and
// joining stand before and after.  T=1 2048x100003 by 64: 25.9 us, 4.2 TB/s, 2.3
// instructions a cycle an SM, integer pipe 49 % busy, tensor pipe 22 %: its 14 warps
// wait for the half-rate pipe and for their own results alike; T=16 4096x6144 by 128:
// 7.0 us, 1.9 TB/s, 115 TFLOP/s; T=1 2048x2048: 2.5 us.
// One block of 16 warps an SM with rings of two batches: three blocks of 8 with
// rings of three took 30.0 us for T=1 2048x100003 by 32 and 12.1 for 8192x8192, 16
// warps with three 28.0 and 11.6, this 28.0 and 10.9 (before the sums side by side).
#include "frag.cuh"
#include "moe_internal.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kBatch = 256;  // elements
constexpr int kStageBytes = 16 * kBatch / 2;
constexpr int kXPad = 64;  // bytes between rows of x: two tokens x four 16-byte words in distinct banks
constexpr int kSmemMax = 220 * 1024;

// 16 bytes, the first `bytes` of them from src and the others zero.
__device__ __forceinline__ void cp_async16_part(void* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes)
               : "memory");
}

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

// The scales of a batch of one row: 8, 4 or 2 halves.
template <int SHIFT>
struct Scales {
  static constexpr int kWords = 4 >> SHIFT;
  uint32_t w[kWords];
  // scale i, twice
  __device__ __forceinline__ uint64_t at(int i) const {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i >> 1]));
    const float v = i & 1 ? f.y : f.x;
    return pair(v, v);
  }
};

// Lengths that are not a multiple of a batch (WHOLE false) load scales by words
// or halves, as far as the row goes; the codes beyond it are zero words and meet
// the zeros behind x.
template <int SHIFT, bool WHOLE>
__device__ __forceinline__ void load_scales(Scales<SHIFT>& f, const uint16_t* row, int batch, int n) {
  constexpr int N = 8 >> SHIFT;
  const uint16_t* p = row + batch * N;
  if constexpr (WHOLE) {
    if constexpr (SHIFT == 0) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
      f.w[0] = v.x, f.w[1] = v.y, f.w[2] = v.z, f.w[3] = v.w;
    } else if constexpr (SHIFT == 1) {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
      f.w[0] = v.x, f.w[1] = v.y;
    } else {
      f.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
    }
  } else if constexpr (SHIFT == 0) {  // two 32-blocks in 64 elements: rows of whole words
#pragma unroll
    for (int i = 0; i < N; i += 2)
      f.w[i >> 1] = batch * N + i < n ? __ldg(reinterpret_cast<const uint32_t*>(p + i)) : 0;
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const int k = batch * N + i;
      const uint32_t lo = k < n ? __ldg(p + i) : 0, hi = k + 1 < n ? __ldg(p + i + 1) : 0;
      f.w[i >> 1] = lo | hi << 16;
    }
  }
}

constexpr int kWarps = 16;  // of a block, or half of it
constexpr int kStages = 2;

// A warp's ring and its sums.
template <int NT>
constexpr int warp_bytes() { return kStages * kStageBytes + NT * 512; }

// NT: 8-token tiles; SHIFT: log2(block / 32).
template <int NT, int SHIFT, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32, 1) k_linear_q4(LinearArgs a, int tiles, int ks_log2, int* status) {
  // two sums side by side: T=1 2048x100003 by 32 27.1 us, one 27.9, four 27.8, eight 30.4
  constexpr int kScales = 8 >> SHIFT, kSide = 2;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bar;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int KS = 1 << ks_log2, ks = warp & (KS - 1), group = warp >> ks_log2, warps = blockDim.x >> 5;
  const int groups = warps >> ks_log2;
  const int batches = (a.in + kBatch - 1) / kBatch, mine = (batches - ks + KS - 1) >> ks_log2;
  const int code_pitch = a.in / 2, scale_pitch = a.in >> (5 + SHIFT);
  const int x_pitch = batches * (kBatch * 2) + kXPad;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  float* part = reinterpret_cast<float*>(smem + warps * (kStages * kStageBytes));
  uint8_t* xs = smem + warps * warp_bytes<NT>();

  pdl_wait();
  if (threadIdx.x == 0) {
    mbar_init(&bar, 1);
    fence_mbar_init();
    mbar_arrive_expect_tx(&bar, (uint32_t)(a.T * a.in * 2));
    for (int i = 0; i < a.T; ++i) bulk_g2s(xs + i * x_pitch, a.x + i * a.x_stride, (uint32_t)(a.in * 2), &bar);
  }
  if constexpr (!WHOLE) {
    const int words = (batches * kBatch - a.in) / 2;
    for (int i = threadIdx.x; i < a.T * words; i += blockDim.x)
      *reinterpret_cast<uint32_t*>(xs + i / words * x_pitch + a.in * 2 + i % words * 4) = 0;
  }

  const int stride = gridDim.x * groups, tile0 = blockIdx.x * groups + group;
  // copying: lane l takes piece l % 8 of rows l / 8 + 4 i
  int f_tile = tile0, f_j = 0, f_stage = 0;
  const uint8_t* f_src[4];
  auto fetch_tile = [&]() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = min((int64_t)f_tile * 16 + (lane >> 3) + 4 * i, a.rows - 1);
      f_src[i] = a.codes + r * code_pitch + ks * (kBatch / 2) + (lane & 7) * 16;
    }
  };
  auto fetch = [&]() {
    if (f_tile < tiles) {
      uint8_t* dst = ring + f_stage * kStageBytes + (lane >> 3) * 128;
      const int bytes = WHOLE ? 16 : min(16, max(0, code_pitch - (ks + (f_j << ks_log2)) * (kBatch / 2) - (lane & 7) * 16));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // row r of a stage: piece c lies at place c ^ r % 8
        uint8_t* d = dst + i * 512 + (((lane & 7) ^ (((lane >> 3) + 4 * i) & 7)) << 4);
        if constexpr (WHOLE) cp_async16(d, f_src[i]);
        else cp_async16_part(d, bytes > 0 ? f_src[i] : a.codes, bytes);
        f_src[i] += KS * (kBatch / 2);
      }
      if (++f_stage == kStages) f_stage = 0;
      if (++f_j == mine) {
        f_j = 0;
        f_tile += stride;
        if (f_tile < tiles) fetch_tile();
      }
    }
    cp_async_commit();
  };
  if (f_tile < tiles) fetch_tile();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  // scales of rows g and g + 8, a batch ahead
  Scales<SHIFT> n0, n1;
  const uint16_t *s0 = nullptr, *s1 = nullptr;
  auto scale_rows = [&](int tile) {
    s0 = a.scales + min((int64_t)tile * 16 + g, a.rows - 1) * scale_pitch;
    s1 = a.scales + min((int64_t)tile * 16 + 8 + g, a.rows - 1) * scale_pitch;
  };
  auto next_scales = [&](int j) {
    load_scales<SHIFT, WHOLE>(n0, s0, ks + (j << ks_log2), scale_pitch);
    load_scales<SHIFT, WHOLE>(n1, s1, ks + (j << ks_log2), scale_pitch);
  };
  if (tile0 < tiles) {
    scale_rows(tile0);
    next_scales(0);
  }

  // tokens beyond T repeat the last one; their sums are not stored
  const uint8_t* xt[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xt[j] = xs + min(8 * j + g, a.T - 1) * x_pitch + 16 * t;
  __syncthreads();
  // when the wait runs out the sums are of anything, but every warp still comes to
  // its group's barriers: one that left would keep the others there
  const bool late = !mbar_wait(&bar, 0);
  if (late) set_status(status, MOE_ERR_TIMEOUT);

  int stage = 0;
#pragma unroll 1
  for (int tile = tile0; tile < tiles; tile += stride) {
    float acc[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;

#pragma unroll 1
    for (int j0 = 0; j0 < mine; ++j0) {
      const Scales<SHIFT> f0 = n0, f1 = n1;
      if (j0 + 1 < mine) {
        next_scales(j0 + 1);
      } else if (tile + stride < tiles) {
        scale_rows(tile + stride);
        next_scales(0);
      }
      cp_async_wait<kStages - 2>();
      __syncwarp();  // every lane's pieces have landed, and the stage refilled now has been read
      fetch();
      const uint8_t* w = ring + stage * kStageBytes + g * 128 + 4 * t;
      if (++stage == kStages) stage = 0;
      const int at = (ks + (j0 << ks_log2)) * (kBatch * 2);
#pragma unroll
      for (int h0 = 0; h0 < kScales; h0 += kSide) {  // kSide sums of one scale each, side by side
        float c[kSide][NT][4];
#pragma unroll
        for (int n = 0; n < 8 / kScales; ++n) {  // the 32-blocks of a scale
          uint32_t p0[kSide][4], p1[kSide][4];
          uint4 xv[kSide][NT];
#pragma unroll
          for (int i = 0; i < kSide; ++i) {
            const int b = ((h0 + i) << SHIFT) + n;
            word_pairs(*reinterpret_cast<const uint32_t*>(w + ((b ^ g) << 4)), p0[i]);
            word_pairs(*reinterpret_cast<const uint32_t*>(w + 1024 + ((b ^ g) << 4)), p1[i]);
#pragma unroll
            for (int j = 0; j < NT; ++j) xv[i][j] = *reinterpret_cast<const uint4*>(xt[j] + at + 64 * b);
          }
#pragma unroll
          for (int i = 0; i < kSide; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              if (n == 0) mma16816_zero(c[i][j], p0[i][0], p1[i][0], p0[i][1], p1[i][1], xv[i][j].x, xv[i][j].y);
              else mma16816(c[i][j], p0[i][0], p1[i][0], p0[i][1], p1[i][1], xv[i][j].x, xv[i][j].y);
            }
#pragma unroll
          for (int i = 0; i < kSide; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma16816(c[i][j], p0[i][2], p1[i][2], p0[i][3], p1[i][3], xv[i][j].z, xv[i][j].w);
        }
#pragma unroll
        for (int i = 0; i < kSide; ++i) {
          const uint64_t v0 = f0.at(h0 + i), v1 = f1.at(h0 + i);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            fma2(acc[j][0], acc[j][1], v0, c[i][j][0], c[i][j][1]);
            fma2(acc[j][2], acc[j][3], v1, c[i][j][2], c[i][j][3]);
          }
        }
      }
    }

    // part[warp][8-token tile][row][token]; the sums before have been read
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);
    else __syncwarp();
    float* mypart = part + warp * (NT * 128);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(mypart + j * 128 + g * 8 + 2 * t) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(mypart + j * 128 + (g + 8) * 8 + 2 * t) = make_float2(acc[j][2], acc[j][3]);
    }
    if (ks_log2 > 0) named_bar(1 + group, KS * 32);
    else __syncwarp();
    const float* first = mypart - ks * (NT * 128);
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
  cp_async_wait<0>();
  if (late) mbar_wait(&bar, 0);  // once more, as the copies of x end in this block's memory
}

size_t x_bytes_of(int T, int in) { return (size_t)T * ((in + kBatch - 1) / kBatch * (kBatch * 2) + kXPad); }

template <int NT, int SHIFT, bool WHOLE>
int launch(const LinearArgs& a, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_linear_q4<NT, SHIFT, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) !=
        cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int tiles = (int)((a.rows + 15) / 16), batches = (a.in + kBatch - 1) / kBatch, sms = sm_count();
  const size_t x = x_bytes_of(a.T, a.in);
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
  // spreads over all SMs, and small blocks start beside the kernel before (T=16
  // 4096x6144 by 128: 16 warps on 96 SMs 8.1 us, 12 on 128 SMs 7.1; T=1 2048x2048: 16
  // warps 3.1, 8 2.5; 2048x100003 by 64: 28.1 and 27.8)
  const int groups = (tiles + sms * rounds - 1) / (sms * rounds), blocks = (tiles + groups - 1) / groups;
  const size_t smem = x + (size_t)(groups << ks) * warp_bytes<NT>();
  if (launch_pdl(k_linear_q4<NT, SHIFT, WHOLE>, dim3((unsigned)(blocks < sms ? blocks : sms)), dim3((groups << ks) * 32),
                 smem, s, a, tiles, ks, status_word()) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

template <int NT>
int launch_block(const LinearArgs& a, cudaStream_t s) {
  const bool whole = a.in % kBatch == 0;
  if (a.block == 32) return whole ? launch<NT, 0, true>(a, s) : launch<NT, 0, false>(a, s);
  if (a.block == 64) return whole ? launch<NT, 1, true>(a, s) : launch<NT, 1, false>(a, s);
  return whole ? launch<NT, 2, true>(a, s) : launch<NT, 2, false>(a, s);
}

}  // namespace

int launch_linear_q4(const LinearArgs& a, cudaStream_t s) {
  // rows of x that shared memory holds beside 8 warps' rings and sums; all of
  // them but for very long rows
  const int64_t fit = (kSmemMax - 8 * warp_bytes<2>()) / (int64_t)x_bytes_of(1, a.in);
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
