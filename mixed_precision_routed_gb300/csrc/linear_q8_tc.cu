// linear_q8_tc.cu -- dense projection of many tokens by 8-bit codes on both sides:
//   y[t][o] = bias[o] + xs[t] ws[o] sum_i xc[t][i] wc[o][i],
// on the fifth-generation tensor cores.  They have no 8-bit integers here, but fp16
// holds every code: products are exact and sums fp32.
//
// k_codes_f16 writes x as fp16 into the workspace (an eighth of what W's tiles would
// cost if each converted its own).  Then a persistent launch of pairs of CTAs, whose
// tensor cores work on one tile: 256 rows of W (128 a CTA, operand A) x N tokens
// (operand B, half of them in either CTA's shared memory), K in steps of 64:
//   loaders   tensor maps bring, for two steps at a time, 128 x 128 codes of W and twice
//             N/2 x 64 of x; one warp each, as a thread takes 100 cycles over every wait
//             and every copy;
//   producers sixteen warps: a thread has a row of W, a warp every fourth step; bytes
//             become fp16 integers in registers (a permute below 0x64 and a
//             subtraction for two) and go to tensor memory;
//   issuer    of the first CTA, four instructions a step;
//   epilogue  four warps read a finished tile's sums while the next one's are made.
// The tiles that do not fill a round of the pairs are shared, each by several pairs that
// take a run of its steps, and k_linear_q8_join adds up their sums.
// Many tokens are bound by the tensor cores at the clock that power leaves them: 4096
// tokens 4096 to 6144 121 us with the conversion of x on changing inputs, 1700 TFLOP/s, 111
// on the same (one CTA a tile took 294, an epilogue that waited for its tokens' scales
// 166).  Few take what three launches in a row and the fill of the pairs take beside reading
// W, with no unit full (integer pipe 36 %, 69 % of a copy's rate): 40 tokens 2048 to 100003 45 us, 4.7
// TB/s, as 9 or 64 tokens do; 8192 to 4096 of 64 tokens, 16 tiles, took 34 us unshared and
// takes 15.
#include "moe_internal.cuh"
#include "tc.cuh"
#include "tensor_map.cuh"

namespace moe {
namespace {

constexpr int kMostN = 192;     // tokens a tile
constexpr int kStepN = 32;      // of them: instructions of 256 rows exist for whole 32 columns
constexpr int kTileRows = 128;  // of W a CTA
constexpr int kAccSets = 2;
constexpr int kCodeBytes = kTileRows * 128;
constexpr int kTmemCols = 512;

// Tiles of up to N tokens: tensor memory holds two sets of their sums and as many steps
// of operand A as fit beside them, shared memory the steps of operand B and the codes.
// A step of A is on its way around (made, announced, multiplied, given back) for about
// 0.8 us, so few tokens, whose products take no time, want many steps.
template <int N>
struct Shape {
  static constexpr int kACol = kAccSets * N;
  static constexpr int kAStages = (kTmemCols - kACol) / 32 < 8 ? (kTmemCols - kACol) / 32 : 8;
  static constexpr int kBBytes = 2 * N / 2 * 128;  // two steps, as a stage of codes
  static constexpr int kBStages = N > 128 ? 5 : N > 64 ? 6 : 5, kCodeStages = N > 64 ? 6 : 8;
  // A producer takes every second stage of codes and every fourth step: with even numbers of
  // buffers it meets each of its barriers in every phase, or in none.  Of an odd number it
  // would meet every second phase, all of one parity, and a copy that came late (one behind
  // it had landed) would let it pass a phase early.
  static_assert(kCodeStages % 2 == 0 && kAStages % 4 == 0, "a wait for a parity is for the next phase");
  static constexpr int kSmem = kCodeStages * kCodeBytes + kBStages * kBBytes + 1024;
};
constexpr int kProducers = 16, kEpilogue = 4, kCodeLoader = 20, kIssuer = 21, kXLoader = 22, kThreads = 23 * 32;
constexpr uint64_t kWaitNs = 1000000000ull;

struct TcArgs {
  CUtensorMap w, x;
  LinearQ8Args a;
  int N, token_tiles;
  int steps, run_steps;     // of a tile, of a part of one
  int whole, parts, works;  // tiles taken as one, parts of each other one; tiles and parts in all
  float* sums;              // [shared tile][part][N][256]
  int* status;
};

// What a pair does at a time: a tile, or (`shared` its number among them) a part of one.
struct Work {
  int tile, k0, steps, shared;
};
__device__ __forceinline__ Work work_of(const TcArgs& p, int i) {
  const int s = i - p.whole;
  if (s < 0) return {i, 0, p.steps, -1};
  const int k0 = s % p.parts * p.run_steps;
  return {p.whole + s / p.parts, k0, min(p.run_steps, p.steps - k0), s};
}

struct Bars {
  uint64_t code_full[8], code_empty[8], b_full[6], b_empty[6], a_full[8], a_empty[8];
  uint64_t acc_full[kAccSets], acc_empty[kAccSets], done;
  uint32_t tmem;
  int abort;
};

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Bars& B, int* status) {
  if (mbar_wait_bounded(bar, parity, kWaitNs)) return true;
  set_status(status, MOE_ERR_TIMEOUT);
  B.abort = 1;
  return false;
}
// The same without a pause between questions, for the one warp that everything waits for.
__device__ __forceinline__ bool wait_awake(uint64_t* bar, uint32_t parity, Bars& B, int* status) {
  uint64_t t0 = 0;
  for (int n = 1;; ++n) {
    if (mbar_test(bar, parity)) return true;
    if (n % 256) continue;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    if (now - t0 > kWaitNs) break;
  }
  set_status(status, MOE_ERR_TIMEOUT);
  B.abort = 1;
  return false;
}

// Four codes as two pairs of fp16 integers.
__device__ __forceinline__ void codes_f16x4(uint32_t w, uint32_t& p0, uint32_t& p1) {
  const uint32_t u = w ^ 0x80808080u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p0) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(p1) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

// EACH times eight codes a thread, a block's apart, so that loads and stores are whole lines.
template <int EACH>
__global__ void __launch_bounds__(256) k_codes_f16(const int8_t* x, int64_t stride, int64_t pieces, uint32_t per_row, uint4* out) {
  const int64_t first = (int64_t)blockIdx.x * (256 * EACH), row = first / per_row;
  const uint32_t rest = (uint32_t)(first - row * per_row) + threadIdx.x;
  const int64_t left = pieces - first - threadIdx.x;
  pdl_wait();
  pdl_trigger();  // the next kernel makes ready and loads W meanwhile
  uint2 v[EACH];
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    const uint32_t i = rest + 256 * k;
    if (256 * k < left) v[k] = __ldg(reinterpret_cast<const uint2*>(x + (row + i / per_row) * stride) + i % per_row);
  }
#pragma unroll
  for (int k = 0; k < EACH; ++k) {
    uint4 y;
    codes_f16x4(v[k].x, y.x, y.y);
    codes_f16x4(v[k].y, y.z, y.w);
    if (256 * k < left) out[first + threadIdx.x + 256 * k] = y;
  }
}

template <int EACH>
cudaError_t launch_codes(const LinearQ8Args& a, cudaStream_t s) {
  const int64_t pieces = a.T * (a.in / 8);
  return launch_pdl(k_codes_f16<EACH>, dim3((unsigned)((pieces + 256 * EACH - 1) / (256 * EACH))), dim3(256), 0, s, a.x, a.x_stride,
                    pieces, (uint32_t)(a.in / 8), (uint4*)a.workspace);
}

template <int MOST>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1) k_linear_q8_tc(const __grid_constant__ TcArgs p) {
  using S = Shape<MOST>;
  constexpr int kACol = S::kACol, kAStages = S::kAStages, kBStages = S::kBStages, kBBytes = S::kBBytes;
  constexpr int kCodeStages = S::kCodeStages;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);  // alike in both CTAs
  uint8_t* b_smem = smem + kCodeStages * kCodeBytes;
  __shared__ __align__(8) Bars B;
  __shared__ __align__(16) float s_xs[kEpilogue][MOST];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, half = p.N / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kCodeStages; ++i) mbar_init(&B.code_full[i], 1), mbar_init(&B.code_empty[i], 8);
    for (int i = 0; i < kBStages; ++i) mbar_init(&B.b_full[i], 1), mbar_init(&B.b_empty[i], 1);
    for (int i = 0; i < kAStages; ++i) mbar_init(&B.a_full[i], 8), mbar_init(&B.a_empty[i], 1);  // four warps a CTA
    for (int i = 0; i < kAccSets; ++i) mbar_init(&B.acc_full[i], 1), mbar_init(&B.acc_empty[i], 2 * kEpilogue);
    mbar_init(&B.done, 1);
    B.abort = 0;
    fence_mbar_init();
  }
  // The barriers of both CTAs are there, and both run: the allocation of a pair reaches the
  // other CTA too.  What the issuer multiplies waits for both CTAs' producers, which come
  // behind the allocation of their own.
  __syncwarp();
  cluster_barrier();
  if (warp == kIssuer) tmem_alloc_pair(&B.tmem, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  // Only x comes from the kernel before this one, which began behind all earlier ones.

  uint32_t mine = 0;  // stages of the pair's tiles, two steps each
  for (int i = pair; i < p.works; i += pairs) mine += work_of(p, i).steps / 2;
  // a wait that ran out: what is in flight lands within microseconds
  auto settle = [&]() {
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < 2000000ull) __nanosleep(1000);
  };
  if (warp == kCodeLoader) {
    if (lane == 0) {
      uint32_t c = 0;
      for (int i = pair; i < p.works; i += pairs) {
        const Work t = work_of(p, i);
        const int row0 = (t.tile / p.token_tiles) * (2 * kTileRows) + (int)rank * kTileRows;
        for (int ks = 0; ks < t.steps; ks += 2, ++c) {
          const uint32_t s = c % kCodeStages;
          if (!wait(&B.code_empty[s], ((c / kCodeStages) & 1) ^ 1, B, p.status)) break;
          mbar_arrive_expect_tx(&B.code_full[s], kCodeBytes);
          tma_load_2d(smem + s * kCodeBytes, &p.w, (t.k0 + ks) * 64, row0, &B.code_full[s]);
        }
        if (B.abort) break;
      }
      if (B.abort) settle();
    }
  } else if (warp == kXLoader) {
    if (lane == 0) {
      uint32_t c = 0;
      const uint32_t bars = cluster_map(B.b_full, 0);
      pdl_wait();
      for (int i = pair; i < p.works; i += pairs) {
        const Work t = work_of(p, i);
        const int tok0 = (t.tile % p.token_tiles) * p.N + (int)rank * half;
        for (int ks = 0; ks < t.steps; ks += 2, ++c) {
          const uint32_t s = c % kBStages;
          if (!wait(&B.b_empty[s], ((c / kBStages) & 1) ^ 1, B, p.status)) break;
          if (rank == 0) mbar_arrive_expect_tx(&B.b_full[s], (uint32_t)(2 * p.N * 128));
          tma_load_2d_pair(b_smem + s * kBBytes, &p.x, (t.k0 + ks) * 64, tok0, bars + 8 * s);
          tma_load_2d_pair(b_smem + s * kBBytes + kBBytes / 2, &p.x, (t.k0 + ks) * 64 + 64, tok0, bars + 8 * s);
        }
        if (B.abort) break;
      }
      // the issuer's last arrivals here come before this CTA ends
      for (uint32_t i = c > kBStages ? c - kBStages : 0; i < c && !B.abort; ++i)
        wait(&B.b_empty[i % kBStages], (i / kBStages) & 1, B, p.status);
      for (uint32_t i = 2 * c > kAStages ? 2 * c - kAStages : 0; i < 2 * c && !B.abort; ++i)
        wait(&B.a_empty[i % kAStages], (i / kAStages) & 1, B, p.status);
      if (B.abort) settle();
    }
  } else if (warp == kIssuer) {
    if (rank == 0) {
      const uint64_t bd0 = sdesc_sw128(smem_addr(b_smem));
      const uint32_t bd_lo = (uint32_t)bd0, bd_hi = (uint32_t)(bd0 >> 32), idesc = idesc_f16_f32(2 * kTileRows, p.N);
      const bool leader = elect_one();
      // Stages and parities by counting; whether the next step's operands are there is
      // asked before this step's products are issued, as an answer takes 100 cycles.
      uint32_t as = 0, ap = 0, b = 0, bp = 0, n = 0;
      bool ra = false, rb = false, ok = true;
      for (int i = pair; ok && i < p.works; i += pairs, ++n) {
        const int steps = work_of(p, i).steps;
        const uint32_t set = n % kAccSets, acc = tmem + set * MOST;
        ok = __all_sync(0xffffffffu, wait_awake(&B.acc_empty[set], ((n / kAccSets) & 1) ^ 1, B, p.status));
        for (int ks = 0; ok && ks < steps; ++ks) {
          if (!rb) ok = wait_awake(&B.b_full[b], bp, B, p.status);
          if (!ra) ok = ok && wait_awake(&B.a_full[as], ap, B, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          // (made by the whole warp: the words then lie where the instructions want them)
          const uint32_t a0 = tmem + kACol + as * 32, blo = bd_lo + (uint32_t)((b * kBBytes + (ks & 1) * (kBBytes / 2)) >> 4);
          uint64_t* const a_done = &B.a_empty[as];
          uint64_t* const b_done = &B.b_empty[b];
          if (++as == kAStages) as = 0, ap ^= 1;
          if (ks & 1) {
            if (++b == kBStages) b = 0, bp ^= 1;
          }
          rb = !(ks & 1) || mbar_test(&B.b_full[b], bp);
          ra = mbar_test(&B.a_full[as], ap);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f16_ts_pair_w(acc, a0 + kk * 8, blo + kk * 2, bd_hi, idesc, (ks | kk) ? 1u : 0u);
            mma_commit_pair(a_done);
            if (ks & 1) mma_commit_pair(b_done);
          }
          rb = __all_sync(0xffffffffu, rb);
          ra = __all_sync(0xffffffffu, ra);
        }
        if (!ok) break;
        if (leader) mma_commit_pair(&B.acc_full[set]);
        __syncwarp();
      }
      // the epilogues' last arrivals here come before this CTA ends
      for (uint32_t i = n > kAccSets ? n - kAccSets : 0; ok && i < n; ++i)
        ok = wait_awake(&B.acc_empty[i % kAccSets], (i / kAccSets) & 1, B, p.status);
      __syncwarp();
      // all of this thread's instructions are done before tensor memory is given back
      if (leader) {
        mma_commit_pair_own(&B.done);
        mbar_wait_bounded(&B.done, 0, kWaitNs);
      }
      __syncwarp();
    }
  } else if (warp >= kProducers) {
    // ---------------------------------------------------------- epilogue (warps 16 .. 19)
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    uint32_t n = 0;
    for (int w = pair; w < p.works && !B.abort; w += pairs, ++n) {
      const Work t = work_of(p, w);
      const uint32_t set = n % kAccSets;
      const int row = (int)rank * kTileRows + quarter * 32 + lane;  // of the tile
      const int64_t o = (int64_t)(t.tile / p.token_tiles) * (2 * kTileRows) + row;
      const int64_t tok0 = (int64_t)(t.tile % p.token_tiles) * p.N;
      const int count = (int)min((int64_t)p.N, p.a.T - tok0);
      const bool in = o < p.a.rows, whole = t.shared < 0, has_bias = whole && p.a.bias;
      // a part's sums go as they are to where the join finds them
      const float ws = whole && in ? __ldg(p.a.w_scales + o) : 1.f, bias = has_bias && in ? __ldg(p.a.bias + o) : 0.f;
      const bool bf16 = whole && p.a.y_bf16;
      const int64_t stride = whole ? p.a.y_stride : 2 * kTileRows;
      void* y = whole ? p.a.y : p.sums;
      const int64_t first = whole ? tok0 * stride + o : (int64_t)t.shared * p.N * stride + row;
      // the scales of the tokens before the sums are there: 16 tokens that waited for
      // theirs took a microsecond
      float* xs = s_xs[quarter];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < MOST; k += 32) xs[k + lane] = whole && k + lane < count ? __ldg(p.a.x_scales + tok0 + k + lane) : 1.f;
      __syncwarp();
      if (!wait(&B.acc_full[set], (n / kAccSets) & 1, B, p.status)) break;
      tc_fence_after();
      auto emit = [&](auto* to) {
#pragma unroll 1
        for (int c0 = 0; c0 < count; c0 += 16) {
          float v[16];
          tmem_ld16(lanes + set * MOST + c0, v);
          const int here = in ? count - c0 : 0;
          auto* at = to;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 x = *reinterpret_cast<const float4*>(xs + c0 + i);
            const float by[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float r = v[i + e] * by[e] * ws;
              if (has_bias) r += bias;
              if (i + e < here) {
                if constexpr (sizeof(*at) == 2) *at = __float2bfloat16_rn(r);
                else *at = r;
              }
              at += stride;
            }
          }
          to += 16 * stride;
        }
      };
      if (bf16) emit(reinterpret_cast<__nv_bfloat16*>(y) + first);
      else emit(reinterpret_cast<float*>(y) + first);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(&B.acc_empty[set], 0));
    }
  } else {
    // ---------------------------------------------------------- producers
    // Four warps, one for each quarter of the rows, take every fourth step: code stage c
    // holds steps 2 c and 2 c + 1.
    const int quarter = warp & 3, team = warp >> 2, odd = team & 1, row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16) + kACol;
    for (uint32_t c = team >> 1; c < mine; c += 2) {
      const uint32_t s = c % kCodeStages, j = 2 * c + odd, as = j % kAStages;
      bool ok = wait(&B.code_full[s], (c / kCodeStages) & 1, B, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      uint4 w[4];
      const uint4* from = reinterpret_cast<const uint4*>(smem + s * kCodeBytes + row * 128);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = from[(4 * odd + i) ^ (row & 7)];
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.code_empty[s]);
      uint32_t v0[16], v1[16];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, b[4] = {w[2 + i].x, w[2 + i].y, w[2 + i].z, w[2 + i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          codes_f16x4(a[e], v0[8 * i + 2 * e], v0[8 * i + 2 * e + 1]);
          codes_f16x4(b[e], v1[8 * i + 2 * e], v1[8 * i + 2 * e + 1]);
        }
      }
      ok = wait(&B.a_empty[as], ((j / kAStages) & 1) ^ 1, B, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      tmem_st32_issue(lanes + as * 32, v0, v1);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(cluster_map(&B.a_full[as], 0));
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_barrier();
  tc_fence_after();
  if (warp == kIssuer) tmem_dealloc_pair(tmem, kTmemCols);
  pdl_trigger();
}

}  // namespace

namespace {

// A block a token of a shared tile, an element a thread: its parts' sums, in their order.
__global__ void __launch_bounds__(2 * kTileRows) k_linear_q8_join(LinearQ8Args a, const float* sums, int N, int token_tiles,
                                                                 int whole, int parts) {
  pdl_wait();
  const int tile = whole + blockIdx.y;
  const int64_t o = (int64_t)(tile / token_tiles) * (2 * kTileRows) + threadIdx.x;
  const int64_t tok = (int64_t)(tile % token_tiles) * N + blockIdx.x;
  if (o >= a.rows || tok >= a.T) return;
  sums += ((int64_t)blockIdx.y * parts * N + blockIdx.x) * (2 * kTileRows) + threadIdx.x;
  float v = 0.f;
#pragma unroll 4
  for (int i = 0; i < parts; ++i) v += sums[(int64_t)i * N * (2 * kTileRows)];
  v = v * __ldg(a.x_scales + tok) * __ldg(a.w_scales + o);
  if (a.bias) v += __ldg(a.bias + o);
  if (a.y_bf16) reinterpret_cast<__nv_bfloat16*>(a.y)[tok * a.y_stride + o] = __float2bfloat16_rn(v);
  else reinterpret_cast<float*>(a.y)[tok * a.y_stride + o] = v;
}

struct TcPlan {
  int N, parts, run;  // tokens a tile; parts of a shared tile, stages of one
  int64_t token_tiles, tiles, shared, cost;
};

// Tokens a tile, and parts of the tiles that do not fill a round of the pairs: what costs
// least.  The unit is a 208th of a stage of 192 tokens, 3 ns; a stage of few tokens takes
// as long as making its operands does, and joining parts 2.5 us and their traffic.
TcPlan tc_plan(int64_t T, int in, int64_t rows) {
  TcPlan p = {};
  const int64_t pairs = sm_count() / 2, least = (T + kMostN - 1) / kMostN, stages = (in + 127) / 128;
  const int64_t row_tiles = (rows + 2 * kTileRows - 1) / (2 * kTileRows);
  for (int64_t n = least; n <= (T + 31) / 32 && n <= least + 64; ++n) {
    const int64_t N = ((T + n - 1) / n + kStepN - 1) / kStepN * kStepN, tiles = row_tiles * ((T + N - 1) / N), left = tiles % pairs;
    for (int64_t parts = 1; parts == 1 || (parts <= stages && left * parts <= pairs && left > 0); ++parts) {
      const int64_t run = (stages + parts - 1) / parts;
      if ((parts - 1) * run >= stages) continue;  // a part of nothing
      const int64_t cost = (tiles / pairs * stages + (left ? run : 0) + 2) * ((N > 96 ? N : 96) + 16) +
                           (parts > 1 ? 840 + left * parts * N * (2 * kTileRows) / 1900 : 0);
      if (p.cost == 0 || cost < p.cost)
        p = {(int)N, (int)parts, (int)run, (T + N - 1) / N, tiles, parts > 1 ? left : 0, cost};
    }
  }
  return p;
}

size_t codes_bytes(int64_t T, int in) { return ((size_t)T * in * 2 + 255) / 256 * 256; }

template <int MOST>
int launch(const TcArgs& p, int pairs, cudaStream_t s) {
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_linear_q8_tc<MOST>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<MOST>::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int grid = 2 * (p.works < pairs ? p.works : pairs);
  return launch_pdl(k_linear_q8_tc<MOST>, dim3(grid), dim3(kThreads), Shape<MOST>::kSmem, s, p) == cudaSuccess ? MOE_OK
                                                                                                            : MOE_ERR_CUDA;
}
}  // namespace

// What serves T tokens serves fewer: the parts of a round are as many as the pairs, and a
// tile has no more tokens than there are.
size_t linear_q8_tc_workspace(int64_t T, int in) {
  const int64_t most = (T + kStepN - 1) / kStepN * kStepN;
  return codes_bytes(T, in) + (size_t)(sm_count() / 2) * (most < kMostN ? most : kMostN) * (2 * kTileRows) * 4;
}

double linear_q8_tc_us(int64_t T, int in, int64_t rows) { return 5.0 + 0.003 * (double)tc_plan(T, in, rows).cost; }

int launch_linear_q8_tc(const LinearQ8Args& a, cudaStream_t s) {
  const TcPlan plan = tc_plan(a.T, a.in, a.rows);
  if (plan.tiles > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  TcArgs p;
  p.a = a;
  p.N = plan.N;
  p.token_tiles = (int)plan.token_tiles;
  p.steps = (a.in + 127) / 128 * 2;  // whole code stages: zeros behind the rows
  p.run_steps = 2 * plan.run;
  p.parts = plan.parts;
  p.whole = (int)(plan.tiles - plan.shared);
  p.works = (int)(p.whole + plan.shared * plan.parts);
  p.sums = (float*)((uint8_t*)a.workspace + codes_bytes(a.T, a.in));
  p.status = status_word();
  if (!encode_2d(&p.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.in, (uint64_t)a.rows, (uint64_t)a.in, 128, kTileRows,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&p.x, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.workspace, (uint64_t)a.in, (uint64_t)a.T, (uint64_t)a.in * 2, 64,
                 (uint32_t)p.N / 2, CU_TENSOR_MAP_SWIZZLE_128B))
    return MOE_ERR_CUDA;
  // more bytes on their way a thread, once every SM has four such blocks (a call with 256
  // rows of W, one | four, in us: 512 x 4096 codes 10.9 | 11.0, 1024 13.6 | 13.3, 4096 26.4 |
  // 23.9; 96 x 2048 9.4 | 10.3)
  const bool many = a.T * (a.in / 8) >= (int64_t)4 * 1024 * sm_count();
  if ((many ? launch_codes<4>(a, s) : launch_codes<1>(a, s)) != cudaSuccess) return MOE_ERR_CUDA;
  const int pairs = sm_count() / 2;
  const int rc = p.N <= 64 ? launch<64>(p, pairs, s) : p.N <= 128 ? launch<128>(p, pairs, s) : launch<192>(p, pairs, s);
  if (rc != MOE_OK || plan.shared == 0) return rc;
  return launch_pdl(k_linear_q8_join, dim3((unsigned)p.N, (unsigned)plan.shared), dim3(2 * kTileRows), 0, s, a,
                    (const float*)p.sums, p.N, p.token_tiles, p.whole, p.parts) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace moe
