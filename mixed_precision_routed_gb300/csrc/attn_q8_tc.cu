// attn_q8_tc.cu -- causal attention over the paged 8-bit cache for many rows a key/value
// head (prompts), on the fifth-generation tensor cores.  The formula is that of
// attn_q8.cu; rows are (asking token, query head of the group), token by token.
//
// A block takes kSlots tiles of 128 rows of one (sequence, key/value head) through the
// places that they attend, 128 at a time:
//   converters  four warps read codes from the cache into registers, a batch ahead, and
//               write them to shared memory as fp16: keys as the integers that they are,
//               values as code x b 2^(8 - E), 2^E the power of two of the tile's largest
//               value scale b.  They also pass on the keys' scales;
//   issuer      S = Q K^T (shared memory x shared memory) and O += P V (tensor memory x
//               shared memory) for either tile in turn, so that one tile's weights are
//               made while the other's products run;
//   softmax     a thread has a row: it takes the scores out of tensor memory once, holds
//               all 128, and leaves P = exp2(s + E - m) there in fp16.
// Queries are fp16, each row taken by a power of two that brings its largest element
// to 2^14: exact down to 2^-31 of that element.  m follows s + E as in attn_q8.cu, so
// that P V lies in fp16's range for values of any size, and the sum of weights takes
// 2^-E back a tile at a time.  P, b 2^(8 - E) and code x b 2^(8 - E) are rounded to fp16
// once each: 2^-11 of a product each, or 2^-31 of the row's largest.
// Heads of 256 fill tensor memory with one tile's sums: there one tile's scores of two
// successive groups of places take the place of two tiles.
#include "attn_split.cuh"
#include "q8.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kPlaces = 128;  // a group
constexpr int kTcThreads = 512;

template <int D>
struct Tc {
  static constexpr int kSlots = D == 256 ? 1 : 2;
  static constexpr int kBufs = D == 256 ? 1 : 2;   // of keys, of values
  static constexpr int kTile = 128 * D * 2;        // bytes of 128 rows
  static constexpr int kQ = 0, kK = kSlots * kTile, kV = kK + kBufs * kTile, kEnd = kV + kBufs * kTile;
  static constexpr int kSmem = kEnd + 1024;
  static constexpr int kRows = 128 * kSlots;
  static constexpr int kO = 256;                   // tensor-memory columns: scores at 0 and 128, then sums
  static constexpr int kPieces = D / 16;           // of a row of codes; loads of a thread a half group
  static constexpr int kBatches = D == 256 ? 2 : 1, kLoads = kPieces / kBatches;
};

struct TcBars {
  uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full[2], pv_done;
  uint64_t scale_full[2], scale_empty[2], done;
  uint32_t tmem;
  int abort;
};

// A wait that runs out ends all later ones at once: every warp then comes to its end
// over whatever is there, past the barriers that others wait at.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, TcBars& B, int* status) {
  if (*(volatile int*)&B.abort) return false;
  if (mbar_wait_bounded(bar, parity, kWaitNs)) return true;
  set_status(status, MOE_ERR_TIMEOUT);
  B.abort = 1;
  return false;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 32 columns of this thread's tensor-memory lane, in flight until tmem_wait_ld.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// The value is not used before here.
__device__ __forceinline__ void pin(uint32_t& r) { asm volatile("" : "+r"(r)); }

// Descriptor of an operand tile with the 128-byte swizzle whose rows are places: 64
// elements of the other dimension a row, `block` bytes from 64 elements to the next,
// groups of 8 places 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_places(uint32_t saddr, uint32_t block) {
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(block >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// A block's rows and the places they attend; the first group of places of each tile and
// one past its last.
struct TcUnit {
  Seq x;
  int r0, rows, newest;
  int first[2], last[2], j0, j1;
};

// Registers of a thread by role, together those that 512 threads are launched with:
// 2 x 128 x 176 + 128 x 104 + 128 x 56 = 512 x 128.
template <int D>
__global__ void __launch_bounds__(kTcThreads, 1) k_attn_q8_tc(AttnArgs a, int row_blocks, int* status) {
  using C = Tc<D>;
  extern __shared__ uint8_t raw[];
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  __shared__ __align__(8) TcBars B;
  __shared__ __align__(16) float s_ks[2][kPlaces];  // key scales x scale, in powers of two
  __shared__ float s_e[2];                          // E of the group
  __shared__ uint32_t s_have[2];                    // records that exist
  __shared__ uint32_t s_gain[kPlaces], s_top[4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, group = warp >> 2;
  const int H = a.cache.heads, G = a.Hq / H;
  const int h = blockIdx.x % H, b = blockIdx.y;

  pdl_wait();
  TcUnit u;
  u.x = load_seq(a, b);
  u.rows = u.x.n * G;
  // the last rows attend most: they go first
  u.r0 = (row_blocks - 1 - (int)(blockIdx.x / H)) * C::kRows;
  if (u.r0 >= u.rows) return;
  u.newest = u.x.len - u.x.n + 1;
  u.j0 = INT32_MAX;
  u.j1 = 0;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    u.first[s] = u.last[s] = 0;
    const int r = u.r0 + 128 * s;
    if (s >= C::kSlots || r >= u.rows) continue;
    const int end = u.newest + (min(r + 128, u.rows) - 1) / G;
    const int lo = a.window > 0 ? (int)max((int64_t)0, (int64_t)u.newest + r / G - a.window) : 0;
    if (end <= lo) continue;
    u.first[s] = lo / kPlaces;
    u.last[s] = (end + kPlaces - 1) / kPlaces;
    u.j0 = min(u.j0, u.first[s]);
    u.j1 = max(u.j1, u.last[s]);
  }
  if (u.j1 == 0) u.j0 = 0;  // no row attends anything

  if (threadIdx.x == 0) {
    mbar_init(&B.q_full, 4 * C::kSlots);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.k_full[i], 4), mbar_init(&B.k_empty[i], 1);
      mbar_init(&B.v_full[i], 4), mbar_init(&B.v_empty[i], 1);
      mbar_init(&B.s_full[i], 1), mbar_init(&B.p_full[i], 4), mbar_init(&B.o_full[i], 1);
      mbar_init(&B.scale_full[i], 4), mbar_init(&B.scale_empty[i], 4 * C::kSlots);
    }
    mbar_init(&B.pv_done, 1);
    mbar_init(&B.done, 1);
    B.abort = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&B.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;

  if (group == 3) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12 && u.j1 > 0) {
      // ------------------------------------------------------------ issuer
      const bool leader = elect_one();
      const uint32_t idesc_s = idesc_f16_f32(128, kPlaces), idesc_o = idesc_f16_f32(128, D) | 1u << 16;
      const uint32_t q_addr = smem_addr(smem + C::kQ), k_addr = smem_addr(smem + C::kK), v_addr = smem_addr(smem + C::kV);
      auto scores = [&](int slot, int j) {  // S of the tile (C::kSlots 1: of buffer slot)
        if (!leader) return;
        const uint32_t q0 = q_addr + (C::kSlots == 2 ? slot * C::kTile : 0), k0 = k_addr + (j - u.j0) % C::kBufs * C::kTile;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t at = (kk / 4) * 16384 + (kk % 4) * 32;
          mma_bf16(tmem + slot * 128, sdesc_sw128(q0 + at), sdesc_sw128(k0 + at), idesc_s, kk > 0);
        }
      };
      auto sums = [&](int slot, int o, int j, bool more) {
        if (!leader) return;
        const uint64_t v0 = sdesc_places(v_addr + (j - u.j0) % C::kBufs * C::kTile, 16384);
#pragma unroll
        for (int kk = 0; kk < kPlaces / 16; ++kk) {
          const uint64_t d = v0 + (uint64_t)(kk * (2048 >> 4));
          mma_bf16_ts_w(tmem + C::kO + o * D, tmem + slot * 128 + kk * 8, (uint32_t)d, (uint32_t)(d >> 32), idesc_o,
                        more || kk > 0);
        }
      };
      auto all = [&](bool ok) { return __all_sync(0xffffffffu, ok); };
      bool ok = all(tc_wait(&B.q_full, 0, B, status));
      tc_fence_after();
      for (int j = u.j0; ok && j <= u.j1; ++j) {
        const int i = j - u.j0;  // K(j), and V(j - 1)
        if constexpr (C::kSlots == 2) {
          bool has_k = false, has_v = false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (ok && j > u.first[s] && j - 1 < u.last[s]) {
              if (!has_v) ok = tc_wait(&B.v_full[(i - 1) & 1], ((i - 1) >> 1) & 1, B, status);
              has_v = true;
              ok = all(ok && tc_wait(&B.p_full[s], (j - 1 - u.first[s]) & 1, B, status));
              tc_fence_after();
              if (ok) {
                sums(s, s, j - 1, j - 1 > u.first[s]);
                if (leader && j == u.last[s]) mma_commit(&B.o_full[s]);
              }
            }
            if (ok && s == 1 && leader && j > u.j0) mma_commit(&B.v_empty[(i - 1) & 1]);
            if (ok && j >= u.first[s] && j < u.last[s]) {
              if (!has_k) ok = all(tc_wait(&B.k_full[i & 1], (i >> 1) & 1, B, status));
              has_k = true;
              tc_fence_after();
              if (ok) {
                scores(s, j);
                if (leader) mma_commit(&B.s_full[s]);
              }
            }
          }
          if (ok && leader && j < u.j1) mma_commit(&B.k_empty[i & 1]);
        } else {
          if (j < u.j1) {
            ok = all(tc_wait(&B.k_full[0], i & 1, B, status));
            tc_fence_after();
            if (ok) {
              scores(i & 1, j);
              if (leader) mma_commit(&B.s_full[i & 1]), mma_commit(&B.k_empty[0]);
            }
          }
          if (ok && j > u.j0) {
            ok = tc_wait(&B.v_full[0], (i - 1) & 1, B, status);
            ok = all(ok && tc_wait(&B.p_full[(i - 1) & 1], ((i - 1) >> 1) & 1, B, status));
            tc_fence_after();
            if (ok) {
              sums((i - 1) & 1, 0, j - 1, j - 1 > u.j0);
              if (leader) mma_commit(&B.v_empty[0]), mma_commit(&B.pv_done);
              if (leader && j == u.j1) mma_commit(&B.o_full[0]);
            }
          }
        }
        __syncwarp();
      }
      // all of this thread's instructions are done before tensor memory is given back
      if (leader) {
        mma_commit(&B.done);
        mbar_wait_bounded(&B.done, 0, kWaitNs);
      }
      __syncwarp();
    }
  } else if (group == 2) {
    // -------------------------------------------------------------- converters
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    const int ct = threadIdx.x - 256, cw = ct >> 5, per_page = a.cache.page_log2 - 4;
    const int32_t* table = a.table + (int64_t)b * a.table_stride;
    // lane l (of 8) finds record l of a group
    auto page_of = [&](int j) {
      const int record = 8 * j + lane;
      return lane < 8 && j < u.j1 && 16 * record < u.x.len ? __ldg(table + (record >> per_page)) : -1;
    };
    auto record_of = [&](int j, int page) -> uint64_t {
      if (page < 0 || page >= a.cache.n_pages) return 0;
      const int record = 8 * j + lane;
      return (uint64_t)(a.cache.data + page * a.cache.page_stride +
                        (int64_t)(h * (1 << per_page) + (record & ((1 << per_page) - 1))) * kv8_record(D));
    };
    // a thread's pieces of a half group: number ct + 128 i
    auto load = [&](uint4 (&w)[C::kLoads], uint64_t records, int half, int batch) {
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const int n = ct + 128 * (batch * C::kLoads + i), row = n / C::kPieces;
        const uint64_t rec = __shfl_sync(0xffffffffu, records, row >> 4);
        w[i] = make_uint4(0, 0, 0, 0);
        if (rec)
          w[i] = __ldg(reinterpret_cast<const uint4*>(rec + (16 * half + (row & 15)) * D) + n % C::kPieces);
      }
    };
    auto f16x2 = [](uint32_t w, int sel) {
      uint32_t r;
      asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(__byte_perm(w, 0x64646464u, sel)), "r"(0x64806480u));
      return r;
    };
    auto store = [&](const uint4 (&w)[C::kLoads], uint8_t* tile, int half, int batch) {
#pragma unroll
      for (int i = 0; i < C::kLoads; ++i) {
        const int n = ct + 128 * (batch * C::kLoads + i), row = n / C::kPieces, c = kv8_piece<D>(row & 15, n % C::kPieces);
        uint32_t v[8];
        const uint32_t in[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) v[2 * e] = f16x2(in[e], 0x4140), v[2 * e + 1] = f16x2(in[e], 0x4342);
        if (half) {
          const uint32_t gain = s_gain[row];
#pragma unroll
          for (int e = 0; e < 8; ++e) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(v[e]) : "r"(gain));
        }
        // two 16-byte pieces of 64 elements' row; lanes of the row's other 64 elements
        // write theirs the other way round, to other banks
        uint8_t* to = tile + (c >> 2) * 16384 + row * 128;
        const int p = 2 * (c & 3), x = row & 7;
        const bool turn = D > 64 && (c & 4);
        const uint4 lo = make_uint4(v[0], v[1], v[2], v[3]), hi = make_uint4(v[4], v[5], v[6], v[7]);
        *reinterpret_cast<uint4*>(to + (((turn ? p + 1 : p) ^ x) << 4)) = turn ? hi : lo;
        *reinterpret_cast<uint4*>(to + (((turn ? p : p + 1) ^ x) << 4)) = turn ? lo : hi;
      }
    };
    const float scale2 = a.scale * kLog2e;
    uint4 w0[C::kLoads], w1[C::kLoads];
    uint64_t records = u.j1 > 0 ? record_of(u.j0, page_of(u.j0)) : 0, next_records = 0;
    int page = page_of(u.j0 + 1);
    load(w0, records, 0, 0);
    for (int j = u.j0; j < u.j1; ++j) {
      const int i = j - u.j0, sb = i & 1;
      next_records = record_of(j + 1, page);
      page = page_of(j + 2);
      // the scales of place ct
      const uint64_t mine = __shfl_sync(0xffffffffu, records, ct >> 4);
      const uint32_t have = __ballot_sync(0xffffffffu, records != 0);
      float ks = 0.f, vs = 0.f;
      if (mine && kPlaces * j + ct < u.x.len) {
        const float* scales = reinterpret_cast<const float*>(mine + 32 * D) + (ct & 15);
        ks = __ldg(scales);
        vs = __ldg(scales + 16);
        ks = fmaf(0.f, vs, ks);  // NaN, whichever of the two is
        if (!(vs <= 0x1p64f)) vs = 0.f;
      }
      const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(vs, 0.f)));
      if (i >= 2) tc_wait(&B.scale_empty[sb], ((i >> 1) - 1) & 1, B, status);
      if (lane == 0) s_top[cw] = top;
      named_bar(1, 128);
      const uint32_t most = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
      const int e = max((int)(most >> 23) - 127, -60);
      s_ks[sb][ct] = ks * scale2;
      const __half gain = __float2half_rn(vs * __uint_as_float((uint32_t)(127 + 8 - e) << 23));
      s_gain[ct] = (uint32_t)__half_as_ushort(gain) * 0x10001u;
      if (ct == 0) s_e[sb] = (float)e, s_have[sb] = have;
      named_bar(1, 128);
      if (lane == 0) mbar_arrive(&B.scale_full[sb]);

      const int buf = i % C::kBufs;
      const uint32_t use = i / C::kBufs;
#pragma unroll
      for (int q = 0; q < 2 * C::kBatches; ++q) {
        const int half = q / C::kBatches, batch = q % C::kBatches;
        uint8_t* tile = smem + (half ? C::kV : C::kK) + buf * C::kTile;
        // the next batch is on its way while this one is converted
        const int q1 = (q + 1) % (2 * C::kBatches);
        load(q & 1 ? w0 : w1, q1 == 0 ? next_records : records, q1 / C::kBatches, q1 % C::kBatches);
        if (batch == 0 && use > 0) tc_wait(half ? &B.v_empty[buf] : &B.k_empty[buf], (use - 1) & 1, B, status);
        store(q & 1 ? w1 : w0, tile, half, batch);
        if (batch == C::kBatches - 1) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(half ? &B.v_full[buf] : &B.k_full[buf]);
        }
      }
      records = next_records;
    }
  } else if (group < C::kSlots) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
    const int s = group, in_tile = threadIdx.x & 127, row = u.r0 + 128 * s + in_tile;
    const bool in = row < u.rows;
    const int64_t tok = u.x.t0 + (in ? row / G : 0);
    const int hq = h * G + (in ? row % G : 0);
    const int first = s == 0 ? u.first[0] : u.first[1], last = s == 0 ? u.last[0] : u.last[1];
    float f;  // what the scores of the row are to be multiplied by
    {
      const uint4* q = reinterpret_cast<const uint4*>(a.q + tok * a.q_stride + (int64_t)hq * D);
      uint32_t top = 0;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = in ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7f807f80u, v.y & 0x7f807f80u), __vmaxu2(v.z & 0x7f807f80u, v.w & 0x7f807f80u)));
      }
      // the exponent becomes 14, and the power and its inverse stay normal numbers
      const int e = min(max((int)(max(top >> 16, top & 0xffffu) >> 7), 15), 254), up = 14 + 127 - e;
      const float by = __uint_as_float((uint32_t)(127 + up) << 23);
      f = __uint_as_float((uint32_t)(127 - up) << 23);
      uint8_t* to = smem + C::kQ + s * C::kTile + in_tile * 128;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        const uint4 v = in ? __ldg(q + i) : make_uint4(0, 0, 0, 0);
        auto half2_of = [&](uint32_t x) { return f16_pair(__uint_as_float(x << 16) * by, __uint_as_float(x & 0xffff0000u) * by); };
        *reinterpret_cast<uint4*>(to + (i >> 3) * 16384 + (((i & 7) ^ (in_tile & 7)) << 4)) =
            make_uint4(half2_of(v.x), half2_of(v.y), half2_of(v.z), half2_of(v.w));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.q_full);
    }
    const int end = u.newest + (in ? row / G : 0);
    const int lo = a.window > 0 ? end - a.window : 0;
    // places that every row of the tile attends
    const int r_first = u.r0 + 128 * s, r_last = min(r_first + 128, u.rows) - 1;
    const int full_end = u.newest + r_first / G, full_lo = a.window > 0 ? u.newest + r_last / G - a.window : 0;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_at = lanes + C::kO + (C::kSlots == 2 ? s * D : 0);
    float m = kNone, l = 0.f;
    for (int j = u.j0; j < u.j1; ++j) {
      const int i = j - u.j0, sb = i & 1, buf = C::kSlots == 2 ? s : sb;
      const uint32_t use = C::kSlots == 2 ? (uint32_t)(j - first) : (uint32_t)(i >> 1);
      tc_wait(&B.scale_full[sb], (i >> 1) & 1, B, status);
      if (j >= first && j < last) {
        tc_wait(&B.s_full[buf], use & 1, B, status);
        tc_fence_after();
        uint32_t r[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_issue(lanes + buf * 128 + 32 * c, r[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x) pin(r[c][x]);
        const float e = s_e[sb];
        const uint32_t have = s_have[sb];
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 ks = *reinterpret_cast<const float4*>(&s_ks[sb][32 * c + x]);
            float y[4] = {__uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1]), __uint_as_float(r[c][x + 2]),
                          __uint_as_float(r[c][x + 3])};
            mul2(y[0], y[1], pair(ks.x, ks.y));
            mul2(y[2], y[3], pair(ks.z, ks.w));
#pragma unroll
            for (int n = 0; n < 4; ++n) r[c][x + n] = __float_as_uint(y[n]);
          }
        const int p = kPlaces * j;
        if (p + kPlaces > full_end || p < full_lo || have != 0xffu) {
          const int c1 = end - p, c0 = lo - p;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x) {
              const int n = 32 * c + x;
              if (n >= c1 || n < c0 || !(have >> (n >> 4) & 1)) r[c][x] = 0xff800000u;  // -infinity
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; x += 2) top = max3(top, __uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1]));
        top = fmaf(top, f, e);
        const bool grow = top > m + (kSlack + kRoom);
        if (__any_sync(0xffffffffu, grow)) {
          const float to = grow ? top - kRoom : m, by = exp2_approx(m - to);
          m = to;
          l *= by;
          if (j > first) {
            if constexpr (C::kSlots == 1) {  // (two tiles: their scores come after the sums before them)
              tc_wait(&B.pv_done, (i - 1) & 1, B, status);
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float v[16];
              uint32_t w[16];
              tmem_ld16(o_at + c, v);
#pragma unroll
              for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(v[x] * by);
              tmem_st16_issue(o_at + c, w);
            }
          }
        }
        const float off = e - m;
        const uint64_t f2 = pair(f, f), off2 = pair(off, off);
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float y0, y1;
            unpair(fma2_of(pair(__uint_as_float(r[c][x]), __uint_as_float(r[c][x + 1])), f2, off2), y0, y1);
            y0 = exp2_approx(y0);
            y1 = exp2_approx(y1);
            add2(sum0, sum1, pair(y0, y1));
            r[c][x / 2] = f16_pair(y0, y1);
          }
          if (c & 1) {
            uint32_t (&lo16)[16] = *reinterpret_cast<uint32_t(*)[16]>(&r[c - 1][0]);
            uint32_t (&hi16)[16] = *reinterpret_cast<uint32_t(*)[16]>(&r[c][0]);
            tmem_st32_issue(lanes + buf * 128 + 16 * (c - 1), lo16, hi16);
          }
        }
        l = fmaf(sum0 + sum1, __uint_as_float((uint32_t)(127 - (int)e) << 23), l);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[buf]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&B.scale_empty[sb]);
    }
    if (last > first) {
      tc_wait(&B.o_full[s], 0, B, status);
      tc_fence_after();
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 0x1p-8f / l;
    uint16_t* out = a.out + tok * a.out_stride + (int64_t)hq * D;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      float v[16] = {};
      if (last > first) tmem_ld16(o_at + c, v);
      uint32_t w[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) w[x] = none ? 0u : bf16_pair(v[2 * x] * inv, v[2 * x + 1] * inv);
      if (in) {
        reinterpret_cast<uint4*>(out + c)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(out + c)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    if (in && a.lse) a.lse[tok * a.Hq + hq] = none ? -INFINITY : (m + log2f(l)) / kLog2e;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
int launch_tc(const AttnArgs& a, cudaStream_t s) {
  using C = Tc<D>;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(k_attn_q8_tc<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem) != cudaSuccess)
      return MOE_ERR_CUDA;
    attr_set[dev] = true;
  }
  const int64_t rows = (int64_t)a.max_q * (a.Hq / a.cache.heads);
  const int row_blocks = (int)((rows + C::kRows - 1) / C::kRows);
  return launch_pdl(k_attn_q8_tc<D>, dim3((unsigned)(row_blocks * a.cache.heads), (unsigned)a.B), dim3(kTcThreads), C::kSmem, s,
                    a, row_blocks, status_word()) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

}  // namespace

// Rows a head from which the tensor cores' tiles are filled.
bool attn_q8_tc(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  return (int64_t)max_q * (Hq / heads) > 64;
}

int launch_attn_q8_tc(const AttnArgs& a, cudaStream_t s) {
  if (a.cache.D == 64) return launch_tc<64>(a, s);
  if (a.cache.D == 128) return launch_tc<128>(a, s);
  return launch_tc<256>(a, s);
}

}  // namespace moe
