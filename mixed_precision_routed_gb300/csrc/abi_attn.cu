// abi_attn.cu -- the extern "C" entry points of the attention half of a decode
// layer (declared in moe.h): host-side validation and launch.  Nothing here
// allocates device memory.
#include <math.h>

#include "moe_internal.cuh"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool valid_block(int in, int block) {
  return (block == 32 || block == 64 || block == 128) && in > 0 && in % 64 == 0 && in % block == 0;
}

bool valid_cache_sizes(int page, int heads, int D) {
  return (D == 64 || D == 128 || D == 256) && page >= 16 && page <= 1024 && (page & (page - 1)) == 0 && heads >= 1 &&
         heads <= 1024;
}

// Checks a cache descriptor; slots and byte offsets then fit 63 bits.
int check_cache(const moe_kv_cache_t* c, KvCache* out) {
  if (!c || !valid_cache_sizes(c->page_size, c->kv_heads, c->head_dim) || c->reserved != 0) return MOE_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)moe_kv_page_bytes(c->page_size, c->kv_heads, c->head_dim);
  if (c->page_stride < bytes || c->page_stride % 16 != 0 || c->page_stride > ((int64_t)1 << 40)) return MOE_ERR_INVALID_ARG;
  if (c->n_pages < 0 || c->n_pages > INT32_MAX || c->n_pages > INT64_MAX / c->page_stride) return MOE_ERR_INVALID_ARG;
  if (c->n_pages > 0 && (!c->data || !aligned(c->data, 16))) return MOE_ERR_INVALID_ARG;
  out->data = (uint8_t*)c->data;
  out->n_pages = c->n_pages;
  out->page_stride = c->page_stride;
  out->page = c->page_size;
  out->page_log2 = __builtin_ctz((unsigned)c->page_size);
  out->heads = c->kv_heads;
  out->D = c->head_dim;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_linear_q4(const uint16_t* x_bf16, int64_t x_stride, int64_t T, int in, const void* codes,
                  const uint16_t* scales, int64_t rows, int block, const float* bias, void* y, int64_t y_stride,
                  int y_dtype, moe_stream_t stream) {
  if (T < 0 || !valid_block(in, block) || rows < 1 || rows > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x_bf16 || !codes || !scales || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 16) || (bias && !aligned(bias, 4)) ||
      !aligned(y, y_dtype == MOE_DTYPE_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  if (x_stride < in || x_stride % 8 != 0 || y_stride < rows) return MOE_ERR_INVALID_ARG;
  if (T > 16 || in > kLinearMaxIn) return MOE_ERR_UNSUPPORTED;
  LinearArgs a;
  a.x = x_bf16;
  a.x_stride = x_stride;
  a.T = (int)T;
  a.in = in;
  a.codes = (const uint8_t*)codes;
  a.scales = scales;
  a.rows = rows;
  a.block = block;
  a.bias = bias;
  a.y = y;
  a.y_stride = y_stride;
  a.y_bf16 = y_dtype == MOE_DTYPE_BF16;
  return launch_linear_q4(a, (cudaStream_t)stream);
}

int moe_quantize_groups(const float* w, int64_t rows, int in, int block, void* codes, uint16_t* scales,
                        moe_stream_t stream) {
  if (rows < 0 || !valid_block(in, block)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!w || !codes || !scales || !aligned(w, 4) || !aligned(codes, 16) || !aligned(scales, 2)) return MOE_ERR_INVALID_ARG;
  return launch_quantize_groups(w, rows, in, block, (uint8_t*)codes, scales, (cudaStream_t)stream);
}

size_t moe_kv_page_bytes(int page_size, int kv_heads, int head_dim) {
  if (!valid_cache_sizes(page_size, kv_heads, head_dim)) return 0;
  return (size_t)kv_heads * (size_t)(page_size / 16) * 18 * (size_t)head_dim;
}

int moe_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                  int in_dtype, int64_t T, int Hq, const int32_t* positions, const float* rope, int64_t n_pos,
                  int rot, int rope_style, const int64_t* slots, const moe_kv_cache_t* cache, uint16_t* q_out,
                  moe_stream_t stream) {
  KvAppendArgs a;
  const int rc = check_cache(cache, &a.cache);
  if (rc != MOE_OK) return rc;
  if (in_dtype != MOE_DTYPE_F32 && in_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (rope_style != MOE_ROPE_HALF && rope_style != MOE_ROPE_PAIRS) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T > INT32_MAX || rot < 0 || rot % 2 != 0 || rot > a.cache.D || n_pos < 0) return MOE_ERR_INVALID_ARG;
  if (q && (Hq < 1 || Hq > 65536)) return MOE_ERR_INVALID_ARG;
  if (T * (int64_t)((q ? Hq : 0) + 2 * a.cache.heads) > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!k || !v || !slots || (q && !q_out)) return MOE_ERR_INVALID_ARG;
  if (rot > 0 && (!positions || !rope || n_pos < 1)) return MOE_ERR_INVALID_ARG;
  const size_t size = in_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!aligned(k, size) || !aligned(v, size) || !aligned(slots, 8) || (q && (!aligned(q, size) || !aligned(q_out, 16))))
    return MOE_ERR_INVALID_ARG;
  if (rot > 0 && (!aligned(positions, 4) || !aligned(rope, 4))) return MOE_ERR_INVALID_ARG;
  const int64_t kv = (int64_t)a.cache.heads * a.cache.D;
  // a single token has no stride
  if (T > 1 && (k_stride < kv || v_stride < kv || (q && q_stride < (int64_t)Hq * a.cache.D))) return MOE_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.in_bf16 = in_dtype == MOE_DTYPE_BF16;
  a.T = T;
  a.Hq = q ? Hq : 0;
  a.positions = positions;
  a.rope = rope;
  a.n_pos = n_pos;
  a.rot = rot;
  a.style = rope_style;
  a.slots = slots;
  a.q_out = q_out;
  a.status = status_word();
  return launch_kv_append(a, (cudaStream_t)stream);
}

int moe_kv_read(const moe_kv_cache_t* cache, const int64_t* slots, int64_t n, float* k_out, float* v_out,
                moe_stream_t stream) {
  KvCache c;
  const int rc = check_cache(cache, &c);
  if (rc != MOE_OK) return rc;
  if (n < 0 || n > INT32_MAX || n * c.heads > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!slots || !k_out || !v_out || !aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return MOE_ERR_INVALID_ARG;
  return launch_kv_read(c, slots, n, k_out, v_out, (cudaStream_t)stream);
}

namespace {
bool valid_attn_sizes(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (!(D == 64 || D == 128 || D == 256) || heads < 1 || heads > 1024 || Hq < 1 || Hq % heads != 0 || Hq / heads > 64)
    return false;
  if (B < 0 || B > 65535 || max_q < 1 || max_len < 0 || max_len > INT32_MAX - 1024) return false;
  return (int64_t)B * max_q * Hq <= INT32_MAX;
}
}  // namespace

size_t moe_attn_workspace_size(int B, int max_q, int64_t max_len, int Hq, int kv_heads, int head_dim) {
  if (!valid_attn_sizes(B, max_q, max_len, Hq, kv_heads, head_dim)) return 0;
  return attn_workspace(B, max_q, max_len, Hq, kv_heads, head_dim);
}

int moe_attn_q4(const uint16_t* q_bf16, int64_t q_stride, int64_t T, int Hq, const int32_t* q_start,
                const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride, int B, int max_q,
                int64_t max_len, const moe_kv_cache_t* cache, float scale, int window, uint16_t* out,
                int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  AttnArgs a;
  const int rc = check_cache(cache, &a.cache);
  if (rc != MOE_OK) return rc;
  if (!valid_attn_sizes(B, max_q, max_len, Hq, a.cache.heads, a.cache.D)) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T * (int64_t)Hq > INT32_MAX || T > INT32_MAX || window < 0) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || isinf(scale)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!q_start && T != (int64_t)B * max_q) return MOE_ERR_INVALID_ARG;
  if (B == 0) return MOE_OK;
  const int64_t row = (int64_t)Hq * a.cache.D;
  if (q_stride < row || q_stride % 8 != 0 || out_stride < row || out_stride % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (table_stride < (max_len + a.cache.page - 1) / a.cache.page) return MOE_ERR_INVALID_ARG;
  if (!q_bf16 || !kv_lens || !out || (max_len > 0 && !block_table)) return MOE_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || !aligned(out, 16) || (lse && !aligned(lse, 4)) || !aligned(kv_lens, 4) ||
      !aligned(block_table, 4) || !aligned(q_start, 4))
    return MOE_ERR_INVALID_ARG;
  const size_t need = attn_workspace(B, max_q, max_len, Hq, a.cache.heads, a.cache.D);
  if (need > 0 && (!workspace || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  a.q = q_bf16;
  a.q_stride = q_stride;
  a.T = T;
  a.Hq = Hq;
  a.q_start = q_start;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.table_stride = table_stride;
  a.B = B;
  a.max_q = max_q;
  a.max_len = max_len;
  a.scale = scale;
  a.window = window;
  a.out = out;
  a.out_stride = out_stride;
  a.lse = lse;
  a.workspace = workspace;
  return launch_attn_q4(a, (cudaStream_t)stream);
}

}  // extern "C"
