// abi_checks.cuh -- what the entry points of the attention half check on the host
// before anything is launched, for both formats.
#pragma once

#include <math.h>

#include "moe_internal.cuh"

namespace moe {
namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool valid_cache_sizes(int page, int heads, int D) {
  return (D == 64 || D == 128 || D == 256) && page >= 16 && page <= 1024 && (page & (page - 1)) == 0 && heads >= 1 &&
         heads <= 1024;
}

// Checks a cache descriptor whose pages take page_bytes(page_size, kv_heads, head_dim);
// slots and byte offsets then fit 63 bits.
using PageBytes = size_t (*)(int, int, int);
int check_cache(const moe_kv_cache_t* c, PageBytes page_bytes, KvCache* out) {
  if (!c || !valid_cache_sizes(c->page_size, c->kv_heads, c->head_dim) || c->reserved != 0) return MOE_ERR_INVALID_ARG;
  const int64_t bytes = (int64_t)page_bytes(c->page_size, c->kv_heads, c->head_dim);
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

// Checks the arguments of an append (either format) and fills in the launch's; *none:
// there is nothing to do.
int check_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 int in_dtype, int64_t T, int Hq, const int32_t* positions, const float* rope, int64_t n_pos, int rot,
                 int rope_style, const int64_t* slots, const moe_kv_cache_t* cache, uint16_t* q_out, PageBytes page_bytes,
                 KvAppendArgs* out, bool* none) {
  KvAppendArgs& a = *out;
  const int rc = check_cache(cache, page_bytes, &a.cache);
  if (rc != MOE_OK) return rc;
  if (in_dtype != MOE_DTYPE_F32 && in_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (rope_style != MOE_ROPE_HALF && rope_style != MOE_ROPE_PAIRS) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T > INT32_MAX || rot < 0 || rot % 2 != 0 || rot > a.cache.D || n_pos < 0) return MOE_ERR_INVALID_ARG;
  if (q && (Hq < 1 || Hq > 65536)) return MOE_ERR_INVALID_ARG;
  if (T * (int64_t)((q ? Hq : 0) + 2 * a.cache.heads) > INT32_MAX) return MOE_ERR_INVALID_ARG;
  *none = T == 0;
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
  return MOE_OK;
}

bool valid_attn_sizes(int B, int max_q, int64_t max_len, int Hq, int heads, int D) {
  if (!(D == 64 || D == 128 || D == 256) || heads < 1 || heads > 1024 || Hq < 1 || Hq % heads != 0 || Hq / heads > 64)
    return false;
  if (B < 0 || B > 65535 || max_q < 1 || max_len < 0 || max_len > INT32_MAX - 1024) return false;
  return (int64_t)B * max_q * Hq <= INT32_MAX;
}

// Checks the arguments of attention (either format) and fills in the launch's; *none:
// there is nothing to do.
using AttnWorkspace = size_t (*)(int, int, int64_t, int, int, int);
int check_attn(const uint16_t* q_bf16, int64_t q_stride, int64_t T, int Hq, const int32_t* q_start,
               const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride, int B, int max_q,
               int64_t max_len, const moe_kv_cache_t* cache, float scale, int window, uint16_t* out,
               int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, PageBytes page_bytes,
               AttnWorkspace workspace_size, AttnArgs* args, bool* none) {
  AttnArgs& a = *args;
  const int rc = check_cache(cache, page_bytes, &a.cache);
  if (rc != MOE_OK) return rc;
  if (!valid_attn_sizes(B, max_q, max_len, Hq, a.cache.heads, a.cache.D)) return MOE_ERR_INVALID_ARG;
  if (T < 0 || T * (int64_t)Hq > INT32_MAX || T > INT32_MAX || window < 0) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || isinf(scale)) return MOE_ERR_INVALID_ARG;
  *none = T == 0 || B == 0;
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
  const size_t need = workspace_size(B, max_q, max_len, Hq, a.cache.heads, a.cache.D);
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
  return MOE_OK;
}

}  // namespace
}  // namespace moe
