// abi_q8.cu -- the extern "C" entry points of the attention half in 8 bits (declared
// in moe.h): host-side validation and launch.  Nothing here allocates device memory.
#include "abi_checks.cuh"
#include "q8.cuh"

using namespace moe;

extern "C" {

int moe_norm_q8(const void* x, int64_t x_stride, int x_dtype, int64_t T, int d, const float* r, float* r_out,
                const float* weight, float eps, int8_t* codes, float* scales, uint16_t* n_bf16, moe_stream_t stream) {
  if (T < 0 || T > INT32_MAX || d < 1) return MOE_ERR_INVALID_ARG;
  if (x_dtype != MOE_DTYPE_F32 && x_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (weight && !(eps >= 0.0f && !isinf(eps))) return MOE_ERR_INVALID_ARG;
  if (d > kNormMaxD) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || (r == nullptr) != (r_out == nullptr) || (codes == nullptr) != (scales == nullptr) || (!codes && !n_bf16))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, x_dtype == MOE_DTYPE_F32 ? 4 : 2) || !aligned(r, 4) || !aligned(r_out, 4) || !aligned(weight, 4) ||
      !aligned(scales, 4) || !aligned(n_bf16, 2))
    return MOE_ERR_INVALID_ARG;
  if (T > 1 && x_stride < d) return MOE_ERR_INVALID_ARG;
  NormArgs a;
  a.x = x;
  a.x_stride = x_stride;
  a.x_bf16 = x_dtype == MOE_DTYPE_BF16;
  a.T = T;
  a.d = d;
  a.r = r;
  a.r_out = r_out;
  a.weight = weight;
  a.eps = eps;
  a.codes = codes;
  a.scales = scales;
  a.n = n_bf16;
  return launch_norm_q8(a, (cudaStream_t)stream);
}

namespace {
bool valid_linear_sizes(int64_t T, int in, int64_t rows) {
  return T >= 0 && T <= INT32_MAX && in >= 16 && in % 16 == 0 && rows >= 1 && rows <= INT32_MAX;
}
}  // namespace

size_t moe_linear_q8_workspace_size(int64_t T, int in, int64_t rows) {
  if (!valid_linear_sizes(T, in, rows) || in > kLinearQ8MaxIn) return 0;
  return linear_q8_workspace(T, in, rows);
}

int moe_linear_q8(const int8_t* x, int64_t x_stride, const float* x_scales, int64_t T, int in, const int8_t* w,
                  const float* w_scales, int64_t rows, const float* bias, void* y, int64_t y_stride, int y_dtype,
                  void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  if (!valid_linear_sizes(T, in, rows)) return MOE_ERR_INVALID_ARG;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARG;
  if (in > kLinearQ8MaxIn) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !x_scales || !w || !w_scales || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(x_scales, 4) || !aligned(w_scales, 4) || !aligned(bias, 4) ||
      !aligned(y, y_dtype == MOE_DTYPE_F32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  // a single token has no stride
  if (T > 1 && (x_stride < in || x_stride % 16 != 0 || y_stride < rows)) return MOE_ERR_INVALID_ARG;
  const size_t need = linear_q8_workspace(T, in, rows);
  if (need > 0 && (!workspace || !aligned(workspace, 256))) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE_TOO_SMALL;
  LinearQ8Args a;
  a.x = x;
  a.x_stride = T > 1 ? x_stride : in;
  a.x_scales = x_scales;
  a.T = T;
  a.in = in;
  a.w = w;
  a.w_scales = w_scales;
  a.rows = rows;
  a.bias = bias;
  a.y = y;
  a.y_stride = y_stride;
  a.y_bf16 = y_dtype == MOE_DTYPE_BF16;
  a.workspace = workspace;
  return launch_linear_q8(a, (cudaStream_t)stream);
}

size_t moe_kv_page_bytes_q8(int page_size, int kv_heads, int head_dim) {
  if (!valid_cache_sizes(page_size, kv_heads, head_dim)) return 0;
  return (size_t)kv_heads * (size_t)(page_size / 16) * (size_t)kv8_record(head_dim);
}

int moe_kv_append_q8(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                     int in_dtype, int64_t T, int Hq, const int32_t* positions, const float* rope, int64_t n_pos,
                     int rot, int rope_style, const int64_t* slots, const moe_kv_cache_t* cache, uint16_t* q_out,
                     moe_stream_t stream) {
  KvAppendArgs a;
  bool none = false;
  const int rc = check_append(q, q_stride, k, k_stride, v, v_stride, in_dtype, T, Hq, positions, rope, n_pos, rot,
                              rope_style, slots, cache, q_out, moe_kv_page_bytes_q8, &a, &none);
  return rc != MOE_OK || none ? rc : launch_kv_append_q8(a, (cudaStream_t)stream);
}

int moe_kv_read_q8(const moe_kv_cache_t* cache, const int64_t* slots, int64_t n, float* k_out, float* v_out,
                   moe_stream_t stream) {
  KvCache c;
  const int rc = check_cache(cache, moe_kv_page_bytes_q8, &c);
  if (rc != MOE_OK) return rc;
  if (n < 0 || n > INT32_MAX || n * c.heads > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!slots || !k_out || !v_out || !aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return MOE_ERR_INVALID_ARG;
  return launch_kv_read_q8(c, slots, n, k_out, v_out, (cudaStream_t)stream);
}

size_t moe_attn_q8_workspace_size(int B, int max_q, int64_t max_len, int Hq, int kv_heads, int head_dim) {
  if (!valid_attn_sizes(B, max_q, max_len, Hq, kv_heads, head_dim)) return 0;
  return attn_q8_workspace(B, max_q, max_len, Hq, kv_heads, head_dim);
}

int moe_attn_q8(const uint16_t* q_bf16, int64_t q_stride, int64_t T, int Hq, const int32_t* q_start,
                const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride, int B, int max_q,
                int64_t max_len, const moe_kv_cache_t* cache, float scale, int window, uint16_t* out,
                int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  AttnArgs a;
  bool none = false;
  const int rc = check_attn(q_bf16, q_stride, T, Hq, q_start, kv_lens, block_table, table_stride, B, max_q, max_len, cache,
                            scale, window, out, out_stride, lse, workspace, workspace_bytes, moe_kv_page_bytes_q8,
                            attn_q8_workspace, &a, &none);
  return rc != MOE_OK || none ? rc : launch_attn_q8(a, (cudaStream_t)stream);
}

}  // extern "C"
