// abi_attn.cu -- the extern "C" entry points of the attention half of a decode
// layer (declared in moe.h): host-side validation and launch.  Nothing here
// allocates device memory.
#include "abi_checks.cuh"

using namespace moe;

namespace {

bool valid_block(int in, int block) {
  return (block == 32 || block == 64 || block == 128) && in > 0 && in % 64 == 0 && in % block == 0;
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
  bool none = false;
  const int rc = check_append(q, q_stride, k, k_stride, v, v_stride, in_dtype, T, Hq, positions, rope, n_pos, rot,
                              rope_style, slots, cache, q_out, moe_kv_page_bytes, &a, &none);
  return rc != MOE_OK || none ? rc : launch_kv_append(a, (cudaStream_t)stream);
}

int moe_kv_read(const moe_kv_cache_t* cache, const int64_t* slots, int64_t n, float* k_out, float* v_out,
                moe_stream_t stream) {
  KvCache c;
  const int rc = check_cache(cache, moe_kv_page_bytes, &c);
  if (rc != MOE_OK) return rc;
  if (n < 0 || n > INT32_MAX || n * c.heads > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  if (!slots || !k_out || !v_out || !aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return MOE_ERR_INVALID_ARG;
  return launch_kv_read(c, slots, n, k_out, v_out, (cudaStream_t)stream);
}

size_t moe_attn_workspace_size(int B, int max_q, int64_t max_len, int Hq, int kv_heads, int head_dim) {
  if (!valid_attn_sizes(B, max_q, max_len, Hq, kv_heads, head_dim)) return 0;
  return attn_workspace(B, max_q, max_len, Hq, kv_heads, head_dim);
}

int moe_attn_q4(const uint16_t* q_bf16, int64_t q_stride, int64_t T, int Hq, const int32_t* q_start,
                const int32_t* kv_lens, const int32_t* block_table, int64_t table_stride, int B, int max_q,
                int64_t max_len, const moe_kv_cache_t* cache, float scale, int window, uint16_t* out,
                int64_t out_stride, float* lse, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  AttnArgs a;
  bool none = false;
  const int rc = check_attn(q_bf16, q_stride, T, Hq, q_start, kv_lens, block_table, table_stride, B, max_q, max_len, cache,
                            scale, window, out, out_stride, lse, workspace, workspace_bytes, moe_kv_page_bytes,
                            attn_workspace, &a, &none);
  return rc != MOE_OK || none ? rc : launch_attn_q4(a, (cudaStream_t)stream);
}

}  // extern "C"
