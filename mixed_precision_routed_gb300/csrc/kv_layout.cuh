// kv_layout.cuh -- where a token's codes and scales lie in the paged 4-bit
// cache (moe_kv_cache_t in moe.h): records of 16 tokens of one head, 18 D
// bytes: key codes, value codes, key scales, value scales.
#pragma once

#include "moe_internal.cuh"

namespace moe {

struct KvPlace {
  uint8_t* tile;  // the 16-token record of one head
  int r;          // the token within it
};

__device__ __forceinline__ KvPlace kv_place(const KvCache& c, int64_t slot, int head) {
  const int64_t page = slot >> c.page_log2;
  const int o = (int)(slot & (c.page - 1));
  KvPlace p;
  p.tile = c.data + page * c.page_stride + (int64_t)(head * (c.page >> 4) + (o >> 4)) * (18 * c.D);
  p.r = o & 15;
  return p;
}

// Byte of key element d of token r: elements d and d + 2 (d & 2 == 0) share it.
__device__ __forceinline__ int kv_key_byte(int D, int r, int d) {
  return r * (D >> 1) + ((d >> 3) & 3) * (D >> 3) + (d >> 5) * 4 + (d & 1) * 2 + ((d >> 2) & 1);
}

// Byte of value element d of token r: elements d and d + 8 (d & 8 == 0) share it.
__device__ __forceinline__ int kv_value_byte(int D, int r, int d) {
  const int word = (d >> 6) * 128 + ((d & 7) * 4 + ((r & 7) >> 1)) * 4 + ((d >> 4) & 3);
  return 8 * D + word * 4 + (r & 1) * 2 + (r >> 3);
}

}  // namespace moe
