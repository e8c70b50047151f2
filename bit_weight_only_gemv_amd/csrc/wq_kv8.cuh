// Shared by the kernels of the 8-bit key/value cache (wq_kv8.hip,
// wq_kv8_attn.hip).  Not part of the public ABI.
#pragma once

#include "wq_kv4.cuh"

namespace wqd {

constexpr int kBlock8 = 16;          // tokens that share an exponent
constexpr int kLeast8 = -24, kMost8 = 10;

// The exponent of block u (0..3) in four of them, whatever the byte holds.
__device__ __forceinline__ int exponent8(uint32_t word, int u) {
  return min(max((int)(word << (24 - 8 * u)) >> 24, kLeast8), kMost8);
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2(int e) {
  return __builtin_bit_cast(float, (uint32_t)(127 + e) << 23);
}

int kv8_check_cache(const wq_kv8_cache* c, const char* who);
// The 8-bit cache as kv4_check_rows takes one (it looks at its heads alone).
inline wq_kv4_cache kv8_shape(const wq_kv8_cache* c) {
  return wq_kv4_cache{c->data, nullptr, c->n_pages, c->n_kv_heads, c->head_dim};
}

}  // namespace wqd
