// Shared by the kernels of the 4-bit key/value cache (wq_kv4.hip,
// wq_kv4_attn.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "wq_common.cuh"
#include "wq_device.h"

namespace wqd {

// wq_kv4_rows as the kernels take it.
struct KvRows {
  const int32_t* table;
  const int32_t* lens;
  const int32_t* cu;
  int64_t width;
  int seqs, rows, heads;
  const uint16_t* q;
  int64_t q_row, q_head;
};

// Division of 0 <= n < 2^31 by a divisor known on the host: one multiplication
// (the device's own division is some 40 instructions, and a short attention call
// would spend a tenth of its time on them).  With l = ceil(log2 d) and m =
// ceil(2^(31 + l) / d) < 2^32, n m / 2^(31 + l) exceeds n / d by less than
// n / 2^31 / d < 1 / d, so the floors agree.
struct Divisor {
  uint32_t d, m, l;
  Divisor() = default;
  explicit Divisor(int64_t by) : d((uint32_t)by), l(0) {
    while ((1ull << l) < (uint64_t)by) ++l;
    m = (uint32_t)(((1ull << (31 + l)) + d - 1) / d);
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)(((uint64_t)(uint32_t)n * m) >> (31 + l));
  }
};

template <int DT>
__device__ __forceinline__ float to_float(uint16_t b) {
  if constexpr (DT == WQ_DT_F16) return h2f(b);
  return __builtin_bit_cast(float, (uint32_t)b << 16);
}
template <int DT>
__device__ __forceinline__ uint16_t from_float(float f) {   // round to nearest even
  if constexpr (DT == WQ_DT_F16) return f2h(f);
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// The sequence of a row and the row's position in it (-1: it sees no token).  No
// difference overflows for any lens and cu_rows.
struct SeqRow {
  int b, pos;
};
__device__ __forceinline__ SeqRow find_row(const KvRows& a, int row) {
  int lo = 0, hi = a.seqs;
  if (row < hi && a.cu[row] == row && a.cu[row + 1] == row + 1)   // one row each: no search
    return {row, max(a.lens[row], 0) - 1};
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.cu[m] <= row) lo = m; else hi = m;
  }
  const int end = a.cu[lo + 1];
  return {lo, row < end ? max(max(a.lens[lo], 0) - (end - row), -1) : -1};
}

// Index arrays (int32) need their own alignment only: a caller's free list or
// table row may start anywhere.
inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int kv4_check_cache(const wq_kv4_cache* c, const char* who);
int kv4_check_rows(const wq_kv4_cache* c, const wq_kv4_rows* a, const char* who);
KvRows kv4_rows(const wq_kv4_rows* a);

// Calls f with the type and the head size as compile-time constants.
template <typename F>
inline void kv4_dispatch(int dtype, int64_t head_dim, F f) {
  auto by_dim = [&](auto dt) {
    if (head_dim == 64) f(dt, std::integral_constant<int, 64>{});
    else if (head_dim == 128) f(dt, std::integral_constant<int, 128>{});
    else f(dt, std::integral_constant<int, 256>{});
  };
  if (dtype == WQ_DT_F16) by_dim(std::integral_constant<int, WQ_DT_F16>{});
  else by_dim(std::integral_constant<int, WQ_DT_BF16>{});
}

}  // namespace wqd
