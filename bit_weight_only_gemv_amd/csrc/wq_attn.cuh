// Shared by the attention kernels of the 4-bit and 8-bit key/value caches
// (wq_kv4_attn.hip, wq_kv8_attn.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

#include "wq_common.cuh"
#include "wq_kv4.cuh"

namespace wqd {

constexpr int kAttnWaves = 4, kAttnMoreWaves = 8;
constexpr float kWeightExp = 10.f;   // a page's largest weight at the reference is 2^10;
constexpr float kRaise = 4.f;        // one of over 2^14 raises the reference,
constexpr float kLower = 8.f;        // one of less than 2^2 lowers it,
constexpr float kBelow = 64.f;       // by no more than 2^64 below the highest

// f(0), ..., f(N - 1) with the index as a compile-time constant.
template <typename F, int... I>
__device__ __forceinline__ void unroll_over(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void unroll(F f) {
  unroll_over(f, std::make_integer_sequence<int, N>{});
}

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Logarithm of a sum of weights that carry 2^kWeightExp, at maximum mx (base 2).
__device__ __forceinline__ float log_sum(float sum, float mx) {
  return sum == 0.f ? -INFINITY
                    : ((mx == -INFINITY ? 0.f : mx) - kWeightExp) * 0.69314718f + __logf(sum);
}

// Joins the splits of one (row, head): split s's weight is 2^(m_s - max m).  16
// bytes a lane and D / 4 lanes a split, so that 1024 / D splits are read at a
// time; their sums are added in order.  With `cu` (then seqs + 1 entries, and the heads of a
// row), rows outside the sequences' have no parts and stay as they are.
template <int DT, int D>
static __global__ void __launch_bounds__(kAttnWaves * kWave)
join_kernel(const float* __restrict__ part, int64_t items, int splits, uint16_t* __restrict__ out,
            float* __restrict__ lse, const int32_t* __restrict__ cu = nullptr, int seqs = 0,
            int heads = 0) {
  constexpr int L = D / 4, S = kAttnWaves * kWave / L;
  __shared__ f4 s_acc[S][L];
  __shared__ float s_sum[S][3];
  const int64_t at = blockIdx.x;
  if (cu != nullptr && (at < (int64_t)cu[0] * heads || at >= (int64_t)cu[seqs] * heads)) return;
  const int x = threadIdx.x % L, y = threadIdx.x / L;
  const f4* ml = reinterpret_cast<const f4*>(part + items * splits * D) + at * splits;
  const f4* o = reinterpret_cast<const f4*>(part + at * splits * D) + x;
  float mx = -INFINITY, sum = 0.f, ex = 0.f;
  f4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int s = y; s < splits; s += S) {
    const f4 h = ml[s], v = o[(int64_t)s * L];
    const float top = fmaxf(mx, h[1]);
    const float f = mx == top ? 1.f : __builtin_amdgcn_exp2f(mx - top);
    const float w = h[1] == top ? 1.f : __builtin_amdgcn_exp2f(h[1] - top);
    mx = top;
    sum = sum * f + w * h[0];
    ex = ex * f + w * h[2];
    acc = acc * f + w * v;
  }
  s_acc[y][x] = acc;
  if (x == 0) {
    s_sum[y][0] = mx;
    s_sum[y][1] = sum;
    s_sum[y][2] = ex;
  }
  __syncthreads();
  if (y != 0) return;
#pragma unroll
  for (int s = 1; s < S; ++s) mx = fmaxf(mx, s_sum[s][0]);
  sum = ex = 0.f;
  acc = f4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const float w = s_sum[s][0] == mx ? 1.f : __builtin_amdgcn_exp2f(s_sum[s][0] - mx);
    sum += w * s_sum[s][1];
    ex += w * s_sum[s][2];
    acc += w * s_acc[s][x];
  }
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = from_float<DT>(sum == 0.f ? 0.f : acc[i] / sum);
  *reinterpret_cast<u2*>(out + at * D + 4 * x) = u2{pack2(h[0], h[1]), pack2(h[2], h[3])};
  if (x == 0 && lse != nullptr) lse[at] = log_sum(ex, mx);
}

}  // namespace wqd
