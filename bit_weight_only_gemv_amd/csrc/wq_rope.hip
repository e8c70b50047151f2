// Norm of every head of queries and keys and the rotation by position, in one pass
// (wq.h, "norm and rotation of queries and keys").
//
//   y_d = x_d / sqrt(mean x^2 + eps) w_d,
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position f.
//
// D / 8 lanes take a head, each 8 channels that are 4 whole pairs, so that a rotation
// stays in its lane; a wave takes 64 / (D / 8) heads of a row at a time, up to
// kRopeTurns times with one set of sines and cosines.
//
// The angle.  t / 2 pi is needed modulo 1 alone, so f / 2 pi is made a 64-bit fraction
// of a turn and multiplied with the position in whole numbers modulo 2^64: no bit
// is lost however far the position (a float32 product is off by 0.004 at position
// 131072).  Sine and cosine are then their Taylor sums over an eighth of a turn
// each way (to x^9 and x^10: off by less than 2 10^-9 and 2 10^-10), in float32: the
// angle there is good to 2^-26 of a turn, the sums to 2^-23.
//
// Memory bounds prompts: 8190 rows of 40 heads of 128 channels (168 MB) take 38 us, a
// plain copy of them 33.  One row: 4.5 us, latency.

#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"

namespace wqd {

constexpr int kRopeWaves = 4, kRopeTurns = 4;

struct RopeSide {
  const uint16_t* x;
  uint16_t* out;
  const uint16_t* weight;
  int64_t row, head, out_row, out_head;
};
struct RopeArgs {
  RopeSide q, k;
  const int32_t* positions;
  const double* freqs;
  int64_t units;
  int heads, kv_heads, n_freq;
  float eps;               // negative: no norm
  Divisor chunks_by;
};

// Sine and cosine of a fraction of a turn, in units of 2^-32.
__device__ __forceinline__ void sine_cosine(uint32_t turn, float& s, float& c) {
  const uint32_t quarter = (turn + 0x20000000u) >> 30;
  const float x = (float)(int)(turn - (quarter << 30)) * (6.28318531f * 0x1p-32f), z = x * x;
  float sn = __builtin_fmaf(z, 2.75573192e-6f, -1.98412698e-4f);
  sn = __builtin_fmaf(z, sn, 8.33333333e-3f);
  sn = __builtin_fmaf(z, sn, -1.66666667e-1f);
  sn = __builtin_fmaf(x * z, sn, x);
  float cs = __builtin_fmaf(z, -2.75573192e-7f, 2.48015873e-5f);
  cs = __builtin_fmaf(z, cs, -1.38888889e-3f);
  cs = __builtin_fmaf(z, cs, 4.16666667e-2f);
  cs = __builtin_fmaf(z, cs, -0.5f);
  cs = __builtin_fmaf(z, cs, 1.f);
  s = quarter & 1 ? cs : sn;
  c = quarter & 1 ? sn : cs;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

// f over the L lanes of a head, in all of them.
template <int L, typename F>
__device__ __forceinline__ float head_reduce(float v, F f) {
  v = f(v, dpp_mov<0xB1>(v));                   // quad_perm [1,0,3,2]
  v = f(v, dpp_mov<0x4E>(v));                   // quad_perm [2,3,0,1]
  v = f(v, dpp_mov<0x141>(v));                  // row_half_mirror
  if constexpr (L >= 16) v = f(v, dpp_mov<0x140>(v));    // row_mirror
  if constexpr (L == 32) v = f(v, __shfl_xor(v, 16));
  return v;
}

template <int L>
__device__ __forceinline__ float head_squares(const float (&a)[4], const float (&b)[4]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s = __builtin_fmaf(a[e], a[e], __builtin_fmaf(b[e], b[e], s));
  return head_reduce<L>(s, [](float x, float y) { return x + y; });
}

// Squares of BF16 values leave float32's range both ways.  Sums from kLargeSquares on, and any
// with an eps that does not outweigh what may be lost, are made again of the head times the power
// of two that brings the larger of its largest channel and sqrt(eps) near 1.  The test costs
// 1 to 2% of a prompt's time, in turn with a build without it; where large channels were
// looked for before the loop it was 3%, and 5 to 16% where such heads waited for a second one.
constexpr float kLargeSquares = 0x1p120f, kSmallEps = 0x1p-60f;

template <int L>
__device__ __forceinline__ void rescale_head(float (&a)[4], float (&b)[4], float& s, float& eps) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(a[e]), fabsf(b[e])));
  top = fmaxf(head_reduce<L>(top, [](float x, float y) { return fmaxf(x, y); }), sqrtf(eps));
  const int by = top > 0.f && top < INFINITY ? -ilogbf(top) : 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    a[e] = ldexpf(a[e], by);
    b[e] = ldexpf(b[e], by);
  }
  s = head_squares<L>(a, b);
  eps = ldexpf(ldexpf(eps, by), by);
}

template <int DT, int D, bool NEIGHBOURS>
__global__ void __launch_bounds__(kRopeWaves * kWave) rope_kernel(RopeArgs p) {
  constexpr int L = D / 8, HP = kWave / L;      // lanes a head, heads at a time
  const int lane = threadIdx.x & 63, i = lane % L;
  const int64_t unit = (int64_t)blockIdx.x * kRopeWaves + (threadIdx.x >> 6);
  if (unit >= p.units) return;
  const int row = p.chunks_by.div((int)unit), chunk = (int)unit - row * (int)p.chunks_by.d;
  const bool turns = 8 * i < 2 * p.n_freq;
  // this lane's channels: a .. a + 3 and b .. b + 3
  const int a = !NEIGHBOURS && turns ? 4 * i : 8 * i;
  const int b = !NEIGHBOURS && turns ? p.n_freq + 4 * i : 8 * i + 4;
  u2 xa[kRopeTurns], xb[kRopeTurns];
  const int all = p.heads + p.kv_heads, h0 = chunk * (HP * kRopeTurns) + lane / L;
#pragma unroll
  for (int t = 0; t < kRopeTurns; ++t) {
    const int h = h0 + t * HP;
    if (h >= all) continue;
    const bool is_q = h < p.heads;
    const uint16_t* const x = is_q ? p.q.x + row * p.q.row + h * p.q.head
                                   : p.k.x + row * p.k.row + (h - p.heads) * p.k.head;
    xa[t] = *reinterpret_cast<const u2*>(x + a);
    xb[t] = *reinterpret_cast<const u2*>(x + b);
  }
  float sn[4], cs[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) { sn[e] = 0.f; cs[e] = 1.f; }
  if (turns) {
    const int64_t pos = p.positions[row];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      double f = p.freqs[4 * i + e] * 0.15915494309189535;      // 1 / 2 pi
      f = (f - __builtin_floor(f)) * 4294967296.0;
      const uint32_t hi = (uint32_t)f, lo = (uint32_t)((f - (double)hi) * 4294967296.0);
      const uint64_t turn = (uint64_t)pos * ((uint64_t)hi << 32 | lo);
      sine_cosine((uint32_t)(turn >> 32), sn[e], cs[e]);
    }
  }
  const bool small_eps = p.eps < kSmallEps;
#pragma unroll
  for (int t = 0; t < kRopeTurns; ++t) {
    const int h = h0 + t * HP;
    if (h - lane / L >= all) break;             // the same for the wave
    const bool is_q = h < p.heads, on = h < all;
    float ya[4], yb[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      ya[e] = to_float<DT>((uint16_t)(xa[t][e >> 1] >> (16 * (e & 1))));
      yb[e] = to_float<DT>((uint16_t)(xb[t][e >> 1] >> (16 * (e & 1))));
    }
    if (p.eps >= 0.f) {
      float s = head_squares<L>(ya, yb), eps = p.eps;
      if constexpr (DT == WQ_DT_BF16) {
        if (small_eps || __any(!(s < kLargeSquares))) {
          asm volatile("");      // stays a branch
          rescale_head<L>(ya, yb, s, eps);
        }
      }
      const float inv = 1.f / sqrtf(__builtin_fmaf(s, 1.f / D, eps));
      const uint16_t* const w = is_q ? p.q.weight : p.k.weight;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        ya[e] *= inv;
        yb[e] *= inv;
      }
      if (w != nullptr) {
        const u2 wa = *reinterpret_cast<const u2*>(w + a), wb = *reinterpret_cast<const u2*>(w + b);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          ya[e] *= to_float<DT>((uint16_t)(wa[e >> 1] >> (16 * (e & 1))));
          yb[e] *= to_float<DT>((uint16_t)(wb[e >> 1] >> (16 * (e & 1))));
        }
      }
    }
    if (turns) {
      if constexpr (NEIGHBOURS) {               // pairs (0, 1), (2, 3) of a and of b
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float& x = e < 2 ? ya[2 * e] : yb[2 * e - 4];
          float& y = e < 2 ? ya[2 * e + 1] : yb[2 * e - 3];
          const float u = x * cs[e] - y * sn[e];
          y = y * cs[e] + x * sn[e];
          x = u;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = ya[e] * cs[e] - yb[e] * sn[e];
          yb[e] = yb[e] * cs[e] + ya[e] * sn[e];
          ya[e] = u;
        }
      }
    }
    if (on) {
      uint16_t* const out = is_q ? p.q.out + row * p.q.out_row + h * p.q.out_head
                                 : p.k.out + row * p.k.out_row + (h - p.heads) * p.k.out_head;
      uint16_t oa[4], ob[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        oa[e] = from_float<DT>(ya[e]);
        ob[e] = from_float<DT>(yb[e]);
      }
      *reinterpret_cast<u2*>(out + a) = u2{pack2(oa[0], oa[1]), pack2(oa[2], oa[3])};
      *reinterpret_cast<u2*>(out + b) = u2{pack2(ob[0], ob[1]), pack2(ob[2], ob[3])};
    }
  }
}

}  // namespace wqd

using namespace wqd;

static bool good_side(const wq_heads* s) {
  return aligned16(s->x) && aligned16(s->out) && aligned16(s->weight) && s->row_stride % 8 == 0 &&
         s->head_stride % 8 == 0 && s->out_row_stride % 8 == 0 && s->out_head_stride % 8 == 0 &&
         s->row_stride >= 0 && s->head_stride >= 0 && s->out_row_stride >= 0 &&
         s->out_head_stride >= 0;
}

extern "C" int wq_qk_norm_rope(int dtype, const wq_heads* q, const wq_heads* k, int64_t n_rows,
                               int64_t head_dim, float eps, const int32_t* positions,
                               const double* inv_freq, int64_t n_freq, int neighbours,
                               void* stream) {
  const char* who = "wq_qk_norm_rope";
  if (!q || !k) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL heads", who);
  if (dtype != WQ_DT_F16 && dtype != WQ_DT_BF16)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: dtype must be WQ_DT_F16 or WQ_DT_BF16", who);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256, got %lld", who,
                    (long long)head_dim);
  if (n_rows < 0 || n_rows > (1 << 24) || q->n_heads < 0 || q->n_heads > 65535 || k->n_heads < 0 ||
      k->n_heads > 65535)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (n_freq < 0 || n_freq % 4 || 2 * n_freq > head_dim)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: n_freq must be a multiple of 4 up to head_dim / 2, got %lld",
                    who, (long long)n_freq);
  if (eps != eps) return wq::fail(WQ_ERR_INVALID_ARG, "%s: eps is NaN", who);
  const int64_t heads = q->n_heads + k->n_heads;
  if (n_rows == 0 || heads == 0) return wq::ok();
  if ((q->n_heads && (!q->x || !q->out)) || (k->n_heads && (!k->x || !k->out)) ||
      (n_freq && (!positions || !inv_freq)))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned4(positions) || ((uintptr_t)inv_freq & 7u))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if ((q->n_heads && !good_side(q)) || (k->n_heads && !good_side(k)))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: pointers must be 16-byte aligned, strides multiples of 8 elements", who);
  for (const wq_heads* s : {q, k})
    if (s->n_heads && s->out == s->x &&
        ((n_rows > 1 && s->out_row_stride != s->row_stride) ||
         (s->n_heads > 1 && s->out_head_stride != s->head_stride)))
      return wq::fail(WQ_ERR_INVALID_ARG, "%s: in place, the output's strides must be the input's", who);
  for (const wq_heads* s : {q, k})
    if (s->n_heads && ((n_rows > 1 && s->out_row_stride < head_dim) ||
                       (s->n_heads > 1 && s->out_head_stride < head_dim)))
      return wq::fail(WQ_ERR_INVALID_ARG, "%s: the output's rows or heads overlap", who);
  const int64_t per = kRopeTurns * (512 / head_dim), chunks = (heads + per - 1) / per;
  const int64_t units = n_rows * chunks;
  if (units > 0x7FFFFFFFll) return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  auto side = [](const wq_heads* s) {
    return RopeSide{s->x, s->out, s->weight, s->row_stride, s->head_stride, s->out_row_stride, s->out_head_stride};
  };
  RopeArgs p{};
  p.q = side(q);
  p.k = side(k);
  p.positions = positions;
  p.freqs = inv_freq;
  p.units = units;
  p.heads = (int)q->n_heads;
  p.kv_heads = (int)k->n_heads;
  p.n_freq = (int)n_freq;
  p.eps = eps;
  p.chunks_by = Divisor(chunks);
  const dim3 grid((unsigned)((units + kRopeWaves - 1) / kRopeWaves));
  kv4_dispatch(dtype, head_dim, [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value;
    if (neighbours) rope_kernel<DT, D, true><<<grid, kRopeWaves * kWave, 0, (hipStream_t)stream>>>(p);
    else rope_kernel<DT, D, false><<<grid, kRopeWaves * kWave, 0, (hipStream_t)stream>>>(p);
  });
  return check_launch(who);
}
