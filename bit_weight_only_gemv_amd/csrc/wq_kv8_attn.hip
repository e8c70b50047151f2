// Attention over the paged 8-bit key/value cache and the softmax weights that its
// tokens get (wq.h, "8-bit key/value cache"), on the matrix cores.
//
// A workgroup takes 16 columns, (row, head) pairs of one key/value head, and its
// waves pages of 64 tokens in turn.  With a block's exponents e (keys) and f (values),
//   logit = scale 2^e (code . Q),   out_d = sum_t (p_t 2^f) code_{t,d},
// both 16x16x32 products of FP16 operands.  A code is an FP16 number (one byte
// permute makes 1024 + 128 + q of two, one packed subtraction q), so its products
// are exact; the powers of two go into the exponential's argument.  Tokens are the
// rows of the first product, so a lane ends with 4 tokens of one column per block,
// and two blocks are just its 8 k of the second product's B operand: the weights
// never leave their registers.
//
// Precision.  Queries are scaled by a power of two, the largest channel to [2^14,
// 2^15), and so are exact in FP16, of either type, down to 2^-24 of the largest;
// smaller ones are off by 2^-35 of it at most.  Logits, maxima and sums are FP32.
// A weight p 2^f is an FP16 number and its FP16 remainder (22 bits): rounded to 11
// bits it shows where values of both signs nearly cancel.  Weights are relative to a
// reference that follows logit + f both ways: a page whose largest weight would
// pass 2^14 or stay below 2^2 sets it to that, where weights carry 2^10.  So 22
// bits hold for what counts in a page, however small the page's share is, and most
// pages are spared the cross-lane maximum and the rescale of the sums.  (Both parts end
// at 2^-24, 2^-26 of 2^2: tokens far below their page's largest weight have fewer bits, which
// shows only where that one's values are nearly zero.)  The
// reference stays within 2^64 of the highest and f within [-24, 10], so that FP32
// holds the sums.
//
// What bounds it (traced times).  One token a sequence over a long cache: the cache's
// bytes.  Four sequences of 131072 tokens, 8 heads of 128 channels, 1074 MB: 185 us,
// 5.8 TB/s, where a plain read reaches 5.6; a page costs a wave 435 vector and 48
// matrix instructions, at two waves a SIMD.  32 sequences of up to 8191 tokens, 361 MB:
// 73 us, the last of it with few workgroups at work (the longest sequences' splits).
// Many rows: instructions of both kinds (617 vector and 96 matrix ones a page and wave
// with two column tiles) and uneven sequences: two prompts, 267 and 458 rows over 6000 and
// 3967 tokens, take 105 us for 54 GFLOP.  Where it takes 110 (runs differ by that much), it
// takes 96 without the remainders' products, 104 without the exponentials, and 110 without
// the conversions of codes.  Short caches: latency, 7.7 us for 500 tokens.

#include "wq_attn.cuh"
#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"
#include "wq_kv8.cuh"

namespace wqd {

// 8 codes (bytes q + 128) as a matrix-core operand.
__device__ __forceinline__ h8 codes8(uint32_t w0, uint32_t w1) {
  const h2 bias = {(_Float16)1152.f, (_Float16)1152.f};
  const uint32_t magic = 0x64646464u;
  const h2 a = as_h2(__builtin_amdgcn_perm(magic, w0, 0x04010400u)) - bias;
  const h2 b = as_h2(__builtin_amdgcn_perm(magic, w0, 0x04030402u)) - bias;
  const h2 c = as_h2(__builtin_amdgcn_perm(magic, w1, 0x04010400u)) - bias;
  const h2 d = as_h2(__builtin_amdgcn_perm(magic, w1, 0x04030402u)) - bias;
  return __builtin_bit_cast(h8, u4v{as_u32(a), as_u32(b), as_u32(c), as_u32(d)});
}

// A column's query: raw as loaded (8 channels 32 g + 8 r of group g), then scaled, and
// its factor: logits to base 2 are factor 2^e (code . Q).
template <int G>
struct Query {
  u4v raw[G];
  h8 q[G];
  float factor;
  __device__ __forceinline__ void load(const uint16_t* __restrict__ src, bool on) {
#pragma unroll
    for (int g = 0; g < G; ++g)
      raw[g] = on ? *reinterpret_cast<const u4v*>(src + 32 * g) : u4v{0, 0, 0, 0};
  }
  template <int DT>
  __device__ __forceinline__ void scale(float by) {
    float top = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        top = fmaxf(top, fabsf(to_float<DT>((uint16_t)(raw[g][i >> 1] >> (16 * (i & 1))))));
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
    e = top == 0.f || e > 127 ? 14 : max(e, -100);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[g][i] = (_Float16)ldexpf(to_float<DT>((uint16_t)(raw[g][i >> 1] >> (16 * (i & 1)))), 14 - e);
    factor = ldexpf(by * 1.44269504f, e - 14);
  }
};

// A page's keys of one head: block u, channels 64 c + 32 (0, 1) + 8 r of token l.
template <int D>
struct Keys8 {
  static constexpr int C = D / 64;
  u4v codes[4][C];
  __device__ __forceinline__ void load(const uint8_t* __restrict__ page, uint32_t lane) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int c = 0; c < C; ++c)
        codes[u][c] = *reinterpret_cast<const u4v*>(page + u * (16 * D) + c * 1024 + lane * 16);
  }
};

// The sequence of place n when they are ordered by length, longest first (of more than
// 64 sequences: the n-th as they come).  Two prompts of 267 and 458 rows over 6000 and
// 3967 tokens take 110 us so, and 115 with both side by side.
__device__ __forceinline__ int nth_longest(const KvRows& a, int n, int lane) {
  if (a.seqs < 2 || a.seqs > kWave) return n;
  const int len = lane < a.seqs ? a.lens[lane] : INT32_MIN;
  int before = 0;
  for (int i = 0; i < a.seqs; ++i) {
    const int x = __builtin_amdgcn_readlane(len, i);
    before += x > len || (x == len && i < lane);
  }
  return __builtin_ctzll(__ballot(lane < a.seqs && before == n));
}

struct Attn8Args {
  KvRows a;
  const uint8_t* data;
  const uint32_t* exps;   // [page][head][2]
  int64_t n_pages;
  Divisor kv_heads_by, group_by, parts_by, splits_by;
  int kv_heads, window, tiles, splits, split_pages;
  float scale;
  uint16_t* out;
  float* lse;
  float* part;            // [row][head][split][D], then [row][head][split][4]: sum, reference, sum
};

template <int DT, int D, int NW, int CT>
__global__ void __launch_bounds__(NW * kWave, D == 256 ? 1 : 2) attn8_kernel(Attn8Args p) {
  constexpr int G = D / 32, J = D / 16;
  constexpr int kPart = (4 * J + 2) * 64;     // floats a wave leaves in LDS, a column tile
  extern __shared__ __attribute__((aligned(16))) float s_merge[];
  const KvRows& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 4, l = lane & 15;
  const int R = (int)p.group_by.d;

  // Heads vary fastest: workgroups that read the same pages are a multiple of the heads
  // apart and so, for 8 heads and their multiples, on the same XCD.  Long sequences
  // come first, and of their column tiles the last, which see the most tokens: what
  // starts late is short.
  const int rest = p.kv_heads_by.div(blockIdx.x), kvh = blockIdx.x - rest * p.kv_heads;
  const int place = p.parts_by.div(rest), part = rest - place * p.parts_by.d;
  const int turn = p.splits_by.div(part), split = part - turn * p.splits;
  const int tile0 = p.tiles - 1 - turn;
  const int b = nth_longest(a, place, lane);
  const int32_t* const table = a.table + (int64_t)b * a.width;
  // the wave's first page numbers, read at the same time as the lengths: where the
  // hints hold, a split starts here
  const int guess_at = split * p.split_pages + wave + NW * lane;
  const int guess = guess_at < a.width ? table[guess_at] : -1;
  const int row0 = max(a.cu[b], 0);
  const int n = max(min(max(a.cu[b + 1], 0), a.rows) - row0, 0);   // rows of the call for any cu_rows
  const int len = max(a.lens[b], 0);
  const int cols = n * R;
  const int64_t stride = (int64_t)p.kv_heads * (128 * D);
  const uint8_t* const base = p.data + (int64_t)kvh * (128 * D);
  const uint32_t* const exps = p.exps + 2 * kvh;

  for (int tile = tile0; tile * (16 * CT) < cols; tile += p.tiles) {
    const int c_hi = min(tile * (16 * CT) + 16 * CT - 1, cols - 1);
    const int pos_lo = len - n + p.group_by.div(tile * (16 * CT));
    const int pos_hi = len - n + p.group_by.div(c_hi);
    const int64_t pages64 = ((int64_t)pos_hi + 64) / 64;
    const int pages = (int)(pages64 < a.width ? pages64 : a.width);
    const int first = p.window > 0 ? max(pos_lo - p.window + 1, 0) / 64 : 0;
    const int total = max(pages - first, 0);
    const int per = max(p.split_pages, p.splits_by.div(total + p.splits - 1));
    const int j0 = min(split * per, total), j1 = min(j0 + per, total);
    const int count = (j1 - j0 - wave + NW - 1) / NW;

    // the wave's next page.  Lanes hold the places, numbers and exponents of 64 pages
    // at a time.
    int k = -1, held_at = 0, held_id = 0, at = -1;
    u2 held_exp = {0, 0};
    uint32_t exp_k = 0, exp_v = 0;
    const uint8_t* src = base;
    auto next = [&]() {
      for (at = -1; ++k < count;) {
        if ((k & 63) == 0) {
          const int j = j0 + wave + NW * (k + lane);
          held_at = j < j1 ? first + j : -1;
          held_id = -1;
          if (held_at >= 0 && held_at < pages)
            held_id = k == 0 && per == p.split_pages && first == 0 ? guess : table[held_at];
          if (held_id < 0 || held_id >= p.n_pages) held_id = -1;
          if (held_id >= 0)
            held_exp = *reinterpret_cast<const u2*>(exps + (int64_t)held_id * (2 * p.kv_heads));
        }
        const int id = __builtin_amdgcn_readlane(held_id, k & 63);
        if (id < 0) continue;      // no tokens there
        at = __builtin_amdgcn_readlane(held_at, k & 63);
        src = base + id * stride;
        break;
      }
    };
    Keys8<D> kt;
    u4v vt[J];
    auto load_values = [&]() {
#pragma unroll
      for (int j = 0; j < J; ++j)
        vt[j] = *reinterpret_cast<const u4v*>(src + 64 * D + j * 1024 + lane * 16);
    };
    auto load_exponents = [&]() {
      exp_k = __builtin_amdgcn_readlane(held_exp[0], k & 63);
      exp_v = __builtin_amdgcn_readlane(held_exp[1], k & 63);
    };
    // this lane's column, its query's loads ahead of the pages' and its scaling behind
    int row[CT], head[CT], pos[CT];
    Query<G> Q[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int col = tile * (16 * CT) + 16 * ct + l;
      const bool on = col < cols;
      const int nth = p.group_by.div(col);
      row[ct] = on ? row0 + nth : -1;
      head[ct] = kvh * R + col - nth * R;
      pos[ct] = on ? len - n + nth : -1;
      Q[ct].load(a.q + (on ? row[ct] * a.q_row + head[ct] * a.q_head : 0) + 8 * r, on);
    }
    next();
    if (at >= 0) {
      kt.load(src, lane);
      load_values();
      load_exponents();
    }
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) Q[ct].template scale<DT>(p.scale);

    f4 O[CT][J];
    float m[CT];            // the reference
    float least[CT];        // the lowest that it may be
    float sum[CT];          // this lane's weights without 2^f
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      m[ct] = least[ct] = -INFINITY;
      sum[ct] = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) O[ct][j] = f4{0, 0, 0, 0};
    }

    while (at >= 0) {
      const int t0 = at * 64;
      f4 sc[CT][4];
      unroll<4>([&](auto u) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) sc[ct][u] = f4{0, 0, 0, 0};
        unroll<G>([&](auto g) {
          const u4v w = kt.codes[u][g / 2];
          const h8 ka = codes8(w[2 * (g % 2)], w[2 * (g % 2) + 1]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) sc[ct][u] = mfma(ka, Q[ct].q[g], sc[ct][u]);
        });
      });
      int ek[4], ev[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ek[u] = exponent8(exp_k, u);
        ev[u] = exponent8(exp_v, u);
      }
      // the keys' registers are free: the next page's keys arrive behind the values'
      // product, its values behind the next logits
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int u = 0; u < 4; ++u) asm volatile("" : "+v"(sc[ct][u]));   // done here, not after the loads
      __builtin_amdgcn_sched_barrier(0);
      auto next_keys = [&]() {
        next();
        kt.load(src, lane);        // past the last page: that page's again, not used
        load_exponents();
        __builtin_amdgcn_sched_barrier(0);
      };
      if constexpr (CT == 1) next_keys();

      // base-2 logits and the values' exponent above the reference, plus kWeightExp
      float y[CT][16], top[CT];
      bool raise = false;
      uint64_t lower = 0;     // bit l: column l's four lanes
      const bool edge = t0 + 63 > pos_lo || (p.window > 0 && t0 <= pos_hi - p.window);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const bool none = m[ct] == -INFINITY;
        const float m8 = none ? -kWeightExp : m[ct] - kWeightExp;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float c = ldexpf(Q[ct].factor, ek[u]), d = (float)ev[u] - m8;
#pragma unroll
          for (int i = 0; i < 4; ++i) y[ct][4 * u + i] = __builtin_fmaf(sc[ct][u][i], c, d);
        }
        if (edge) {
          // stays a branch: few pages have an edge.  The distance of the column's position
          // from the lane's first token
          int rel = pos[ct] - t0 - 4 * r;
          asm volatile("" : "+v"(rel));
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int t = 16 * (i >> 2) + (i & 3);
            if (t > rel || (p.window > 0 && t <= rel - p.window)) y[ct][i] = -INFINITY;
          }
        }
        top[ct] = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) top[ct] = fmaxf(top[ct], y[ct][i]);
        raise |= top[ct] > (none ? -INFINITY : kWeightExp + kRaise);
        const uint64_t low = __ballot(top[ct] < kWeightExp - kLower && m[ct] > least[ct]);
        lower |= low & low >> 16 & low >> 32 & low >> 48;
      }
      if (__any(raise) || (lower & 0xFFFFu) != 0) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const bool none = m[ct] == -INFINITY;
          float most = fmaxf(top[ct], __shfl_xor(top[ct], 16));
          most = fmaxf(most, __shfl_xor(most, 32));
          // the reference in y's scale stands at kWeightExp
          float up = most == -INFINITY ? 0.f : most - kWeightExp;
          if (!none && up < 0.f) up = up < -kLower ? fmaxf(up, least[ct] - m[ct]) : 0.f;
          const float f = none ? 0.f : __builtin_amdgcn_exp2f(-up);
          if (!none) m[ct] += up;
          else if (most != -INFINITY) m[ct] = up;
          least[ct] = fmaxf(least[ct], m[ct] - kBelow);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[ct][i] -= up;
#pragma unroll
          for (int j = 0; j < J; ++j) O[ct][j] *= f;
          sum[ct] *= f;
        }
      }
      h8 wh[CT][2], wl[CT][2];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int i = 0; i < 16; ++i) y[ct][i] = __builtin_amdgcn_exp2f(y[ct][i]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          sum[ct] = __builtin_fmaf((y[ct][4 * u] + y[ct][4 * u + 1]) + (y[ct][4 * u + 2] + y[ct][4 * u + 3]),
                                   pow2(-ev[u]), sum[ct]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u4v wv, rv;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            // both parts cut, not rounded: the remainder takes what the first leaves, and
            // the second's error is below 2^-21
            const float y0 = y[ct][8 * h + 2 * x], y1 = y[ct][8 * h + 2 * x + 1];
            const h2 w = __builtin_bit_cast(h2, __builtin_amdgcn_cvt_pkrtz(y0, y1));
            wv[x] = as_u32(w);
            rv[x] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(
                __builtin_fmaf((float)w[0], -1.f, y0), __builtin_fmaf((float)w[1], -1.f, y1)));
          }
          wh[ct][h] = __builtin_bit_cast(h8, wv);
          wl[ct][h] = __builtin_bit_cast(h8, rv);
        }
      }
      if constexpr (CT > 1) {      // here, where the logits have left their registers
        __builtin_amdgcn_sched_barrier(0);
        next_keys();
      }
      unroll<J>([&](auto j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const h8 va = codes8(vt[j][2 * h], vt[j][2 * h + 1]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            O[ct][j] = mfma(va, wh[ct][h], O[ct][j]);
            O[ct][j] = mfma(va, wl[ct][h], O[ct][j]);
          }
        }
      });
      __builtin_amdgcn_sched_barrier(0);
      load_values();
    }

    // the waves' parts joined in order
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float* const s = s_merge + (wave * CT + ct) * kPart;
      sum[ct] += __shfl_xor(sum[ct], 16);
      sum[ct] += __shfl_xor(sum[ct], 32);
#pragma unroll
      for (int j = 0; j < J; ++j) reinterpret_cast<f4*>(s)[j * 64 + lane] = O[ct][j];
      s[4 * J * 64 + lane] = sum[ct];
      s[(4 * J + 1) * 64 + lane] = m[ct];
    }
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (row[ct] < 0) continue;
      auto part_of = [&](int w) { return s_merge + (w * CT + ct) * kPart; };
      float mw[NW], mx = -INFINITY, all = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        mw[w] = part_of(w)[(4 * J + 1) * 64 + lane];
        mx = fmaxf(mx, mw[w]);
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        mw[w] = mw[w] == mx ? 1.f : __builtin_amdgcn_exp2f(mw[w] - mx);
        all += mw[w] * part_of(w)[4 * J * 64 + lane];
      }
      const int64_t out_at = (int64_t)row[ct] * a.heads + head[ct];
      const float inv = all == 0.f ? 0.f : 1.f / all;
      for (int j = wave; j < J; j += NW) {
        f4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) o += mw[w] * reinterpret_cast<const f4*>(part_of(w))[j * 64 + lane];
        const int d = 16 * j + 4 * r;
        if (p.splits == 1) {
          uint16_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = from_float<DT>(all == 0.f ? 0.f : o[i] * inv);
          *reinterpret_cast<u2*>(p.out + out_at * D + d) = u2{pack2(h[0], h[1]), pack2(h[2], h[3])};
        } else {
          *reinterpret_cast<f4*>(p.part + (out_at * p.splits + split) * D + d) = o;
        }
      }
      if (wave == 0 && r == 0) {
        if (p.splits == 1) {
          if (p.lse != nullptr) p.lse[out_at] = log_sum(all, mx);
        } else {
          reinterpret_cast<f4*>(p.part + (int64_t)a.rows * a.heads * p.splits *
                                             D)[out_at * p.splits + split] = f4{all, mx, all, 0.f};
        }
      }
    }
    __syncthreads();
  }
}

// How a call is split: column tiles of a sequence and splits of its pages.  Hints
// past what the call can have count as that, so that nothing overflows; there is at
// least one row and one sequence.
struct Attn8Plan {
  int64_t pairs, tiles, splits, split_pages;
  int waves, ct;            // waves a workgroup, column tiles a wave
};
static Attn8Plan attn8_plan(const wq_kv8_cache* c, const wq_kv4_rows* a, int64_t max_rows,
                            int64_t max_len) {
  Attn8Plan p{};
  const int64_t R = a->n_heads / c->n_kv_heads;
  if (max_rows > a->n_rows) max_rows = a->n_rows;
  if (max_len > 64 * a->table_width) max_len = 64 * a->table_width;
  const int64_t cols = (max_rows < 1 ? 1 : max_rows) * R;
  // Two column tiles share the codes' conversion where there are enough of them: the same
  // prompts take 110 us with two, 128 with one, and 384 with four, whose registers spill.
  // Heads of 256 channels would not fit either.
  p.ct = c->head_dim <= 128 && cols >= 64 ? 2 : 1;
  p.tiles = (cols + 16 * p.ct - 1) / (16 * p.ct);
  p.pairs = a->n_seqs * c->n_kv_heads;
  int64_t pages = (max_len + 63) / 64;
  if (pages < 1) pages = 1;
  // Two workgroups of 4 waves for every compute unit, as many as run at once (one with
  // heads of 256 channels): finer splits cost more in parts to be joined than they even
  // out (32 sequences of up to 8191 tokens: 78 us, in one and a half to three rounds 81 to
  // 87).  A split has at least two pages a wave, one while that leaves compute units idle.
  // All sequences have as many tiles and splits as the largest could need: a few rows beside
  // a prompt's many, or tokens far fewer than max_len, leave compute units idle.
  const int64_t items = p.pairs * p.tiles, at_once = c->head_dim == 256 ? 256 : 512;
  int64_t splits = (at_once + items - 1) / items;
  const int64_t waves = items * ((pages + kAttnWaves - 1) / kAttnWaves) <= 256 ? kAttnWaves : 2 * kAttnWaves;
  const int64_t most = (pages + waves - 1) / waves;
  if (splits > most) splits = most;
  // few pages for few workgroups: one workgroup of up to 8 waves, and no second launch
  p.waves = kAttnWaves;
  if (items <= 256 && pages <= 2 * kAttnMoreWaves) {
    splits = 1;
    if (pages > kAttnWaves && p.ct == 1 && c->head_dim <= 128) p.waves = kAttnMoreWaves;
  }
  p.split_pages = (pages + splits - 1) / splits;
  p.splits = (pages + p.split_pages - 1) / p.split_pages;
  return p;
}

// ------------------------------------------------------------- accumulate
// mass[b][kvh][t] += sum over the rows' heads of the group of exp(logit - lse).  Every
// page belongs to one wave (few columns) or workgroup (many), so no sum crosses
// workgroups and the order is fixed; keys alone are read.
struct Mass8Args {
  KvRows a;
  const uint8_t* data;
  const uint32_t* exps;
  int64_t n_pages;
  Divisor kv_heads_by, group_by, pairs_by;
  int kv_heads, window;
  float scale;
  const float* lse;
  const int32_t* held;
  float* mass;
  int64_t mass_tokens;
  // scaled queries in the order of the matrix cores' operands, and a column's factor, lse to
  // base 2 and position: per key/value head `col_tiles` column tiles, of which those of
  // sequence b begin at mass8_first_tile
  h8* queries;            // [kvh][tile][D / 32][64 lanes]
  f4* columns;            // [kvh][tile][16]
  int64_t col_tiles;
};

// The column tiles of the rows before a sequence's, each sequence's last one partly used:
// no more than this.
__device__ __forceinline__ int64_t mass8_first_tile(int row0, int R, int b) {
  return (int64_t)row0 * R / 16 + b;
}

// Sums of v[0..15] over the 16 lanes of a row: lane l ends with that of v[l].  Each
// step leaves a lane the half of the sums that its bit of l names.
__device__ __forceinline__ float row16_transposed(const float (&v)[16], int l) {
  float a[8], b[4], c[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = (l & 8 ? v[i + 8] : v[i]) + dpp_mov<0x128>(l & 8 ? v[i] : v[i + 8]);   // row_ror:8
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = (l & 4 ? a[i + 4] : a[i]) + dpp_mov<0x141>(l & 4 ? a[i] : a[i + 4]);   // row_half_mirror
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = (l & 2 ? b[i + 2] : b[i]) + dpp_mov<0x4E>(l & 2 ? b[i] : b[i + 2]);    // quad_perm [2,3,0,1]
  return (l & 1 ? c[1] : c[0]) + dpp_mov<0xB1>(l & 1 ? c[0] : c[1]);                                         // quad_perm [1,0,3,2]
}

// A pair's (sequence and key/value head) part of the call.
struct Mass8Pair {
  int b, kvh, row0, n, len, held, cols, pages;
  int skip;               // the first pages of these have left the window, and their masses stay
  int64_t tokens;
  const int32_t* table;
  float* mass;
  __device__ __forceinline__ Mass8Pair(const Mass8Args& p, int pair) {
    const KvRows& a = p.a;
    b = p.kv_heads_by.div(pair);
    kvh = pair - b * p.kv_heads;
    row0 = max(a.cu[b], 0);
    n = max(min(max(a.cu[b + 1], 0), a.rows) - row0, 0);   // rows of the call for any cu_rows
    len = max(a.lens[b], 0);
    held = p.held[b];
    cols = n * (int)p.group_by.d;
    tokens = min((int64_t)len, p.mass_tokens);
    pages = (int)min((tokens + 63) / 64, a.width);
    skip = p.window > 0 ? max(min(len - n - p.window + 1, min(held, len)), 0) / 64 : 0;
    table = a.table + (int64_t)b * a.width;
    mass = p.mass + ((int64_t)b * p.kv_heads + kvh) * p.mass_tokens;
  }
};

// The weights of a block's four tokens in a lane, added to acc.
template <bool EDGE>
__device__ __forceinline__ void add_weights(f4 sc, float c, float lse, int t, int pos, int window, float* acc) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float y = __builtin_fmaf(sc[i], c, -lse);
    if (EDGE && (t + i > pos || (window > 0 && t + i <= pos - window))) y = -INFINITY;
    acc[i] += __builtin_amdgcn_exp2f(y);
  }
}

// Few columns (decoding): up to CT column tiles of queries stay in registers, every wave
// takes pages of its own, the next page's keys under way behind this one's logits.
// Bytes and latency: 32 sequences of up to 8191 tokens, 8 heads of 128 channels, 191 MB
// in 42 us (4.5 TB/s; 55 with the queries made anew for every page).
template <int DT, int D, int CT>
__global__ void __launch_bounds__(kAttnWaves * kWave, 2) mass8_few_kernel(Mass8Args p) {
  constexpr int G = D / 32;
  const KvRows& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 4, l = lane & 15;
  const int R = (int)p.group_by.d;
  const int rest = p.pairs_by.div(blockIdx.x);
  const Mass8Pair o(p, blockIdx.x - rest * p.pairs_by.d);
  const int step = (gridDim.x / p.pairs_by.d) * kAttnWaves, first = o.skip + rest * kAttnWaves + wave;
  const int count = first < o.pages ? (o.pages - first + step - 1) / step : 0;
  if (count == 0) return;
  const int64_t stride = (int64_t)p.kv_heads * (128 * D);
  const uint8_t* const base = p.data + (int64_t)o.kvh * (128 * D);
  const int tok = 16 * (l >> 2) + 4 * r + (l & 3);       // the token whose sum this lane ends with

  // more columns than the hint promised take more rounds over the pages
  for (int tile = 0; tile == 0 || tile * 16 < o.cols; tile += CT) {
    Query<G> Q[CT];
    float lse[CT];
    int pos[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int col = (tile + ct) * 16 + l, nth = p.group_by.div(col);
      const int row = o.row0 + nth, head = o.kvh * R + col - nth * R;
      const bool in = col < o.cols;
      const float x = in ? p.lse[(int64_t)row * a.heads + head] : INFINITY;
      const bool on = in && fabsf(x) < INFINITY;         // else its weights are exp(0 - inf)
      lse[ct] = on ? x * 1.44269504f : INFINITY;
      pos[ct] = on ? o.len - o.n + nth : -1;
      Q[ct].load(a.q + (on ? row * a.q_row + head * a.q_head : 0) + 8 * r, on);
    }
    const int c_lo = min(tile * 16, max(o.cols - 1, 0)), c_hi = max(min((tile + CT) * 16, o.cols) - 1, 0);
    const int pos_lo = o.len - o.n + p.group_by.div(c_lo), pos_hi = o.len - o.n + p.group_by.div(c_hi);

    int k = -1, held_id = -1, id = -1, at = -1;
    uint32_t held_exp = 0, exp_k = 0;
    float old = 0.f;
    Keys8<D> kt;
    auto next = [&]() {      // the wave's next page (at: past the last, -1), its keys' loads
      if (++k >= count) {
        at = -1;
        return;
      }
      if ((k & 63) == 0) {
        const int j = first + step * (k + lane);
        held_id = k + lane < count ? o.table[j] : -1;
        if (held_id < 0 || held_id >= p.n_pages) held_id = -1;
        if (held_id >= 0) held_exp = p.exps[2 * ((int64_t)held_id * p.kv_heads + o.kvh)];
      }
      at = first + step * k;
      id = __builtin_amdgcn_readlane(held_id, k & 63);
      if (p.window > 0 && at * 64 + 63 <= pos_lo - p.window) id = -1;     // none of these rows sees it
      exp_k = __builtin_amdgcn_readlane(held_exp, k & 63);
      if (id >= 0) kt.load(base + id * stride, lane);
      const int t = at * 64 + tok;
      old = t < o.tokens && (t < o.held || tile > 0) ? o.mass[t] : 0.f;
    };
    next();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) Q[ct].template scale<DT>(p.scale);
    while (at >= 0) {
      const int t0 = at * 64, id_now = id;
      const uint32_t exp_now = exp_k;
      const float old_now = old;
      f4 sc[CT][4];
      unroll<4>([&](auto u) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) sc[ct][u] = f4{0, 0, 0, 0};
        unroll<G>([&](auto g) {
          const u4v w = kt.codes[u][g / 2];
          const h8 ka = codes8(w[2 * (g % 2)], w[2 * (g % 2) + 1]);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) sc[ct][u] = mfma(ka, Q[ct].q[g], sc[ct][u]);
        });
      });
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int u = 0; u < 4; ++u) asm volatile("" : "+v"(sc[ct][u]));   // done here, not after the loads
      __builtin_amdgcn_sched_barrier(0);
      next();
      __builtin_amdgcn_sched_barrier(0);
      float acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = 0.f;
      if (id_now >= 0) {
        const bool edge = t0 + 63 > pos_lo || (p.window > 0 && t0 <= pos_hi - p.window);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float c = ldexpf(Q[ct].factor, exponent8(exp_now, u));
            const int t = t0 + 16 * u + 4 * r;
            if (edge) add_weights<true>(sc[ct][u], c, lse[ct], t, pos[ct], p.window, acc + 4 * u);
            else add_weights<false>(sc[ct][u], c, lse[ct], t, pos[ct], p.window, acc + 4 * u);
          }
      }
      const float s = row16_transposed(acc, l);
      if (t0 + tok < o.tokens) o.mass[t0 + tok] = old_now + s;
    }
  }
}

// Many columns (prompts): the queries scaled and laid out once.
template <int DT, int D>
__global__ void __launch_bounds__(kAttnWaves * kWave) scale8_kernel(Mass8Args p) {
  constexpr int G = D / 32;
  const KvRows& a = p.a;
  const int lane = threadIdx.x & 63, r = lane >> 4, l = lane & 15;
  const int R = (int)p.group_by.d;
  const int rest = p.pairs_by.div(blockIdx.x);
  const Mass8Pair o(p, blockIdx.x - rest * p.pairs_by.d);
  const int64_t at = (int64_t)o.kvh * p.col_tiles + mass8_first_tile(o.row0, R, o.b);
  const int step = (gridDim.x / p.pairs_by.d) * kAttnWaves;
  for (int tile = rest * kAttnWaves + (threadIdx.x >> 6); tile * 16 < o.cols; tile += step) {
    const int col = tile * 16 + l, nth = p.group_by.div(col);
    const int row = o.row0 + nth, head = o.kvh * R + col - nth * R;
    const float x = col < o.cols ? p.lse[(int64_t)row * a.heads + head] : INFINITY;
    const bool on = fabsf(x) < INFINITY;               // else its weights are exp(0 - inf)
    Query<G> q;
    q.load(a.q + (on ? row * a.q_row + head * a.q_head : 0) + 8 * r, on);
    q.template scale<DT>(p.scale);
#pragma unroll
    for (int g = 0; g < G; ++g) p.queries[((at + tile) * G + g) * kWave + lane] = q.q[g];
    if (r == 0)
      p.columns[(at + tile) * 16 + l] = f4{q.factor, on ? x * 1.44269504f : INFINITY,
                                           __builtin_bit_cast(float, on ? o.len - o.n + nth : -1), 0.f};
  }
}

// Two pages a workgroup, two waves each: a page's keys stay in a wave's registers as
// FP16 numbers while it goes through every second column tile, the next one's loads
// ahead.  Vector instructions bound it, 73 a tile and page, 16 of them exponentials,
// beside 16 matrix ones: 267 and 458 rows over 6000 and 3967 tokens, 27 GFLOP, take 42 us
// with the scaling (one page a workgroup 50, four waves a page 52, one wave a page 58 to
// 68; with the columns' places found in the loop 76).
constexpr int kMass8Pages = 2, kMass8Turns = 2;
template <int D>
__global__ void __launch_bounds__(kMass8Pages* kMass8Turns* kWave, 2) mass8_many_kernel(Mass8Args p) {
  constexpr int G = D / 32;
  __shared__ float s_sum[kMass8Pages][kMass8Turns][kWave];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 4, l = lane & 15;
  const int R = (int)p.group_by.d;
  const int rest = p.pairs_by.div(blockIdx.x);
  const Mass8Pair o(p, blockIdx.x - rest * p.pairs_by.d);
  const int step = (gridDim.x / p.pairs_by.d) * kMass8Pages;
  const int pg = wave / kMass8Turns, turn = wave % kMass8Turns;
  const int tok = 16 * (l >> 2) + 4 * r + (l & 3);
  const int64_t first = (int64_t)o.kvh * p.col_tiles + mass8_first_tile(o.row0, R, o.b);
  const h8* const queries = p.queries + first * (G * kWave) + lane;
  const f4* const columns = p.columns + first * 16 + l;

  for (int at0 = o.skip + rest * kMass8Pages; at0 < o.pages; at0 += step) {
    const int at = at0 + pg, t0 = at * 64;
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    const int id = at < o.pages ? __builtin_amdgcn_readfirstlane(o.table[at]) : -1;
    if (id >= 0 && id < p.n_pages) {
      const int64_t ph = (int64_t)id * p.kv_heads + o.kvh;
      Keys8<D> kt;
      kt.load(p.data + ph * (128 * D), lane);
      const uint32_t exp_k = p.exps[2 * ph];
      // the rows that see some of the page, from the first one on to where the window
      // has passed it; of those [whole0, whole1) see all of it
      const int64_t from = (int64_t)t0 - (o.len - o.n), n = o.n;
      auto row_in = [&](int64_t row) { return min(max(row, (int64_t)0), n); };
      const int64_t to = p.window > 0 ? row_in(from + 63 + p.window) : n;
      const int tile0 = (int)(row_in(from) * R / 16), tiles = (int)((to * R + 15) / 16);
      const int whole0 = (int)((row_in(from + 63) * R + 15) / 16);
      const int whole1 = p.window > 0 ? (int)(row_in(from + p.window) * R / 16) : tiles;
      h8 q_next[G];
      f4 col_next;
      auto load = [&](int tile) {
#pragma unroll
        for (int g = 0; g < G; ++g) q_next[g] = queries[((int64_t)tile * G + g) * kWave];
        col_next = columns[(int64_t)tile * 16];
      };
      int tile = tile0 + turn;
      if (tile < tiles) load(tile);
      h8 ka[4][G];
      float by[4];
      unroll<4>([&](auto u) {
        by[u] = pow2(exponent8(exp_k, u));
        unroll<G>([&](auto g) {
          const u4v w = kt.codes[u][g / 2];
          ka[u][g] = codes8(w[2 * (g % 2)], w[2 * (g % 2) + 1]);
        });
      });
      for (; tile < tiles; tile += kMass8Turns) {
        h8 q[G];
#pragma unroll
        for (int g = 0; g < G; ++g) q[g] = q_next[g];
        const f4 col = col_next;
        if (tile + kMass8Turns < tiles) load(tile + kMass8Turns);
        const float pos_bits = col[2];       // a bit cast of the element itself takes the first one
        const int pos = __builtin_bit_cast(int, pos_bits);
        const bool edge = tile < whole0 || tile >= whole1;
        unroll<4>([&](auto u) {
          f4 sc = {0, 0, 0, 0};
          unroll<G>([&](auto g) { sc = mfma(ka[u][g], q[g], sc); });
          const float c = col[0] * by[u];
          const int t = t0 + 16 * u + 4 * r;
          if (edge) add_weights<true>(sc, c, col[1], t, pos, p.window, acc + 4 * u);
          else add_weights<false>(sc, c, col[1], t, pos, p.window, acc + 4 * u);
        });
      }
    }
    s_sum[pg][turn][lane] = row16_transposed(acc, l);
    __syncthreads();
    if (turn == 0 && at < o.pages) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kMass8Turns; ++i) s += s_sum[pg][i][lane];
      const int t = t0 + tok;
      if (t < o.tokens) o.mass[t] = t < o.held ? o.mass[t] + s : s;
    }
    __syncthreads();
  }
}

// Up to two column tiles stay in registers; more are many.
static int mass8_tiles(const wq_kv8_cache* c, const wq_kv4_rows* a, int64_t max_rows) {
  if (max_rows > a->n_rows) max_rows = a->n_rows;
  const int64_t cols = (max_rows < 1 ? 1 : max_rows) * (a->n_heads / c->n_kv_heads);
  return cols <= 16 ? 1 : cols <= 32 ? 2 : 3;
}

}  // namespace wqd

using namespace wqd;

static int check_attention8(const wq_kv8_cache* cache, const wq_kv4_rows* rows, int64_t max_rows,
                            int64_t max_len, const char* who) {
  if (int e = kv8_check_cache(cache, who)) return e;
  const wq_kv4_cache shape = kv8_shape(cache);
  if (int e = kv4_check_rows(&shape, rows, who)) return e;
  if (max_rows < 0 || max_len < 0) return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  return WQ_OK;
}

extern "C" int64_t wq_kv8_attention_workspace(const wq_kv8_cache* cache, const wq_kv4_rows* rows,
                                              int64_t max_rows, int64_t max_len) {
  if (int e = check_attention8(cache, rows, max_rows, max_len, "wq_kv8_attention_workspace")) return e;
  wq::ok();
  if (rows->n_rows == 0 || rows->n_seqs == 0) return 0;
  const Attn8Plan p = attn8_plan(cache, rows, max_rows, max_len);
  if (p.splits == 1) return 0;
  return (rows->n_rows * rows->n_heads * p.splits * (cache->head_dim + 4) * 4 + 15) / 16 * 16;
}

extern "C" int wq_kv8_attention(const wq_kv8_cache* cache, const wq_kv4_rows* rows,
                                int64_t max_rows, int64_t max_len, float scale, int64_t window,
                                uint16_t* out, float* lse, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  const char* who = "wq_kv8_attention";
  if (int e = check_attention8(cache, rows, max_rows, max_len, who)) return e;
  if (window < 0) return wq::fail(WQ_ERR_INVALID_ARG, "%s: window must be at least 0", who);
  if (rows->n_rows == 0 || rows->n_seqs == 0) return wq::ok();
  const int64_t need = wq_kv8_attention_workspace(cache, rows, max_rows, max_len);
  if (!out || (need && !workspace)) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (workspace_bytes < need)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                    (long long)workspace_bytes, (long long)need);
  if (!aligned16(out) || !aligned4(lse) || !aligned16(workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  const Attn8Plan plan = attn8_plan(cache, rows, max_rows, max_len);
  const int64_t grid = plan.pairs * plan.tiles * plan.splits;
  const int64_t items = rows->n_rows * rows->n_heads;
  if (grid > 0x7FFFFFFFll || items > 0x7FFFFF00ll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  Attn8Args p{};
  p.a = kv4_rows(rows);
  p.data = cache->data;
  p.exps = reinterpret_cast<const uint32_t*>(cache->exponents);
  p.n_pages = cache->n_pages;
  p.kv_heads = (int)cache->n_kv_heads;
  p.kv_heads_by = Divisor(cache->n_kv_heads);
  p.group_by = Divisor(rows->n_heads / cache->n_kv_heads);
  p.parts_by = Divisor(plan.tiles * plan.splits);
  p.splits_by = Divisor(plan.splits);
  p.window = window > 0x40000000 ? 0 : (int)window;
  p.tiles = (int)plan.tiles;
  p.splits = (int)plan.splits;
  p.split_pages = (int)plan.split_pages;
  p.scale = scale;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  int status = WQ_OK;
  kv4_dispatch(rows->dtype, cache->head_dim, [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value;
    auto launch = [&](auto kernel) {
      const size_t lds = (size_t)plan.waves * plan.ct * (D / 4 + 2) * 64 * 4;
      if (!allow_lds((const void*)kernel, lds)) {
        status = wq::fail(WQ_ERR_HIP, "%s: cannot use %zu bytes of LDS", who, lds);
        return;
      }
      kernel<<<dim3((unsigned)grid), plan.waves * kWave, lds, (hipStream_t)stream>>>(p);
    };
    if (plan.ct == 2) {
      if constexpr (D <= 128) launch(attn8_kernel<DT, D, kAttnWaves, 2>);
    } else if (plan.waves == kAttnWaves) {
      launch(attn8_kernel<DT, D, kAttnWaves, 1>);
    } else {
      if constexpr (D <= 128) launch(attn8_kernel<DT, D, kAttnMoreWaves, 1>);
    }
    if (status == WQ_OK && plan.splits > 1)
      join_kernel<DT, D><<<dim3((unsigned)items), kAttnWaves * kWave, 0, (hipStream_t)stream>>>(
          p.part, items, p.splits, out, lse, rows->cu_rows, (int)rows->n_seqs, (int)rows->n_heads);
  });
  return status == WQ_OK ? check_launch(who) : status;
}

// Column tiles of a key/value head that hold any division of the rows into sequences.
static int64_t mass8_col_tiles(const wq_kv8_cache* c, const wq_kv4_rows* a) {
  return a->n_rows * (a->n_heads / c->n_kv_heads) / 16 + a->n_seqs + 1;
}
static int64_t mass8_queries_bytes(const wq_kv8_cache* c, const wq_kv4_rows* a) {
  return c->n_kv_heads * mass8_col_tiles(c, a) * 32 * c->head_dim;
}

extern "C" int64_t wq_kv8_accumulate_workspace(const wq_kv8_cache* cache, const wq_kv4_rows* rows,
                                               int64_t max_rows, int64_t max_len) {
  if (int e = check_attention8(cache, rows, max_rows, max_len, "wq_kv8_accumulate_workspace")) return e;
  wq::ok();
  if (rows->n_rows == 0 || rows->n_seqs == 0 || mass8_tiles(cache, rows, max_rows) < 3) return 0;
  return mass8_queries_bytes(cache, rows) + cache->n_kv_heads * mass8_col_tiles(cache, rows) * 256;
}

extern "C" int wq_kv8_accumulate(const wq_kv8_cache* cache, const wq_kv4_rows* rows,
                                 int64_t max_rows, int64_t max_len, const float* lse, float scale,
                                 int64_t window, const int32_t* held, float* mass,
                                 int64_t mass_tokens, void* workspace, int64_t workspace_bytes,
                                 void* stream) {
  const char* who = "wq_kv8_accumulate";
  if (int e = check_attention8(cache, rows, max_rows, max_len, who)) return e;
  if (window < 0 || mass_tokens < 1)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad window or mass size", who);
  if (rows->n_rows == 0 || rows->n_seqs == 0) return wq::ok();
  const int64_t need = wq_kv8_accumulate_workspace(cache, rows, max_rows, max_len);
  if (!lse || !held || !mass || (need && !workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (workspace_bytes < need)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                    (long long)workspace_bytes, (long long)need);
  if (!aligned4(lse) || !aligned4(held) || !aligned4(mass) || !aligned16(workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (max_len > 64 * rows->table_width) max_len = 64 * rows->table_width;
  const int tiles = mass8_tiles(cache, rows, max_rows);
  const int64_t pairs = rows->n_seqs * cache->n_kv_heads, items = rows->n_rows * rows->n_heads;
  const int64_t pages = max_len < 1 ? 1 : (max_len + 63) / 64;
  // Few columns: a wave has several pages where there are enough, so that its queries are
  // made once, but not so many that uneven lengths leave compute units idle (32 sequences of
  // up to 8191 tokens, 8 heads: 42 us in up to 12 workgroups a compute unit, 46 in 3, 6 or 32).
  const int64_t each = tiles < 3 ? kAttnWaves : kMass8Pages, most = 12 * 256;
  int64_t groups = (pages + each - 1) / each;
  if (tiles < 3 && pairs * groups > most) groups = (most + pairs - 1) / pairs;
  const int64_t most_rows = max_rows > rows->n_rows ? rows->n_rows : max_rows;
  const int64_t scalers = (most_rows * (rows->n_heads / cache->n_kv_heads) + 16 * kAttnWaves - 1) / (16 * kAttnWaves) + 1;
  if (pairs * groups > 0x7FFFFFFFll || pairs * scalers > 0x7FFFFFFFll || items > 0x7FFFFF00ll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  Mass8Args p{};
  p.a = kv4_rows(rows);
  p.data = cache->data;
  p.exps = reinterpret_cast<const uint32_t*>(cache->exponents);
  p.n_pages = cache->n_pages;
  p.kv_heads = (int)cache->n_kv_heads;
  p.kv_heads_by = Divisor(cache->n_kv_heads);
  p.group_by = Divisor(rows->n_heads / cache->n_kv_heads);
  p.pairs_by = Divisor(pairs);
  p.window = window > 0x40000000 ? 0 : (int)window;
  p.scale = scale;
  p.lse = lse;
  p.held = held;
  p.mass = mass;
  p.mass_tokens = mass_tokens;
  p.queries = static_cast<h8*>(workspace);
  p.col_tiles = mass8_col_tiles(cache, rows);
  p.columns = reinterpret_cast<f4*>(static_cast<uint8_t*>(workspace) + mass8_queries_bytes(cache, rows));
  const dim3 grid((unsigned)(pairs * groups));
  hipStream_t st = (hipStream_t)stream;
  kv4_dispatch(rows->dtype, cache->head_dim, [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value;
    if (tiles == 1) {
      mass8_few_kernel<DT, D, 1><<<grid, kAttnWaves * kWave, 0, st>>>(p);
    } else if (tiles == 2) {
      mass8_few_kernel<DT, D, 2><<<grid, kAttnWaves * kWave, 0, st>>>(p);
    } else {
      scale8_kernel<DT, D><<<dim3((unsigned)(pairs * scalers)), kAttnWaves * kWave, 0, st>>>(p);
      mass8_many_kernel<D><<<grid, kMass8Pages * kMass8Turns * kWave, 0, st>>>(p);
    }
  });
  return check_launch(who);
}
