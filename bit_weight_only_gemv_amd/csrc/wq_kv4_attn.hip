// Attention over the paged 4-bit key/value cache (wq.h, "4-bit key/value
// cache"), on the matrix cores.
//
// A workgroup takes 16 columns, (row, head) pairs of one key/value head, and its
// waves pages of 64 tokens in turn.  With key code c, scale S and offset Z of a token and
// group g, and the group's part of the query Q_g,
//   logit = scale (sum_g S_g (c_g . Q_g) + sum_g Z_g sum(Q_g)),
// and with the softmax weights p,
//   out_d = sum_t p_t (S_{t,g(d)} c_{t,d}) + sum_t p_t Z_{t,g(d)}.
// Both are 16x16x32 products.  The first one's A operand is the codes: one mask per
// two codes makes FP16 subnormals c 2^-24 (or 16 c 2^-24; B carries the 1/16).  The
// second one's is S c.  Tokens are the rows of the first product, so a lane ends with
// 4 tokens of one column per 16, and two such tiles are just its 8 k of the second
// product's B operand: the weights never leave their registers.
//
// Precision.  Queries are scaled by a power of two, the largest channel to [2^14,
// 2^15), and so are exact in FP16, of either type, down to 2^-24 of the largest;
// smaller ones are off by 2^-35 of it at most.  Logits, maxima and sums are FP32.
// A softmax weight is an FP16 number and its FP16 remainder (22 bits), for BF16
// outputs too: rounded to 11 bits it shows where values of both signs nearly cancel.
// S c is an FP16 number and its remainder, which is exact; the product of the two
// remainders, 2^-22 of the whole, is left out.  Scales stay off the weights: a small
// weight times a small scale would fall below FP16, and its token would count as its
// group's minimum.  For the same reason the weights are relative to a
// reference that follows the logits both ways: a page whose largest weight would
// pass 2^14 or stay below 2^2 sets it to that logit, where weights carry 2^10.  So
// 22 bits hold for what counts in a page, however small the page's share is
// (behind a strong first token, say), and most pages are spared the cross-lane
// maximum and the rescale of the sums.  The reference stays within 2^64 of the
// highest, so that FP32 holds the sums.
//
// What bounds it (traced times).  One token a sequence over a long cache: the
// cache's bytes and the instructions nearly alike.  Four sequences of 131072 tokens,
// 8 heads of 128 channels, 671 MB: 137 us, where a plain read of as many bytes takes
// 119; a page costs a wave 775 vector and 72 matrix instructions, which issue in 60%
// and keep the matrix cores for 22% of the time at two waves a SIMD, and its loads are
// under way while the one before is computed (keys are loaded into the registers
// that the logits have just freed, values into those of the values' product).
// Many rows: the vector instructions (1197 a page and wave with two column tiles, 422
// of them for each tile alone), 251 us for 54 GFLOP of a 512-token piece of two
// prompts over 6000 tokens.  Short caches: latency, 8 us for one page a wave (lengths and page numbers, then the page, the dependent steps of its
// computation, the join).

#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"

#include <utility>

namespace wqd {

constexpr int kAttnWaves = 4, kAttnMoreWaves = 8;
constexpr int kFoldPages = 8;        // at 2 the long case takes 158 us instead of 137, and is no closer
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

// Lane N of every row of 16 lanes, in all of the row's lanes.
template <int N>
__device__ __forceinline__ uint32_t row_lane(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x150 + N, 0xF, 0xF, false);
}

// 8 codes of a word as a matrix-core operand: slots 0, 1, 4, 5 hold c 2^-24,
// slots 2, 3, 6, 7 hold 16 c 2^-24.
__device__ __forceinline__ h8 code_operand(uint32_t w) {
  uint32_t lo0, hi0, lo1, hi1;
  w4_word_sub(w, lo0, hi0, lo1, hi1);
  return __builtin_bit_cast(h8, u4v{lo0, hi0, lo1, hi1});
}

// Codes of a word's slots 2 x and 2 x + 1 as FP16 numbers (a subnormal S c would not
// be exact), from numbers of which they are the last bits: 1024 + c, and 64 + c
// where they stand 4 bits higher.
template <int X>
__device__ __forceinline__ h2 code_pair(uint32_t w, uint32_t magic, uint32_t magic16) {
  if constexpr (X >= 2) w >>= 8;
  if constexpr (X & 1)
    return as_h2((w & 0x00F000F0u) | magic16) - h2{(_Float16)64.f, (_Float16)64.f};
  return as_h2((w & 0x000F000Fu) | magic) - h2{(_Float16)1024.f, (_Float16)1024.f};
}

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// One tile of 32 tokens of one head in registers: lane (row r = lane / 16,
// l = lane % 16).
template <int D>
struct TileShape {
  static constexpr int G = D / 32, W = G < 4 ? G : 4, J = D / 16, M = G == 8 ? 2 : 1, ZN = G / 2;
  // Byte of row r's scales that lane l holds: M dwords (2 slots each) of 4 G.
  static __device__ __forceinline__ uint32_t scale_at(uint32_t r, uint32_t l) {
    return r * (16 * G) + (G == 2 ? (l & 7) * 4 : l * (4 * M));
  }
  // Dword j (slots 2j, 2j + 1) of group g of row r's scales (GJ = 4 g + j), in all lanes.
  template <int GJ>
  static __device__ __forceinline__ h2 scale2(const uint32_t (&s)[M]) {
    if constexpr (M == 1) return as_h2(row_lane<GJ>(s[0]));
    else return as_h2(row_lane<GJ / 2>(s[GJ & 1]));
  }
};

template <int D>
struct KeyTile : TileShape<D> {
  using S = TileShape<D>;
  uint32_t codes[2][S::G];      // 16-token part, group: 8 codes of token l
  uint32_t scales[S::M];
  uint32_t offsets[2][S::ZN];   // token l's, all groups
  __device__ __forceinline__ void load(const uint8_t* __restrict__ q, uint32_t lane) {
    constexpr int G = S::G, W = S::W;
    const uint32_t r = lane >> 4, l = lane & 15;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int c = 0; c < G / W; ++c)
        __builtin_memcpy(&codes[u][c * W], q + u * (8 * D) + c * (256 * W) + lane * (4 * W), 4 * W);
    __builtin_memcpy(&scales[0], q + 32 * D + S::scale_at(r, l), 4 * S::M);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      __builtin_memcpy(&offsets[u][0], q + 34 * D + (16 * u + l) * (2 * G), 2 * G);
  }
};

template <int D>
struct ValueTile : TileShape<D> {
  using S = TileShape<D>;
  uint32_t codes[S::J];         // 16 channels: 8 codes of channel l
  uint32_t scales[S::M];
  u4v offsets;                  // group l's, of 8 tokens
  __device__ __forceinline__ void load(const uint8_t* __restrict__ q, uint32_t lane) {
    const uint32_t r = lane >> 4, l = lane & 15;
#pragma unroll
    for (int c = 0; c < S::J / 4; ++c)
      __builtin_memcpy(&codes[c * 4], q + 16 * D + c * 1024 + lane * 16, 16);
    __builtin_memcpy(&scales[0], q + 36 * D + S::scale_at(r, l), 4 * S::M);
    __builtin_memcpy(&offsets, q + 38 * D + r * (16 * S::G) + (l < S::G ? l : 0) * 16, 16);
  }
  // Clears the scales and offsets of tokens n and later (they were never
  // written and may be anything).
  __device__ __forceinline__ void cut(int n, int lane) {
    const int r = lane >> 4, l = lane & 15;
#pragma unroll
    for (int x = 0; x < S::M; ++x) {
      const int j = (S::M == 1 ? l : 2 * l + x) & 3;
      const int tok = 16 * (j >> 1) + 4 * r + 2 * (j & 1);
      scales[x] = tok >= n ? 0 : tok + 1 >= n ? scales[x] & 0xFFFFu : scales[x];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int tok = 16 * (j >> 1) + 4 * r + 2 * (j & 1);
      offsets[j] = tok >= n ? 0 : tok + 1 >= n ? offsets[j] & 0xFFFFu : offsets[j];
    }
  }
};

// Logarithm of a sum of weights that carry 2^kWeightExp, at maximum mx (base 2).
__device__ __forceinline__ float log_sum(float sum, float mx) {
  return sum == 0.f ? -INFINITY
                    : ((mx == -INFINITY ? 0.f : mx) - kWeightExp) * 0.69314718f + __logf(sum);
}

struct AttnArgs {
  KvRows a;
  const uint8_t* data;
  int64_t n_pages;
  Divisor kv_heads_by, group_by, pairs_by, splits_by;
  int kv_heads, window, n_sel, tiles, splits, split_pages;
  float scale;
  const int32_t* sel;
  uint16_t* out;
  float* lse;
  float* part;            // [row][head][split][D], then [row][head][split][4]: sum, maximum, exact sum
};

template <int DT, int D, bool SEL, int NW, int CT>
__global__ void __launch_bounds__(NW * kWave, 2) attn_kernel(AttnArgs p) {
  using TS = TileShape<D>;
  constexpr int G = TS::G, J = TS::J;
  constexpr int NT = D <= 128 && CT == 1 ? 2 : 1;        // tiles taken together
  constexpr int kPart = (4 * J + 3) * 64;     // floats a wave keeps in LDS, a column tile
  extern __shared__ __attribute__((aligned(16))) float s_merge[];
  const KvRows& a = p.a;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 4, l = lane & 15;
  const int R = (int)p.group_by.d;

  // pairs (sequence or row, key/value head) vary fastest: workgroups that read
  // the same pages are a multiple of the pairs apart and so, for 8 pairs and
  // their multiples, on the same XCD; the last column tiles, which see the most
  // tokens, come first
  const int rest = p.pairs_by.div(blockIdx.x), pair = blockIdx.x - rest * p.pairs_by.d;
  const int of = p.kv_heads_by.div(pair), kvh = pair - of * p.kv_heads;
  const int turn = p.splits_by.div(rest), split = rest - turn * p.splits;
  const int tile0 = p.tiles - 1 - turn;
  int b, row0, n, len;
  // The wave's first page numbers (or their places in the row's list), read at
  // the same time as the lengths: where the hints hold, a split starts here.
  const int guess_at = split * p.split_pages + wave + NW * lane;
  int guess = -1;
  if constexpr (SEL) {
    row0 = of;
    if (guess_at < p.n_sel) guess = p.sel[((int64_t)row0 * p.kv_heads + kvh) * p.n_sel + guess_at];
    const SeqRow sr = find_row(a, row0);
    b = sr.b;
    n = 1;
    len = sr.pos + 1;
    if (row0 >= a.cu[b + 1]) return;
  } else {
    b = of;
    if (guess_at < a.width) guess = a.table[(int64_t)b * a.width + guess_at];
    row0 = max(a.cu[b], 0);
    n = max(min(max(a.cu[b + 1], 0), a.rows) - row0, 0);     // rows of the call for any cu_rows
    len = max(a.lens[b], 0);
  }
  const int cols = n * R;
  const int written = SEL ? a.lens[b] : len;      // tokens that the cache holds
  const int32_t* const table = a.table + (int64_t)b * a.width;
  const int32_t* const list = SEL ? p.sel + ((int64_t)row0 * p.kv_heads + kvh) * p.n_sel : nullptr;
  const int64_t stride = (int64_t)p.kv_heads * (80 * D);
  const uint8_t* const base = p.data + (int64_t)kvh * (80 * D);
  uint32_t magic = 0x64006400u, magic16 = 0x54005400u;   // in VGPRs: a mask and one are then one instruction
  asm("" : "+v"(magic), "+v"(magic16));

  for (int tile = tile0; tile * (16 * CT) < cols; tile += p.tiles) {
    // positions of the tile's columns, and this workgroup's pages: positions in
    // the block table, or in the row's list; a wave takes every NW-th
    const int c_hi = min(tile * (16 * CT) + 16 * CT - 1, cols - 1);
    const int pos_lo = SEL ? len - 1 : len - n + p.group_by.div(tile * (16 * CT));
    const int pos_hi = SEL ? len - 1 : len - n + p.group_by.div(c_hi);
    const int64_t pages64 = ((int64_t)pos_hi + 64) / 64;
    const int pages = (int)(pages64 < a.width ? pages64 : a.width);
    const int first = !SEL && p.window > 0 ? max(pos_lo - p.window + 1, 0) / 64 : 0;
    const int total = SEL ? p.n_sel : max(pages - first, 0);
    const int per = max(p.split_pages, p.splits_by.div(total + p.splits - 1));
    const int j0 = min(split * per, total), j1 = min(j0 + per, total);
    const int count = (j1 - j0 - wave + NW - 1) / NW;

    // the next step of this wave: a page, or where NT is 1 a tile of it.  Lanes
    // hold the places and numbers of 64 pages at a time.
    int k = -1, held_at = 0, held_id = 0, at = -1, part = 2 / NT - 1;
    const uint8_t* src = base;
    auto next = [&]() {
      if (NT == 1 && part == 0) {
        part = 1;
        src += 40 * D;
        return;
      }
      part = 0;
      for (at = -1; ++k < count;) {
        if ((k & 63) == 0) {
          const int j = j0 + wave + NW * (k + lane);
          const bool guessed = k == 0 && per == p.split_pages && first == 0;
          held_at = j < j1 ? (SEL ? (guessed ? guess : list[j]) : first + j) : -1;
          held_id = -1;
          if (held_at >= 0 && held_at < pages)
            held_id = !SEL && guessed ? guess : table[held_at];
        }
        const int id = __builtin_amdgcn_readlane(held_id, k & 63);
        if (id < 0 || id >= p.n_pages) continue;      // no tokens there
        at = __builtin_amdgcn_readlane(held_at, k & 63);
        src = base + id * stride;
        break;
      }
    };
    KeyTile<D> kt[NT];
    ValueTile<D> vt[NT];
    auto load_keys = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t) kt[t].load(src + t * (40 * D), lane);
    };
    auto load_values = [&]() {
#pragma unroll
      for (int t = 0; t < NT; ++t) vt[t].load(src + t * (40 * D), lane);
    };
    // this lane's column, its query's loads ahead of the pages' and its scaling
    // behind them
    int row[CT], head[CT], pos[CT];
    u4v qv[CT][G];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const int col = tile * (16 * CT) + 16 * ct + l;
      const bool on = col < cols;
      const int nth = p.group_by.div(col);
      row[ct] = on ? row0 + nth : -1;
      head[ct] = kvh * R + col - nth * R;
      pos[ct] = on ? (SEL ? len - 1 : len - n + nth) : -1;
      const uint16_t* q = a.q + (on ? row[ct] * a.q_row + head[ct] * a.q_head : 0) + 8 * r;
#pragma unroll
      for (int g = 0; g < G; ++g)
        qv[ct][g] = on ? *reinterpret_cast<const u4v*>(q + 32 * g) : u4v{0, 0, 0, 0};
    }
    next();
    if (at >= 0) {
      load_keys();
      load_values();
    }
    h8 Q[CT][G], SQ[CT];
    float c1[CT], c2[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      float top = 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          top = fmaxf(top, fabsf(to_float<DT>((uint16_t)(qv[ct][g][i >> 1] >> (16 * (i & 1))))));
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      int e = (int)(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
      e = top == 0.f || e > 127 ? 14 : max(e, -100);
      uint32_t sq[4] = {0, 0, 0, 0};
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float y =
              ldexpf(to_float<DT>((uint16_t)(qv[ct][g][i >> 1] >> (16 * (i & 1)))), 14 - e);
          sum += y;
          Q[ct][g][i] = (_Float16)(i & 2 ? y * 0.0625f : y);
        }
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        sum *= 0.015625f;
        const _Float16 hi = (_Float16)sum, lo = (_Float16)(sum - (float)hi);
        const uint32_t bits = r == 0 ? __builtin_bit_cast(uint16_t, hi)
                                     : r == 1 ? __builtin_bit_cast(uint16_t, lo) : 0u;
        sq[g >> 1] |= bits << (16 * (g & 1));
      }
      SQ[ct] = __builtin_bit_cast(h8, u4v{sq[0], sq[1], sq[2], sq[3]});
      const float f = p.scale * 1.44269504f;
      c1[ct] = ldexpf(f, e - 14 + 24);
      c2[ct] = ldexpf(f, e - 14 + 6);
    }

    f4 O[CT][J], OZ[CT];
    float m[CT], m_kept[CT];      // the reference, now and at the last fold
    float least[CT];        // the lowest that it may be
    float exact[CT];        // this lane's weights before their rounding, for lse
    bool kept = false;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      m[ct] = m_kept[ct] = least[ct] = -INFINITY;
      exact[ct] = 0.f;
      OZ[ct] = f4{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < J; ++j) O[ct][j] = f4{0, 0, 0, 0};
    }
    // Folds code sums and offsets into the wave's values in LDS.  The two nearly
    // cancel, and a matrix-core sum loses a little to every addition: over a long
    // cache what they have in common would swallow the result's last bits.
    auto fold = [&]() {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float* const s = s_merge + (wave * CT + ct) * kPart;
        f4* const s4 = reinterpret_cast<f4*>(s) + lane;
        const float f = m_kept[ct] == m[ct] ? 1.f : __builtin_amdgcn_exp2f(m_kept[ct] - m[ct]);
        float z[G];
#pragma unroll
        for (int g = 0; g < G; ++g) z[g] = __shfl(OZ[ct][g & 3], (g >> 2) * 16 + l);
        float sum = __shfl(OZ[ct][0], 32 + l);
#pragma unroll
        for (int j = 0; j < J; ++j) {
          f4 v = O[ct][j] + z[j >> 1];
          if (kept) v += s4[j * 64] * f;
          s4[j * 64] = v;
          O[ct][j] = f4{0, 0, 0, 0};
        }
        if (kept) sum += s[4 * J * 64 + lane] * f;
        s[4 * J * 64 + lane] = sum;
        s[(4 * J + 1) * 64 + lane] = m[ct];
        OZ[ct] = f4{0, 0, 0, 0};
        m_kept[ct] = m[ct];
      }
      kept = true;
    };

    int since = 0;          // steps since the last fold
    while (at >= 0) {
      if (since == kFoldPages * (2 / NT)) {
        fold();
        since = 0;
      }
      ++since;
      const int t0 = at * 64 + part * 32;
      // logits: sums of codes times queries by group, and of offsets
      f4 sc[CT][2 * NT], zt[CT][2 * NT];
      unroll<2 * NT>([&](auto uu) {
        constexpr int u = uu, t = u / 2, h = u % 2;
        uint32_t zw[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < TS::ZN; ++i) zw[i] = kt[t].offsets[h][i];
        if (u == 2) __builtin_amdgcn_sched_barrier(0);
        const h8 za = __builtin_bit_cast(h8, u4v{zw[0], zw[1], zw[2], zw[3]});
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          zt[ct][u] = mfma(za, SQ[ct], f4{0, 0, 0, 0});
          sc[ct][u] = f4{0, 0, 0, 0};
        }
        unroll<G>([&](auto g) {
          const h8 ka = code_operand(kt[t].codes[h][g]);
          const h2 s0 = TS::template scale2<g * 4 + 2 * h>(kt[t].scales);
          const h2 s1 = TS::template scale2<g * 4 + 2 * h + 1>(kt[t].scales);
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            const f4 d = mfma(ka, Q[ct][g], f4{0, 0, 0, 0});
            f4& s = sc[ct][u];
            s[0] = __builtin_fmaf((float)s0[0], d[0], s[0]);
            s[1] = __builtin_fmaf((float)s0[1], d[1], s[1]);
            s[2] = __builtin_fmaf((float)s1[0], d[2], s[2]);
            s[3] = __builtin_fmaf((float)s1[1], d[3], s[3]);
          }
        });
      });
      // the keys' registers are free: the next step's keys arrive behind the
      // values' product, its values behind the next logits
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int u = 0; u < 2 * NT; ++u)
          asm volatile("" : "+v"(sc[ct][u]), "+v"(zt[ct][u]));   // done here, not after the loads
      __builtin_amdgcn_sched_barrier(0);
      next();
      load_keys();           // past the last step: that step's again, not used
      __builtin_amdgcn_sched_barrier(0);

      // base-2 logits above the reference, plus kWeightExp
      constexpr int NY = 8 * NT;
      float y[CT][NY], top[CT];
      bool raise = false;
      uint64_t lower = 0;     // bit l: column l's four lanes
      const bool edge = t0 + 32 * NT - 1 > pos_lo || (p.window > 0 && t0 <= pos_hi - p.window);
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const bool none = m[ct] == -INFINITY;
        const float m8 = none ? -kWeightExp : m[ct] - kWeightExp;
#pragma unroll
        for (int i = 0; i < NY; ++i)
          y[ct][i] = __builtin_fmaf(sc[ct][i >> 2][i & 3], c1[ct],
                                    __builtin_fmaf(zt[ct][i >> 2][i & 3], c2[ct], -m8));
        if (edge) {
          asm volatile("");      // stays a branch: few pages have an edge
#pragma unroll
          for (int i = 0; i < NY; ++i) {
            const int t = t0 + 16 * (i >> 2) + 4 * r + (i & 3);
            if (t > pos[ct] || (p.window > 0 && t <= pos[ct] - p.window)) y[ct][i] = -INFINITY;
          }
        }
        top[ct] = -INFINITY;
#pragma unroll
        for (int i = 0; i < NY; ++i) top[ct] = fmaxf(top[ct], y[ct][i]);
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
          for (int i = 0; i < NY; ++i) y[ct][i] -= up;
#pragma unroll
          for (int j = 0; j < J; ++j) O[ct][j] *= f;
          OZ[ct] *= f;
          exact[ct] *= f;
        }
      }
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
        for (int i = 0; i < NY; ++i) y[ct][i] = __builtin_amdgcn_exp2f(y[ct][i]);
        if (p.lse != nullptr) {
          asm volatile("");      // stays a branch
#pragma unroll
          for (int i = 0; i < NY; ++i) exact[ct] += y[ct][i];
        }
      }

      if (t0 + 32 * NT > written) {
        asm volatile("");
#pragma unroll
        for (int t = 0; t < NT; ++t) vt[t].cut(written - t0 - 32 * t, lane);
      }
      const uint32_t fill = l == 8 ? 0x3C003C00u : 0u;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        u4v z = vt[t].offsets;
        if (l >= G) z = u4v{fill, fill, fill, fill};
        const h8 za = __builtin_bit_cast(h8, z);
        h8 wh[CT], wl[CT];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          u4v wv, rv;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float y0 = y[ct][8 * t + 2 * x], y1 = y[ct][8 * t + 2 * x + 1];
            const h2 w = {(_Float16)y0, (_Float16)y1};
            const h2 rest = {(_Float16)(y0 - (float)w[0]), (_Float16)(y1 - (float)w[1])};
            wv[x] = as_u32(w);
            rv[x] = as_u32(rest);
          }
          wh[ct] = __builtin_bit_cast(h8, wv);
          wl[ct] = __builtin_bit_cast(h8, rv);
          OZ[ct] = mfma(za, wh[ct], OZ[ct]);
          OZ[ct] = mfma(za, wl[ct], OZ[ct]);
        }
        // 15 S passes FP16's range from 4096 on: such scales enter as four quarters
        uint32_t wide = 0, quarters[TS::M];
#pragma unroll
        for (int x = 0; x < TS::M; ++x) wide |= (vt[t].scales[x] + 0x14001400u) & 0x80008000u;
        int times = 1;
        if (__any(wide != 0)) {
          times = 4;
#pragma unroll
          for (int x = 0; x < TS::M; ++x) {
            quarters[x] = ((vt[t].scales[x] + 0x14001400u) >> 15 & 0x00010001u) * 0xFFFFu;
            vt[t].scales[x] -= quarters[x] & 0x08000800u;
          }
        }
        for (;;) {
          unroll<G>([&](auto g) {
            uint32_t (&codes)[TS::J] = vt[t].codes;
            asm volatile("" : "+v"(codes[2 * g]), "+v"(codes[2 * g + 1]));   // unpacked here, not ahead of the loop
            u4v hi[2], lo[2];
            unroll<4>([&](auto x) {
              const h2 s = TS::template scale2<g * 4 + x>(vt[t].scales);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const h2 c = code_pair<x>(codes[2 * g + i], magic, magic16), h = c * s;
                hi[i][(int)x] = as_u32(h);
                lo[i][(int)x] = as_u32(__builtin_elementwise_fma(c, s, -h));
              }
            });
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
              for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                  O[ct][2 * g + i] = mfma(__builtin_bit_cast(h8, k == 1 ? lo[i] : hi[i]),
                                          k == 2 ? wl[ct] : wh[ct], O[ct][2 * g + i]);
          });
          if (--times == 0) break;
#pragma unroll
          for (int x = 0; x < TS::M; ++x) vt[t].scales[x] &= quarters[x];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      load_values();
    }

    fold();
    if (p.lse != nullptr) {
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        exact[ct] += __shfl_xor(exact[ct], 16);
        exact[ct] += __shfl_xor(exact[ct], 32);
        s_merge[(wave * CT + ct) * kPart + (4 * J + 2) * 64 + lane] = exact[ct];
      }
    }
    // the waves' parts joined in order
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      if (row[ct] < 0) continue;
      auto part_of = [&](int w) { return s_merge + (w * CT + ct) * kPart; };
      float mw[NW], mx = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        mw[w] = part_of(w)[(4 * J + 1) * 64 + lane];
        mx = fmaxf(mx, mw[w]);
      }
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        mw[w] = mw[w] == mx ? 1.f : __builtin_amdgcn_exp2f(mw[w] - mx);
        sum += mw[w] * part_of(w)[4 * J * 64 + lane];
      }
      const int64_t out_at = (int64_t)row[ct] * a.heads + head[ct];
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      for (int j = wave; j < J; j += NW) {
        f4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) o += mw[w] * reinterpret_cast<const f4*>(part_of(w))[j * 64 + lane];
        const int d = 16 * j + 4 * r;
        if (p.splits == 1) {
          uint16_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = from_float<DT>(sum == 0.f ? 0.f : o[i] * inv);
          *reinterpret_cast<u2*>(p.out + out_at * D + d) = u2{pack2(h[0], h[1]), pack2(h[2], h[3])};
        } else {
          *reinterpret_cast<f4*>(p.part + (out_at * p.splits + split) * D + d) = o;
        }
      }
      if (wave == 0 && r == 0) {
        float ex = 0.f;
        if (p.lse != nullptr)
#pragma unroll
          for (int w = 0; w < NW; ++w) ex += mw[w] * part_of(w)[(4 * J + 2) * 64 + lane];
        if (p.splits == 1) {
          if (p.lse != nullptr) p.lse[out_at] = log_sum(ex, mx);
        } else {
          reinterpret_cast<f4*>(p.part + (int64_t)a.rows * a.heads * p.splits *
                                             D)[out_at * p.splits + split] = f4{sum, mx, ex, 0.f};
        }
      }
    }
    __syncthreads();
  }
}

// Joins the splits of one (row, head): split s's weight is 2^(m_s - max m).  16
// bytes a lane and D / 4 lanes a split, so that 1024 / D splits are read at a
// time; their sums are added in order.
template <int DT, int D>
__global__ void __launch_bounds__(kAttnWaves * kWave)
join_kernel(const float* __restrict__ part, int64_t items, int splits, uint16_t* __restrict__ out,
            float* __restrict__ lse) {
  constexpr int L = D / 4, S = kAttnWaves * kWave / L;
  __shared__ f4 s_acc[S][L];
  __shared__ float s_sum[S][3];
  const int64_t at = blockIdx.x;
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

// How a call is split: column tiles of a sequence (or row) and splits of its pages.
// Hints past what the call can have count as that, so that nothing overflows; there
// is at least one row and one sequence.
struct AttnPlan {
  int64_t pairs, tiles, splits, split_pages;
  int waves, ct;            // waves a workgroup, column tiles a wave
};
static AttnPlan attn_plan(const wq_kv4_cache* c, const wq_kv4_rows* a, int64_t max_rows,
                          int64_t max_len, int64_t n_sel, bool sel) {
  AttnPlan p{};
  const int64_t R = a->n_heads / c->n_kv_heads;
  if (max_rows > a->n_rows) max_rows = a->n_rows;
  if (max_len > 64 * a->table_width) max_len = 64 * a->table_width;
  const int64_t cols = (sel || max_rows < 1 ? 1 : max_rows) * R;
  // Two column tiles share the codes' unpacking where there are enough of them: a
  // 512-token piece of two prompts over 6000 tokens takes 251 us with two, 298 with
  // one.  Heads of 256 channels would not fit their registers.
  p.ct = !sel && c->head_dim <= 128 && cols >= 64 ? 2 : 1;
  p.tiles = (cols + 16 * p.ct - 1) / (16 * p.ct);
  p.pairs = (sel ? a->n_rows : a->n_seqs) * c->n_kv_heads;
  int64_t pages = sel ? n_sel : (max_len + 63) / 64;
  if (pages < 1) pages = 1;
  // Two workgroups of 4 waves for every compute unit, as many as run at once:
  // a second round costs more than uneven lengths do (32 sequences of up to 8191
  // tokens: 67 us, in two rounds 72).  A split has at least two pages a wave, one
  // while that leaves compute units idle (64 chosen pages: 8.6 us, 11.8 with two).
  const int64_t items = p.pairs * p.tiles;
  int64_t splits = (512 + items - 1) / items;
  const int64_t waves = items * ((pages + kAttnWaves - 1) / kAttnWaves) <= 256 ? kAttnWaves : 2 * kAttnWaves;
  const int64_t most = (pages + waves - 1) / waves;
  if (splits > most) splits = most;
  // Few pages for few workgroups: one workgroup of up to 8 waves, and no second
  // launch.  500 tokens of one sequence: 9.9 us with 8 waves, 11.0 with 4, 8.6 and
  // 2.7 in two launches; 1000 tokens: 13.2, 14.8, 8.4 and 2.6, where the second launch's
  // own 2 to 3 us make up for it; 2000 tokens: 8.7 and 2.9 in two.
  p.waves = kAttnWaves;
  if (items <= 256 && pages <= 2 * kAttnMoreWaves) {
    splits = 1;
    if (pages > kAttnWaves && p.ct == 1) p.waves = kAttnMoreWaves;
  }
  p.split_pages = (pages + splits - 1) / splits;
  p.splits = (pages + p.split_pages - 1) / p.split_pages;
  return p;
}

}  // namespace wqd

using namespace wqd;

static int check_attention(const wq_kv4_cache* cache, const wq_kv4_rows* rows, int64_t max_rows,
                           int64_t max_len, int64_t n_sel, const char* who) {
  if (int e = kv4_check_cache(cache, who)) return e;
  if (int e = kv4_check_rows(cache, rows, who)) return e;
  if (max_rows < 0 || max_len < 0 || n_sel < 0 || n_sel > (1 << 20))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  return WQ_OK;
}

extern "C" int64_t wq_kv4_attention_workspace(const wq_kv4_cache* cache, const wq_kv4_rows* rows,
                                              int64_t max_rows, int64_t max_len, int64_t n_sel) {
  if (int e = check_attention(cache, rows, max_rows, max_len, n_sel, "wq_kv4_attention_workspace"))
    return e;
  wq::ok();
  if (rows->n_rows == 0 || rows->n_seqs == 0) return 0;
  const AttnPlan p = attn_plan(cache, rows, max_rows, max_len, n_sel, n_sel > 0);
  if (p.splits == 1) return 0;
  return (rows->n_rows * rows->n_heads * p.splits * (cache->head_dim + 4) * 4 + 15) / 16 * 16;
}

extern "C" int wq_kv4_attention(const wq_kv4_cache* cache, const wq_kv4_rows* rows,
                                int64_t max_rows, int64_t max_len, float scale, int64_t window,
                                const int32_t* sel, int64_t n_sel, uint16_t* out, float* lse,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "wq_kv4_attention";
  if (int e = check_attention(cache, rows, max_rows, max_len, n_sel, who)) return e;
  if (window < 0) return wq::fail(WQ_ERR_INVALID_ARG, "%s: window must be at least 0", who);
  const bool empty = rows->n_rows == 0 || rows->n_seqs == 0;   // its sel may be NULL
  if (sel != nullptr ? n_sel == 0 : n_sel > 0 && !empty)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: sel and n_sel go together", who);
  if (empty) return wq::ok();
  const int64_t need = wq_kv4_attention_workspace(cache, rows, max_rows, max_len, n_sel);
  if (!out || (need && !workspace)) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (workspace_bytes < need)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                    (long long)workspace_bytes, (long long)need);
  if (!aligned16(out) || !aligned4(lse) || !aligned4(sel) || !aligned16(workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  const AttnPlan plan = attn_plan(cache, rows, max_rows, max_len, n_sel, sel != nullptr);
  const int64_t grid = plan.pairs * plan.tiles * plan.splits;
  const int64_t items = rows->n_rows * rows->n_heads;
  if (grid > 0x7FFFFFFFll || items > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  AttnArgs p{};
  p.a = kv4_rows(rows);
  p.data = cache->data;
  p.n_pages = cache->n_pages;
  p.kv_heads = (int)cache->n_kv_heads;
  p.kv_heads_by = Divisor(cache->n_kv_heads);
  p.group_by = Divisor(rows->n_heads / cache->n_kv_heads);
  p.pairs_by = Divisor(plan.pairs);
  p.splits_by = Divisor(plan.splits);
  p.window = window > 0x40000000 ? 0 : (int)window;
  p.n_sel = (int)n_sel;
  p.tiles = (int)plan.tiles;
  p.splits = (int)plan.splits;
  p.split_pages = (int)plan.split_pages;
  p.scale = scale;
  p.sel = sel;
  p.out = out;
  p.lse = lse;
  p.part = static_cast<float*>(workspace);
  int status = WQ_OK;
  kv4_dispatch(rows->dtype, cache->head_dim, [&](auto dt, auto d) {
    constexpr int DT = decltype(dt)::value, D = decltype(d)::value;
    auto launch = [&](auto kernel) {
      const size_t lds = (size_t)plan.waves * plan.ct * (D / 4 + 3) * 64 * 4;
      if (!allow_lds((const void*)kernel, lds)) {
        status = wq::fail(WQ_ERR_HIP, "%s: cannot use %zu bytes of LDS", who, lds);
        return;
      }
      kernel<<<dim3((unsigned)grid), plan.waves * kWave, lds, (hipStream_t)stream>>>(p);
    };
    if (plan.ct == 2) {
      if constexpr (D <= 128) launch(attn_kernel<DT, D, false, kAttnWaves, 2>);
    } else if (plan.waves == kAttnWaves) {
      if (sel != nullptr) launch(attn_kernel<DT, D, true, kAttnWaves, 1>);
      else launch(attn_kernel<DT, D, false, kAttnWaves, 1>);
    } else {
      if (sel != nullptr) launch(attn_kernel<DT, D, true, kAttnMoreWaves, 1>);
      else launch(attn_kernel<DT, D, false, kAttnMoreWaves, 1>);
    }
    if (status == WQ_OK && plan.splits > 1)
      join_kernel<DT, D><<<dim3((unsigned)items), kAttnWaves * kWave, 0, (hipStream_t)stream>>>(
          p.part, items, p.splits, out, lse);
  });
  return status == WQ_OK ? check_launch(who) : status;
}
