// The paged 4-bit key/value cache (wq.h, "4-bit key/value cache"): where new
// tokens go, writing them, and the choice of pages for sparse attention.
// Attention itself is in wq_kv4_attn.hip.

#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"
#include "wq_select.cuh"

namespace wqd {

// ------------------------------------------------------------------- plan
// Block table, slots and runs from request lengths.  Every workgroup scans the
// sequences for itself (page needs and run counts, exclusive sums in LDS), so
// one launch without any exchange between workgroups does it all: a scan of
// 1000 sequences is 4 loads a thread, less than a second launch.  Table
// entries, slots and runs are then found by binary search in those sums.  Latency
// bounds it: 4.5 us for 64 decoding sequences, 6.5 us for 1000 sequences with 50000
// new tokens.
constexpr int kPlanThreads = 1024;
constexpr int kMaxLen = 1 << 30;
constexpr int kMaxPage = (1 << 25) - 1;   // slots stay below 2^31

__device__ __forceinline__ int upper_index(const int* sums, int n, int x) {
  // the last b in [0, n) with sums[b] <= x, for rising sums and sums[0] <= x
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (sums[m] <= x) lo = m; else hi = m;
  }
  return lo;
}

// New tokens of a sequence, 0 .. T for any cu_rows: the difference of two int32 need
// not be one, and of a signed one that overflows the compiler assumes that it does not.
__device__ __forceinline__ int new_tokens(int from, int to, int T) {
  return to > from ? (int)min((uint32_t)to - (uint32_t)from, (uint32_t)T) : 0;
}

__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const int32_t* __restrict__ lens, const int32_t* __restrict__ cu, int B, int T,
            int32_t* __restrict__ table, int64_t width, const int32_t* __restrict__ free_pages,
            int n_free, int32_t* __restrict__ new_lens, int32_t* __restrict__ slots,
            int32_t* __restrict__ runs, int n_runs, int32_t* __restrict__ taken) {
  extern __shared__ int s_plan[];
  int* s_len = s_plan;                 // [B]
  int* s_cu = s_len + B;               // [B + 1]
  int* s_need = s_cu + B + 1;          // [B + 1] exclusive sums of pages needed
  int* s_runs = s_need + B + 1;        // [B + 1] exclusive sums of runs
  __shared__ uint32_t s_wave[2][kPlanThreads / kWave];
  const int tid = threadIdx.x;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(tid * per, B), b1 = min(b0 + per, B);
  uint32_t need = 0, nruns = 0;        // sums of bad cu_rows may wrap, so unsigned
  for (int b = b0; b < b1; ++b) {
    const int len = min(max(lens[b], 0), kMaxLen);
    const int c = cu[b], n = new_tokens(c, cu[b + 1], T);
    s_len[b] = len;
    s_cu[b] = c;
    if (b == B - 1) s_cu[B] = cu[B];
    s_need[b] = (int)need;
    s_runs[b] = (int)nruns;
    need += (len + n + 63) / 64 - (len + 63) / 64;
    nruns += n > 0 ? (len + n - 1) / 64 - len / 64 + 1 : 0;
  }
  uint32_t ni = need, ri = nruns;      // inclusive sums over the wave's lanes
  for (int d = 1; d < kWave; d <<= 1) {
    const uint32_t a = __shfl_up(ni, d), b = __shfl_up(ri, d);
    if ((tid & 63) >= d) { ni += a; ri += b; }
  }
  if ((tid & 63) == 63) { s_wave[0][tid >> 6] = ni; s_wave[1][tid >> 6] = ri; }
  __syncthreads();
  uint32_t nbase = ni - need, rbase = ri - nruns;
  for (int w = 0; w < tid >> 6; ++w) { nbase += s_wave[0][w]; rbase += s_wave[1][w]; }
  for (int b = b0; b < b1; ++b) {
    s_need[b] = (int)((uint32_t)s_need[b] + nbase);
    s_runs[b] = (int)((uint32_t)s_runs[b] + rbase);
  }
  if (tid == kPlanThreads - 1) { s_need[B] = (int)(nbase + need); s_runs[B] = (int)(rbase + nruns); }
  __syncthreads();
  const int total = s_need[B], total_runs = s_runs[B];
  const int g0 = blockIdx.x * kPlanThreads + tid, step = gridDim.x * kPlanThreads;

  if (g0 == 0) taken[0] = total;
  for (int b = g0; b < B; b += step) new_lens[b] = s_len[b] + new_tokens(s_cu[b], s_cu[b + 1], T);
  for (int i = g0; i < min(total, T / 64 + B); i += step) {    // rising cu_rows need no more
    const int b = upper_index(s_need, B, i);
    const uint32_t p = (uint32_t)((s_len[b] + 63) / 64) + ((uint32_t)i - (uint32_t)s_need[b]);
    if (p < width) table[b * width + p] = i < n_free ? free_pages[i] : -1;
  }
  for (int row = g0; row < T; row += step) {
    int slot = -1;
    const int b = upper_index(s_cu, B, row);
    // any cu_rows: no position past kMaxLen + T, no page outside the list
    const uint32_t off = (uint32_t)row - (uint32_t)s_cu[b];
    if (row >= s_cu[b] && row < s_cu[b + 1] && off < (uint32_t)T) {
      const int pos = s_len[b] + (int)off, p = pos / 64;
      const int fresh = p - (s_len[b] + 63) / 64;   // pages this call adds start at 0
      const uint32_t at = (uint32_t)s_need[b] + (uint32_t)fresh;
      int page = -1;
      if (p < width) {
        if (fresh < 0) page = table[b * width + p];
        else if (at < (uint32_t)n_free) page = free_pages[at];
      }
      if (page >= 0 && page <= kMaxPage) slot = page * 64 + (pos & 63);
    }
    slots[row] = slot;
  }
  for (int j = g0; j < n_runs; j += step) {
    int first = -1, count = 0;
    if (j < total_runs) {
      const int b = upper_index(s_runs, B, j);
      const int len = s_len[b], end = len + new_tokens(s_cu[b], s_cu[b + 1], T);
      const int64_t start = 64 * (int64_t)(len / 64 + ((int64_t)j - s_runs[b]));
      const int lo = (int)max(start, (int64_t)len), hi = (int)min(start + 64, (int64_t)end);
      first = (int)((uint32_t)s_cu[b] + (uint32_t)lo - (uint32_t)len);
      count = (int)((uint32_t)hi - (uint32_t)lo);
    }
    reinterpret_cast<int2*>(runs)[j] = make_int2(first, count);
  }
}

// ----------------------------------------------------------------- append
// One workgroup per (run, head, keys or values).  A thread takes 8 channels of
// a token at a time, 4 neighbouring lanes one group of 32; all of a page's
// loads are in flight before the first is used.  Keys leave as whole words.
// Values go through LDS as bytes, 4 channels of 8 tokens to a thread, and come
// out as 4 words by a byte transpose.  Vector instructions bound it: 23300 tokens of
// 8 heads of 128 channels (126 MB) take 30 us, 22 as a plain read and write of
// these bytes; a lane issues 20 instructions a value, which at four cycles each take
// 24 us, and LDS bank conflicts are below 1 us.  One token: 3.8 us.
constexpr int kAppendThreads = 256;

// Codes as floats of 8 channels, in the header's arithmetic.  (w - Z) / S is
// first taken with the reciprocal, which is within 2^-16 of the rounded
// quotient (|q| < 32, three roundings of 2^-23); where that lies so near to a
// half that rounding could go another way, the wave divides.
__device__ __forceinline__ void codes_of(const float (&x)[8], float z, float s, float (&q)[8]) {
  const float inv = s > 0.f ? __builtin_amdgcn_rcpf(s) : 0.f;
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = (x[i] - z) * inv;
    q[i] = rintf(t);
    far = fmaxf(far, fabsf(t - q[i]));
  }
  if (__any(far > 0.5f - 0x1p-16f)) {
    asm volatile("");          // stays a branch
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = s > 0.f ? rintf((x[i] - z) / s) : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __builtin_amdgcn_fmed3f(q[i], 0.f, 15.f);
}

// Whether one of a word's two values is NaN, infinite or past 65504 (its exponent
// field reaches the highest, for BF16 that of 65536).
template <int DT>
__device__ __forceinline__ uint32_t out_of_range(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + (DT == WQ_DT_F16 ? 0x04000400u : 0x38803880u)) & 0x80008000u;
}

// d / 15 rounded to nearest: the quotient by the rounded reciprocal, corrected
// once by its exact remainder.
__device__ __forceinline__ float fifteenth(float d) {
  const float c = 1.0f / 15.0f, q = d * c;
  return __builtin_fmaf(__builtin_fmaf(-15.0f, q, d), c, q);
}

constexpr int append_lds_words(int D) { return 16 * D > 2048 ? 16 * D : 2048; }

// FULL: the run is a whole page, so nothing is masked.
template <int DT, int D, bool VALUES, bool FULL>
__device__ __forceinline__ void append_run(const uint16_t* __restrict__ src, int64_t row, int o,
                                           int count, uint8_t* __restrict__ page,
                                           uint16_t* __restrict__ summary, uint32_t* s_mem) {
  constexpr int G = D / 32, W = G < 4 ? G : 4, O = D / 8, TS = kAppendThreads / O, IT = 64 / TS;
  const int tid = threadIdx.x, oc = tid % O, g = oc >> 2, r8 = oc & 3;
  u4v raw[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int n = tid / O + it * TS;
    if (FULL || n < count) raw[it] = *reinterpret_cast<const u4v*>(src + n * row + oc * 8);
  }
  float lo8[8], hi8[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) { lo8[i] = INFINITY; hi8[i] = -INFINITY; }
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int n = tid / O + it * TS;
    if (!FULL && n >= count) continue;     // the 4 lanes of a group go together
    const int t = o + n, tt = t & 31, u = tt >> 4, r = (tt >> 2) & 3, e = 4 * u + (tt & 3);
    float x[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = to_float<DT>((uint16_t)(raw[it][i >> 1] >> (16 * (i & 1))));
    if (__any((out_of_range<DT>(raw[it][0]) | out_of_range<DT>(raw[it][1]) |
               out_of_range<DT>(raw[it][2]) | out_of_range<DT>(raw[it][3])) != 0)) {
      asm volatile("");        // stays a branch
#pragma unroll
      for (int i = 0; i < 8; ++i)
        x[i] = x[i] != x[i] ? 0.f : fminf(fmaxf(x[i], -65504.f), 65504.f);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      if (!VALUES) {
        lo8[i] = fminf(lo8[i], x[i]);
        hi8[i] = fmaxf(hi8[i], x[i]);
      }
    }
    lo = fminf(lo, dpp_mov<0xB1>(lo));   // quad_perm [1,0,3,2]
    hi = fmaxf(hi, dpp_mov<0xB1>(hi));
    lo = fminf(lo, dpp_mov<0x4E>(lo));   // quad_perm [2,3,0,1]
    hi = fmaxf(hi, dpp_mov<0x4E>(hi));
    const uint16_t zb = f2h(h2f(f2h(lo)) + 0.0f), sb = f2h(fifteenth(hi - lo));
    codes_of(x, h2f(zb), h2f(sb), q);
    uint8_t* const tile = page + (t >> 5) * (40 * D);
    if (!VALUES) {
      // slots 0, 2, 4, 6 are the low half's nibbles, 1, 3, 5, 7 the high half's
      const float a = __builtin_fmaf(4096.f, q[6], __builtin_fmaf(256.f, q[4], __builtin_fmaf(16.f, q[2], q[0])));
      const float b = __builtin_fmaf(4096.f, q[7], __builtin_fmaf(256.f, q[5], __builtin_fmaf(16.f, q[3], q[1])));
      *reinterpret_cast<uint32_t*>(tile + u * (8 * D) + (g / W) * (256 * W) +
                                   ((r8 * 16 + (tt & 15)) * W + g % W) * 4) =
          (uint32_t)a | (uint32_t)b << 16;
    } else {
      // bytes from sums that stay below 2^24
      const uint32_t w0 = (uint32_t)__builtin_fmaf(65536.f, q[2], __builtin_fmaf(256.f, q[1], q[0])) | (uint32_t)q[3] << 24;
      const uint32_t w1 = (uint32_t)__builtin_fmaf(65536.f, q[6], __builtin_fmaf(256.f, q[5], q[4])) | (uint32_t)q[7] << 24;
      *reinterpret_cast<u2*>(s_mem + t * (D / 4) + oc * 2) = u2{w0, w1};
    }
    // lane 0 of the group stores the scale, lane 1 the offset
    const int at = r * 8 * G + g * 8 + e;
    uint16_t* const meta = reinterpret_cast<uint16_t*>(tile + (VALUES ? 36 : 32) * D);
    if (r8 < 2) meta[r8 == 0 ? at : D + (VALUES ? at : tt * G + g)] = r8 == 0 ? sb : zb;
  }
  if constexpr (!VALUES) {
    if (summary == nullptr) return;
    // FP16 minima and maxima of the threads' tokens, [2][TS][D], then over those:
    // rounding is monotonic, so it may come first
    u4v lv, hv;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      lv[x] = pack2(f2h(lo8[2 * x]), f2h(lo8[2 * x + 1]));
      hv[x] = pack2(f2h(hi8[2 * x]), f2h(hi8[2 * x + 1]));
    }
    u4v* const s4 = reinterpret_cast<u4v*>(s_mem);
    s4[tid] = lv;
    s4[kAppendThreads + tid] = hv;
    __syncthreads();
    for (int c = tid; c < D; c += kAppendThreads) {      // two channels of one of the two
      const bool mx = c >= D / 2;
      const uint32_t* const from = s_mem + (mx ? 4 * kAppendThreads : 0) + c % (D / 2);
      uint32_t* const at = reinterpret_cast<uint32_t*>(summary) + c;
      h2 m = as_h2(from[0]);
#pragma unroll
      for (int j = 1; j < TS; ++j) {
        const h2 y = as_h2(from[j * (D / 2)]);
        m = mx ? __builtin_elementwise_max(m, y) : __builtin_elementwise_min(m, y);
      }
      if (o > 0) {
        const h2 y = as_h2(*at);
        m = mx ? __builtin_elementwise_max(m, y) : __builtin_elementwise_min(m, y);
      }
      *at = as_u32(m);
    }
    return;
  }
  __syncthreads();
  // a thread: tile, row r, 64 channels c, 4 channels at d4 and every 16th (j); the
  // bits of tokens outside the run stay
  for (int c = tid; c < 2 * D; c += kAppendThreads) {
    const int j = c & 3, d4 = (c >> 2) & 3, r = (c >> 4) & 3, c64 = (c >> 6) % (D / 64),
              tile = (c >> 6) / (D / 64);
    uint32_t mask = 0, A[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int t = tile * 32 + (e >> 2) * 16 + r * 4 + (e & 3);
      const uint32_t in = FULL || (t >= o && t < o + count) ? 0xFFFFFFFFu : 0u;
      A[e] = s_mem[t * (D / 4) + c64 * 16 + j * 4 + d4] & in;
      mask |= in & 15u << (4 * ((e >> 1) + 4 * (e & 1)));
    }
    if (mask == 0) continue;
    const uint32_t b0 = A[0] | A[2] << 4, b1 = A[4] | A[6] << 4, b2 = A[1] | A[3] << 4,
                   b3 = A[5] | A[7] << 4;
    uint32_t* const at = reinterpret_cast<uint32_t*>(page + tile * (40 * D) + 16 * D + c64 * 1024 +
                                                     (r * 16 + d4 * 4) * 16 + j * 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w = (b0 >> (8 * i) & 255u) | (b1 >> (8 * i) & 255u) << 8 |
                         (b2 >> (8 * i) & 255u) << 16 | (b3 >> (8 * i) & 255u) << 24;
      at[4 * i] = FULL || mask == 0xFFFFFFFFu ? w : (at[4 * i] & ~mask) | w;
    }
  }
}

template <int DT, int D>
__global__ void __launch_bounds__(kAppendThreads)
append_kernel(const uint16_t* __restrict__ k, int64_t k_row, int64_t k_head,
              const uint16_t* __restrict__ v, int64_t v_row, int64_t v_head, int T,
              const int32_t* __restrict__ slots, const int2* __restrict__ runs,
              uint8_t* __restrict__ data, uint16_t* __restrict__ summary, int64_t n_pages,
              int heads, Divisor by) {
  __shared__ __attribute__((aligned(16))) uint32_t s_mem[append_lds_words(D)];
  const bool values = blockIdx.x & 1;
  const int run = by.div(blockIdx.x >> 1), head = (int)(blockIdx.x >> 1) - run * heads;
  const int2 rc = runs[run];
  if (rc.x < 0 || rc.y <= 0 || rc.y > 64 || rc.x > T - rc.y) return;
  const int slot = slots[rc.x], last = slots[rc.x + rc.y - 1], o = slot & 63;
  if (slot < 0 || (slot >> 6) >= n_pages || o + rc.y > 64 || last != slot + rc.y - 1) return;
  const int64_t ph = (int64_t)(slot >> 6) * heads + head;
  uint8_t* const page = data + ph * (80 * D);
  uint16_t* const sm = summary == nullptr ? nullptr : summary + ph * (2 * D);
  if (values) {
    const uint16_t* const src = v + rc.x * v_row + head * v_head;
    if (rc.y == 64) append_run<DT, D, true, true>(src, v_row, 0, 64, page, sm, s_mem);
    else append_run<DT, D, true, false>(src, v_row, o, rc.y, page, sm, s_mem);
  } else {
    const uint16_t* const src = k + rc.x * k_row + head * k_head;
    if (rc.y == 64) append_run<DT, D, false, true>(src, k_row, 0, 64, page, sm, s_mem);
    else append_run<DT, D, false, false>(src, k_row, o, rc.y, page, sm, s_mem);
  }
}

// ----------------------------------------------------------------- select
// Scores (float32 in the workspace, [row][head][page]), then the n_sel highest.
//
// A page's bound is sum_d max(q min, q max) = sum_d q' (max + min) + |q'| (max -
// min) with q' = q / 2.  FP16 values and their products are
// far inside 64 bits, so those sums are exact but for operands that lie 2^20
// apart, and the choice does not depend on their order: two fused multiply-adds
// a channel and head, at the rate of 32-bit ones.  They are finite unless the head's
// query is not (0 times infinity included), and such a head takes no part.  A wave takes 512 / D pages at
// a time, 8 channels a lane, up to 8 heads' queries in registers.  16 sequences of
// up to 65001 tokens, 64 heads over 8 (43 MB of summaries, 8 us as a read): 25 us,
// half of it the multiply-adds, the rest conversions and sums across lanes.
constexpr int kScoreWaves = 4;
constexpr int kScoreHeads = 8;       // heads of one pass
constexpr int kScoreTurns = 8;       // most turns of a wave
constexpr float kMostScore = 0x1.fffffep127f;

__device__ __forceinline__ double lane_add(double v, int d) { return v + __shfl_xor(v, d); }

// v + v of the lane at the DPP control, within rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ double row_add(double v) {
  const u2 b = __builtin_bit_cast(u2, v);
  const u2 m = {dpp_mov<CTRL>(b[0]), dpp_mov<CTRL>(b[1])};
  return v + __builtin_bit_cast(double, m);
}

template <int DT, int D>
__global__ void __launch_bounds__(kScoreWaves * kWave)
score_kernel(KvRows a, Divisor by, const uint16_t* __restrict__ summary, int64_t n_pages,
             int kv_heads, int R, int n_sel, int chunk, float* __restrict__ scores) {
  constexpr int L = D / 8, P = kWave / L;   // lanes a page, pages a wave
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = by.div(blockIdx.x), head = blockIdx.x - row * kv_heads;
  const SeqRow sr = find_row(a, row);
  const int pages = sr.pos >= 0 ? (int)min((int64_t)(sr.pos / 64 + 1), a.width) : 0;
  if (pages <= n_sel) return;               // all of them are taken
  const int p_end = min((int)(blockIdx.y + 1) * chunk, pages);
  const int p_first = blockIdx.y * chunk + wave * P + lane / L;
  if ((int)blockIdx.y * chunk >= pages) return;
  const int c0 = (lane % L) * 8;
  const int32_t* const table = a.table + (int64_t)sr.b * a.width;
  float* const out = scores + ((int64_t)row * kv_heads + head) * a.width;
  // the pages of this wave's turns: P of each, a lane's own in every turn
  constexpr int kStep = kScoreWaves * P;
  int ids[kScoreTurns];
#pragma unroll
  for (int t = 0; t < kScoreTurns; ++t) {
    const int p = p_first + t * kStep;
    ids[t] = p < p_end ? table[p] : -1;
    if (ids[t] >= n_pages) ids[t] = -1;
  }
  auto load = [&](int id, u4v& lo, u4v& hi) {
    const uint16_t* sm = summary + ((int64_t)max(id, 0) * kv_heads + head) * (2 * D) + c0;
    lo = *reinterpret_cast<const u4v*>(sm);
    hi = *reinterpret_cast<const u4v*>(sm + D);
  };
  for (int h0 = 0; h0 < R; h0 += kScoreHeads) {
    u4v lo, hi;
    load(ids[0], lo, hi);
    double q[kScoreHeads][8];
#pragma unroll
    for (int h = 0; h < kScoreHeads; ++h) {
      // heads past the last repeat it, which changes no maximum
      const uint16_t* src = a.q + row * a.q_row + (head * R + min(h0 + h, R - 1)) * a.q_head + c0;
      const u4v v = *reinterpret_cast<const u4v*>(src);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[h][i] = 0.5 * (double)to_float<DT>((uint16_t)(v[i >> 1] >> (16 * (i & 1))));
    }
#pragma unroll
    for (int t = 0; t < kScoreTurns; ++t) {
      const int p = p_first + t * kStep;
      if (p - lane / L >= p_end) break;     // the same for the wave
      const u4v lo_now = lo, hi_now = hi;
      if (t + 1 < kScoreTurns) load(ids[t + 1 < kScoreTurns ? t + 1 : t], lo, hi);
      double s[kScoreHeads];
#pragma unroll
      for (int h = 0; h < kScoreHeads; ++h) s[h] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double mn = (double)h2f((uint16_t)(lo_now[i >> 1] >> (16 * (i & 1))));
        const double mx = (double)h2f((uint16_t)(hi_now[i >> 1] >> (16 * (i & 1))));
        const double sum = mx + mn, span = mx - mn;
#pragma unroll
        for (int h = 0; h < kScoreHeads; ++h) {
          s[h] = __builtin_fma(q[h][i], sum, s[h]);
          s[h] = __builtin_fma(__builtin_fabs(q[h][i]), span, s[h]);
        }
      }
      double best = -INFINITY;
#pragma unroll
      for (int h = 0; h < kScoreHeads; ++h) {
        double v = s[h];
        v = row_add<0xB1>(v);                 // quad_perm [1,0,3,2]
        v = row_add<0x4E>(v);                 // quad_perm [2,3,0,1]
        v = row_add<0x141>(v);                // row_half_mirror
        if constexpr (L >= 16) v = row_add<0x140>(v);   // row_mirror
        if constexpr (L == 32) v = lane_add(v, 16);
        best = fmax(best, __builtin_fma(v, 0.0, v));   // NaN unless finite, and then passed over
      }
      if (lane % L == 0 && p < p_end) {
        // infinite for the two that are always taken, and for no other
        float f = p == 0 || p == pages - 1 ? INFINITY
                                           : (ids[t] >= 0 ? fminf((float)best, kMostScore) : -INFINITY);
        if (h0 > 0) f = fmaxf(f, out[p]);
        out[p] = f;
      }
    }
  }
}

// Order of a float32 score as an unsigned key (NaN lowest).
__device__ __forceinline__ uint32_t score_key(float f) {
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  if (f != f) return 0;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The n_sel highest scores of one (row, head), rising: the n_sel-th highest key
// 8 bits at a time from histograms in LDS, then each thread a stretch of pages
// with its place from sums over the threads before it.  6 us for 512 pages, 7 for
// 1000: four passes of two barriers each.
constexpr int kPickThreads = 256;
constexpr int kPickHeld = 8192;      // keys held in LDS; more are read again

// Sum of v over the threads before this one, and over all in `total`.
__device__ __forceinline__ uint32_t block_before(uint32_t v, uint32_t* s_wave, uint32_t& total) {
  uint32_t t;
  const uint32_t in_wave = wave_excl_sum(v, t);
  const int w = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_wave[w] = t;
  __syncthreads();
  uint32_t base = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kPickThreads / kWave; ++i) {
    if (i < w) base += s_wave[i];
    total += s_wave[i];
  }
  return base + in_wave;
}

__global__ void __launch_bounds__(kPickThreads)
pick_kernel(KvRows a, Divisor by, const float* __restrict__ scores, int n_sel,
            int32_t* __restrict__ sel) {
  __shared__ uint32_t s_hist[4][256];
  __shared__ uint32_t s_found[2], s_wave[kPickThreads / kWave];
  extern __shared__ uint32_t s_key[];
  const int tid = threadIdx.x, row = by.div(blockIdx.x);
  const SeqRow sr = find_row(a, row);
  const int pages = sr.pos >= 0 ? (int)min((int64_t)(sr.pos / 64 + 1), a.width) : 0;
  const float* sc = scores + (int64_t)blockIdx.x * a.width;
  int32_t* out = sel + (int64_t)blockIdx.x * n_sel;
  const int n = min(n_sel, pages);
  for (int j = n + tid; j < n_sel; j += kPickThreads) out[j] = -1;
  if (n == pages) {
    for (int j = tid; j < n; j += kPickThreads) out[j] = j;
    return;
  }
  const bool held = pages <= kPickHeld;
#pragma unroll
  for (int i = 0; i < 4; ++i) s_hist[i][tid] = 0;
  __syncthreads();
  auto key_at = [&](int p) { return held ? s_key[p] : score_key(sc[p]); };
  uint32_t cut = 0, rank = (uint32_t)n;
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    for (int p = tid; p < pages; p += kPickThreads) {
      uint32_t key;
      if (pass == 0) {
        key = score_key(sc[p]);
        if (held) s_key[p] = key;
      } else {
        key = key_at(p);
        if ((key >> (shift + 8)) != cut) continue;
      }
      atomicAdd(&s_hist[pass][(key >> shift) & 255], 1u);
    }
    __syncthreads();
    // thread t holds bin 255 - t: the one where the sum from above reaches the rank
    uint32_t total;
    const uint32_t mine = s_hist[pass][255 - tid];
    const uint32_t above = block_before(mine, s_wave, total);
    if (above < rank && rank <= above + mine) {
      s_found[0] = (cut << 8) | (uint32_t)(255 - tid);
      s_found[1] = rank - above;
    }
    __syncthreads();
    cut = s_found[0];
    rank = s_found[1];
  }
  // keys above the cut, and of those equal to it the first `rank`
  const int per = (pages + kPickThreads - 1) / kPickThreads;
  const int p0 = min(tid * per, pages), p1 = min(p0 + per, pages);
  uint32_t above = 0, equal = 0, total;
  for (int p = p0; p < p1; ++p) {
    const uint32_t key = key_at(p);
    above += key > cut;
    equal += key == cut;
  }
  uint32_t at = block_before(above, s_wave, total);
  uint32_t eq = block_before(equal, s_wave, total);
  at += min(eq, rank);
  for (int p = p0; p < p1; ++p) {
    const uint32_t key = key_at(p);
    if (key > cut) out[at++] = p;
    else if (key == cut && eq++ < rank) out[at++] = p;
  }
}

// -------------------------------------------------------------- host side

int kv4_check_cache(const wq_kv4_cache* c, const char* who) {
  if (c == nullptr || c->data == nullptr) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL cache", who);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: head_dim must be 64, 128 or 256, got %lld", who,
                    (long long)c->head_dim);
  if (c->n_pages < 1 || c->n_pages > kMaxPage + 1 || c->n_kv_heads < 1 || c->n_kv_heads > 65535)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad cache shape (%lld pages, %lld heads)", who,
                    (long long)c->n_pages, (long long)c->n_kv_heads);
  if (!aligned16(c->data) || !aligned16(c->summary))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: cache pointers must be 16-byte aligned", who);
  return WQ_OK;
}

int kv4_check_rows(const wq_kv4_cache* c, const wq_kv4_rows* a, const char* who) {
  if (a == nullptr) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL rows", who);
  if (a->dtype != WQ_DT_F16 && a->dtype != WQ_DT_BF16)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: dtype must be WQ_DT_F16 or WQ_DT_BF16", who);
  if (a->n_seqs < 0 || a->n_rows < 0 || a->n_rows > (1 << 24) || a->n_seqs > (1 << 24) ||
      a->n_heads < 1 || a->n_heads > 65535 || a->table_width < 1 || a->table_width > (1 << 24))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (a->n_heads % c->n_kv_heads)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: %lld heads do not divide into %lld key/value heads",
                    who, (long long)a->n_heads, (long long)c->n_kv_heads);
  if (a->n_rows == 0 || a->n_seqs == 0) return WQ_OK;
  if (!a->block_table || !a->lens || !a->cu_rows || !a->q)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned4(a->block_table) || !aligned4(a->lens) || !aligned4(a->cu_rows) ||
      !aligned16(a->q))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (a->q_row_stride % 8 || a->q_head_stride % 8 || a->q_row_stride < 0 || a->q_head_stride < 0)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: q strides must be multiples of 8 elements", who);
  return WQ_OK;
}

KvRows kv4_rows(const wq_kv4_rows* a) {
  return KvRows{a->block_table, a->lens,          a->cu_rows,       a->table_width,
                (int)a->n_seqs, (int)a->n_rows,   (int)a->n_heads,  a->q,
                a->q_row_stride, a->q_head_stride};
}

}  // namespace wqd

using namespace wqd;

extern "C" int64_t wq_kv4_max_runs(int64_t n_seqs, int64_t n_rows) {
  if (n_seqs < 0 || n_rows < 0 || n_rows > (1 << 24) || n_seqs > WQ_KV4_MAX_SEQS)
    return wq::fail(WQ_ERR_INVALID_ARG, "wq_kv4_max_runs: bad sizes");
  wq::ok();
  const int64_t n = n_rows / WQ_KV4_PAGE + 2 * n_seqs;
  return n < n_rows ? n : n_rows;
}

extern "C" int wq_kv4_plan(const int32_t* lens, const int32_t* cu_rows, int64_t n_seqs,
                           int64_t n_rows, int32_t* block_table, int64_t table_width,
                           const int32_t* free_pages, int64_t n_free, int32_t* new_lens,
                           int32_t* slots, int32_t* runs, int64_t n_runs, int32_t* taken,
                           void* stream) {
  const char* who = "wq_kv4_plan";
  if (n_seqs > WQ_KV4_MAX_SEQS)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: at most %d sequences", who, WQ_KV4_MAX_SEQS);
  if (n_seqs < 0 || n_rows < 0 || n_rows > (1 << 24) || table_width < 1 ||
      table_width > (1 << 24) || n_free < 0 || n_free > kMaxPage + 1)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (n_seqs == 0 && n_rows > 0) return wq::ok();
  const int64_t want = wq_kv4_max_runs(n_seqs, n_rows);
  if (n_runs < want)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: runs holds %lld, %lld needed", who, (long long)n_runs,
                    (long long)want);
  if (n_runs > (1 << 25)) return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  if ((n_seqs && (!lens || !cu_rows || !block_table || !new_lens)) || !taken ||
      (n_rows && !slots) || (n_runs && !runs) || (n_free && !free_pages))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned4(lens) || !aligned4(cu_rows) || !aligned4(block_table) || !aligned4(new_lens) ||
      !aligned4(taken) || !aligned4(slots) || ((uintptr_t)runs & 7u) || !aligned4(free_pages))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  const size_t lds = (size_t)(4 * n_seqs + 3) * 4;
  if (!allow_lds((const void*)plan_kernel, lds))
    return wq::fail(WQ_ERR_HIP, "%s: cannot use %zu bytes of LDS", who, lds);
  int64_t most = n_rows > n_runs ? n_rows : n_runs;
  if (n_seqs > most) most = n_seqs;
  int64_t wgs = (most + kPlanThreads - 1) / kPlanThreads;   // one at least, for `taken`
  wgs = wgs > 256 ? 256 : wgs < 1 ? 1 : wgs;
  plan_kernel<<<dim3((unsigned)wgs), kPlanThreads, lds, (hipStream_t)stream>>>(
      lens, cu_rows, (int)n_seqs, (int)n_rows, block_table, table_width, free_pages, (int)n_free,
      new_lens, slots, runs, (int)n_runs, taken);
  return check_launch(who);
}

extern "C" int wq_kv4_append(const wq_kv4_cache* cache, int dtype, const uint16_t* k,
                             int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                             int64_t v_row_stride, int64_t v_head_stride, int64_t n_rows,
                             const int32_t* slots, const int32_t* runs, int64_t n_runs,
                             void* stream) {
  const char* who = "wq_kv4_append";
  if (int e = kv4_check_cache(cache, who)) return e;
  if (dtype != WQ_DT_F16 && dtype != WQ_DT_BF16)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: dtype must be WQ_DT_F16 or WQ_DT_BF16", who);
  if (n_rows < 0 || n_rows > (1 << 24) || n_runs < 0 ||
      n_runs * cache->n_kv_heads * 2 > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  if (n_rows == 0 || n_runs == 0) return wq::ok();
  if (!k || !v || !slots || !runs) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots) || ((uintptr_t)runs & 7u))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (k_row_stride % 8 || k_head_stride % 8 || v_row_stride % 8 || v_head_stride % 8 ||
      k_row_stride < 0 || k_head_stride < 0 || v_row_stride < 0 || v_head_stride < 0)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements", who);
  const dim3 grid((unsigned)(n_runs * cache->n_kv_heads * 2));
  kv4_dispatch(dtype, cache->head_dim, [&](auto dt, auto d) {
    append_kernel<decltype(dt)::value, decltype(d)::value>
        <<<grid, kAppendThreads, 0, (hipStream_t)stream>>>(
            k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, (int)n_rows, slots,
            reinterpret_cast<const int2*>(runs), cache->data, cache->summary, cache->n_pages,
            (int)cache->n_kv_heads, Divisor(cache->n_kv_heads));
  });
  return check_launch(who);
}

extern "C" int64_t wq_kv4_select_workspace(int64_t n_rows, int64_t n_kv_heads,
                                           int64_t table_width) {
  if (n_rows < 0 || n_rows > (1 << 24) || n_kv_heads < 1 || n_kv_heads > 65535 ||
      table_width < 1 || table_width > (1 << 24))
    return wq::fail(WQ_ERR_INVALID_ARG, "wq_kv4_select_workspace: bad sizes");
  if (n_rows * n_kv_heads > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "wq_kv4_select_workspace: too many rows");
  wq::ok();
  return (n_rows * n_kv_heads * table_width * 4 + 15) / 16 * 16;
}

extern "C" int wq_kv4_select(const wq_kv4_cache* cache, const wq_kv4_rows* rows, int64_t n_sel,
                             int32_t* sel, void* workspace, int64_t workspace_bytes,
                             void* stream) {
  const char* who = "wq_kv4_select";
  if (int e = kv4_check_cache(cache, who)) return e;
  if (int e = kv4_check_rows(cache, rows, who)) return e;
  if (cache->summary == nullptr)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: the cache has no summary", who);
  if (n_sel < 2 || n_sel > (1 << 20))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: n_sel must be at least 2 (the first and last page)", who);
  if (rows->n_rows == 0 || rows->n_seqs == 0) return wq::ok();
  if (rows->n_rows * cache->n_kv_heads > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  const int64_t need = wq_kv4_select_workspace(rows->n_rows, cache->n_kv_heads, rows->table_width);
  if (!sel || !workspace) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (workspace_bytes < need)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                    (long long)workspace_bytes, (long long)need);
  if (!aligned4(sel) || !aligned16(workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  const KvRows a = kv4_rows(rows);
  const Divisor by(cache->n_kv_heads);
  float* scores = static_cast<float*>(workspace);
  // a workgroup takes `chunk` pages of a (row, head): up to 8 of its waves' turns
  // (the queries' conversion is spread over them), fewer where that would leave
  // compute units idle
  const int64_t turn = kScoreWaves * (512 / cache->head_dim);
  const int64_t pairs = rows->n_rows * cache->n_kv_heads;
  int64_t turns = pairs * rows->table_width / (turn * 512);
  turns = turns < 1 ? 1 : turns > kScoreTurns ? kScoreTurns : turns;
  if (rows->table_width > turn * turns * 65535)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: table of %lld pages", who,
                    (long long)rows->table_width);
  const int64_t chunk = turn * turns;
  const dim3 grid((unsigned)pairs, (unsigned)((rows->table_width + chunk - 1) / chunk));
  kv4_dispatch(rows->dtype, cache->head_dim, [&](auto dt, auto d) {
    score_kernel<decltype(dt)::value, decltype(d)::value>
        <<<grid, kScoreWaves * kWave, 0, (hipStream_t)stream>>>(
            a, by, cache->summary, cache->n_pages, (int)cache->n_kv_heads,
            (int)(rows->n_heads / cache->n_kv_heads), (int)n_sel, (int)chunk, scores);
  });
  const int64_t held = rows->table_width < kPickHeld ? rows->table_width : kPickHeld;
  pick_kernel<<<dim3((unsigned)pairs), kPickThreads, (size_t)held * 4, (hipStream_t)stream>>>(
      a, by, scores, (int)n_sel, sel);
  return check_launch(who);
}
