// The paged 8-bit key/value cache (wq.h, "8-bit key/value cache"): writing tokens
// and moving the most attended ones to fresh pages.  Attention is in
// wq_kv8_attn.hip.

#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"
#include "wq_kv8.cuh"
#include "wq_select.cuh"

namespace wqd {

typedef unsigned short us2 __attribute__((ext_vector_type(2)));

// v + 2^23 + 128 in float32 is rounded to a whole number, ties to even, and its last
// byte is that number, + 128: a code as the cache holds it.
constexpr float kRound8 = 8388608.f + 128.f;

// The last bytes of four numbers as one word.
__device__ __forceinline__ uint32_t bytes4(float a, float b, float c, float d) {
  const uint32_t lo = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x0C0C0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, d), __builtin_bit_cast(uint32_t, c), 0x04000C0Cu);
  return lo | hi;
}

// Four codes at an exponent `by` powers of two higher: rint(q / 2^by).
__device__ __forceinline__ uint32_t raise4(uint32_t w, int by) {
  const float f = pow2(-by);
  float q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q[i] = __builtin_fmaf((float)((w >> (8 * i)) & 255u) - 128.f, f, kRound8);
  return bytes4(q[0], q[1], q[2], q[3]);
}

// ----------------------------------------------------------------- append
// One workgroup per (run, head, keys or values).  A thread takes 8 channels of a
// token at a time; all of a page's loads are in flight before the first is used.
// Keys leave as 8 bytes a thread; values go through LDS, where a thread then gathers
// 16 tokens of a channel.  Memory bounds prompts: 23145 tokens of 8 heads of 128
// channels (142 MB) take 31 us, 28 as a plain copy of as many bytes.  Single tokens:
// latency of run, slot, token and bytes in turn, with 256 of them 8.9 us a call in
// workgroups of one wave and 10.4 in four.
constexpr int kAppend8Threads = 256, kAppend8Few = 64;

// 16-bit values past +-65504 (BF16: 65536, whose code is the same) and infinities
// as that, NaN as 0.
template <int DT>
__device__ __forceinline__ uint32_t within16(uint32_t w) {
  constexpr uint32_t kInf = DT == WQ_DT_F16 ? 0x7C00u : 0x7F80u, kTop = DT == WQ_DT_F16 ? 0x7BFFu : 0x4780u;
  uint32_t out = 0;
#pragma unroll
  for (int s = 0; s < 32; s += 16) {
    const uint32_t h = (w >> s) & 0xFFFFu, m = h & 0x7FFFu;
    out |= (m > kInf ? 0u : m > kTop ? (h & 0x8000u) | kTop : h) << s;
  }
  return out;
}

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2, a), __builtin_bit_cast(us2, b)));
}

// The largest of the wave's values.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  auto dpp = [](uint32_t x, auto c) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, decltype(c)::value, 0xF, 0xF, false);
  };
  v = max(v, dpp(v, std::integral_constant<int, 0xB1>{}));    // quad_perm [1,0,3,2]
  v = max(v, dpp(v, std::integral_constant<int, 0x4E>{}));    // quad_perm [2,3,0,1]
  v = max(v, dpp(v, std::integral_constant<int, 0x124>{}));   // row_ror:4
  v = max(v, dpp(v, std::integral_constant<int, 0x128>{}));   // row_ror:8
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}

// The smallest exponent from kLeast8 on with most 2^-e < 127.5 = 1.9921875 2^6: adding
// 2^-7 of the leading bit carries where the significand reaches 1.9921875.
__device__ __forceinline__ int exponent_of(float most) {
  return max((int)((__builtin_bit_cast(uint32_t, most) + 0x10000u) >> 23) - 133, kLeast8);
}

// FULL: the run is a whole page, so nothing is masked.
template <int DT, int D, int NT, bool VALUES, bool FULL>
__device__ __forceinline__ void append8_run(const uint16_t* __restrict__ src, int64_t row, int o,
                                            int count, uint8_t* __restrict__ page,
                                            uint8_t* __restrict__ exps, uint32_t* s_mem) {
  constexpr int O = D / 8, TS = NT / O, IT = 64 / TS;
  __shared__ uint32_t s_most[4];
  const int tid = threadIdx.x, oc = tid % O;
  u4v raw[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    const int t = tid / O + it * TS;
    const bool in = FULL || (t >= o && t < o + count);
    raw[it] = in ? *reinterpret_cast<const u4v*>(src + (t - o) * row + oc * 8) : u4v{0, 0, 0, 0};
  }
  const int u0 = o / kBlock8, u1 = (o + count - 1) / kBlock8;     // the blocks with new tokens
  const bool older = !FULL && o % kBlock8 != 0;                    // block u0 has some from before
  const int was = older ? min(max((int)(int8_t)exps[u0], kLeast8), kMost8) : kLeast8;
  if (tid < 4) s_most[tid] = 0;
  lds_barrier();
  // turns without a token of the run are passed over
  auto idle = [&](int it) { return !FULL && (it * TS + TS <= o || it * TS >= o + count); };
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    if (idle(it)) continue;
    uint32_t m = max_halves(max_halves(raw[it][0] & 0x7FFF7FFFu, raw[it][1] & 0x7FFF7FFFu),
                            max_halves(raw[it][2] & 0x7FFF7FFFu, raw[it][3] & 0x7FFF7FFFu));
    m = max(m & 0xFFFFu, m >> 16);
    if (__any(m > (DT == WQ_DT_F16 ? 0x7BFFu : 0x4780u))) {
      asm volatile("");        // stays a branch
      m = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        raw[it][x] = within16<DT>(raw[it][x]);
        m = max_halves(m, raw[it][x] & 0x7FFF7FFFu);
      }
      m = max(m & 0xFFFFu, m >> 16);
    }
    m = wave_max(m);
    // a wave's tokens of one turn are of one block
    if ((tid & 63) == 0) atomicMax(&s_most[(tid / O + it * TS) / kBlock8], m);
  }
  __syncthreads();
  auto exponent = [&](int u) {
    const int e = exponent_of(to_float<DT>((uint16_t)s_most[u]));
    return older && u == u0 ? max(e, was) : e;
  };
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    if (idle(it)) continue;
    const int t = tid / O + it * TS;
    if (!FULL && (t < o || t >= o + count)) continue;
    const float by = pow2(-exponent(t / kBlock8));
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      q[i] = __builtin_fmaf(to_float<DT>((uint16_t)(raw[it][i >> 1] >> (16 * (i & 1)))), by, kRound8);
    const u2 w = {bytes4(q[0], q[1], q[2], q[3]), bytes4(q[4], q[5], q[6], q[7])};
    if (VALUES)
      *reinterpret_cast<u2*>(s_mem + t * (D / 4) + oc * 2) = w;
    else
      *reinterpret_cast<u2*>(page + (t / 16) * (16 * D) + (oc / 8) * 1024 +
                             ((oc & 3) * 16 + (t & 15)) * 16 + ((oc >> 2) & 1) * 8) = w;
  }
  if (tid >= u0 && tid <= u1) exps[tid] = (uint8_t)exponent(tid);
  const int by = older ? exponent(u0) - was : 0;     // the block's older tokens move by this
  if constexpr (!VALUES) {
    if (by > 0) {
      const int nt = o % kBlock8;
      uint32_t* const block = reinterpret_cast<uint32_t*>(page + u0 * (16 * D));
      for (int c = tid; c < nt * (D / 4); c += NT) {
        const int x = c >> 2, l = x % nt, cr = x / nt;
        uint32_t* const at = block + cr * 64 + l * 4 + (c & 3);
        *at = raise4(*at, by);
      }
    }
    return;
  }
  __syncthreads();
  // a thread: row r of the page's blocks, one channel: 4 bytes of each block, from LDS
  const uint8_t* const bytes = reinterpret_cast<const uint8_t*>(s_mem);
  for (int c = tid; c < 4 * D; c += NT) {
    const int d = c % D, r = c / D;
    uint32_t* const at = reinterpret_cast<uint32_t*>(page + 64 * D + ((d / 16 * 4 + r) * 16 + d % 16) * 16);
    u4v w;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint8_t* const from = bytes + (16 * u + 4 * r) * D + d;
      if (FULL) {
        w[u] = from[0] | (uint32_t)from[D] << 8 | (uint32_t)from[2 * D] << 16 | (uint32_t)from[3 * D] << 24;
        continue;
      }
      if (u < u0 || u > u1) continue;
      const int t = 16 * u + 4 * r;
      const bool moves = by > 0 && u == u0 && t < o;
      if (!moves && (t + 3 < o || t >= o + count)) continue;
      const uint32_t old = at[u], moved = moves ? raise4(old, by) : old;
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool in = t + i >= o && t + i < o + count;
        const uint32_t keep = t + i < o ? moved : old;
        v |= in ? (uint32_t)from[i * D] << (8 * i) : keep & 255u << (8 * i);
      }
      at[u] = v;
    }
    if (FULL) *reinterpret_cast<u4v*>(at) = w;
  }
}

template <int DT, int D, int NT>
__global__ void __launch_bounds__(NT)
append8_kernel(const uint16_t* __restrict__ k, int64_t k_row, int64_t k_head,
               const uint16_t* __restrict__ v, int64_t v_row, int64_t v_head, int T,
               const int32_t* __restrict__ slots, const int2* __restrict__ runs,
               uint8_t* __restrict__ data, uint8_t* __restrict__ exps, int64_t n_pages, int heads,
               Divisor by) {
  __shared__ __attribute__((aligned(16))) uint32_t s_mem[16 * D];
  const bool values = blockIdx.x & 1;
  const int run = by.div(blockIdx.x >> 1), head = (int)(blockIdx.x >> 1) - run * heads;
  const int2 rc = runs[run];
  if (rc.x < 0 || rc.y <= 0 || rc.y > 64 || rc.x > T - rc.y) return;
  const int slot = slots[rc.x], last = slots[rc.x + rc.y - 1], o = slot & 63;
  if (slot < 0 || (slot >> 6) >= n_pages || o + rc.y > 64 || last != slot + rc.y - 1) return;
  const int64_t ph = (int64_t)(slot >> 6) * heads + head;
  uint8_t* const page = data + ph * (128 * D);
  uint8_t* const ex = exps + ph * 8;
  if (values) {
    const uint16_t* const src = v + rc.x * v_row + head * v_head;
    if (rc.y == 64) append8_run<DT, D, NT, true, true>(src, v_row, 0, 64, page, ex + 4, s_mem);
    else append8_run<DT, D, NT, true, false>(src, v_row, o, rc.y, page, ex + 4, s_mem);
  } else {
    const uint16_t* const src = k + rc.x * k_row + head * k_head;
    if (rc.y == 64) append8_run<DT, D, NT, false, true>(src, k_row, 0, 64, page, ex, s_mem);
    else append8_run<DT, D, NT, false, false>(src, k_row, o, rc.y, page, ex, s_mem);
  }
}

// ------------------------------------------------------------------ evict
// Which tokens stay (pick8_kernel, with the tables), then their move (move8_kernel).

constexpr int kPick8Threads = 1024, kPick8Waves = kPick8Threads / kWave;
constexpr int kPick8Bins = 2048;
constexpr int kPick8Held = 16;         // masses a thread holds; those of longer sequences are read again,
constexpr int kPick8Again = 8;         // so many at a time
constexpr int kPick8Few = 4;           // masses a thread whose keys are made anew each time

struct Evict8Args {
  const int32_t *table, *lens, *free_pages;
  int64_t width, mass_tokens, new_tokens;
  const float* mass;
  int32_t *new_table, *new_lens, *taken, *kept;
  float* new_mass;
  int seqs, heads, keep, recent, n_free, pages;   // pages: those of `keep` tokens
  Divisor heads_by;
};

// Tokens of a sequence: those with a place in the table.
__device__ __forceinline__ int evict_len(const Evict8Args& p, int b) {
  return (int)min((int64_t)max(p.lens[b], 0), 64 * p.width);
}

// Order of a mass as an unsigned key: NaN lowest, -0 as 0.
__device__ __forceinline__ uint32_t mass_key(float f) {
  if (f != f) return 0;
  const uint32_t b = __builtin_bit_cast(uint32_t, f + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the workgroup, in all threads.
__device__ __forceinline__ uint32_t block_sum(uint32_t v, uint32_t* s_wave) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s_wave[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t all = 0;
#pragma unroll
  for (int w = 0; w < kPick8Waves; ++w) all += s_wave[w];
  return all;
}

// A sequence's new table row and length, and the pages taken.
__device__ __forceinline__ void evict_tables(const Evict8Args& p, int b, uint32_t* s_wave) {
  const int tid = threadIdx.x, len = evict_len(p, b);
  const bool over = len > p.keep;
  uint32_t before = 0, all = 0;
  for (int s = tid; s < p.seqs; s += kPick8Threads) {
    const uint32_t need = evict_len(p, s) > p.keep ? p.pages : 0;
    all += need;
    if (s < b) before += need;
  }
  before = block_sum(before, s_wave);
  if (b == 0) {
    all = block_sum(all, s_wave);
    if (tid == 0) p.taken[0] = (int)all;
  }
  if (tid == 0) p.new_lens[b] = min(len, p.keep);
  for (int64_t i = tid; i < p.width; i += kPick8Threads) {
    int page = -1;
    if (!over) page = p.table[b * p.width + i];
    else if (i < p.pages && before + i < (uint32_t)p.n_free) page = p.free_pages[before + i];
    p.new_table[b * p.width + i] = page;
  }
}

// A batch without sequences takes no pages.
__global__ void none_taken_kernel(int32_t* taken) { taken[0] = 0; }

// One workgroup a sequence for the tables, and one a (sequence, head) for the tokens:
// the room-th highest key 11 bits at a time from histograms in LDS (four of them for
// the first bits, which many masses share), then every wave a stretch of the tokens
// with its place from the counts of the waves before it.  Masses stay in registers: in
// tables of up to 16384 tokens all of them, and their keys too, unless the table has no more
// than 4096 (4 x 16384 tokens take 42 us, 45 with keys made anew each time; 1000 take 16, 15).
// LONG: of any length.
// Latency, with the move: 4500 tokens 18 us; 16384 of 131072 172 us, 195 where a load waits
// for the one before and 237 where masses that are not held are read one at a time.
enum Pick8 { kPick8Short, kPick8Keys, kPick8Long };
template <Pick8 HOW>
__global__ void __launch_bounds__(kPick8Threads) pick8_kernel(Evict8Args p) {
  constexpr bool LONG = HOW == kPick8Long, KEYS = HOW == kPick8Keys;
  __shared__ uint32_t s_hist[6 * kPick8Bins];      // four of the first bits, one of the next each
  __shared__ uint32_t s_wave[kPick8Waves], s_count[kPick8Waves][2], s_found[2];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if ((int)blockIdx.x < p.seqs) {
    evict_tables(p, blockIdx.x, s_wave);
    return;
  }
  const int item = blockIdx.x - p.seqs, b = p.heads_by.div(item), head = item - b * p.heads;
  const int len = evict_len(p, b);
  const bool over = len > p.keep;
  const int64_t pair = (int64_t)b * p.heads + head;
  const float* const masses = p.mass + pair * p.mass_tokens;
  auto mass_of = [&](int t) { return t < p.mass_tokens ? masses[t] : 0.f; };
  float* const new_mass = p.new_mass + pair * p.new_tokens;
  int32_t* const kept = p.kept + pair * p.keep;
  const int room = over ? p.keep - p.recent : 0, old = over ? len - p.recent : 0;
  // the last tokens (all of a sequence within its budget)
  for (int i = room + tid; i < p.keep; i += kPick8Threads) {
    const int t = old + (i - room);
    kept[i] = t < len ? t : -1;
    if (t < len) new_mass[i] = mass_of(t);
  }
  if (room == 0) return;
  // every wave a stretch of the tokens, 64 at a time
  const int turns = (old + kPick8Threads - 1) / kPick8Threads;
  const int t0 = wave * turns * kWave + lane;
  // without a branch, so that no load waits for another
  const int have = (int)min((int64_t)old, p.mass_tokens);
  auto load = [&](int i) {
    const int t = t0 + i * kWave;
    const float m = masses[min(t, have - 1)];
    return t < have ? m : 0.f;
  };
  float held[kPick8Held];
#pragma unroll
  for (int i = 0; i < kPick8Held; ++i) held[i] = load(i);
  uint32_t keys[kPick8Held];
  // f(mass, its key, token) of the stretch's tokens, all lanes together (a token past
  // the last: old or more); those that are not held are read again, several at a time
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < kPick8Held; ++i)
      if (i < turns) f(held[i], KEYS ? keys[i] : mass_key(held[i]), t0 + i * kWave);
    for (int i0 = kPick8Held; LONG && i0 < turns; i0 += kPick8Again) {
      float m[kPick8Again];
#pragma unroll
      for (int i = 0; i < kPick8Again; ++i) m[i] = load(i0 + i);
#pragma unroll
      for (int i = 0; i < kPick8Again; ++i)
        if (i0 + i < turns) f(m[i], mass_key(m[i]), t0 + (i0 + i) * kWave);
    }
  };
  for (int i = tid; i < 6 * kPick8Bins; i += kPick8Threads) s_hist[i] = 0;
  __syncthreads();
  if constexpr (KEYS) {
#pragma unroll
    for (int i = 0; i < kPick8Held; i += 4) {
      if (i >= turns) break;
#pragma unroll
      for (int x = i; x < i + 4; ++x) {
        keys[x] = mass_key(held[x]);
        asm volatile("" : "+v"(keys[x]));        // kept, not made again
      }
    }
  }
  uint32_t cut = 0, rank = (uint32_t)room;     // 0 < room < old
  int bits = 0;
  for (int pass = 0; pass < 3; ++pass) {
    const int width = pass < 2 ? 11 : 10, shift = 32 - bits - width;
    const int copies = pass == 0 ? 4 : 1, first_copy = pass == 0 ? 0 : pass + 3;
    uint32_t* const hist = s_hist + (pass == 0 ? lane & 3 : first_copy) * kPick8Bins;
    each([&](float, uint32_t key, int t) {
      if (t < old && (pass == 0 || (key >> (shift + width)) == cut))
        atomicAdd(&hist[(key >> shift) & ((1u << width) - 1)], 1u);
    });
    __syncthreads();
    // thread t holds the bins 2047 - 2 t and 2046 - 2 t: where the sum from above
    // reaches the rank
    uint32_t c0 = 0, c1 = 0;
    for (int i = first_copy; i < first_copy + copies; ++i) {
      c0 += s_hist[(i + 1) * kPick8Bins - 1 - 2 * tid];
      c1 += s_hist[(i + 1) * kPick8Bins - 2 - 2 * tid];
    }
    uint32_t total;
    uint32_t above = wave_excl_sum(c0 + c1, total);
    if (lane == 0) s_wave[wave] = total;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kPick8Waves; ++w) above += w < wave ? s_wave[w] : 0;
    if (above < rank && rank <= above + c0 + c1) {
      const bool first = rank <= above + c0;
      s_found[0] = (cut << width) | (uint32_t)(kPick8Bins - 1 - 2 * tid - (first ? 0 : 1));
      s_found[1] = rank - above - (first ? 0 : c0);
    }
    __syncthreads();
    cut = s_found[0];
    rank = s_found[1];
    bits += width;
  }
  // keys above the cut, and of those equal to it the first `rank`
  uint32_t above = 0, equal = 0;
  each([&](float, uint32_t key, int t) {
    above += __popcll(__ballot(t < old && key > cut));
    equal += __popcll(__ballot(t < old && key == cut));
  });
  if (lane == 0) { s_count[wave][0] = above; s_count[wave][1] = equal; }
  __syncthreads();
  uint32_t at = 0, eq = 0;
#pragma unroll
  for (int w = 0; w < kPick8Waves; ++w) {
    at += w < wave ? s_count[w][0] : 0;
    eq += w < wave ? s_count[w][1] : 0;
  }
  at += min(eq, rank);
  const uint64_t below = (1ull << lane) - 1;
  each([&](float m, uint32_t key, int t) {
    const uint64_t same = __ballot(t < old && key == cut);
    const bool take = t < old && (key > cut || (key == cut && eq + __popcll(same & below) < rank));
    const uint64_t took = __ballot(take);
    if (take) {
      const uint32_t i = at + __popcll(took & below);
      kept[i] = t;
      new_mass[i] = m;
    }
    at += __popcll(took);
    eq += __popcll(same);
  });
}

// The kept tokens of a sequence over its budget, in fresh pages: one workgroup per
// (page, head).  Keys move by 16 bytes of a token.  A value's bytes stand with those
// of 15 other tokens, so that a token touches every line of its page's values: the
// source pages go through LDS, 24 KB of them at a time (D = 256: 16), and a lane gathers the 16
// bytes of a channel from there (the lanes of a wave the same tokens, 16 bytes
// apart).  Memory bounds it: 12 sequences of 6001 to 16000 tokens, 6000 kept, 8 heads
// of 128 channels read 350 MB (nearly every source line has a kept token, and a source
// page at the border of two fresh ones is read twice) and write 180 in 109 us, 4.9 TB/s;
// a plain copy reaches 5.2.  Stores that stay in the caches cost 4 us more.
constexpr int kMove8Threads = 256;
template <int D>
__global__ void __launch_bounds__(kMove8Threads)
move8_kernel(Evict8Args p, Divisor pairs_by, uint8_t* __restrict__ data,
             uint8_t* __restrict__ exps, int64_t n_pages) {
  constexpr int kPages = D == 256 ? 1 : 384 / D, kBytes = 64 * D;     // source pages in LDS, a page's bytes there
  constexpr int kChunks = 4 * D / kMove8Threads;       // 16-byte chunks of a page that a thread writes
  __shared__ __attribute__((aligned(16))) uint8_t s_values[kPages * kBytes];
  __shared__ int64_t s_src[64];       // page and head of a token, times 64, + its place; -1: none
  __shared__ __attribute__((aligned(16))) int s_at[64];      // byte of a token's first value, pages in a row
  __shared__ __attribute__((aligned(16))) int s_by[2][64];   // what its exponents rise by
  __shared__ int64_t s_page[64];
  __shared__ int s_pages, s_rise;
  const int tid = threadIdx.x;
  // pages of a pair (sequence, head) share source pages: for 8 pairs and their
  // multiples they are on one XCD
  const int pg = pairs_by.div(blockIdx.x), pair = blockIdx.x - pg * (int)pairs_by.d;
  const int b = p.heads_by.div(pair), head = pair - b * p.heads;
  const int n = min(p.keep - 64 * pg, 64);
  const int kept = tid < n ? p.kept[(int64_t)pair * p.keep + 64 * pg + tid] : -1;
  const int to = pg < p.width ? p.new_table[(int64_t)b * p.width + pg] : -1;
  if (evict_len(p, b) <= p.keep || to < 0 || to >= n_pages) return;
  const int64_t dst = (int64_t)to * p.heads + head;
  if (tid < 64) {
    int64_t src = -1;
    int place = -1;
    u2 ex = {0, 0};
    if (tid < n) {
      place = kept / 64;
      const int page = p.table[(int64_t)b * p.width + place];
      if (page >= 0 && page < n_pages) {
        const int64_t ph = (int64_t)page * p.heads + head;
        src = ph * 64 + (kept & 63);
        ex = *reinterpret_cast<const u2*>(exps + ph * 8);
      }
    }
    const int s = (int)(src & 63);
    bool rise = false;
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const int e = src < 0 ? kLeast8 : exponent8(ex[v], s / kBlock8);
      int most = e;                   // of the block's 16 lanes
#pragma unroll
      for (int d = 1; d < kBlock8; d <<= 1) most = max(most, __shfl_xor(most, d));
      s_by[v][tid] = most - e;
      if (tid % kBlock8 == 0 && tid < n) exps[dst * 8 + 4 * v + tid / kBlock8] = (uint8_t)most;
      rise |= v && most > e;
    }
    rise = __any(rise);
    // source pages in the order of their tokens
    const int prev = __shfl_up(place, 1);
    const bool first = tid < n && (tid == 0 || place != prev);
    const uint64_t firsts = __ballot(first);
    const int nth = __popcll(firsts & ((2ull << tid) - 1)) - 1;
    s_src[tid] = src;
    s_at[tid] = src < 0 ? -1 : nth * kBytes + ((s >> 2) & 3) * 256 + (s / 16) * 4 + (s & 3);
    if (first) s_page[nth] = src < 0 ? -1 : src >> 6;
    if (tid == 0) {
      s_pages = __popcll(firsts);
      s_rise = rise;
    }
  }
  __syncthreads();
  uint8_t* const page = data + dst * (128 * D);
  const u4v zeros = {0x80808080u, 0x80808080u, 0x80808080u, 0x80808080u};
  u4v key[kChunks], w[kChunks];
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int c = tid + k * kMove8Threads, t = c & 63, cr = c >> 6;
    const int64_t src = s_src[t];
    const int s = (int)(src & 63);
    key[k] = w[k] = zeros;
    if (src >= 0)
      key[k] = *reinterpret_cast<const u4v*>(data + (src >> 6) * (128 * D) + (s / 16) * (16 * D) +
                                             cr * 256 + (s & 15) * 16);
  }
  for (int q = 0; q < s_pages; q += kPages) {
    if (q > 0) __syncthreads();
    u4v got[kPages * kChunks];
#pragma unroll
    for (int x = 0; x < kPages * kChunks; ++x) {
      const int c = tid + x * kMove8Threads, slot = c / (4 * D);
      const int64_t from = q + slot < s_pages ? s_page[q + slot] : -1;
      got[x] = from >= 0 ? *reinterpret_cast<const u4v*>(data + from * (128 * D) + kBytes + (c % (4 * D)) * 16)
                         : zeros;
    }
    if (q == 0) {
#pragma unroll
      for (int k = 0; k < kChunks; ++k) {
        const int c = tid + k * kMove8Threads, t = c & 63, cr = c >> 6, by = s_by[0][t];
        if (by > 0) {
#pragma unroll
          for (int x = 0; x < 4; ++x) key[k][x] = raise4(key[k][x], by);
        }
        if (t < n)
          __builtin_nontemporal_store(
              key[k], reinterpret_cast<u4v*>(page + (t / 16) * (16 * D) + cr * 256 + (t & 15) * 16));
      }
    }
#pragma unroll
    for (int x = 0; x < kPages * kChunks; ++x)
      reinterpret_cast<u4v*>(s_values)[tid + x * kMove8Threads] = got[x];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kChunks; ++k) {
      const int c = tid + k * kMove8Threads, d = c % D, r = c / D;
      const int of = (d / 16) * 1024 + (d % 16) * 16;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int4 at = *reinterpret_cast<const int4*>(&s_at[16 * u + 4 * r]);
        const int a[4] = {at.x, at.y, at.z, at.w};
        // four tokens in a row: mostly of one round
        const int lo = q * kBytes, hi = lo + kPages * kBytes;
        if (max(max(a[0], a[1]), max(a[2], a[3])) < lo) continue;
        uint32_t v[4];
        bool in[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          in[i] = a[i] >= lo && a[i] < hi;
          v[i] = s_values[in[i] ? a[i] - lo + of : of];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (in[i]) w[k][u] = (w[k][u] & ~(255u << (8 * i))) | v[i] << (8 * i);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int c = tid + k * kMove8Threads, d = c % D, r = c / D;
    u4v* const out = reinterpret_cast<u4v*>(page + kBytes + (d / 16) * 1024 + (d % 16) * 16 + r * 256);
    if (4 * r >= n) continue;
    if (s_rise) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int4 by = *reinterpret_cast<const int4*>(&s_by[1][16 * u + 4 * r]);
        const int f[4] = {by.x, by.y, by.z, by.w};
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = __builtin_fmaf((float)((w[k][u] >> (8 * i)) & 255u) - 128.f, pow2(-f[i]), kRound8);
        w[k][u] = bytes4(v[0], v[1], v[2], v[3]);
      }
    }
    if (n < 64) {                     // the bytes of tokens past the last stay
      const u4v old = *out;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int have = min(max(n - (16 * u + 4 * r), 0), 4);
        const uint32_t m = have == 4 ? 0xFFFFFFFFu : (1u << (8 * have)) - 1;
        w[k][u] = (w[k][u] & m) | (old[u] & ~m);
      }
    }
    __builtin_nontemporal_store(w[k], out);
  }
}

// -------------------------------------------------------------- host side

int kv8_check_cache(const wq_kv8_cache* c, const char* who) {
  if (c == nullptr || c->exponents == nullptr) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL cache", who);
  const wq_kv4_cache shape = kv8_shape(c);
  if (int e = kv4_check_cache(&shape, who)) return e;
  if ((uintptr_t)c->exponents & 7u)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: exponents must be 8-byte aligned", who);
  return WQ_OK;
}

}  // namespace wqd

using namespace wqd;

extern "C" int wq_kv8_append(const wq_kv8_cache* cache, int dtype, const uint16_t* k,
                             int64_t k_row_stride, int64_t k_head_stride, const uint16_t* v,
                             int64_t v_row_stride, int64_t v_head_stride, int64_t n_rows,
                             const int32_t* slots, const int32_t* runs, int64_t n_runs,
                             void* stream) {
  const char* who = "wq_kv8_append";
  if (int e = kv8_check_cache(cache, who)) return e;
  if (dtype != WQ_DT_F16 && dtype != WQ_DT_BF16)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: dtype must be WQ_DT_F16 or WQ_DT_BF16", who);
  if (n_rows < 0 || n_rows > (1 << 24) || n_runs < 0 || n_runs > 0x7FFFFFFF ||
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
    auto launch = [&](auto kernel, int threads) {
      kernel<<<grid, threads, 0, (hipStream_t)stream>>>(
          k, k_row_stride, k_head_stride, v, v_row_stride, v_head_stride, (int)n_rows, slots,
          reinterpret_cast<const int2*>(runs), cache->data,
          reinterpret_cast<uint8_t*>(cache->exponents), cache->n_pages, (int)cache->n_kv_heads,
          Divisor(cache->n_kv_heads));
    };
    // runs of less than four tokens on average: a wave each
    if (n_rows < 4 * n_runs)
      launch(append8_kernel<decltype(dt)::value, decltype(d)::value, kAppend8Few>, kAppend8Few);
    else
      launch(append8_kernel<decltype(dt)::value, decltype(d)::value, kAppend8Threads>, kAppend8Threads);
  });
  return check_launch(who);
}

extern "C" int wq_kv8_evict(const wq_kv8_cache* cache, const float* mass, int64_t mass_tokens,
                            const int32_t* block_table, int64_t table_width, const int32_t* lens,
                            int64_t n_seqs, int64_t keep, int64_t recent,
                            const int32_t* free_pages, int64_t n_free, int32_t* new_table,
                            int32_t* new_lens, float* new_mass, int64_t new_tokens,
                            int32_t* taken, int32_t* kept, void* stream) {
  const char* who = "wq_kv8_evict";
  if (int e = kv8_check_cache(cache, who)) return e;
  if (n_seqs > WQ_KV4_MAX_SEQS)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: at most %d sequences", who, WQ_KV4_MAX_SEQS);
  if (n_seqs < 0 || table_width < 1 || table_width > (1 << 24) || mass_tokens < 1 ||
      mass_tokens > (1 << 30) || keep < 1 || keep > (1 << 30) || keep > 64 * table_width ||
      recent < 0 || recent > keep || n_free < 0 || n_free > (1 << 25) || new_tokens < keep ||
      new_tokens > (1 << 30))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: bad sizes", who);
  const int64_t pages = (keep + WQ_KV4_PAGE - 1) / WQ_KV4_PAGE, pairs = n_seqs * cache->n_kv_heads;
  if (pairs * pages > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many pages", who);
  if (!taken) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned4(taken)) return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (n_seqs && (!mass || !block_table || !lens || !new_table || !new_lens || !new_mass || !kept ||
                 (n_free && !free_pages)))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (!aligned4(mass) || !aligned4(block_table) || !aligned4(lens) || !aligned4(free_pages) ||
      !aligned4(new_table) || !aligned4(new_lens) || !aligned4(new_mass) || !aligned4(kept))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (n_seqs == 0) {
    none_taken_kernel<<<dim3(1), 1, 0, (hipStream_t)stream>>>(taken);
    return check_launch(who);
  }
  if (new_table == block_table || new_mass == mass || new_lens == lens)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: the new table, lengths and masses need memory of their own", who);
  Evict8Args p{};
  p.table = block_table;
  p.lens = lens;
  p.free_pages = free_pages;
  p.width = table_width;
  p.mass_tokens = mass_tokens;
  p.new_tokens = new_tokens;
  p.mass = mass;
  p.new_table = new_table;
  p.new_lens = new_lens;
  p.taken = taken;
  p.kept = kept;
  p.new_mass = new_mass;
  p.seqs = (int)n_seqs;
  p.heads = (int)cache->n_kv_heads;
  p.keep = (int)keep;
  p.recent = (int)recent;
  p.n_free = (int)n_free;
  p.pages = (int)pages;
  p.heads_by = Divisor(cache->n_kv_heads);
  const dim3 picks((unsigned)(n_seqs + pairs));
  const int64_t most = 64 * table_width;
  if (most <= kPick8Few * kPick8Threads)
    pick8_kernel<kPick8Short><<<picks, kPick8Threads, 0, (hipStream_t)stream>>>(p);
  else if (most <= kPick8Held * kPick8Threads)
    pick8_kernel<kPick8Keys><<<picks, kPick8Threads, 0, (hipStream_t)stream>>>(p);
  else
    pick8_kernel<kPick8Long><<<picks, kPick8Threads, 0, (hipStream_t)stream>>>(p);
  uint8_t* const exps = reinterpret_cast<uint8_t*>(cache->exponents);
  const dim3 grid((unsigned)(pairs * pages));
  const Divisor pairs_by(pairs);
  if (cache->head_dim == 64)
    move8_kernel<64><<<grid, kMove8Threads, 0, (hipStream_t)stream>>>(p, pairs_by, cache->data, exps, cache->n_pages);
  else if (cache->head_dim == 128)
    move8_kernel<128><<<grid, kMove8Threads, 0, (hipStream_t)stream>>>(p, pairs_by, cache->data, exps, cache->n_pages);
  else
    move8_kernel<256><<<grid, kMove8Threads, 0, (hipStream_t)stream>>>(p, pairs_by, cache->data, exps, cache->n_pages);
  return check_launch(who);
}
