// Attention over the paged 4-bit key/value cache (wq.h, "4-bit key/value
// cache").

#include "wq_common.cuh"
#include "wq_device.h"
#include "wq_kv4.cuh"

namespace wqd {

constexpr int kAttnThreads = 256;

// One workgroup per (row, head): 256 tokens at a time, a thread's logit each,
// then a thread's channel each over those tokens.
template <int DT, int D>
__global__ void __launch_bounds__(kAttnThreads)
attn_kernel(KvRows a, const uint8_t* __restrict__ data, int64_t n_pages, int kv_heads, float scale,
            int window, const int32_t* __restrict__ sel, int n_sel, uint16_t* __restrict__ out,
            float* __restrict__ lse) {
  constexpr int G = D / 32, W = G < 4 ? G : 4;
  __shared__ float s_q[D], s_p[kAttnThreads], s_red[kAttnThreads];
  __shared__ int64_t s_page[kAttnThreads / 64];
  const int row = blockIdx.x / a.heads, h = blockIdx.x % a.heads;
  const int kvh = h / (a.heads / kv_heads), tid = threadIdx.x;
  const SeqRow sr = find_row(a, row);
  if (row >= a.cu[sr.b + 1]) return;
  for (int d = tid; d < D; d += kAttnThreads)
    s_q[d] = to_float<DT>(a.q[row * a.q_row + h * a.q_head + d]);
  const int first = window > 0 ? max(sr.pos - window + 1, 0) : 0;
  const int pages = (int)min((int64_t)((sr.pos + 64) / 64), a.width);
  const int n = sel != nullptr ? n_sel : pages;
  const int32_t* pick =
      sel != nullptr ? sel + ((int64_t)row * kv_heads + kvh) * n_sel : nullptr;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int j0 = 0; j0 < n; j0 += 4) {
    __syncthreads();
    const int j = j0 + tid / 64;
    const int p = j < n ? (pick != nullptr ? pick[j] : j) : -1;
    const int page = p >= 0 && p < pages ? a.table[sr.b * a.width + p] : -1;
    const bool ok = page >= 0 && page < n_pages;
    const int t = p * 64 + (tid & 63);
    if ((tid & 63) == 0) s_page[tid / 64] = ok ? page : -1;
    float x = -INFINITY;
    if (ok && t <= sr.pos && t >= first) {
      const int tt = t & 31, u = tt >> 4, r = (tt >> 2) & 3, e = 4 * u + (tt & 3);
      const uint8_t* tile = data + ((int64_t)page * kv_heads + kvh) * (80 * D) + ((t >> 5) & 1) * (40 * D);
      const uint16_t* meta = reinterpret_cast<const uint16_t*>(tile + 32 * D);
      x = 0.f;
      for (int g = 0; g < G; ++g) {
        float dot = 0.f, sum = 0.f;
        for (int c = 0; c < 4; ++c) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(
              tile + u * (8 * D) + (g / W) * (256 * W) + ((c * 16 + (tt & 15)) * W + g % W) * 4);
          for (int i = 0; i < 8; ++i) {
            const float q = s_q[g * 32 + c * 8 + i];
            dot += q * (float)((w >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15u);
            sum += q;
          }
        }
        x += h2f(meta[r * 8 * G + g * 8 + e]) * dot + h2f(meta[D + tt * G + g]) * sum;
      }
      x *= scale;
    }
    s_red[tid] = x != x ? INFINITY : x;   // a NaN logit makes its row NaN
    __syncthreads();
    for (int w = kAttnThreads / 2; w > 0; w >>= 1) {
      if (tid < w) s_red[tid] = fmaxf(s_red[tid], s_red[tid + w]);
      __syncthreads();
    }
    const float m_new = fmaxf(m, s_red[0]);
    if (m_new == -INFINITY) continue;   // the same for every thread
    s_p[tid] = __expf(x - m_new);
    __syncthreads();
    const float f = __expf(m - m_new);
    m = m_new;
    l *= f;
    o *= f;
    for (int i = 0; i < kAttnThreads; ++i) {
      const float pv = s_p[i];
      if (pv == 0.f) continue;
      l += pv;
      if (tid < D) {
        const int tt = i & 31, u = tt >> 4, r = (tt >> 2) & 3, e = 4 * u + (tt & 3), d = tid;
        const uint8_t* tile = data + (s_page[i / 64] * kv_heads + kvh) * (80 * D) + ((i >> 5) & 1) * (40 * D);
        const uint16_t* meta = reinterpret_cast<const uint16_t*>(tile + 36 * D);
        const uint32_t w = *reinterpret_cast<const uint32_t*>(
            tile + 16 * D + (d >> 6) * 1024 + (r * 16 + (d & 15)) * 16 + ((d >> 4) & 3) * 4);
        const int at = r * 8 * G + (d / 32) * 8 + e;
        o += pv * (h2f(meta[at]) * (float)((w >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u) + h2f(meta[D + at]));
      }
    }
  }
  if (tid < D) out[((int64_t)row * a.heads + h) * D + tid] = from_float<DT>(l == 0.f ? 0.f : o / l);
  if (tid == 0 && lse != nullptr)
    lse[(int64_t)row * a.heads + h] = l == 0.f ? -INFINITY : m + __logf(l);
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
  return 0;
}

extern "C" int wq_kv4_attention(const wq_kv4_cache* cache, const wq_kv4_rows* rows,
                                int64_t max_rows, int64_t max_len, float scale, int64_t window,
                                const int32_t* sel, int64_t n_sel, uint16_t* out, float* lse,
                                void* workspace, int64_t workspace_bytes, void* stream) {
  const char* who = "wq_kv4_attention";
  if (int e = check_attention(cache, rows, max_rows, max_len, n_sel, who)) return e;
  if (window < 0) return wq::fail(WQ_ERR_INVALID_ARG, "%s: window must be at least 0", who);
  if (rows->n_rows == 0 || rows->n_seqs == 0) return wq::ok();
  const int64_t need = wq_kv4_attention_workspace(cache, rows, max_rows, max_len, n_sel);
  if (!out || (need && !workspace)) return wq::fail(WQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
  if (workspace_bytes < need)
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: workspace of %lld bytes, %lld needed", who,
                    (long long)workspace_bytes, (long long)need);
  if (!aligned16(out) || !aligned4(lse) || !aligned4(sel) || !aligned16(workspace))
    return wq::fail(WQ_ERR_INVALID_ARG, "%s: misaligned device pointer", who);
  if (rows->n_rows * rows->n_heads > 0x7FFFFFFFll)
    return wq::fail(WQ_ERR_UNSUPPORTED, "%s: too many rows", who);
  const KvRows a = kv4_rows(rows);
  const int win = window > 0x40000000 ? 0 : (int)window;
  kv4_dispatch(rows->dtype, cache->head_dim, [&](auto dt, auto d) {
    attn_kernel<decltype(dt)::value, decltype(d)::value>
        <<<dim3((unsigned)(rows->n_rows * rows->n_heads)), kAttnThreads, 0, (hipStream_t)stream>>>(
            a, cache->data, cache->n_pages, (int)cache->n_kv_heads, scale, win, sel, (int)n_sel,
            out, lse);
  });
  return check_launch(who);
}
