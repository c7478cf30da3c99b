// Attention of a step's new tokens over the paged cache.
//
// One warp per (token, query head): every lane holds D / 32 of the query, a
// key's logit is one warp-wide sum, and the softmax runs with a running
// maximum and sum (one pass over the keys).
#include "seq_batch.cuh"

namespace qz {
namespace {

__device__ int g_attn_error = 0;

constexpr int kWarps = 4;

struct AttnParams {
  const __half *q;
  __half *out;
  int64_t q_token, q_head, o_token, o_head;
  int hq;
  float scale, softcap;
  int64_t window;
  PagedView c;
  SeqView s;
};

template <int D>
__global__ void __launch_bounds__(32 * kWarps) attn_warp_kernel(const AttnParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t t = blockIdx.x;
  const int g = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int seq = seq_of_token(p.s, t);
  if (seq < 0 || g >= p.hq) return;
  const int64_t kv = __ldg(p.s.kv_len + seq);
  const int64_t pos = kv - __ldg(p.s.cu_q + seq + 1) + t;
  const int h = g / (p.hq / p.c.hkv);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __half2float(p.q[t * p.q_token + g * p.q_head + lane + 32 * e]) * p.scale;
    o[e] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  const int64_t lo = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
  for (int64_t j = lo; j <= pos && j < kv; ++j) {
    const int64_t pi = j >> p.c.page_shift;
    const int page = pi < p.s.ld_table ? __ldg(p.s.table + seq * p.s.ld_table + pi) : -1;
    const bool ok = page >= 0 && page < p.c.n_pages;
    if (!ok && lane == 0) atomicOr(&g_attn_error, 4);
    const int64_t slot = j & (p.c.page_size - 1);
    float x = 0.0f, v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float k = ok ? __half2float(p.c.k[page * p.c.k_page + h * p.c.k_head +
                                              slot * p.c.k_token + lane + 32 * e])
                         : 0.0f;
      v[e] = ok ? __half2float(p.c.v[page * p.c.v_page + h * p.c.v_head + slot * p.c.v_token +
                                     lane + 32 * e])
                : 0.0f;
      x = fmaf(q[e], k, x);
    }
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    if (p.softcap > 0.0f) x = p.softcap * tanhf(x / p.softcap);
    const float mn = fmaxf(m, x), c = expf(m - mn), w = expf(x - mn);
    l = l * c + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * c + w * v[e];
    m = mn;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.out[t * p.o_token + g * p.o_head + lane + 32 * e] = __float2half_rn(o[e] * inv);
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

qz_status launch_attention(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                           const PagedView &c, const SeqView &sv, float scale, float softcap,
                           int64_t window, __half *out, int64_t o_token, int64_t o_head, void *,
                           cudaStream_t s) {
  const AttnParams p = {q,     out,     q_token, q_head, o_token, o_head, (int)hq,
                        scale, softcap, window,  c,      sv};
  const dim3 grid((unsigned)sv.n_tokens, (unsigned)((hq + kWarps - 1) / kWarps));
  if (c.D == 64)
    attn_warp_kernel<64><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (c.D == 128)
    attn_warp_kernel<128><<<grid, 32 * kWarps, 0, s>>>(p);
  else
    attn_warp_kernel<256><<<grid, 32 * kWarps, 0, s>>>(p);
  return launch_status();
}

qz_status read_attn_error(int *code, int clear) {
  return read_error_word(g_attn_error, code, clear);
}

}  // namespace qz
