// Rotary embedding of a step's new queries and keys and storage of its keys
// and values into the paged cache.
//
// Every value is read and written once; a thread takes the 8 + 8 values that
// rotate into one another (j.., j + D/2..) as two 16-byte loads and stores, or
// copies 16 of a value row.  A token's position and page come from one warp-wide
// search of the sequence boundaries (seq_of_token).  HBM bounds long steps, launch
// latency a decode step.  Measured (GB300): 1854 packed tokens, 64 heads, 8 KV
// heads of 128 14.8 us, 5.2 TB/s (78% of a plain copy's rate; the fp32 cosines are
// as many loads as the values, read from L2); 64 single tokens, 32 heads 2.9 us.
#include "seq_batch.cuh"

namespace qz {
namespace {

__device__ int g_rope_error = 0;

constexpr int kThreads = 128;

struct RopeParams {
  const __half *q, *k, *v;
  __half *qo;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, qo_token, qo_head;
  int hq;
  const float *rope;
  int64_t rope_len;
  PagedView c;
  SeqView s;
};

// Items of a token: (head, 8-column group of the first half), query heads
// first, then key heads, then value heads.  A thread takes U of them with the
// same columns, so it reads their cosines and sines once.
template <int U>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(const RopeParams p) {
  const int64_t t = blockIdx.x;
  const int seq = seq_of_token(p.s, t);
  if (seq < 0) return;
  const int end = __ldg(p.s.cu_q + seq + 1);
  const int64_t pos = (int64_t)__ldg(p.s.kv_len + seq) - end + t;
  bool ok = pos >= 0;
  int page = -1;
  if (ok) {
    const int64_t pi = pos >> p.c.page_shift;
    if (pi < p.s.ld_table) page = __ldg(p.s.table + seq * p.s.ld_table + pi);
    ok = page >= 0 && page < p.c.n_pages && (!p.rope || pos < p.rope_len);
    if (!ok && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_rope_error, 4);
  }
  const int half = p.c.D / 2, shift = 31 - __clz(half / 8);  // 4, 8 or 16 groups
  const int slot = (int)(pos & (p.c.page_size - 1));
  const int hq = p.qo ? p.hq : 0, heads = hq + 2 * p.c.hkv;
  const int j = (threadIdx.x & ((1 << shift) - 1)) * 8;
  const int step = kThreads >> shift;  // heads a CTA takes at once
  const int first = (int)blockIdx.y * U * step + (threadIdx.x >> shift);
  uint4 a[U], b[U];
  __half *dst[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    int head = first + i * step;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    dst[i] = nullptr;
    const __half *src;
    if (head < hq) {
      src = p.q + t * p.q_token + head * p.q_head;
      dst[i] = p.qo + t * p.qo_token + head * p.qo_head + j;
    } else if (ok && head < heads) {
      head -= hq;
      if (head < p.c.hkv) {
        src = p.k + t * p.k_token + head * p.k_head;
        dst[i] = p.c.k + page * p.c.k_page + head * p.c.k_head + slot * p.c.k_token + j;
      } else {
        head -= p.c.hkv;
        src = p.v + t * p.v_token + head * p.v_head;
        dst[i] = p.c.v + page * p.c.v_page + head * p.c.v_head + slot * p.c.v_token + j;
      }
    }
    if (ok && dst[i]) {
      a[i] = *reinterpret_cast<const uint4 *>(src + j);
      b[i] = *reinterpret_cast<const uint4 *>(src + j + half);
    }
  }
  const bool rotate = ok && p.rope;
  float c[8], s[8];
  if (rotate) {
    const float4 *cs = reinterpret_cast<const float4 *>(p.rope + pos * p.c.D + j);
    const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);
    const float4 s0 = __ldg(cs + half / 4), s1 = __ldg(cs + half / 4 + 1);
    c[0] = c0.x, c[1] = c0.y, c[2] = c0.z, c[3] = c0.w;
    c[4] = c1.x, c[5] = c1.y, c[6] = c1.z, c[7] = c1.w;
    s[0] = s0.x, s[1] = s0.y, s[2] = s0.z, s[3] = s0.w;
    s[4] = s1.x, s[5] = s1.y, s[6] = s1.z, s[7] = s1.w;
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    if (rotate && first + i * step < hq + p.c.hkv) {
      uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 u = h2f(av[k]), w = h2f(bv[k]);
        av[k] = f2h(u.x * c[2 * k] - w.x * s[2 * k], u.y * c[2 * k + 1] - w.y * s[2 * k + 1]);
        bv[k] = f2h(w.x * c[2 * k] + u.x * s[2 * k], w.y * c[2 * k + 1] + u.y * s[2 * k + 1]);
      }
      a[i] = make_uint4(av[0], av[1], av[2], av[3]);
      b[i] = make_uint4(bv[0], bv[1], bv[2], bv[3]);
    }
    if (dst[i]) {
      *reinterpret_cast<uint4 *>(dst[i]) = a[i];
      *reinterpret_cast<uint4 *>(dst[i] + half) = b[i];
    }
  }
}

template <int U>
qz_status launch(const RopeParams &p, int items, cudaStream_t s) {
  const int per = kThreads * U;
  const dim3 grid((unsigned)p.s.n_tokens, (unsigned)((items + per - 1) / per));
  rope_append_kernel<U><<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

}  // namespace

qz_status launch_rope_append(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                             const __half *k, int64_t k_token, int64_t k_head, const __half *v,
                             int64_t v_token, int64_t v_head, const float *rope, int64_t rope_len,
                             const PagedView &c, const SeqView &sv, __half *qo, int64_t qo_token,
                             int64_t qo_head, cudaStream_t s) {
  RopeParams p = {q,      k,      v,      qo,      q_token, q_head, k_token, k_head, v_token,
                  v_head, qo_token, qo_head, (int)hq, rope,    rope_len, c,     sv};
  const int items = ((qo ? (int)hq : 0) + 2 * c.hkv) * (c.D / 16);
  DeviceInfo di;
  const qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  // One item a thread while the GPU holds all CTAs of the call at once (64 tokens,
  // 32 heads: 2.9 us, three items 3.15), three once it does not (1854 tokens: 14.9
  // us with one, 14.6 with two or five, 14.5 with three).
  const int64_t ctas = sv.n_tokens * ((items + kThreads - 1) / kThreads);
  return ctas > (int64_t)di.sms * 16 ? launch<3>(p, items, s) : launch<1>(p, items, s);
}

qz_status read_rope_error(int *code, int clear) {
  return read_error_word(g_rope_error, code, clear);
}

}  // namespace qz
