// Rotary embedding of a step's new queries and keys and storage of its keys
// and values into the paged cache.
//
// Every value is read and written once; a thread takes the 8 + 8 values that
// rotate into one another (j.., j + D/2..) as two 16-byte loads and stores, or
// copies 16 of a value row.  HBM bounds long steps, launch latency a decode
// step.  A token's position and page come from one warp-wide search of the
// sequence boundaries (seq_of_token).  One item a thread: 2, 4 or 8 in flight
// per thread took as long or longer.  Measured
// (GB300): 1854 packed tokens, 64 heads, 8 KV heads of 128 15.6 us, 4.9 TB/s; 64
// single tokens, 32 heads 3.4 us.
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

__device__ __forceinline__ float2 h2f(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
__device__ __forceinline__ uint32_t f2h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Items of a token: (head, 8-column group of the first half), query heads
// first, then key heads, then value heads.
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
  const int half = p.c.D / 2, groups = half / 8;
  const int slot = (int)(pos & (p.c.page_size - 1));
  const int items = ((p.qo ? p.hq : 0) + 2 * p.c.hkv) * groups;
  for (int it = blockIdx.y * kThreads + threadIdx.x; it < items; it += gridDim.y * kThreads) {
    int head = it / groups;
    const int j = (it - head * groups) * 8;
    const __half *src;
    __half *dst;
    bool rotate = p.rope != nullptr;
    if (p.qo && head < p.hq) {
      src = p.q + t * p.q_token + head * p.q_head;
      dst = p.qo + t * p.qo_token + head * p.qo_head;
    } else {
      if (!ok) continue;
      head -= p.qo ? p.hq : 0;
      if (head < p.c.hkv) {
        src = p.k + t * p.k_token + head * p.k_head;
        dst = p.c.k + page * p.c.k_page + head * p.c.k_head + slot * p.c.k_token;
      } else {
        head -= p.c.hkv;
        src = p.v + t * p.v_token + head * p.v_head;
        dst = p.c.v + page * p.c.v_page + head * p.c.v_head + slot * p.c.v_token;
        rotate = false;
      }
    }
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (ok) {
      a = *reinterpret_cast<const uint4 *>(src + j);
      b = *reinterpret_cast<const uint4 *>(src + j + half);
    }
    if (ok && rotate) {
      const float4 *cs = reinterpret_cast<const float4 *>(p.rope + pos * p.c.D + j);
      const float4 c0 = __ldg(cs), c1 = __ldg(cs + 1);
      const float4 s0 = __ldg(cs + half / 4), s1 = __ldg(cs + half / 4 + 1);
      const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
      const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
      uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 u = h2f(av[i]), w = h2f(bv[i]);
        av[i] = f2h(u.x * c[2 * i] - w.x * s[2 * i], u.y * c[2 * i + 1] - w.y * s[2 * i + 1]);
        bv[i] = f2h(w.x * c[2 * i] + u.x * s[2 * i], w.y * c[2 * i + 1] + u.y * s[2 * i + 1]);
      }
      a = make_uint4(av[0], av[1], av[2], av[3]);
      b = make_uint4(bv[0], bv[1], bv[2], bv[3]);
    }
    *reinterpret_cast<uint4 *>(dst + j) = a;
    *reinterpret_cast<uint4 *>(dst + j + half) = b;
  }
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
  const dim3 grid((unsigned)sv.n_tokens, (unsigned)((items + kThreads - 1) / kThreads));
  rope_append_kernel<<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

qz_status read_rope_error(int *code, int clear) {
  return read_error_word(g_rope_error, code, clear);
}

}  // namespace qz
