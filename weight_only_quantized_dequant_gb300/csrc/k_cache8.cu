// A step's new keys and values into a paged cache of INT8 rows, and rows of
// such a cache back as fp16.
//
// A row (one token and KV head) is D codes and one fp32 scale, by the rule of the
// quantizer: scale = max|y| / 127, code = rint(y / scale), with y the value or the
// rotated key in fp32.  Codes that are decided by a rounding have to be the same
// wherever they are computed, so the rotation is rounded once (its two products
// and their sum carry their errors along) and the divisions are IEEE's.
//
// Append: a thread takes the 8 + 8 values that rotate into one another, as in the
// fp16 append; the D / 16 threads of a row share its largest value by shuffles.
// Longer steps take three items a thread, and warps of queries leave before the rows' part:
// 1854 tokens, 64 heads on 8, D 128, 18.9 us, 3.9 TB/s (with the 3600 rows that their
// sequences hold read back 24.3; with two items 25.3, with one 27.2, and 30.3 when queries
// went through the rows' part).  What is left over HBM's 10.8 us is latency: the place is
// looked up, then loads, divisions and shuffles, one chain.  64 tokens, 32 heads: 4.3 us, the
// launch's.
// Read: 16 codes a thread, one 16-byte load and two 16-byte stores; a CTA takes 8 tokens,
// whose sequences and pages its first threads look up at once.  8 sequences of up to 16384
// tokens, 8 heads of 128: 95 us, 5.6 TB/s, HBM's; 199 tokens 4.5 us, the launch's.
#include "seq_batch.cuh"

namespace qz {
namespace {

__device__ int g_cache8_error = 0;

constexpr int kThreads = 128;

struct AppendParams {
  const __half *q, *k, *v;
  __half *qo;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head, qo_token, qo_head;
  int hq;
  const float *rope;
  int64_t rope_len;
  PagedInt8View c;
  SeqView s;
};

// a c - b s rounded to fp32: the products' errors by FMA, the difference's exactly
// (Knuth's two-sum); what is left of the error is below 2^-46 of the larger product.  (The
// products by intrinsics: joined with a sum, a product's error would be in it twice.)
__device__ __forceinline__ float rotated(float a, float c, float b, float s) {
  const float h = __fmul_rn(a, c), g = __fmul_rn(-b, s);
  const float eh = fmaf(a, c, -h), eg = fmaf(-b, s, -g);
  const float sum = h + g, t = sum - h;
  const float e = (h - (sum - t)) + (g - t);
  return sum + (e + (eh + eg));
}

// Eight codes of the scale s (0 or not finite: zeros) as 8 bytes.
__device__ __forceinline__ uint2 codes(const float *y, float s) {
  uint32_t w[2] = {0, 0};
  if (s > 0.0f && s < INFINITY) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = fminf(fmaxf(rintf(__fdiv_rn(y[i], s)), -127.0f), 127.0f);
      w[i >> 2] |= (uint32_t)((int)r & 255) << (8 * (i & 3));
    }
  }
  return make_uint2(w[0], w[1]);
}

// Items of a token: (head, 8-column group of the first half), query heads
// first, then key heads, then value heads.  A thread takes U of them with the
// same columns, so it reads their cosines and sines once.
template <int U>
__global__ void __launch_bounds__(kThreads) append_int8_kernel(const AppendParams p) {
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
    if (!ok && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(&g_cache8_error, 4);
  }
  const int half = p.c.D / 2, shift = 31 - __clz(half / 8);  // 4, 8 or 16 groups
  const int slot = (int)(pos & (p.c.page_size - 1));
  const int hq = p.qo ? p.hq : 0, heads = hq + 2 * p.c.hkv;
  const int j = (threadIdx.x & ((1 << shift) - 1)) * 8;
  const int step = kThreads >> shift;  // heads a CTA takes at once
  const int first = (int)blockIdx.y * U * step + (threadIdx.x >> shift);
  uint4 a[U], b[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    int head = first + i * step;
    a[i] = b[i] = make_uint4(0, 0, 0, 0);
    if (!ok || head >= heads) continue;
    const __half *src;
    if (head < hq)
      src = p.q + t * p.q_token + head * p.q_head;
    else if ((head -= hq) < p.c.hkv)
      src = p.k + t * p.k_token + head * p.k_head;
    else
      src = p.v + t * p.v_token + (head - p.c.hkv) * p.v_head;
    a[i] = *reinterpret_cast<const uint4 *>(src + j);
    b[i] = *reinterpret_cast<const uint4 *>(src + j + half);
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
    const int head = first + i * step;
    const uint32_t av[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t bv[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
    if (head < hq) {  // a query: fp16, as in the fp16 append
      uint32_t x[4], y[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 u = h2f(av[k]), w = h2f(bv[k]);
        x[k] = rotate ? f2h(u.x * c[2 * k] - w.x * s[2 * k],
                            u.y * c[2 * k + 1] - w.y * s[2 * k + 1])
                      : av[k];
        y[k] = rotate ? f2h(w.x * c[2 * k] + u.x * s[2 * k],
                            w.y * c[2 * k + 1] + u.y * s[2 * k + 1])
                      : bv[k];
      }
      __half *dst = p.qo + t * p.qo_token + head * p.qo_head + j;
      *reinterpret_cast<uint4 *>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<uint4 *>(dst + half) = make_uint4(y[0], y[1], y[2], y[3]);
    }
    // (whole warps from here on: a row's threads share its largest value)
    const bool key = head < hq + p.c.hkv;
    float x[8], y[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 u = h2f(av[k]), w = h2f(bv[k]);
      x[2 * k] = u.x, x[2 * k + 1] = u.y, y[2 * k] = w.x, y[2 * k + 1] = w.y;
    }
    if (rotate && key && head >= hq) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float u = x[k], w = y[k];
        x[k] = rotated(u, c[k], w, s[k]);
        y[k] = rotated(w, c[k], -u, s[k]);
      }
    }
    if (!__any_sync(0xffffffffu, ok && head >= hq && head < heads)) continue;  // queries
    uint32_t mx = 0;  // magnitudes' bits: a NaN is larger than any value
#pragma unroll
    for (int k = 0; k < 8; ++k)
      mx = max(mx, max(__float_as_uint(x[k]) & 0x7fffffffu, __float_as_uint(y[k]) & 0x7fffffffu));
    for (int o = 1; o < (1 << shift); o <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (!ok || head < hq || head >= heads) continue;
    const float scale = __fdiv_rn(__uint_as_float(mx), 127.0f);
    int8_t *row;
    float *at;
    if (key) {
      const int h = head - hq;
      row = p.c.k + page * p.c.k_page + h * p.c.k_head + slot * p.c.k_token;
      at = p.c.ks + page * p.c.ks_page + h * p.c.ks_head + slot * p.c.ks_token;
    } else {
      const int h = head - hq - p.c.hkv;
      row = p.c.v + page * p.c.v_page + h * p.c.v_head + slot * p.c.v_token;
      at = p.c.vs + page * p.c.vs_page + h * p.c.vs_head + slot * p.c.vs_token;
    }
    *reinterpret_cast<uint2 *>(row + j) = codes(x, scale);
    *reinterpret_cast<uint2 *>(row + j + half) = codes(y, scale);
    if (j == 0) *at = scale;
  }
}

template <int U>
qz_status launch(const AppendParams &p, int items, cudaStream_t s) {
  const int per = kThreads * U;
  const dim3 grid((unsigned)p.s.n_tokens, (unsigned)((items + per - 1) / per));
  append_int8_kernel<U><<<grid, kThreads, 0, s>>>(p);
  return launch_status();
}

// ------------------------------------------------------------------- read --
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 8;  // of a CTA

struct ReadParams {
  PagedInt8View c;
  SeqView s;
  __half *k, *v;
  int64_t k_token, k_head, v_token, v_head;
};

// The last sequence whose first row is not after t, or -1 where t is in none.
__device__ __forceinline__ int seq_of_lane(const SeqView &s, int64_t t) {
  int lo = 0, hi = s.n_seqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if ((int64_t)__ldg(s.cu_q + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  return (int64_t)__ldg(s.cu_q + lo) <= t && t < (int64_t)__ldg(s.cu_q + lo + 1) ? lo : -1;
}

__device__ __forceinline__ uint32_t two_codes(uint32_t w, int at, float s) {
  const float a = (float)(int8_t)(w >> at) * s, b = (float)(int8_t)(w >> (at + 8)) * s;
  return f2h(a, b);
}

__global__ void __launch_bounds__(kReadThreads) read_int8_kernel(const ReadParams p) {
  __shared__ int place[kReadTokens][2];  // page (-1: zeros; -2: not written) and slot
  const int64_t t0 = (int64_t)blockIdx.x * kReadTokens;
  if (threadIdx.x < kReadTokens) {
    const int64_t t = t0 + threadIdx.x;
    int page = -2, slot = 0;
    const int seq = t < p.s.n_tokens ? seq_of_lane(p.s, t) : -1;
    if (seq >= 0) {
      const int end = __ldg(p.s.cu_q + seq + 1);
      const int64_t pos = (int64_t)__ldg(p.s.kv_len + seq) - end + t;
      page = -1;
      if (pos >= 0) {
        const int64_t pi = pos >> p.c.page_shift;
        if (pi < p.s.ld_table) page = __ldg(p.s.table + seq * p.s.ld_table + pi);
        if (page < 0 || page >= p.c.n_pages) {
          page = -1;
          if (blockIdx.y == 0) atomicOr(&g_cache8_error, 4);
        }
        slot = (int)(pos & (p.c.page_size - 1));
      }
    }
    place[threadIdx.x][0] = page;
    place[threadIdx.x][1] = slot;
  }
  __syncthreads();
  // items: (token, keys or values, head, 16 codes)
  const int shift = 31 - __clz(p.c.D / 16), per = 2 * p.c.hkv << shift;
  const int items = kReadTokens * per;
  const int stride = gridDim.y * kReadThreads;
  for (int i = blockIdx.y * kReadThreads + threadIdx.x; i < items; i += stride) {
    const int tok = i / per, rest = i - tok * per;
    const int j = (rest & ((1 << shift) - 1)) * 16;
    int head = rest >> shift;
    const bool key = head < p.c.hkv;
    if (!key) head -= p.c.hkv;
    const int64_t page = place[tok][0];
    const int slot = place[tok][1];
    if (page == -2) continue;
    uint4 w = make_uint4(0, 0, 0, 0);
    float s = 0.0f;
    if (page >= 0) {
      const int8_t *row = key ? p.c.k + page * p.c.k_page + head * p.c.k_head + slot * p.c.k_token
                              : p.c.v + page * p.c.v_page + head * p.c.v_head + slot * p.c.v_token;
      w = __ldcs(reinterpret_cast<const uint4 *>(row + j));
      s = __ldg(key ? p.c.ks + page * p.c.ks_page + head * p.c.ks_head + slot * p.c.ks_token
                    : p.c.vs + page * p.c.vs_page + head * p.c.vs_head + slot * p.c.vs_token);
    }
    __half *dst = (key ? p.k + (t0 + tok) * p.k_token + head * p.k_head
                       : p.v + (t0 + tok) * p.v_token + head * p.v_head) + j;
    __stcs(reinterpret_cast<uint4 *>(dst),
           make_uint4(two_codes(w.x, 0, s), two_codes(w.x, 16, s), two_codes(w.y, 0, s),
                      two_codes(w.y, 16, s)));
    __stcs(reinterpret_cast<uint4 *>(dst) + 1,
           make_uint4(two_codes(w.z, 0, s), two_codes(w.z, 16, s), two_codes(w.w, 0, s),
                      two_codes(w.w, 16, s)));
  }
}

}  // namespace

qz_status launch_rope_append_int8(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                                  const __half *k, int64_t k_token, int64_t k_head,
                                  const __half *v, int64_t v_token, int64_t v_head,
                                  const float *rope, int64_t rope_len, const PagedInt8View &c,
                                  const SeqView &sv, __half *qo, int64_t qo_token,
                                  int64_t qo_head, cudaStream_t s) {
  AppendParams p = {q,      k,      v,        qo,      q_token, q_head,   k_token, k_head, v_token,
                    v_head, qo_token, qo_head, (int)hq, rope,    rope_len, c,       sv};
  const int items = ((qo ? (int)hq : 0) + 2 * c.hkv) * (c.D / 16);
  DeviceInfo di;
  const qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  const int64_t ctas = sv.n_tokens * ((items + kThreads - 1) / kThreads);
  return ctas > (int64_t)di.sms * 16 ? launch<3>(p, items, s) : launch<1>(p, items, s);
}

qz_status launch_cache_read_int8(const PagedInt8View &c, const SeqView &sv, __half *k,
                                 int64_t k_token, int64_t k_head, __half *v, int64_t v_token,
                                 int64_t v_head, cudaStream_t s) {
  ReadParams p = {c, sv, k, v, k_token, k_head, v_token, v_head};
  const int64_t tiles = (sv.n_tokens + kReadTokens - 1) / kReadTokens;
  const int64_t items = (int64_t)kReadTokens * 2 * c.hkv * (c.D / 16);
  const int64_t y = (items + kReadThreads * 4 - 1) / (kReadThreads * 4);
  const dim3 grid((unsigned)tiles, (unsigned)(y < 65535 ? y : 65535));
  read_int8_kernel<<<grid, kReadThreads, 0, s>>>(p);
  return launch_status();
}

qz_status read_cache8_error(int *code, int clear) {
  return read_error_word(g_cache8_error, code, clear);
}

}  // namespace qz
