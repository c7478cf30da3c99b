// Choice of a step's next tokens: temperature, top-k, top-p and min-p over rows
// of logits, and one token a row from one uniform random number.
//
// With m the row's largest logit, w_i = e^{(x_i - m) / T}.  Each filter keeps the
// first so many tokens in the order (value descending, index ascending), so the
// kept set is one prefix of that order: all tokens above a cut value and the
// lowest-indexed so many of those that equal it.  The token is the first, by
// index, at which the running sum of the kept weights passes u * total.
//
// Sums.  A border between two tokens moves with every rounding of every weight,
// and a vocabulary of 256000 lies within 1e-5 of a border at almost any u.  So
// weights are 64-bit integers, 2^45 at the largest logit (good to 2^-28, zero 46
// octaves below), and their sums are exact: neither the order of the atomics nor
// the split of a row shows in a result.  Weights come from fp32 pairs and integer
// products; through fp64 and conversions to integers, both slow here, 64 rows of
// 256000 took 147 us where the same passes took 112, and 16 rows of 128000 65 and 36.
//
// A row is a cluster of CTAs that keep their slices in shared memory: one read of
// HBM and one pass for the maximum.  Then
//  * top-k: the largest logits of groups of the row bound the k-th from below, and
//    the tokens above that bound (some more than k) go to the first CTA's list,
//    which it sorts and answers from;
//  * top-p of a whole row: a histogram of a quarter of the tokens (and of all groups'
//    largest), sixteenths of a logit wide, says about where the cut is; one pass sums
//    all weights and those above the bins around the cut, and lists the places of the
//    tokens in them, warp by warp; the lists are what the histogram by steps of the key
//    (the fp32 value's bits in their order), its refinement and the sums below the bins go
//    through, so the cut is exact whatever the estimate was (64 rows of 256000: 100 us with
//    a branch for those tokens in each pass, 84 with the lists); where few tokens may be
//    kept they are listed as for top-k;
//  * what the estimate misses (logits of 63 and more, lists that overflow, a cut
//    outside) takes the general way, histograms of 2048 steps of the key, refined
//    until a step is one value;
//  * the kept weights are summed warp by warp, and the warp that the answer is in goes
//    through its tokens again.
//
// What bounds it: with many rows the instructions (83 a logit in all, of which a weight is
// about 25; at full issue they would take 36 us of 84) and barriers, at which a cluster waits
// for its first CTA's scans of the bins; with few the chain of cluster barriers (about 1 us
// each).  Measured: 64 rows of 256000 fp16, top-p 0.95, 84 us, by the general way (a row
// whose largest logit is 63 or more) 274, equal logits 381; greedy 29, a temperature alone 49,
// top-k 50 32, top-k 4000 (more than a list holds) 99.  16 of 128000 fp32 with options of each
// row 30; one of 32000, top-k 50 and top-p 0.9, 12.
// Clusters of 8 with 64 KB slices leave some SMs without work; slices of 128 KB (one CTA an
// SM) took 150 us for 64 rows where these took 103, and 1024 threads a CTA 116.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "qz_internal.cuh"

namespace qz {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;       // tokens that a CTA can list
constexpr int kFew = 112;         // of a row, that are listed in any case (and sorted at once)
constexpr int kMine = kList * 8 / kWarps / 2;  // a warp's share of the list, as 16-bit places
constexpr int kMaxCluster = 8;
constexpr int kUnitBits = 45;     // the largest logit's weight is 2^45
constexpr int kSliceBytes = 64 << 10;  // two CTAs an SM
using u64 = unsigned long long;

struct SampleParams {
  const void *logits;
  int64_t ld;
  int V, slice;  // tokens of a row; of a CTA (a multiple of 16 bytes)
  int vec;       // rows may be read 16 bytes at a time
  const float *u;
  const float *temperature, *top_p, *min_p;  // of every row, or NULL: the values below
  const int32_t *top_k;
  float temperature_all, top_p_all, min_p_all;
  int32_t top_k_all;
  int32_t *token;
  float *logprob;
};

// --------------------------------------------------------------- clusters --
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// The address of this CTA's shared variable p in the CTA of the given rank.
template <typename T>
__device__ __forceinline__ uint32_t remote(const T *p, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(a)
      : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ uint32_t ld_remote32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ u64 ld_remote64(uint32_t a) {
  u64 v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_remote64(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
__device__ __forceinline__ void add_remote32(uint32_t a, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void add_remote64(uint32_t a, u64 v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// ------------------------------------------------------------------ values --
// Logits as fp32, NaN as -inf and -0 as 0 (the order of values is that of keys).
__device__ __forceinline__ float clean(float x) { return fmaxf(x, -INFINITY) + 0.0f; }

// Four logits at a time (more at once would not leave 64 registers a thread).
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  using Word = uint4;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__half> {
  using Word = uint2;
  static __device__ __forceinline__ void get(uint2 v, float (&x)[4]) {
    const float2 a = h2f(v.x), b = h2f(v.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
};
template <>
struct Vec<__nv_bfloat16> {
  using Word = uint2;
  static __device__ __forceinline__ void get(uint2 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  }
};
constexpr int N = 4;

// Larger values have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// What a row's tokens are weighed by.
struct Scale {
  float m;           // largest logit
  float c_hi, c_lo;  // log2(e) / T
  float far;         // 46 octaves
};

// 2^(-i/32), i < 32, in units of 2^-45.
__constant__ u64 kPower[32] = {
    35184372088832ull, 34430443548229ull, 33692670141585ull, 32970705697691ull, 32264211463077ull,
    31572855943056ull, 30896314746195ull, 30234270432094ull, 29586412362452ull, 28952436555301ull,
    28332045542385ull, 27724948229574ull, 27130859760289ull, 26549501381838ull, 25980600314626ull,
    25423889624159ull, 24879108095804ull, 24346000112214ull, 23824315533396ull, 23313809579344ull,
    22814242715178ull, 22325380538761ull, 21846993670708ull, 21378857646762ull, 20920752812471ull,
    20472464220127ull, 20033781527906ull, 19604498901178ull, 19184414915921ull, 18773332464219ull,
    18371058661769ull, 17977404757381ull,
};
// In shared memory, a bank each: 32-bit halves of it, less what kMagic adds in units of
// 2^17, and 2^28 times it.
struct Powers {
  uint32_t lo[32], hi[32];
  float flt[32];
};
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: a sum with it has whole numbers as low bits
constexpr uint32_t kMagicBits = 0x4b400000u;

// A number near 1 / (1 + (i + 1/2) / 32), and minus its logarithm in two parts.
__constant__ float kLog[32][3] = {
    {0.984615386f, 0.015504186f, -4.37010483e-10f},
    {0.955223858f, 0.0458095595f, -2.09700451e-10f},
    {0.927536249f, 0.0752234012f, 1.42228584e-09f},
    {0.901408434f, 0.10379681f, 2.39636733e-09f},
    {0.876712322f, 0.131576359f, 5.96729688e-09f},
    {0.853333354f, 0.158605009f, -3.35514616e-09f},
    {0.83116883f, 0.184922338f, 1.89329108e-09f},
    {0.810126603f, 0.210564747f, -3.49109541e-09f},
    {0.790123463f, 0.235566065f, -8.53199122e-10f},
    {0.771084309f, 0.259957552f, 9.73365299e-09f},
    {0.752941191f, 0.283768147f, 6.34272235e-09f},
    {0.735632181f, 0.307025045f, -6.13627682e-09f},
    {0.719101131f, 0.32975328f, -3.55805452e-09f},
    {0.703296721f, 0.351976395f, 3.35814865e-09f},
    {0.688172042f, 0.373716414f, -3.24985527e-09f},
    {0.673684239f, 0.394993752f, 1.31588971e-08f},
    {0.659793794f, 0.41582793f, -4.09624601e-09f},
    {0.646464646f, 0.436236769f, -1.25471211e-09f},
    {0.633663356f, 0.456237435f, 1.39731897e-08f},
    {0.621359229f, 0.475845903f, -7.60144925e-09f},
    {0.609523833f, 0.495077223f, 6.02794836e-09f},
    {0.598130822f, 0.513945758f, 2.44244589e-08f},
    {0.587155938f, 0.532464862f, -2.01595007e-08f},
    {0.576576591f, 0.55064708f, 1.37936649e-08f},
    {0.566371679f, 0.568504751f, -1.16506484e-08f},
    {0.556521714f, 0.58604908f, 1.07433662e-08f},
    {0.547008574f, 0.603290796f, 5.79808201e-09f},
    {0.537815154f, 0.620240331f, 2.78330106e-08f},
    {0.528925598f, 0.636907518f, -1.3763418e-08f},
    {0.520325184f, 0.653301299f, 1.06473328e-08f},
    {0.512000024f, 0.669430614f, -7.07258208e-09f},
    {0.503937006f, 0.685303986f, 2.07516688e-08f},
};
// minus ln(2^-t total / 2^45), t = t_hi + t_lo, to 2^-29 and rounded once: total = 2^e z,
// z kLog = 1 + r (|r| < 1/60, its logarithm by the series), and whatever rounding drops is
// carried along.
__device__ __forceinline__ float log_share(float t_hi, float t_lo, u64 total) {
  const int e = 63 - __clzll(total);
  const u64 m = total << (63 - e);  // z 2^63
  const float z = (float)(uint32_t)(m >> 40) * 0x1p-23f;
  const float y = (float)(uint32_t)(m >> 16 & 0xffffff) * 0x1p-47f;
  const int i = (int)(m >> 58) & 31;
  const float r = fmaf(y, kLog[i][0], fmaf(z, kLog[i][0], -1.0f));
  float s = fmaf(r, 0.2f, -0.25f);
  s = fmaf(r, s, 1.0f / 3.0f);
  s = fmaf(r, s, -0.5f);
  s = fmaf(r * r, s, r) + kLog[i][2];
  // 0.693145751953125 = 22713 / 2^15 is ln 2 to 15 bits: exact with e
  const float n = (float)(e - kUnitBits), a = n * 0.693145751953125f, b = kLog[i][1];
  s = fmaf(n, 1.42860677e-06f, s);
  const float ab = a + b, abv = ab - a;
  s += (a - (ab - abv)) + (b - abv);
  const float x = __fmul_rn(t_hi, 0.693147182f);  // (never joined with the sums)
  s += fmaf(t_hi, 0.693147182f, -x) + fmaf(t_hi, -1.90465421e-09f, t_lo * 0.693147182f);
  const float sum = ab + x, sv = sum - ab;
  return -(sum + (((ab - (sum - sv)) + (x - sv)) + s));
}

// 2^45 e^{(x - m)/T}, x <= m.  With t = (m - x) c as an fp32 pair, q = rint(32 t) and
// f = t - q/32: 2^-t = 2^-(q>>5) 2^-((q&31)/32) 2^-f, the last by its series to f^4 (|f| <=
// 1/64: the next term is below 2^-39).  What the shift drops is taken as half a unit (the
// last bit is set), so that it does not add up; 46 octaves below m nothing is left.
// EXACT: m - x loses nothing that matters (16-bit logits).
template <bool EXACT>
__device__ __forceinline__ u64 weight(const Scale &s, const Powers &pw, float x) {
  const float d = fminf(s.m - x, s.far);
  const float t = d * s.c_hi;
  float lo = fmaf(d, s.c_lo, fmaf(d, s.c_hi, -t));
  if (!EXACT) {
    const float xv = s.m - d;
    const float e = (s.m - (d + xv)) + (xv - x);
    lo = d < s.far ? fmaf(e, s.c_hi, lo) : 0.0f;
  }
  const float qf = fmaf(t, 32.0f, kMagic);
  const uint32_t qb = __float_as_uint(qf), i = qb & 31;
  const float f = fmaf(qf - kMagic, -0.03125f, t) + lo;
  // 2^-f - 1: powers of ln 2 over factorials
  float p = fmaf(f, 9.6181291e-3f, -5.5504109e-2f);
  p = fmaf(f, p, 2.4022651e-1f);
  p = fmaf(f, p, -6.9314718e-1f) * f;
  const uint32_t z = __float_as_uint(fmaf(p, pw.flt[i], kMagic));
  const u64 w = ((u64)pw.hi[i] << 32 | pw.lo[i]) + (u64)z * 131072u;
  const uint32_t some = (qb - (kMagicBits + 46 * 32)) >> 31;  // t < 46
  return w >> ((qb >> 5) & 63) | some;
}

// Logits in sixteenths, from the largest (64) down; the last bin has everything from -64
// on, and rows with logits of 63 and more are not estimated.
constexpr float kPerLogit = 16.0f;
__device__ __forceinline__ int bin_of(float x) {
  const float t = fminf(fmaxf(x * -kPerLogit, -1023.0f), 1024.0f) + 1023.0f;
  return (int)(__float_as_uint(t + kMagic) & (kBins - 1));
}
__device__ __forceinline__ float middle_of(float bin) { return (1023.0f - bin) / kPerLogit; }

// v * f for 0 <= f < 1, rounded down (the rest in *more).
__device__ __forceinline__ u64 times(u64 v, float f, bool *more) {
  const uint32_t b = __float_as_uint(f);
  const int e = (int)(b >> 23);
  const u64 mant = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = 150 - (e ? e : 1);  // f = mant 2^-sh, sh >= 24
  const u64 lo = v * mant, hi = __umul64hi(v, mant);
  if (sh >= 128) {
    *more = (lo | hi) != 0;
    return 0;
  }
  if (sh >= 64) {
    *more = lo != 0 || (sh > 64 && (hi << (128 - sh)) != 0);
    return sh == 64 ? hi : hi >> (sh - 64);
  }
  *more = (lo << (64 - sh)) != 0;
  return (lo >> sh) | (hi << (64 - sh));
}

// A prefix of the tokens by (value descending, index ascending): those with a
// larger key, and the first `ties` of those that have it.
struct Cut {
  uint32_t key;
  int ties;
};

// A row's options, and what follows from them alone.
struct Options {
  float temp, top_p, min_p;
  int top_k;
  float c_hi, c_lo;  // log2(e) / T, 1 where the largest logit is taken
  float l_hi, l_lo;  // T ln(min_p), for 0 < min_p < 1
};
__device__ __forceinline__ Options read_options(const SampleParams &p, int64_t row) {
  Options o;
  o.temp = p.temperature ? p.temperature[row] : p.temperature_all;
  o.top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  o.min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  o.top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  if (!(o.temp > 0.0f)) o.temp = 0.0f;
  // the quotient's fp32 remainder is exact: (c_hi + c_lo) T = log2(e) to 2^-46
  o.c_hi = 1.0f, o.c_lo = 0.0f;
  if (o.temp > 0.0f) {
    o.c_hi = fmaxf(fminf(__fdiv_rn(1.44269502e+00f, o.temp), FLT_MAX), 0x1p-120f);
    const float left = fmaf(-o.c_hi, o.temp, 1.44269502e+00f) + 1.92596303e-08f;
    o.c_lo = o.c_hi < 1e30f && o.c_hi > 1e-30f ? __fdiv_rn(left, o.temp) : 0.0f;
  }
  o.l_hi = o.l_lo = 0.0f;
  if (o.temp > 0.0f && o.min_p > 0.0f && o.min_p < 1.0f) {
    const double l = (double)o.temp * log((double)o.min_p);
    o.l_hi = (float)l;
    o.l_lo = isfinite(o.l_hi) ? (float)(l - (double)o.l_hi) : 0.0f;
  }
  return o;
}
// The key of the smallest value with x >= m + T ln(min_p) (m itself for min_p >= 1).
__device__ __forceinline__ uint32_t key_of_min_p(const Options &o, float m) {
  if (!(o.min_p < 1.0f) || o.temp == 0.0f) return key_of(m);
  const float h = m + o.l_hi, v = h - m;  // the sum's error, exactly
  const float e = ((m - (h - v)) + (o.l_hi - v)) + o.l_lo;
  return key_of(clean(e > 0.0f ? nextafterf(h, INFINITY) : h));
}

struct Shared {
  uint32_t count[kBins];
  u64 mass[kBins];
  u64 list[kList];
  Powers pw;
  Options opt;
  uint32_t cta_max[kMaxCluster];  // largest key of every CTA's slice
  uint32_t n_list;
  u64 warp_mass[kWarps];  // kept weights above the cut, of every warp's tokens
  u64 warp_ties[kWarps];  // tokens at the cut
  u64 warp_all[kWarps];   // all weights
  u64 scan[kWarps];
  u64 found[5];           // what the first CTA found, in every CTA
};

template <typename T>
struct Row {
  Shared *sm;
  const T *x;  // this CTA's tokens, in shared memory, behind the last -inf for whole warps
  int n, seg;  // how many; tokens of a warp
  int first;   // the first one's index
  uint32_t rank, ranks;

  __device__ __forceinline__ void load(int i, float (&v)[N]) const {
    Vec<T>::get(*reinterpret_cast<const typename Vec<T>::Word *>(x + i), v);
  }
  // f(value, index in the slice, place in its vector) for this warp's tokens (as they are:
  // a NaN compares with nothing and has no weight).
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int a = (threadIdx.x >> 5) * seg, b = a + seg;
    for (int i = a + (threadIdx.x & 31) * N; i < b; i += 32 * N) {
      float v[N];
      load(i, v);
#pragma unroll
      for (int j = 0; j < N; ++j) f(v[j], i + j, j);
    }
  }
  __device__ __forceinline__ void sync() const {
    if (ranks > 1)
      cluster_sync();
    else
      __syncthreads();
  }
  // What the first CTA's thread 0 has in found goes to all.
  __device__ __forceinline__ void tell() const {
    if (rank == 0) {
      __syncthreads();
      if (ranks > 1 && threadIdx.x < 5 * ranks)
        st_remote64(remote(&sm->found[threadIdx.x % 5], threadIdx.x / 5),
                    sm->found[threadIdx.x % 5]);
    }
    sync();
  }
};

// Sum over the block of one value a thread, exclusive before this thread's.
__device__ __forceinline__ u64 block_scan(Shared *sm, u64 v, u64 *total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  u64 in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, in, o);
    if (lane >= o) in += t;
  }
  if (lane == 31) sm->scan[warp] = in;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const u64 t = sm->scan[w];
    if (w < warp) before += t;
    all += t;
  }
  __syncthreads();
  *total = all;
  return before + in - v;
}

__device__ __forceinline__ u64 fraction_of(u64 total, float f) {  // rounded up, 1 at least
  bool more;
  const u64 v = times(total, f, &more);
  return max(v + more, (u64)1);
}

__device__ __forceinline__ void add_mass(u64 *m, u64 w) {
  const uint32_t lo = (uint32_t)w;
  uint32_t *p = reinterpret_cast<uint32_t *>(m);
  const uint32_t was = atomicAdd(p, lo);
  const uint32_t hi = (uint32_t)(w >> 32) + (was + lo < lo ? 1u : 0u);
  if (hi) atomicAdd(p + 1, hi);
}

__device__ __forceinline__ void clear_bins(Shared *sm) {
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm->count[i] = 0, sm->mass[i] = 0;
}

// The bin where the running count (MASS: sum of weights) reaches `target`: found gets it,
// what is missing where it begins, what it has and how many tokens, and 1 (first CTA).
template <bool MASS>
__device__ __forceinline__ void find_bin(Shared *sm, u64 target) {
  constexpr int P = kBins / kThreads;
  u64 v[P], sum = 0, total;
  uint32_t n[P];
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const int i = threadIdx.x * P + e;
    n[e] = sm->count[i];
    v[e] = MASS ? sm->mass[i] : (u64)n[e];
    sum += v[e];
  }
  u64 at = block_scan(sm, sum, &total);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (at < target && target <= at + v[e]) {
      sm->found[0] = (u64)(threadIdx.x * P + e);
      sm->found[1] = target - at;
      sm->found[2] = v[e];
      sm->found[3] = n[e];
      sm->found[4] = 1;
    }
    at += v[e];
  }
}

// The cut in a bin of one value, whose steps end at the key hi.
template <typename T, bool MASS>
__device__ __forceinline__ Cut last_cut(uint32_t hi, int shift, u64 target, u64 in_bin, u64 n) {
  // zeros (or, of a negative value's key, ones) behind a 16-bit value
  const uint32_t rest = sizeof(T) == 4 ? 0 : (1u << 13) - 1;
  const u64 one = MASS ? max(in_bin / max(n, (u64)1), (u64)1) : 1;
  return {shift == 0 ? hi : hi & 0x80000000u ? hi & ~rest : ((hi + 1) & ~rest) - 1,
          (int)((target + one - 1) / one)};
}

// The cut at which the running count (MASS: sum of weights) of the tokens with keys in
// [lo, hi] first reaches `target`; with MASS, of those inside `in` only, and with a
// fraction >= 0 target is that fraction of all their weights.  each(f) calls f(value) for
// this CTA's tokens, those outside [lo, hi] among them or not.  A histogram of 2048 steps
// of the key in the first CTA (FEW: straight there; else by way of one in every CTA), then
// of the steps in the one that was found.  The bins are clear before and after, in every
// CTA.  False: they do not reach it.
template <typename T, bool MASS, bool FEW, typename E>
__device__ bool find_cut(const Row<T> &r, const Scale &s, E each, uint32_t lo, uint32_t hi,
                         const Cut &in, u64 target, float fraction, Cut *cut) {
  constexpr bool kExact = sizeof(T) == 2;
  constexpr int kGrain = sizeof(T) == 4 ? 0 : 13;  // zeros behind a 16-bit value
  Shared *sm = r.sm;
  const uint32_t count_at = remote(sm->count, 0), mass_at = remote(sm->mass, 0);
  const bool straight = FEW || r.rank == 0;
  for (;;) {
    const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
    each([&](float x) {
      const uint32_t key = key_of(clean(x));
      if (key < lo || key > hi || (MASS && key <= in.key)) return;
      const uint32_t b = (hi - key) >> shift;
      const u64 w = MASS ? weight<kExact>(s, sm->pw, x) : 0;
      if (straight) {
        add_remote32(count_at + b * 4, 1u);
        if (MASS && w) add_remote64(mass_at + b * 8, w);
      } else {
        atomicAdd(&sm->count[b], 1u);
        if (MASS && w) add_mass(&sm->mass[b], w);
      }
    });
    // the tokens at the cut of `in`: so many of them, counted by the first CTA
    if (MASS && r.rank == 0 && threadIdx.x == 0 && in.ties && in.key >= lo && in.key <= hi) {
      const uint32_t b = (hi - in.key) >> shift;
      add_remote32(count_at + b * 4, (uint32_t)in.ties);
      add_remote64(mass_at + b * 8,
                   (u64)in.ties * weight<kExact>(s, sm->pw, value_of(in.key)));
    }
    if (!straight) {
      __syncthreads();
      for (int i = threadIdx.x; i < kBins; i += kThreads)
        if (sm->count[i]) {
          add_remote32(count_at + i * 4, sm->count[i]);
          if (MASS) add_remote64(mass_at + i * 8, sm->mass[i]);
          sm->count[i] = 0;
          sm->mass[i] = 0;
        }
    }
    if (r.rank == 0 && threadIdx.x == 0) sm->found[4] = 0;
    r.sync();
    if (r.rank == 0) {
      if (MASS && fraction >= 0.0f) {
        u64 sum = 0, total;
        for (int i = threadIdx.x; i < kBins; i += kThreads) sum += sm->mass[i];
        block_scan(sm, sum, &total);
        target = fraction_of(total, fraction);
      }
      find_bin<MASS>(sm, target);
      clear_bins(sm);
    }
    r.tell();
    const uint32_t b = (uint32_t)sm->found[0];
    const u64 in_bin = sm->found[2], n = sm->found[3];
    const bool ok = sm->found[4] != 0;
    target = sm->found[1];
    fraction = -1.0f;
    __syncthreads();
    if (!ok) return false;
    hi -= b << shift;
    lo = max(lo, hi - ((1u << shift) - 1));
    if (shift <= kGrain) {
      *cut = last_cut<T, MASS>(hi, shift, target, in_bin, n);
      return true;
    }
  }
}

// The shorter of two prefixes.
__device__ __forceinline__ Cut shorter(const Cut &a, const Cut &b) {
  if (a.key != b.key) return a.key > b.key ? a : b;
  return a.ties < b.ties ? a : b;
}

// Sorts n <= kList different numbers in shared memory (one CTA): few of them by how many are
// smaller, four threads a number, more as a bitonic network over a power of two.
__device__ __forceinline__ void sort_list(u64 *v, int n) {
  if (n <= kThreads / 4) {
    const int i = threadIdx.x >> 2, part = threadIdx.x & 3;
    u64 x = 0;
    int at = 0;
    __syncthreads();
    if (i < n) {
      x = v[i];
      for (int j = part; j < n; j += 4) at += v[j] < x;
    }
    at += __shfl_xor_sync(0xffffffffu, at, 1);
    at += __shfl_xor_sync(0xffffffffu, at, 2);
    __syncthreads();
    if (i < n && part == 0) v[at] = x;
    __syncthreads();
    return;
  }
  int size = 2;
  while (size < n) size *= 2;
  for (int i = n + (int)threadIdx.x; i < size; i += kThreads) v[i] = ~0ull;
  for (int k = 2; k <= size; k *= 2)
    for (int j = k / 2; j > 0; j /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < size / 2; i += kThreads) {
        const int a = 2 * i - (i & (j - 1)), b = a + j;
        const u64 x = v[a], y = v[b];
        if ((x > y) == ((a & k) == 0)) v[a] = y, v[b] = x;
      }
    }
  __syncthreads();
}

__device__ __forceinline__ void answer(const SampleParams &p, int64_t row, int token, float x,
                                       const Scale &s, const Options &o, u64 total) {
  p.token[row] = token;
  if (!p.logprob) return;
  float t = 0.0f, lo = 0.0f;  // (m - x) / T in powers of two
  if (x != s.m && o.temp > 0.0f) {
    const float d = s.m - x, v = s.m - d, e = (s.m - (d + v)) + (v - x);
    t = d * s.c_hi;
    lo = fmaf(e, s.c_hi, fmaf(d, s.c_lo, fmaf(d, s.c_hi, -t)));
  }
  // (a token alone has probability 1, not the half unit less)
  const bool alone = t == 0.0f && total == ((1ull << kUnitBits) | 1);
  p.logprob[row] = alone ? 0.0f : log_share(t, lo, total);
}

// The whole choice from the list of all tokens that any filter may keep, n in the first
// CTA's shared memory as (~key, index): in order of value for the filters, then of index.
// target: the sum of weights that top-p asks for, 0 for that share of the list's.
template <typename T>
__device__ void solve_list(const SampleParams &p, const Row<T> &r, const Scale &s,
                           const Options &o, uint32_t min_key, int64_t row, int n, u64 target) {
  constexpr bool kExact = sizeof(T) == 2;
  constexpr int P = kList / kThreads;
  Shared *sm = r.sm;
  sort_list(sm->list, n);
  auto value = [&](int i) { return value_of(~(uint32_t)(sm->list[i] >> 32)); };
  const int a = threadIdx.x * P;
  int kept = o.top_k > 0 ? min(n, o.top_k) : n;
  if (o.top_p < 1.0f) {
    u64 w[P], sum = 0, total;
#pragma unroll
    for (int e = 0; e < P; ++e) {
      w[e] = a + e < kept ? weight<kExact>(s, sm->pw, value(a + e)) : 0;
      sum += w[e];
    }
    u64 at = block_scan(sm, sum, &total);
    if (target == 0) target = fraction_of(total, fmaxf(o.top_p, 0.0f));
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (at < target && target <= at + w[e]) sm->found[0] = (u64)(a + e + 1);
      at += w[e];
    }
    __syncthreads();
    kept = (int)sm->found[0];
  }
  if (min_key) {
    int mine = 0;
#pragma unroll
    for (int e = 0; e < P; ++e) mine += a + e < kept && key_of(value(a + e)) >= min_key;
    u64 total;
    block_scan(sm, (u64)mine, &total);
    kept = (int)total;
  }
  for (int i = threadIdx.x; i < kept; i += kThreads)
    sm->mass[i] = (sm->list[i] << 32) | (u64)i;
  sort_list(sm->mass, kept);
  u64 w[P], sum = 0, total;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    w[e] = a + e < kept ? weight<kExact>(s, sm->pw, value((int)(uint32_t)sm->mass[a + e])) : 0;
    sum += w[e];
  }
  u64 at = block_scan(sm, sum, &total);
  bool more;
  const u64 goal = times(total, fminf(fmaxf(p.u[row], 0.0f), 0.99999994f), &more);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (at <= goal && goal < at + w[e])
      answer(p, row, (int)(sm->mass[a + e] >> 32), value((int)(uint32_t)sm->mass[a + e]), s, o,
             total);
    at += w[e];
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleParams p) {
  constexpr bool kExact = sizeof(T) == 2;
  extern __shared__ __align__(16) uint8_t smem[];
  Shared *sm = reinterpret_cast<Shared *>(smem);
  T *slice = reinterpret_cast<T *>(smem + (sizeof(Shared) + 15) / 16 * 16);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Row<T> r;
  r.sm = sm;
  r.x = slice;
  r.rank = cluster_rank();
  r.ranks = cluster_size();
  const int64_t row = blockIdx.x / r.ranks;
  r.first = (int)r.rank * p.slice;
  r.n = max(0, min(p.V - r.first, p.slice));
  r.seg = (p.slice + kWarps * 32 * N - 1) / (kWarps * 32 * N) * (32 * N);

  // ---- the slice, and the largest logit of each of four groups a thread
  const T *src = static_cast<const T *>(p.logits) + row * p.ld + r.first;
  float g[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  constexpr int kCopy = 16 / sizeof(T);
  const int whole = p.vec ? r.n / kCopy * kCopy : 0;  // tokens that come 16 bytes at a time
  for (int i = threadIdx.x * kCopy; i < whole; i += kThreads * kCopy)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(slice + i)),
                 "l"(src + i)
                 : "memory");
  for (int i = whole + (int)threadIdx.x; i < r.seg * kWarps; i += kThreads) {
    const T x = i < r.n ? src[i] : (T)-INFINITY;
    slice[i] = x;
    g[0] = fmaxf(g[0], (float)x);
  }
  if (threadIdx.x < 32) {
    const u64 w = kPower[threadIdx.x], v = w - ((u64)kMagicBits << 17);
    sm->pw.lo[threadIdx.x] = (uint32_t)v;
    sm->pw.hi[threadIdx.x] = (uint32_t)(v >> 32);
    sm->pw.flt[threadIdx.x] = (float)w * 0x1p-17f;
  }
  clear_bins(sm);
  if (threadIdx.x == 0) {
    sm->n_list = 0;
    sm->opt = read_options(p, row);
  }
  // (others may write to this CTA's shared memory once it has come here)
  if (r.ranks > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  asm volatile("cp.async.wait_all;" ::: "memory");
  for (int i = threadIdx.x * kCopy; i < whole; i += kThreads * kCopy)  // (its own)
#pragma unroll
    for (int k = 0; k < kCopy; k += N) {
      float v[N];
      r.load(i + k, v);
#pragma unroll
      for (int j = 0; j < N; ++j) g[j] = fmaxf(g[j], v[j]);
    }
  const uint32_t top = __reduce_max_sync(
      0xffffffffu, key_of(clean(fmaxf(fmaxf(g[0], g[1]), fmaxf(g[2], g[3])))));
  if (lane == 0) sm->scan[warp] = top;
  __syncthreads();
  Options o = sm->opt;
  if (o.top_k >= p.V) o.top_k = 0;
  const bool one = o.temp == 0.0f || o.top_k == 1;
  const bool small = p.V <= kList && r.ranks == 1 && !one;
  const bool by_k = !one && !small && o.top_k > 0;
  const bool by_p = !one && !small && o.top_k <= 0 && o.top_p < 1.0f;
  if (by_k || by_p) {
    // top-k: the groups' largest logits; top-p: those (the few tokens with most of the
    // weight are among them), and for the others those of the first group, four times
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (const int b = bin_of(g[j]); b < kBins - 1) atomicAdd(&sm->count[b], 1u);
    if (by_p)
      r.each([&](float x, int, int j) {
        if (j == 0) {
          const int b = bin_of(x);
          if (b < kBins - 1 && x < g[0]) atomicAdd(&sm->count[b], 4u);
        }
      });
  }
  if (r.ranks > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();
  if (by_k || by_p) {
    // (a CTA clears what it passes on; the first one's own are in `mass` meanwhile)
    const uint32_t mass_at = remote(sm->mass, 0);
    for (int i = threadIdx.x; i < kBins; i += kThreads)
      if (sm->count[i]) {
        add_remote32(mass_at + i * 8, sm->count[i]);
        sm->count[i] = 0;
      }
  }
  if (threadIdx.x < r.ranks) {  // this CTA's largest to all
    uint32_t k = 0;
    for (int w = 0; w < kWarps; ++w) k = max(k, (uint32_t)sm->scan[w]);
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                     remote(&sm->cta_max[r.rank], threadIdx.x)),
                 "r"(k)
                 : "memory");
  }
  r.sync();
  uint32_t max_key = 0;
  for (uint32_t i = 0; i < r.ranks; ++i) max_key = max(max_key, sm->cta_max[i]);
  Scale s;
  s.m = value_of(max_key);

  if (s.m == INFINITY) {  // they share all the weight: 0, and the others -inf
    for (int i = threadIdx.x; i < r.seg * kWarps; i += kThreads)
      slice[i] = (float)slice[i] == INFINITY ? (T)0.0f : (T)-INFINITY;
    s.m = 0.0f;
    max_key = key_of(0.0f);
    __syncthreads();
  }
  s.c_hi = o.c_hi;
  s.far = 46.0f / o.c_hi;
  s.c_lo = o.c_lo;
  const uint32_t min_key = o.min_p > 0.0f ? key_of_min_p(o, s.m) : 0;

  if (s.m == -INFINITY) {  // no token may be chosen
    if (r.rank == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
    if (r.ranks > 1) cluster_sync();
    return;
  }

  bool listed = small;  // the first CTA's list holds all that may be kept
  int n_listed = p.V;
  u64 p_target = 0;
  auto entry = [&](float x, int i) {
    return (u64)(uint32_t)~key_of(clean(x)) << 32 | (u64)(uint32_t)(r.first + i);
  };
  if (small)
    for (int i = threadIdx.x; i < r.n; i += kThreads) sm->list[i] = entry((float)slice[i], i);
  __syncthreads();

  // ---- what the first CTA looks for in the histogram: top-k, a bin up to which that many
  // groups have their largest; top-p, the bins of its cut
  bool found = false;
  float edge_hi = 0.0f, edge_lo = 0.0f;  // values that bound what was found
  if (by_k || by_p) {
    if (r.rank == 0) {
      constexpr int P = kBins / kThreads;
      u64 v[P], k[P], sum = 0, n = 0, total, total_n;
      if (threadIdx.x == 0) sm->found[3] = sm->found[4] = 0;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int i = threadIdx.x * P + e;
        k[e] = sm->mass[i];
        v[e] = by_k ? k[e]
                    : (u64)((float)k[e] *
                            exp2f(40.0f - fmaxf(s.m - middle_of((float)i), 0.0f) * s.c_hi));
        sum += v[e];
        n += k[e];
      }
      u64 at = block_scan(sm, sum, &total), at_n = block_scan(sm, n, &total_n);
      // top-p: the share above a bin is off by what its weights' places in their bins and
      // the tokens that were not counted leave open, some hundredths of share times rest
      const float q = fminf(fmaxf(o.top_p, 0.0f), 1.0f), off = 0.06f * q * (1.0f - q);
      const u64 deep = by_k ? (u64)o.top_k : fraction_of(total, fminf(q + off, 0.99999994f));
      const u64 near = by_k ? (u64)1 : fraction_of(total, q - off);
      const bool ok = s.m < 63.0f;
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const int i = threadIdx.x * P + e;
        // (few tokens are listed whatever weight they have)
        if (by_p && at_n <= kFew && kFew < at_n + k[e] && i > 0) sm->found[3] = (u64)(i - 1);
        at_n += k[e];
        if (at < near && near <= at + v[e]) sm->found[1] = (u64)i;
        if (at < deep && deep <= at + v[e] && i < kBins - 1 && ok) {
          sm->found[0] = (u64)i;
          sm->found[2] = at_n;
          sm->found[4] = 1;
        }
        at += v[e];
      }
      clear_bins(sm);
    }
    r.tell();
    found = sm->found[4] != 0;
    // half a bin to each side, and what rounding may have moved
    const float b = (float)max(sm->found[0], sm->found[3]), b1 = (float)sm->found[1];
    edge_lo = middle_of(b + 0.6f);
    edge_hi = by_k || sm->found[2] <= kList / 2 ? INFINITY : middle_of(b1 - 0.6f);
    if (edge_hi > s.m) edge_hi = INFINITY;
    __syncthreads();
  }

  // ---- top-k: the tokens that may be among them, to the first CTA's list
  const uint32_t n_at = remote(&sm->n_list, 0), list_at = remote(sm->list, 0);
  auto push = [&](float x, int i) {
    uint32_t at;
    asm volatile("atom.relaxed.cluster.shared::cluster.add.u32 %0, [%1], 1;"
                 : "=r"(at)
                 : "r"(n_at)
                 : "memory");
    if (at < kList) st_remote64(list_at + at * 8, entry(x, i));
  };
  if (by_k && found) {
    r.each([&](float x, int i, int) {
      if (x >= edge_lo) push(x, i);
    });
    r.sync();
    n_listed = (int)ld_remote32(n_at);
    listed = n_listed <= kList && n_listed >= o.top_k;
  }
  if (listed) {
    if (r.rank == 0) solve_list(p, r, s, o, min_key, row, n_listed, p_target);
    if (r.ranks > 1) cluster_sync();  // the others have read how many there are
    return;
  }

  // ---- the cut
  constexpr int kGrain = sizeof(T) == 4 ? 0 : 13;
  // This warp's kept weights above the cut, some of them summed already, and tokens at it.
  auto put_sums = [&](u64 had, u64 mass, uint32_t ties) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, d);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
      sm->warp_mass[warp] = had + mass;
      sm->warp_ties[warp] = ties;
    }
  };
  Cut cut = {0, 0};      // every token
  bool summed = false;   // the weights above the cut are, warp by warp
  auto slice_each = [&](auto f) { r.each([&](float x, int, int) { f(x); }); };
  if (one) {
    cut = {max_key, 1};
  } else {
    if (o.top_k > 0)
      find_cut<T, false, false>(r, s, slice_each, 0u, max_key, cut, (u64)o.top_k, -1.0f, &cut);
    Cut last = cut;
    if (o.top_p < 1.0f) {
      bool done = false;
      if (by_p && found) {
        // Few tokens may be kept: all weights, and those tokens to the first CTA's list.
        // Else: all weights, those above the bins around the cut, and a histogram of those
        // in them, by steps of the key.
        const bool few = edge_hi == INFINITY;
        uint32_t hi = few ? max_key : key_of(clean(edge_hi)), lo = key_of(clean(edge_lo));
        const int bits = 32 - __clz(hi - lo), shift = bits > 11 ? bits - 11 : 0;
        const uint32_t count_at = remote(sm->count, 0), mass_at = remote(sm->mass, 0);
        u64 all = 0, above = 0;
        // this warp's tokens in the bins, as places in the slice (below 2^15: 64 KB of
        // 16-bit logits, an eighth of QZ_MAX_VOCAB); more than fit are looked for again
        uint16_t *const in_bins = reinterpret_cast<uint16_t *>(sm->list) + warp * kMine;
        uint32_t n_in = 0;
        auto each_in_bins = [&](auto f) {
          if (n_in <= kMine) {
            for (uint32_t k = lane; k < n_in; k += 32) f((float)slice[in_bins[k]]);
          } else {
            r.each([&](float x, int, int) {
              if (x >= edge_lo && x <= edge_hi) f(x);
            });
          }
        };
        if (few) {
          r.each([&](float x, int i, int) {
            all += weight<kExact>(s, sm->pw, x);
            if (x >= edge_lo) push(x, i);
          });
        } else {
          r.each([&](float x, int i, int) {
            const u64 w = weight<kExact>(s, sm->pw, x);
            all += w;
            above += x > edge_hi ? w : 0;
            const bool in = x >= edge_lo && x <= edge_hi;
            const uint32_t m = __ballot_sync(0xffffffffu, in);  // (whole warps)
            if (m == 0) return;
            const uint32_t at = n_in + __popc(m & ((1u << lane) - 1));
            if (in && at < kMine) in_bins[at] = (uint16_t)i;
            n_in += __popc(m);
          });
          __syncwarp();
          each_in_bins([&](float x) {
            const u64 z = weight<kExact>(s, sm->pw, x);
            const uint32_t b = (hi - key_of(clean(x))) >> shift;
            if (r.rank == 0) {
              add_remote32(count_at + b * 4, 1u);
              if (z) add_remote64(mass_at + b * 8, z);
            } else {
              atomicAdd(&sm->count[b], 1u);
              if (z) add_mass(&sm->mass[b], z);
            }
          });
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          all += __shfl_xor_sync(0xffffffffu, all, d);
          above += __shfl_xor_sync(0xffffffffu, above, d);
        }
        if (lane == 0) {
          sm->warp_all[warp] = all;
          sm->warp_mass[warp] = above;
        }
        if (!few && r.rank != 0) {
          __syncthreads();
          for (int i = threadIdx.x; i < kBins; i += kThreads)
            if (sm->count[i]) {
              add_remote32(count_at + i * 4, sm->count[i]);
              add_remote64(mass_at + i * 8, sm->mass[i]);
              sm->count[i] = 0;
              sm->mass[i] = 0;
            }
        }
        r.sync();
        if (r.rank == 0) {
          u64 t_all = 0, t_above = 0, total, total_above;
          if (threadIdx.x < kWarps * r.ranks) {
            const uint32_t w = threadIdx.x % kWarps, from = threadIdx.x / kWarps;
            t_all = ld_remote64(remote(&sm->warp_all[w], from));
            t_above = ld_remote64(remote(&sm->warp_mass[w], from));
          }
          if (threadIdx.x == 0) sm->found[4] = 0;
          block_scan(sm, t_all, &total);
          block_scan(sm, t_above, &total_above);
          const u64 target = fraction_of(total, fmaxf(o.top_p, 0.0f));
          if (few) {
            const int n = (int)sm->n_list;
            u64 sum = 0;
            if (n <= kList)
              for (int i = threadIdx.x; i < n; i += kThreads)
                sum += weight<kExact>(s, sm->pw, value_of(~(uint32_t)(sm->list[i] >> 32)));
            block_scan(sm, sum, &sum);
            if (sum >= target) solve_list(p, r, s, o, min_key, row, n, target);
            if (threadIdx.x == 0) sm->found[4] = sum >= target;
          } else {
            if (total_above < target) find_bin<true>(sm, target - total_above);
            clear_bins(sm);
          }
        }
        r.tell();
        const bool ok = sm->found[4] != 0;
        if (ok && few) return;
        const u64 left = sm->found[1], in_bin = sm->found[2], n = sm->found[3];
        hi -= (uint32_t)sm->found[0] << shift;
        lo = max(lo, hi - ((1u << shift) - 1));
        __syncthreads();
        if (ok) {
          done = shift <= kGrain
                     ? (last = last_cut<T, true>(hi, shift, left, in_bin, n), true)
                     : find_cut<T, true, true>(r, s, each_in_bins, lo, hi, Cut{0, 0}, left,
                                               -1.0f, &last);
          if (done && (min_key == 0 || min_key <= last.key)) {
            // the kept ones among the tokens of those bins
            const float at = value_of(last.key);
            u64 mass = 0;
            uint32_t ties = 0;
            each_in_bins([&](float x) {
              if (x > at) mass += weight<kExact>(s, sm->pw, x);
              ties += x == at;
            });
            put_sums(above, mass, ties);
            summed = true;
          }
        }
      }
      if (!done)
        find_cut<T, true, false>(r, s, slice_each, 0u, max_key, cut, 0, fmaxf(o.top_p, 0.0f),
                                 &last);
    }
    if (min_key) last = shorter(last, Cut{min_key, INT32_MAX});
    cut = last;
  }

  // ---- kept weights and tokens at the cut, warp by warp
  if (!summed) {
    u64 mass = 0;
    uint32_t ties = 0;
    if (cut.key == 0) {
      r.each([&](float x, int, int) { mass += weight<kExact>(s, sm->pw, x); });
    } else {
      const float at = value_of(cut.key);
      r.each([&](float x, int, int) {
        if (x > at) mass += weight<kExact>(s, sm->pw, x);
        ties += x == at;
      });
    }
    put_sums(0, mass, ties);
  }
  r.sync();
  // Every CTA sums all of them; thread i has warp i of the row.
  const u64 cut_weight = cut.key ? weight<kExact>(s, sm->pw, value_of(cut.key)) : 0;
  const bool live = threadIdx.x < kWarps * r.ranks;
  u64 w_mass = 0, w_ties = 0, total;
  if (live) {
    w_mass = ld_remote64(remote(&sm->warp_mass[threadIdx.x % kWarps], threadIdx.x / kWarps));
    w_ties = ld_remote64(remote(&sm->warp_ties[threadIdx.x % kWarps], threadIdx.x / kWarps));
  }
  const u64 t_before = block_scan(sm, w_ties, &total);
  const u64 left = (u64)cut.ties > t_before ? (u64)cut.ties - t_before : 0;
  const u64 mine = w_mass + min(w_ties, left) * cut_weight;
  const u64 before = block_scan(sm, mine, &total);
  bool more;
  const u64 goal = times(total, fminf(fmaxf(p.u[row], 0.0f), 0.99999994f), &more);
  if (live && before <= goal && goal < before + mine) {
    sm->found[0] = threadIdx.x;
    sm->found[1] = goal - before;
    sm->found[2] = left;
  }
  __syncthreads();
  const int at = (int)sm->found[0];
  if (at / kWarps == (int)r.rank) {
    // that warp's tokens again, by all threads
    u64 want = sm->found[1], rest = sm->found[2];
    const int a = at % kWarps * r.seg, b = a + r.seg;
    for (int i0 = a; i0 < b; i0 += kThreads * N) {
      const int i = i0 + (int)threadIdx.x * N;
      float v[N];
      r.load(min(i, b - N), v);
      u64 w[N], sum = 0, t = 0, all_t, all_w;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[j] = i < b ? clean(v[j]) : -INFINITY;
        t += i < b && key_of(v[j]) == cut.key;
      }
      u64 t_at = block_scan(sm, t, &all_t);  // tokens at the cut before this thread's
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t key = key_of(v[j]);
        w[j] = 0;
        if (key > cut.key) {
          w[j] = weight<kExact>(s, sm->pw, v[j]);
        } else if (key == cut.key) {
          if (t_at < rest) w[j] = cut_weight;
          ++t_at;
        }
        sum += w[j];
      }
      u64 run = block_scan(sm, sum, &all_w);
      if (want < all_w) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (run <= want && want < run + w[j])
            answer(p, row, r.first + i + j, v[j], s, o, total);
          run += w[j];
        }
        break;
      }
      want -= all_w;
      rest = rest > all_t ? rest - all_t : 0;
    }
  }
  if (r.ranks > 1) cluster_sync();  // others may still read this CTA's shared memory
}

template <typename T>
qz_status launch(SampleParams p, int64_t B, cudaStream_t s) {
  DeviceInfo di;
  qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  const size_t head = (sizeof(Shared) + 15) / 16 * 16;
  // CTAs of a row: as many as let two of them share an SM, and more while they have 2048
  // tokens each and the GPU is not full
  constexpr int kWhole = kWarps * 32 * N;  // in shared memory every warp has as many
  constexpr int kCopy = 16 / sizeof(T);
  auto slice_of = [&](int n) { return ((p.V + n - 1) / n + kCopy - 1) / kCopy * kCopy; };
  auto bytes_of = [&](int n) {
    return (size_t)((slice_of(n) + kWhole - 1) / kWhole * kWhole) * sizeof(T);
  };
  int ranks = 1;
  while (ranks < kMaxCluster &&
         (bytes_of(ranks) > kSliceBytes || (B * ranks <= di.sms && p.V > 2048 * ranks)))
    ranks *= 2;
  p.slice = slice_of(ranks);
  const size_t smem = head + bytes_of(ranks);
  if (smem > (size_t)di.max_smem_optin) return QZ_ERR_UNSUPPORTED;
  const cudaError_t e = allow_smem<sample_kernel<T>>(smem);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, sample_kernel<T>, p));
}

}  // namespace

qz_status launch_sample(const void *logits, int dtype, int64_t ld, int64_t B, int64_t V,
                        const float *u, const qz_sampling &o, int32_t *token, float *logprob,
                        cudaStream_t s) {
  SampleParams p = {};
  p.logits = logits;
  p.ld = ld;
  p.V = (int)V;
  const int64_t size = dtype == QZ_FP32 ? 4 : 2;
  p.vec = ((uintptr_t)logits & 15u) == 0 && ld * size % 16 == 0;
  p.u = u;
  p.temperature = o.temperature;
  p.top_k = o.top_k;
  p.top_p = o.top_p;
  p.min_p = o.min_p;
  p.temperature_all = o.temperature_all;
  p.top_k_all = o.top_k_all;
  p.top_p_all = o.top_p_all;
  p.min_p_all = o.min_p_all;
  p.token = token;
  p.logprob = logprob;
  if (dtype == QZ_FP32) return launch<float>(p, B, s);
  if (dtype == QZ_BF16) return launch<__nv_bfloat16>(p, B, s);
  return launch<__half>(p, B, s);
}

}  // namespace qz
