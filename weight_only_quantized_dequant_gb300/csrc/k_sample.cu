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
// weights are 64-bit integers, 2^44 at the largest logit (good to 2^-30, zero
// below 2^-45), and their sums are exact: neither the order of the atomics nor
// the split of a row shows in a result.
//
// A row is a cluster of CTAs that keep their slices in shared memory: one read
// of HBM, one pass for the maximum, then per filter a histogram of distances
// from the maximum, whose crossing bin is refined by digits of the key (the
// bits of the fp32 value in its order), and a last pass that sums the kept
// weights warp by warp.
#include <cuda_bf16.h>

#include <cfloat>
#include <cmath>

#include "qz_internal.cuh"

namespace qz {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kUnitBits = 44;  // the largest logit's weight is 2^44
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

template <typename T>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = h2f(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// Larger values have larger keys.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// What a row's tokens are weighed and binned by.
struct Scale {
  float m;          // largest logit
  float c_hi, c_lo; // log2(e) / T
  float bins;       // bins per unit of the logits
};

// 2^(i/32), i < 32, in units of 2^-44 and as 2^37 times the value (shared memory).
struct Powers {
  u64 fix[32];
  float flt[32];
};

// 2^44 e^{(x - m)/T}, to the nearest integer.  With t = (m - x) c as an fp32
// pair, q = rint(32 t) and f = t - q/32: 2^-t = 2^-(q>>5) 2^-((q&31)/32) 2^-f, the
// last by its series to f^4 (|f| <= 1/64: the next term is below 2^-39).
__device__ __forceinline__ u64 weight(const Scale &s, const Powers &pw, float x) {
  const float d = x == s.m ? 0.0f : s.m - x;
  const float t = d * s.c_hi;
  if (!(t < 46.0f)) return 0;  // (x = -inf with c = 0 gives NaN)
  // m - x is exact for 16-bit logits of like size; what fp32 lost else
  const float xv = s.m - d;
  const float e = (s.m - (d + xv)) + (xv - x);
  const float lo = fmaf(d, s.c_lo, fmaf(d, s.c_hi, -t)) + (x == s.m ? 0.0f : e * s.c_hi);
  const float magic = 12582912.0f;  // 1.5 * 2^23
  const float qf = fmaf(t, 32.0f, magic);
  const int q = (int)(__float_as_uint(qf) & 0x3fffffu);
  const float f = fmaf(qf - magic, -0.03125f, t) + lo;
  // 2^-f - 1, f = g / ln 2
  const float g = -f * 0.69314718055994531f;
  // (the product's own rounding, below 2^-30, aside)
  float p = fmaf(g, 1.0f / 24.0f, 1.0f / 6.0f);
  p = fmaf(g, p, 0.5f);
  p = fmaf(g * g, p, g);
  const int i = q & 31, n = q >> 5;
  const int add = __float2int_rn(p * pw.flt[i]);  // below 2^31.6 / 64
  const u64 w = pw.fix[i] + (u64)((long long)add * 128);
  return n == 0 ? w : ((w >> (n - 1)) + 1) >> 1;
}

__device__ __forceinline__ int bin_of(const Scale &s, float x) {
  const float t = (s.m - x) * s.bins;  // NaN for x = m = inf
  return x == s.m ? 0 : (int)fminf(t, (float)(kBins - 1));
}

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

struct Shared {
  uint32_t count[kBins];
  u64 mass[kBins];
  Powers pw;
  uint32_t max_key;      // of this CTA's slice
  u64 warp_mass[kWarps]; // kept weights above the cut, of every warp's tokens
  u64 warp_ties[kWarps]; // tokens at the cut
  u64 scan[kWarps];
  u64 found[4];          // what the first CTA found: bin, sum before it, sum, count in it
};

template <typename T>
struct Row {
  Shared *sm;
  const T *x;  // this CTA's tokens, in shared memory, padded with -inf to whole vectors
  int n, seg;  // how many; tokens of a warp
  uint32_t rank, ranks;

  // f(value, index in the slice) for this warp's tokens, lane by lane in order.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int N = Vec<T>::N;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int a = warp * seg, b = min(n, a + seg);
    for (int i = a + lane * N; i < b; i += 32 * N) {
      float v[N];
      Vec<T>::get(*reinterpret_cast<const uint4 *>(x + i), v);
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (i + j < b) f(clean(v[j]), i + j);
    }
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

// The cut at which the running count (MASS: sum of weights) of the row's tokens
// first reaches `target`; with MASS, of the tokens inside `in` only, and target
// is that fraction of all of theirs.
template <typename T, bool MASS>
__device__ Cut find_cut(const Row<T> &r, const Scale &s, const Cut &in, u64 target, float fraction) {
  Shared *sm = r.sm;
  constexpr int kLevels = 1 + (sizeof(T) == 4 ? 3 : 2);  // bins, then digits of the key
  int bin = 0;            // found at level 0
  uint32_t prefix = 0;    // digits of the key found since
  int bits = 0;           // how many bits
  u64 last = 0;           // the weight, or count, of one token at the cut
  for (int level = 0; level < kLevels; ++level) {
    const int take = level == 3 ? 10 : 11;
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      sm->count[i] = 0;
      if (MASS) sm->mass[i] = 0;
    }
    __syncthreads();
    r.each([&](float x, int) {
      const uint32_t key = key_of(x);
      int b = bin_of(s, x);
      if (MASS && key < in.key) return;
      if (level > 0) {
        if (b != bin || (level > 1 && key >> (32 - bits) != prefix)) return;
        b = kBins - 1 - (int)((key >> (32 - bits - take)) & ((1u << take) - 1));
      }
      if (!MASS || key > in.key) atomicAdd(&sm->count[b], 1u);
      if (MASS && key > in.key) {
        const u64 w = weight(s, sm->pw, x);
        if (w) {
          const uint32_t lo = (uint32_t)w;
          uint32_t *m = reinterpret_cast<uint32_t *>(&sm->mass[b]);
          const uint32_t was = atomicAdd(m, lo);
          const uint32_t hi = (uint32_t)(w >> 32) + (was + lo < lo ? 1u : 0u);
          if (hi) atomicAdd(m + 1, hi);
        }
      }
    });
    // the tokens at the cut of `in`: so many of them, counted by the first CTA
    __syncthreads();
    if (MASS && r.rank == 0 && threadIdx.x == 0) {
      const float x = value_of(in.key);
      int b = bin_of(s, x);
      bool of = true;
      if (level > 0) {
        of = b == bin && (level == 1 || in.key >> (32 - bits) == prefix);
        b = kBins - 1 - (int)((in.key >> (32 - bits - take)) & ((1u << take) - 1));
      }
      if (of) {
        sm->count[b] += (uint32_t)in.ties;
        sm->mass[b] += (u64)in.ties * weight(s, sm->pw, x);
      }
    }
    if (r.ranks > 1) {
      cluster_sync();
      if (r.rank != 0) {
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
          if (sm->count[i]) {
            add_remote32(remote(&sm->count[i], 0), sm->count[i]);
            if (MASS) add_remote64(remote(&sm->mass[i], 0), sm->mass[i]);
          }
        }
      }
      cluster_sync();
    } else {
      __syncthreads();
    }
    if (r.rank == 0) {
      constexpr int E = kBins / kThreads;
      u64 v[E], sum = 0, total;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int i = threadIdx.x * E + e;
        v[e] = MASS ? sm->mass[i] : (u64)sm->count[i];
        sum += v[e];
      }
      u64 at = block_scan(sm, sum, &total);
      if (MASS && level == 0) {
        bool more;
        target = times(total, fraction, &more);
        target = max(target + more, (u64)1);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (at < target && target <= at + v[e]) {
          sm->found[0] = (u64)(threadIdx.x * E + e);
          sm->found[1] = target - at;
          sm->found[2] = v[e];
          sm->found[3] = sm->count[threadIdx.x * E + e];
        }
        at += v[e];
      }
      __syncthreads();
      if (r.ranks > 1 && threadIdx.x < 4 * r.ranks)
        st_remote64(remote(&sm->found[threadIdx.x & 3], threadIdx.x >> 2),
                    sm->found[threadIdx.x & 3]);
    }
    if (r.ranks > 1)
      cluster_sync();
    else
      __syncthreads();
    const uint32_t b = (uint32_t)sm->found[0];
    target = sm->found[1];
    last = sm->found[3] ? sm->found[2] / sm->found[3] : 0;
    if (level == 0) {
      bin = (int)b;
    } else {
      prefix = (prefix << take) | (uint32_t)(kBins - 1 - b);
      bits += take;
    }
    __syncthreads();
  }
  Cut c;
  // a 16-bit value has zeros in the bits that are left, a negative one's key has ones
  const int rest = 32 - bits;
  c.key = rest == 0 ? prefix : prefix << rest | (prefix >> (bits - 1) ? 0u : (1u << rest) - 1);
  c.ties = MASS ? (int)((target + last - 1) / max(last, (u64)1)) : (int)target;
  return c;
}

// The shorter of two prefixes.
__device__ __forceinline__ Cut shorter(const Cut &a, const Cut &b) {
  if (a.key != b.key) return a.key > b.key ? a : b;
  return a.ties < b.ties ? a : b;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) sample_kernel(const SampleParams p) {
  constexpr int N = Vec<T>::N;
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
  const int first = (int)r.rank * p.slice;
  r.n = max(0, min(p.V - first, p.slice));
  r.seg = (r.n + kWarps * 32 * N - 1) / (kWarps * 32 * N) * (32 * N);
  if (threadIdx.x < 32) {
    const double e = exp2(-(double)threadIdx.x / 32.0);
    sm->pw.fix[threadIdx.x] = (u64)rint(e * (double)(1ull << kUnitBits));
    sm->pw.flt[threadIdx.x] = (float)(e * (double)(1ull << (kUnitBits - 7)));
  }
  if (threadIdx.x == 0) sm->max_key = 0;
  __syncthreads();

  // ---- the slice, and its largest logit
  const T *src = static_cast<const T *>(p.logits) + row * p.ld + first;
  float m = -INFINITY;
  if (p.vec) {
    for (int i = threadIdx.x * N; i < r.n; i += kThreads * N) {
      uint4 w;
      if (i + N <= r.n) {
        w = __ldcs(reinterpret_cast<const uint4 *>(src + i));
        float v[N];
        Vec<T>::get(w, v);
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
        *reinterpret_cast<uint4 *>(slice + i) = w;
      } else {
        for (int j = 0; i + j < r.n; ++j) {
          slice[i + j] = src[i + j];
          m = fmaxf(m, (float)src[i + j]);
        }
      }
    }
  } else {
    for (int i = threadIdx.x; i < r.n; i += kThreads) {
      slice[i] = src[i];
      m = fmaxf(m, (float)src[i]);
    }
  }
  const uint32_t k = __reduce_max_sync(0xffffffffu, key_of(clean(m)));
  if (lane == 0) atomicMax(&sm->max_key, k);
  __syncthreads();
  uint32_t max_key = sm->max_key;
  if (r.ranks > 1) {
    cluster_sync();
    for (uint32_t i = 0; i < r.ranks; ++i)
      max_key = max(max_key, ld_remote32(remote(&sm->max_key, i)));
  }
  Scale s;
  s.m = value_of(max_key);

  // ---- the row's options
  const float temp = p.temperature ? p.temperature[row] : p.temperature_all;
  const float top_p = p.top_p ? p.top_p[row] : p.top_p_all;
  const float min_p = p.min_p ? p.min_p[row] : p.min_p_all;
  int top_k = p.top_k ? p.top_k[row] : p.top_k_all;
  const bool greedy = !(temp > 0.0f);
  if (greedy) top_k = 1;
  const double c = greedy ? 1.0 : 1.4426950408889634074 / (double)temp;
  s.c_hi = (float)fmin(c, (double)FLT_MAX);
  s.c_lo = c < 1e30 ? (float)(c - (double)s.c_hi) : 0.0f;
  s.bins = fminf(fmaxf(16.0f * s.c_hi, 32.0f), 75.0f);

  if (s.m == -INFINITY) {  // no token may be chosen
    if (r.rank == 0 && threadIdx.x == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = -INFINITY;
    }
  } else {
    Cut cut = {0, 0};  // every token
    if (top_k == 1) {
      cut = {max_key, 1};
    } else {
      if (top_k > 0 && top_k < p.V)
        cut = find_cut<T, false>(r, s, cut, (u64)top_k, 0.0f);
      Cut last = cut;
      if (top_p < 1.0f)
        last = find_cut<T, true>(r, s, cut, 0, fmaxf(top_p, 0.0f));
      if (min_p > 0.0f) {
        // x >= m + T ln(min_p), compared in 64 bits; the smallest fp32 value that is
        const double least = min_p < 1.0f ? (double)s.m + (double)temp * log((double)min_p)
                                          : (double)s.m;
        float v = (float)least;
        if ((double)v < least) v = nextafterf(v, INFINITY);
        const Cut b = {s.m == INFINITY ? max_key : key_of(clean(v)), INT32_MAX};
        last = shorter(last, b);
      }
      cut = last;
    }
    // ---- kept weights and tokens at the cut, warp by warp
    u64 mass = 0;
    uint32_t ties = 0;
    r.each([&](float x, int) {
      const uint32_t key = key_of(x);
      if (key > cut.key)
        mass += weight(s, sm->pw, x);
      else
        ties += key == cut.key;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) {
      sm->warp_mass[warp] = mass;
      sm->warp_ties[warp] = ties;
    }
    if (r.ranks > 1)
      cluster_sync();
    else
      __syncthreads();
    // Every CTA sums all of them; thread i has warp i of the row.
    const u64 cut_weight = weight(s, sm->pw, value_of(cut.key));
    const bool live = threadIdx.x < kWarps * r.ranks;
    u64 w_mass = 0, w_ties = 0, all;
    if (live) {
      w_mass = ld_remote64(remote(&sm->warp_mass[threadIdx.x % kWarps], threadIdx.x / kWarps));
      w_ties = ld_remote64(remote(&sm->warp_ties[threadIdx.x % kWarps], threadIdx.x / kWarps));
    }
    const u64 t_before = block_scan(sm, w_ties, &all);
    const u64 left = (u64)cut.ties > t_before ? (u64)cut.ties - t_before : 0;
    const u64 mine = w_mass + min(w_ties, left) * cut_weight;
    u64 total;
    const u64 before = block_scan(sm, mine, &total);
    const float u = fminf(fmaxf(p.u[row], 0.0f), 0.99999994f);
    bool more;
    const u64 goal = times(total, u, &more);  // the first running sum above it
    if (live && before <= goal && goal < before + mine) {
      sm->found[0] = threadIdx.x;
      sm->found[1] = goal - before;
      sm->found[2] = left;
    }
    __syncthreads();
    const int at = (int)sm->found[0];
    if (at / kWarps == (int)r.rank && at % kWarps == warp) {
      // this warp's tokens again, 32 lanes of N at a time
      u64 want = sm->found[1], rest = sm->found[2];
      const int a = warp * r.seg, b = min(r.n, a + r.seg);
      for (int i = a + lane * N; i - lane * N < b; i += 32 * N) {
        float v[N];
        Vec<T>::get(*reinterpret_cast<const uint4 *>(slice + min(i, p.slice - N)), v);
        uint32_t t = 0;
        u64 w[N], sum = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) t += i + j < b && key_of(clean(v[j])) == cut.key;
        uint32_t t_in = t;
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t z = __shfl_up_sync(0xffffffffu, t_in, o);
          if (lane >= o) t_in += z;
        }
        u64 t_at = t_in - t;  // tokens at the cut before this lane's
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint32_t key = key_of(clean(v[j]));
          w[j] = 0;
          if (i + j < b) {
            if (key > cut.key) {
              w[j] = weight(s, sm->pw, clean(v[j]));
            } else if (key == cut.key) {
              if (t_at < rest) w[j] = cut_weight;
              ++t_at;
            }
          }
          sum += w[j];
        }
        u64 in = sum;
        for (int o = 1; o < 32; o <<= 1) {
          const u64 z = __shfl_up_sync(0xffffffffu, in, o);
          if (lane >= o) in += z;
        }
        const u64 lane_at = in - sum;
        const uint32_t hit = __ballot_sync(0xffffffffu, lane_at <= want && want < in);
        if (hit) {
          if (lane == __ffs(hit) - 1) {
            u64 run = lane_at;
            bool done = false;
#pragma unroll
            for (int j = 0; j < N; ++j) {
              run += w[j];
              if (!done && run > want) {
                done = true;
                const float x = clean(v[j]);
                p.token[row] = first + i + j;
                if (p.logprob) {
                  const double z = x == s.m || greedy ? 0.0 : ((double)x - (double)s.m) / (double)temp;
                  p.logprob[row] =
                      (float)(z - log((double)total / (double)(1ull << kUnitBits)));
                }
              }
            }
          }
          break;
        }
        const u64 all_w = __shfl_sync(0xffffffffu, in, 31);
        const uint32_t all_t = __shfl_sync(0xffffffffu, t_in, 31);
        want -= all_w;
        rest = rest > all_t ? rest - all_t : 0;
      }
    }
  }
  if (r.ranks > 1) cluster_sync();  // others may still read this CTA's shared memory
}

template <typename T>
qz_status launch(SampleParams p, int64_t B, cudaStream_t s) {
  DeviceInfo di;
  qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  constexpr int N = Vec<T>::N;
  const size_t head = (sizeof(Shared) + 15) / 16 * 16;
  int ranks = 1;
  // CTAs of a row: while they have 4096 tokens each and the GPU is not full, and as many
  // as their shared memory asks for
  auto slice_of = [&](int n) { return ((p.V + n - 1) / n + N - 1) / N * N; };
  auto bytes_of = [&](int n) { return head + (size_t)slice_of(n) * sizeof(T); };
  while (ranks < kMaxCluster &&
         (bytes_of(ranks) > (size_t)di.max_smem_optin ||
          (B * ranks < 2 * di.sms && p.V / ranks > 8192)))
    ranks *= 2;
  if (bytes_of(ranks) > (size_t)di.max_smem_optin) return QZ_ERR_UNSUPPORTED;
  p.slice = slice_of(ranks);
  const size_t smem = bytes_of(ranks);
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
