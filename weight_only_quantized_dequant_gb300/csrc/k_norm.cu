// Residual addition, root-mean-square normalisation and, optionally, INT8
// rows with a scale each:
//   h = x + r,  y = h * rsqrt(mean(h^2) + eps) * (w_bias + w),
//   s = max|y| / 127,  q = rint(y / s).
//
// One pass over memory: a row's h stays on chip (registers, fp32) between the
// sum of squares, the maximum and the store, so the traffic is the floor's
// (x, r in; y or q, h out) and HBM bounds long calls, launch latency short ones.
// The threads of a row are the fewest that hold it in kMaxVec 16-byte vectors each,
// all loaded before the first use.  Measured (GB300): 2048 x 8192 with residual
// 21.3 us, 6.3 TB/s (94% of a plain copy's rate); 16 x 8192 2.4 us; 1021 x 3584
// to INT8 rows 8.4 us, 3.1 TB/s: its CTAs are little more than the GPU holds at once, so
// it is a row's own chain, the maximum and a division a value included.
#include "qz_internal.cuh"

namespace qz {
namespace {

constexpr int kMaxVec = 4;  // 16-byte vectors of a row that one thread holds

struct NormParams {
  const __half *x, *r, *w;
  int64_t ldx, ldr;
  float bias, eps;
  int64_t T, K;
  __half *y;
  int64_t ldy;
  int8_t *q;
  int64_t ldq;
  float *scale;
  __half *sum;
  int64_t lds;
};

// 1 / sqrt(mean + eps); a row of zeros with eps = 0 stays zeros where it becomes codes.
template <bool INT8>
__device__ __forceinline__ float inv_rms(float ss, int K, float eps) {
  const float d = ss / (float)K + eps;
  return INT8 && d == 0.0f ? 0.0f : rsqrtf(d);
}

// The larger value, or NaN where either is one: a row with a NaN must not pass for one
// without (fmaxf drops it).
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sum or maximum over the TPR threads of a row, in a fixed order.
template <int TPR, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float *part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xffffffffu, v, o);
    v = MAX ? max_nan(v, u) : v + u;
  }
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < TPR / 32; ++i) v = MAX ? max_nan(v, part[i]) : v + part[i];
  }
  return v;
}

// q = clamp(rint(y / s)): the IEEE division of the quantizers, so that codes
// follow the same rule; 0 beside a scale of 0, infinity or NaN.
__device__ __forceinline__ uint32_t code(float y, float s) {
  if (!(s > 0.0f && s < INFINITY)) return 0u;
  return (uint32_t)(int)fminf(fmaxf(rintf(__fdiv_rn(y, s)), -127.0f), 127.0f) & 0xFFu;
}

// TPR threads hold one row, kMaxVec vectors of 8 each at most.
template <int TPR, bool INT8>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR) norm_vec_kernel(const NormParams p) {
  __shared__ float part[2][32];
  constexpr int RPB = TPR < 128 ? 128 / TPR : 1;
  const int64_t t = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const int me = threadIdx.x % TPR;
  const int nv = (int)(p.K / 8);
  const bool live = t < p.T;
  const uint4 *x = reinterpret_cast<const uint4 *>(p.x + (live ? t : 0) * p.ldx);
  const uint4 *r = reinterpret_cast<const uint4 *>(p.r + (live ? t : 0) * p.ldr);
  const uint4 *w = reinterpret_cast<const uint4 *>(p.w);
  uint4 xv[kMaxVec], rv[kMaxVec], wv[kMaxVec];
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const int c = i * TPR + me;
    xv[i] = rv[i] = wv[i] = make_uint4(0, 0, 0, 0);
    if (live && c < nv) {
      xv[i] = x[c];
      if (p.r) rv[i] = r[c];
      wv[i] = __ldg(w + c);
    }
  }
  float h[kMaxVec][8];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const uint32_t a[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w};
    const uint32_t b[4] = {rv[i].x, rv[i].y, rv[i].z, rv[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 u = h2f(a[k]), v = h2f(b[k]);
      h[i][2 * k] = u.x + v.x;
      h[i][2 * k + 1] = u.y + v.y;
      ss = fmaf(h[i][2 * k], h[i][2 * k], ss);
      ss = fmaf(h[i][2 * k + 1], h[i][2 * k + 1], ss);
    }
  }
  if (p.sum && live) {
    uint4 *o = reinterpret_cast<uint4 *>(p.sum + t * p.lds);
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
      const int c = i * TPR + me;
      if (c < nv)
        o[c] = make_uint4(f2h(h[i][0], h[i][1]), f2h(h[i][2], h[i][3]), f2h(h[i][4], h[i][5]),
                          f2h(h[i][6], h[i][7]));
    }
  }
  ss = row_reduce<TPR, false>(ss, part[0]);
  const float rs = inv_rms<INT8>(ss, (int)p.K, p.eps);
  float mx = 0.0f;
#pragma unroll
  for (int i = 0; i < kMaxVec; ++i) {
    const uint32_t a[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 u = h2f(a[k]);
      h[i][2 * k] *= rs * (p.bias + u.x);
      h[i][2 * k + 1] *= rs * (p.bias + u.y);
      if (INT8) mx = max_nan(mx, max_nan(fabsf(h[i][2 * k]), fabsf(h[i][2 * k + 1])));
    }
  }
  if (INT8) {
    mx = row_reduce<TPR, true>(mx, part[1]);
    if (!live) return;
    const float s = __fdiv_rn(mx, 127.0f);
    if (me == 0) p.scale[t] = s;
    uint2 *o = reinterpret_cast<uint2 *>(p.q + t * p.ldq);
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
      const int c = i * TPR + me;
      if (c >= nv) continue;
      uint32_t v[2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        v[k] = code(h[i][4 * k], s) | code(h[i][4 * k + 1], s) << 8 |
               code(h[i][4 * k + 2], s) << 16 | code(h[i][4 * k + 3], s) << 24;
      o[c] = make_uint2(v[0], v[1]);
    }
  } else {
    if (!live) return;
    uint4 *o = reinterpret_cast<uint4 *>(p.y + t * p.ldy);
#pragma unroll
    for (int i = 0; i < kMaxVec; ++i) {
      const int c = i * TPR + me;
      if (c < nv)
        o[c] = make_uint4(f2h(h[i][0], h[i][1]), f2h(h[i][2], h[i][3]), f2h(h[i][4], h[i][5]),
                          f2h(h[i][6], h[i][7]));
    }
  }
}

// Rows that are not 16-byte aligned, or longer than the registers hold: h in
// shared memory, one element at a time.
constexpr int kRowThreads = 512;
template <bool INT8>
__global__ void __launch_bounds__(kRowThreads) norm_row_kernel(const NormParams p) {
  extern __shared__ float row[];  // [K]
  __shared__ float part[2][32];
  const int64_t t = blockIdx.x;
  const int K = (int)p.K;
  const __half *x = p.x + t * p.ldx, *r = p.r + t * p.ldr;
  float ss = 0.0f;
  for (int j = threadIdx.x; j < K; j += kRowThreads) {
    const float v = __half2float(x[j]) + (p.r ? __half2float(r[j]) : 0.0f);
    if (p.sum) p.sum[t * p.lds + j] = __float2half_rn(v);
    row[j] = v;  // read again by this thread only
    ss = fmaf(v, v, ss);
  }
  ss = row_reduce<kRowThreads, false>(ss, part[0]);
  const float rs = inv_rms<INT8>(ss, K, p.eps);
  float mx = 0.0f;
  for (int j = threadIdx.x; j < K; j += kRowThreads) {
    const float v = row[j] * (rs * (p.bias + __half2float(p.w[j])));
    if (INT8) {
      row[j] = v;
      mx = max_nan(mx, fabsf(v));
    } else {
      p.y[t * p.ldy + j] = __float2half_rn(v);
    }
  }
  if (INT8) {
    mx = row_reduce<kRowThreads, true>(mx, part[1]);
    const float s = __fdiv_rn(mx, 127.0f);
    if (threadIdx.x == 0) p.scale[t] = s;
    for (int j = threadIdx.x; j < K; j += kRowThreads)
      p.q[t * p.ldq + j] = (int8_t)code(row[j], s);
  }
}

bool fits16(const void *p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

template <bool INT8>
qz_status launch_row(const NormParams &p, cudaStream_t s) {
  const size_t bytes = (size_t)p.K * sizeof(float);
  const cudaError_t e = allow_smem<norm_row_kernel<INT8>>(bytes);
  if (e != cudaSuccess) return cuda_status(e);
  norm_row_kernel<INT8><<<(unsigned)p.T, kRowThreads, bytes, s>>>(p);
  return launch_status();
}

template <int TPR>
qz_status launch_vec(const NormParams &p, cudaStream_t s) {
  constexpr int threads = TPR < 128 ? 128 : TPR, rpb = threads / TPR;
  const unsigned grid = (unsigned)((p.T + rpb - 1) / rpb);
  if (p.q)
    norm_vec_kernel<TPR, true><<<grid, threads, 0, s>>>(p);
  else
    norm_vec_kernel<TPR, false><<<grid, threads, 0, s>>>(p);
  return launch_status();
}

}  // namespace

qz_status launch_rmsnorm(const __half *x, int64_t ldx, const __half *r, int64_t ldr,
                         const __half *w, float bias, float eps, int64_t T, int64_t K, __half *y,
                         int64_t ldy, int8_t *q, int64_t ldq, float *scale, __half *sum,
                         int64_t lds, cudaStream_t s) {
  const NormParams p = {x, r, w, ldx, r ? ldr : 0, bias, eps, T, K,
                        y, ldy, q, ldq, scale, sum, lds};
  const bool vec = K % 8 == 0 && K <= 8 * kMaxVec * 512 && fits16(x, ldx) &&
                   (!r || fits16(r, ldr)) && fits16(w, 0) && (!sum || fits16(sum, lds)) &&
                   (q ? ((uintptr_t)q & 7u) == 0 && ldq % 8 == 0 : fits16(y, ldy));
  if (!vec) return q ? launch_row<true>(p, s) : launch_row<false>(p, s);
  if (K <= 8 * kMaxVec * 32) return launch_vec<32>(p, s);
  if (K <= 8 * kMaxVec * 128) return launch_vec<128>(p, s);
  if (K <= 8 * kMaxVec * 256) return launch_vec<256>(p, s);
  return launch_vec<512>(p, s);
}

}  // namespace qz
