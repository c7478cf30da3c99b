// Low-rank adapters beside a shared projection: out = y + s_a B_a (A_a x).
//
// Two launches over the same rows, on warp-level matrix instructions (rank and
// run lengths are far below a tcgen05 tile; HBM or launch latency bounds every
// size, not the products):
//   down: u = A_a x.  A CTA takes a few rows and a slice of K; neighbouring rows
//     of one adapter (a run) are the 8 columns of m16n8k16 products whose 16
//     rows are ranks, so one request a run wastes columns, not reads.  Its 8
//     warps split the slice, add up through shared memory in warp order, and
//     leave one fp32 partial of u per slice in the workspace.
//   up: B_a u.  A CTA adds the slices' partials in order, then its warps take 64
//     outputs each.  u enters as two fp16 parts of its value scaled by a power of
//     two per row (22 bits and more, any fp32 range); sums stay fp32 and y is
//     added before the one rounding.  The launch overlaps the first one's tail
//     and prefetches B meanwhile.
// In both, a thread's 16-byte load holds 8 consecutive k of its fragment row:
// the two operands use the same order of k, so no shuffle is needed; likewise the
// rows of B_a are dealt so that a thread ends with 8 consecutive outputs.
// Operands without 16-byte rows take the same path with 2-byte loads.
#include "qz_internal.cuh"

namespace qz {
namespace {

__device__ int g_lora_error = 0;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kSub = 64;                    // k per warp and step
constexpr int kSlice = kSub * kWarps;       // k per CTA and step
constexpr int kMaxRows = 32;                // rows of a CTA (one per lane when runs are found)
constexpr int kRowRanks = 2048;             // rows x padded rank of a CTA (shared memory)
constexpr int kMaxSlices = 16;              // partials of u per row
constexpr int kOut = 64;                    // outputs per warp and step

struct LoraParams {
  const __half *a, *b, *x, *y;
  __half *out;
  const float *scale;
  const int32_t *rank, *index;
  int n_adapters, R, Rp, K, N;  // Rp: R rounded up to 16
  int64_t T, a_adapter, a_row, b_adapter, b_row, ldx, ldy, ldo;
  float *u;       // [slices][T][Rp]
  int slices;     // partials per row
  int k_slice;    // k per CTA (a multiple of kSlice)
  int rows_down, rows_up;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Elements [at, at + 8) of a row with n elements; zeros past its end.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __half *row, int at, int n) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (VEC && at + 8 <= n) return __ldg(reinterpret_cast<const uint4 *>(row + at));
  if (at < n) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = at + 2 * i < n ? __half_as_ushort(row[at + 2 * i]) : 0;
      const uint32_t hi = at + 2 * i + 1 < n ? __half_as_ushort(row[at + 2 * i + 1]) : 0;
      h[i] = lo | hi << 16;
    }
    v = make_uint4(h[0], h[1], h[2], h[3]);
  }
  return v;
}

// Runs of equal adapters among rows [t0, t0 + n), n <= 32; every warp holds
// the same: lane i the adapter of row i, and the mask of rows that start a run.
struct Runs {
  int adapter;      // of this lane's row
  unsigned starts;  // run starts, and one bit at n (if n < 32)
  int n;
  __device__ __forceinline__ Runs(const LoraParams &p, int64_t t0, int rows) : n(rows) {
    const int lane = threadIdx.x & 31;
    const int raw = lane < n ? __ldg(p.index + t0 + lane) : -1;
    adapter = raw >= 0 && raw < p.n_adapters ? raw : -1;
    if (adapter != raw && raw != -1) atomicOr(&g_lora_error, 4);
    const int prev = __shfl_up_sync(0xffffffffu, adapter, 1);
    starts = __ballot_sync(0xffffffffu, lane < n && (lane == 0 || adapter != prev));
  }
  // The next run from row `at` on: its adapter and end.
  __device__ __forceinline__ int run(int at, int &end) const {
    const unsigned later = at + 1 < 32 ? starts & (0xffffffffu << (at + 1)) : 0u;
    end = later ? __ffs(later) - 1 : n;
    return __shfl_sync(0xffffffffu, adapter, at);
  }
};

__device__ __forceinline__ int rank_of(const LoraParams &p, int a) {
  return p.rank ? min(max(__ldg(p.rank + a), 0), p.R) : p.R;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads) lora_down_kernel(const LoraParams p) {
  extern __shared__ float part[];  // [kWarps][rows][Rp]
  asm volatile("griddepcontrol.launch_dependents;");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int64_t t0 = (int64_t)blockIdx.x * p.rows_down;
  const int rows = (int)min((int64_t)p.rows_down, p.T - t0);
  const int k_begin = blockIdx.y * p.k_slice, k_end = min(k_begin + p.k_slice, p.K);
  const Runs runs(p, t0, rows);
  for (int at = 0, end; at < rows; at = end) {
    const int a = runs.run(at, end);
    if (a < 0) continue;
    const int rank = rank_of(p, a);
    const __half *A = p.a + a * p.a_adapter;
    for (int m0 = 0; m0 < rank; m0 += 16) {
      float c[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) c[n][i] = 0.0f;
      const int r0 = m0 + g, r1 = m0 + g + 8;
      for (int k0 = k_begin + warp * kSub; k0 < k_end; k0 += kSlice) {
        uint4 av[2][2], xv[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + 32 * h + 8 * tig;
          const uint4 z = make_uint4(0, 0, 0, 0);
          av[h][0] = r0 < rank ? load8<VEC>(A + r0 * p.a_row, k, k_end) : z;
          av[h][1] = r1 < rank ? load8<VEC>(A + r1 * p.a_row, k, k_end) : z;
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            const int t = at + 8 * n + g;
            xv[h][n] = t < end ? load8<VEC>(p.x + (t0 + t) * p.ldx, k, k_end) : z;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            if (at + 8 * n >= end) break;
            mma16816(c[n], av[h][0].x, av[h][1].x, av[h][0].y, av[h][1].y, xv[h][n].x, xv[h][n].y);
            mma16816(c[n], av[h][0].z, av[h][1].z, av[h][0].w, av[h][1].w, xv[h][n].z, xv[h][n].w);
          }
      }
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = at + 8 * n + 2 * tig + (i & 1);
          if (t < end) part[(warp * rows + t) * p.Rp + (i & 2 ? r1 : r0)] = c[n][i];
        }
    }
  }
  __syncthreads();
  // rows without an adapter and ranks past an adapter's own are never read again
  float *u = p.u + ((int64_t)blockIdx.y * p.T + t0) * p.Rp;
  for (int i = threadIdx.x; i < rows * p.Rp; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w * rows * p.Rp + i];
    u[i] = v;
  }
}

__device__ __forceinline__ uint32_t pack2(__half a, __half b) {
  return (uint32_t)__half_as_ushort(a) | (uint32_t)__half_as_ushort(b) << 16;
}

template <bool VEC>
__global__ void __launch_bounds__(kThreads, 2) lora_up_kernel(const LoraParams p) {
  // Per row of Rk ranks (R rounded up to 32, a pad against bank conflicts): u
  // in two fp16 parts; then the factor that undoes the scaling.
  extern __shared__ __align__(16) uint8_t sm[];
  const int Rk = (p.R + 31) / 32 * 32, pitch = Rk + 8;
  __half *uh = reinterpret_cast<__half *>(sm);
  __half *ul = uh + p.rows_up * pitch;
  float *fs = reinterpret_cast<float *>(ul + p.rows_up * pitch);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int64_t t0 = (int64_t)blockIdx.x * p.rows_up;
  const int rows = (int)min((int64_t)p.rows_up, p.T - t0);
  const Runs runs(p, t0, rows);
  const int i_step = gridDim.y * kWarps * kOut;
  const int i_first = (blockIdx.y * kWarps + warp) * kOut;

  {  // B of the first run and y of its row, ahead of the wait for u
    int end;
    const int a = runs.run(0, end);
    if (a >= 0 && i_first < p.N) {
      const char *b = reinterpret_cast<const char *>(p.b + a * p.b_adapter +
                                                     (int64_t)i_first * p.b_row);
      const int64_t bytes = (int64_t)(min(kOut, p.N - i_first) - 1) * p.b_row * 2 + p.R * 2;
      for (int64_t o = lane * 128; o < bytes; o += 32 * 128)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(b + o));
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // One warp a row: sum of the slices, largest magnitude, two fp16 parts.
  for (int t = warp; t < rows; t += kWarps) {
    const int a = __shfl_sync(0xffffffffu, runs.adapter, t);
    if (a < 0) continue;
    const int rank = rank_of(p, a);
    float v[4], mx = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // R <= 128
      const int r = lane + 32 * q;
      v[q] = 0.0f;
      if (r < rank) {
        const float *u = p.u + (t0 + t) * p.Rp + r;
        for (int s = 0; s < p.slices; ++s) v[q] += __ldcg(u + (int64_t)s * p.T * p.Rp);
      }
      mx = fmaxf(mx, fabsf(v[q]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^e brings the largest into [2^9, 2^10); |e| <= 126 keeps both powers normal
    int e = mx > 0.0f ? 10 - ilogbf(mx) - 1 : 0;
    e = min(max(e, -126), 126);
    const float up = __int_as_float((127 + e) << 23), down = __int_as_float((127 - e) << 23);
    if (lane == 0) fs[t] = down * __ldg(p.scale + a);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = lane + 32 * q;
      if (r < Rk) {
        const float w = v[q] * up;
        const __half h = __float2half_rn(w);
        uh[t * pitch + r] = h;
        ul[t * pitch + r] = __float2half_rn(w - __half2float(h));
      }
    }
  }
  __syncthreads();

  for (int i0 = i_first; i0 < p.N; i0 += i_step) {
    const int i = i0 + g * 8;  // this thread's 8 outputs
    for (int at = 0, end; at < rows; at = end) {
      const int a = runs.run(at, end);
      const int rank = a < 0 ? 0 : rank_of(p, a);
      const __half *B = p.b + (a < 0 ? 0 : a) * p.b_adapter;
      for (int n0 = at; n0 < end; n0 += 16) {  // 2 x 8 rows at a time
        uint4 yv[2][2];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = n0 + 8 * n + 2 * tig + k;
            yv[n][k] = t < end ? load8<VEC>(p.y + (t0 + t) * p.ldy, i, p.N) : make_uint4(0, 0, 0, 0);
          }
        float c[2][4][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) c[n][j][q] = 0.0f;
        for (int r0 = 0; r0 < rank; r0 += 32) {
          const int r = r0 + 8 * tig;
          uint4 bv[4][2];
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              bv[j][k] = i + 2 * j + k < p.N
                             ? load8<VEC>(B + (int64_t)(i + 2 * j + k) * p.b_row, r, rank)
                             : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            if (n0 + 8 * n >= end) break;
            const int t = min(n0 + 8 * n + g, rows - 1);  // columns past the run are not stored
            const uint4 hv = *reinterpret_cast<const uint4 *>(uh + t * pitch + r);
            const uint4 lv = *reinterpret_cast<const uint4 *>(ul + t * pitch + r);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              mma16816(c[n][j], bv[j][0].x, bv[j][1].x, bv[j][0].y, bv[j][1].y, hv.x, hv.y);
              mma16816(c[n][j], bv[j][0].z, bv[j][1].z, bv[j][0].w, bv[j][1].w, hv.z, hv.w);
              mma16816(c[n][j], bv[j][0].x, bv[j][1].x, bv[j][0].y, bv[j][1].y, lv.x, lv.y);
              mma16816(c[n][j], bv[j][0].z, bv[j][1].z, bv[j][0].w, bv[j][1].w, lv.z, lv.w);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = n0 + 8 * n + 2 * tig + k;
            if (t >= end || i >= p.N) continue;
            uint4 o = yv[n][k];
            if (a >= 0) {
              const float f = fs[t];
              uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 yy = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
                w[j] = pack2(__float2half_rn(fmaf(f, c[n][j][k], yy.x)),
                             __float2half_rn(fmaf(f, c[n][j][2 + k], yy.y)));
              }
              o = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __half *dst = p.out + (t0 + t) * p.ldo + i;
            if (VEC && i + 8 <= p.N) {
              *reinterpret_cast<uint4 *>(dst) = o;
            } else {
              const uint32_t w[4] = {o.x, o.y, o.z, o.w};
              for (int q = 0; q < 8 && i + q < p.N; ++q)
                dst[q] = __ushort_as_half((unsigned short)(w[q >> 1] >> (16 * (q & 1))));
            }
          }
      }
    }
  }
}

bool rows16(const void *p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

int pow2_at_least(int64_t v, int hi) {
  int r = 1;
  while (r < v && r < hi) r *= 2;
  return r;
}

int padded_rank(int64_t R) { return (int)((R + 15) / 16 * 16); }

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t K, int64_t R) {
  const int64_t slices = (K + kSlice - 1) / kSlice;
  return (size_t)((slices < kMaxSlices ? slices : kMaxSlices) * (T > 0 ? T : 1) * padded_rank(R)) *
         sizeof(float);
}

qz_status launch_lora(const qz_lora_adapters &ad, const int32_t *index, int64_t T, const __half *x,
                      int64_t ldx, const __half *y, int64_t ldy, __half *out, int64_t ldo,
                      void *workspace, cudaStream_t s) {
  DeviceInfo di;
  const qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  LoraParams p;
  p.a = reinterpret_cast<const __half *>(ad.a);
  p.b = reinterpret_cast<const __half *>(ad.b);
  p.x = x;
  p.y = y;
  p.out = out;
  p.scale = ad.scale;
  p.rank = ad.rank;
  p.index = index;
  p.n_adapters = (int)ad.n_adapters;
  p.R = (int)ad.R;
  p.Rp = padded_rank(ad.R);
  p.K = (int)ad.K;
  p.N = (int)ad.N;
  p.T = T;
  p.a_adapter = ad.a_adapter;
  p.a_row = ad.a_row;
  p.b_adapter = ad.b_adapter;
  p.b_row = ad.b_row;
  p.ldx = ldx;
  p.ldy = ldy;
  p.ldo = ldo;
  p.u = static_cast<float *>(workspace);
  // Slices of K: as many as there are steps of kSlice, at most kMaxSlices.
  const int64_t steps = (ad.K + kSlice - 1) / kSlice;
  p.slices = (int)(steps < kMaxSlices ? steps : kMaxSlices);
  p.k_slice = (int)((steps + p.slices - 1) / p.slices) * kSlice;
  p.slices = (int)((ad.K + p.k_slice - 1) / p.k_slice);
  // Rows per CTA: one while that still leaves few CTAs per SM (a decode step's
  // adapters are read by the whole GPU at once), more as calls grow, so that a
  // run's adapter is read by fewer CTAs.
  const int64_t want = (int64_t)di.sms * 4;
  const int cap = kRowRanks / p.Rp < kMaxRows ? kRowRanks / p.Rp : kMaxRows;
  p.rows_down = pow2_at_least((T * p.slices + want - 1) / want, cap);
  const int64_t chunks = (ad.N + kOut * kWarps - 1) / (kOut * kWarps);
  p.rows_up = pow2_at_least((T * chunks + want - 1) / want, kMaxRows);
  const bool va = rows16(p.a, p.a_row) && p.a_adapter % 8 == 0 && rows16(x, ldx) && p.K % 8 == 0;
  const bool vb = rows16(p.b, p.b_row) && p.b_adapter % 8 == 0 && rows16(y, ldy) && rows16(out, ldo);

  const int down_sm = kWarps * p.rows_down * p.Rp * (int)sizeof(float);
  auto down = va ? lora_down_kernel<true> : lora_down_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (down_sm > 48 * 1024)
    e = cudaFuncSetAttribute(down, cudaFuncAttributeMaxDynamicSharedMemorySize, down_sm);
  if (e != cudaSuccess) return cuda_status(e);
  const dim3 gd((unsigned)((T + p.rows_down - 1) / p.rows_down), (unsigned)p.slices);
  down<<<gd, kThreads, down_sm, s>>>(p);
  qz_status launched = launch_status();
  if (launched != QZ_OK) return launched;

  const int pitch = (p.R + 31) / 32 * 32 + 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((T + p.rows_up - 1) / p.rows_up), (unsigned)chunks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)p.rows_up * (2 * pitch * sizeof(__half) + sizeof(float));
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, vb ? lora_up_kernel<true> : lora_up_kernel<false>, p));
}

qz_status read_lora_error(int *code, int clear) {
  return read_error_word(g_lora_error, code, clear);
}

}  // namespace qz
