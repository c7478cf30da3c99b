// Low-rank adapters beside a shared projection: out = y + s_a B_a (A_a x).
//
// Two products over the same rows, on warp-level matrix instructions (rank and
// run lengths are far below a tcgen05 tile):
//   down: u = A_a x.  A CTA takes a few rows and a slice of K; neighbouring rows
//     of one adapter (a run) are the 8 columns of m16n8k16 products whose 16
//     rows are ranks, so one request a run wastes columns, not reads.  Its 8
//     warps split the slice and add up through shared memory, the slices of a
//     row are a cluster and add up through distributed shared memory, always in
//     the same order.
//   up: B_a u.  A CTA keeps its rows' u in shared memory; a warp takes 64 outputs
//     at a time.  The launch overlaps the first one, and its first B and y are on
//     their way before u is.
// Precision of u: its fp32 sum is scaled by a power of two per row (any fp32
// range) and enters the second product as two fp16 parts, which hold it to 22 bits of
// the row's largest.  One part would be off by up to 2^-11 of it, as much as out's own
// rounding at every K; it took 48.4 us where two take 52.8 (1500 rows of ranks up to 64,
// below), 10.4 for 11.3 (32 rows of rank 16).
// In both, a thread's 16-byte load holds 8 consecutive k of its fragment row:
// the two operands use the same order of k, so no shuffle is needed; likewise the
// rows of B_a are dealt so that a thread ends with 8 consecutive outputs.
// Operands without 16-byte rows take the same path with 2-byte loads.
//
// From kOrderRows rows on, the rows are sorted by adapter first (a third launch, which
// the others overlap), so that an adapter is read for up to 32 of its rows at once
// however they come.
//
// Measured (GB300): 32 rows of 32 adapters of rank 16, 8192 x 8192: 11.3 us with the
// adapters in the L2 (down 5, up 3.5 after it), 13 without; the chain index, adapter,
// products, cluster, u, products is latency.  1500 rows of 8 adapters of ranks up to 64 in runs of 300,
// 4096 x 11008: 52.5-55.8 us by GPU, 2 of them the sort, down 19 (one wave of CTAs with fewer
// slices takes as long), up the rest: each step of 64 outputs waits for its own loads
// (about half of its 4 us; a product is 8 clocks of a scheduler, so the matrix
// instructions are a fifth of the time), twice in the few row tiles that two runs
// share.  1500 rows of 48 adapters of rank 16 in turn: 50.3 us.
#include "lora_plan.h"
#include "qz_internal.cuh"

namespace qz {
namespace {

__device__ int g_lora_error = 0;

constexpr int kWarps = kLoraWarps, kUpWarps = kLoraUpWarps, kSub = kLoraSub, kSlice = kLoraSlice;
constexpr int kMaxRows = kLoraMaxRows, kOut = kLoraOut, kMaxSlices = kLoraMaxSlices;
constexpr int kThreads = 32 * kWarps;       // down
// Rows from which they are sorted first.  Unsorted and sorted, rows in turn: 1500 of 48
// adapters, rank 16, 4096 x 11008: 275 and 50.2 us; 128 of 16, rank 64: 50.1 and 21.0;
// 128 of 128, rank 16, 4096 x 4096: 19.7 and 21.5; 64 of 4: 13.0 and 12.0.  Rows that come
// grouped pay 1.6 us for it (1500 in runs of 300: 50.9 and 52.5).
constexpr int64_t kOrderRows = 128;
constexpr int kBins = 1024;                 // of the sort by adapter
constexpr int kSegment = 2048;              // rows sorted together

struct LoraParams {
  const __half *a, *b, *x, *y;
  __half *out;
  const float *scale;
  const int32_t *rank, *index;
  int n_adapters, R, Rp, Rk, K, N;  // Rp, Rk: R rounded up to 16 and 32
  int64_t T, a_adapter, a_row, b_adapter, b_row, ldx, ldy, ldo;
  __half *uh, *ul;  // [T][Rk] u 2^e and its remainder
  int2 *order;      // [T] (row, index) sorted by adapter, or null: rows as they come
  float *fs;        // [T] scale_a 2^-e
  int slices;
  int k_slice;    // k per CTA (a multiple of kSlice)
  int rows_down, rows_up;
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
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
  int64_t row;      // of x, y and out, for this lane's place
  int adapter;      // of this lane's row
  unsigned starts;  // run starts, and one bit at n (if n < 32)
  int n;
  __device__ __forceinline__ Runs(const LoraParams &p, int64_t t0, int rows) : n(rows) {
    const int lane = threadIdx.x & 31;
    int raw = -1;
    row = t0 + lane;
    if (lane < n) {
      if (p.order) {
        const int2 v = __ldcg(p.order + t0 + lane);
        row = v.x;
        raw = v.y;
      } else {
        raw = __ldg(p.index + t0 + lane);
      }
    }
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
  // The row at place t (a place past the end: that of the last).
  __device__ __forceinline__ int64_t row_at(int t) const {
    return __shfl_sync(0xffffffffu, (int)row, min(t, n - 1));
  }
};

// Rows of a segment sorted by adapter, so that the CTAs below read an adapter
// once for many of them however the rows come (a counting sort; adapters that
// share a bin only make more runs).  The order within a bin is that in which
// warps arrive: no row's sums depend on it.
__global__ void __launch_bounds__(1024) lora_order_kernel(const LoraParams p) {
  __shared__ int count[kBins];
  __shared__ int warp_sum[32];
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  count[tid] = 0;
  __syncthreads();
  int raw[kSegment / 1024], bin[kSegment / 1024], at[kSegment / 1024];
  const int64_t t0 = (int64_t)blockIdx.x * kSegment + tid;
#pragma unroll
  for (int i = 0; i < kSegment / 1024; ++i)
    raw[i] = t0 + i * 1024 < p.T ? __ldg(p.index + t0 + i * 1024) : -1;
#pragma unroll
  for (int i = 0; i < kSegment / 1024; ++i) {
    const bool on = t0 + i * 1024 < p.T;
    bin[i] = !on ? kBins : raw[i] >= 0 && raw[i] < p.n_adapters ? (raw[i] + 1) & (kBins - 1) : 0;
    const unsigned same = __match_any_sync(0xffffffffu, bin[i]);
    const int first = __ffs(same) - 1;
    at[i] = on && lane == first ? atomicAdd(count + bin[i], __popc(same)) : 0;
    at[i] = __shfl_sync(0xffffffffu, at[i], first) + __popc(same & ((1u << lane) - 1));
  }
  __syncthreads();
  const int own = count[tid];
  int sum = own;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int v = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += v;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  if (warp == 0) {
    int v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  count[tid] = sum - own + (warp > 0 ? warp_sum[warp - 1] : 0);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSegment / 1024; ++i)
    if (t0 + i * 1024 < p.T)
      p.order[(int64_t)blockIdx.x * kSegment + count[bin[i]] + at[i]] =
          make_int2((int)(t0 + i * 1024), raw[i]);
}

__device__ __forceinline__ int rank_of(const LoraParams &p, int a) {
  return p.rank ? min(max(__ldg(p.rank + a), 0), p.R) : p.R;
}

__device__ __forceinline__ float ld_cluster(uint32_t addr, int rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [a];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// NT: 8-row column tiles of a CTA (1: at most 8 rows, where latency counts and
// the registers hold more of K at a time; 4: up to 32 rows).
template <bool VEC, int NT>
__global__ void __launch_bounds__(kThreads, 2) lora_down_kernel(const LoraParams p) {
  extern __shared__ float part[];  // [kWarps][rows][Rp]
  // The up product starts once every CTA is past this: the order is then complete.
  if (p.order) asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int MT = NT == 1 ? 2 : 1, KU = NT == 1 ? 2 : 1;  // 16-rank tiles, steps of K at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int64_t t0 = (int64_t)blockIdx.x * p.rows_down;
  const int rows = (int)min((int64_t)p.rows_down, p.T - t0);
  const int k_begin = blockIdx.y * p.k_slice, k_end = min(k_begin + p.k_slice, p.K);
  const Runs runs(p, t0, rows);
  const uint4 z = make_uint4(0, 0, 0, 0);
  for (int at = 0, end; at < rows; at = end) {
    const int a = runs.run(at, end);
    if (a < 0) continue;
    const int rank = rank_of(p, a);
    const __half *A = p.a + a * p.a_adapter + g * p.a_row;
    const __half *X[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) X[n] = p.x + runs.row_at(at + 8 * n + g) * p.ldx;
    for (int m0 = 0; m0 < rank; m0 += 16 * MT) {
      float c[MT][NT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) c[m][n][i] = 0.0f;
      for (int k0 = k_begin + warp * kSub; k0 < k_end; k0 += KU * kSlice) {
        uint4 av[KU][2][MT][2], xv[KU][2][NT];
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = k0 + u * kSlice + 32 * h + 8 * tig;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r = m0 + 16 * m + 8 * i;
                av[u][h][m][i] = r + g < rank ? load8<VEC>(A + r * p.a_row, k, k_end) : z;
              }
#pragma unroll
            for (int n = 0; n < NT; ++n)
              xv[u][h][n] = at + 8 * n + g < end ? load8<VEC>(X[n], k, k_end) : z;
          }
#pragma unroll
        for (int u = 0; u < KU; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              if (n > 0 && at + 8 * n >= end) break;
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                const uint4 a0 = av[u][h][m][0], a1 = av[u][h][m][1], b = xv[u][h][n];
                mma16816(c[m][n], a0.x, a1.x, a0.y, a1.y, b.x, b.y);
                mma16816(c[m][n], a0.z, a1.z, a0.w, a1.w, b.z, b.w);
              }
            }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = at + 8 * n + 2 * tig + (i & 1), r = m0 + 16 * m + g + (i & 2 ? 8 : 0);
            if (t < end && r < rank) part[(warp * rows + t) * p.Rp + r] = c[m][n][i];
          }
    }
  }
  __syncthreads();
  // ranks past an adapter's own, and rows without one, are never written or read
  for (int i = threadIdx.x; i < rows * p.Rp; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += part[w * rows * p.Rp + i];
    part[i] = v;  // this thread alone reads and writes element i
  }
  if (p.slices > 1) cluster_sync();
  else __syncthreads();
  // One warp a row: sum of the slices, largest magnitude, two fp16 parts.
  const uint32_t sums = (uint32_t)__cvta_generic_to_shared(part);
  for (int t = blockIdx.y + p.slices * warp; t < rows; t += p.slices * kWarps) {
    const int a = __shfl_sync(0xffffffffu, runs.adapter, t);
    if (a < 0) continue;
    const int rank = rank_of(p, a);
    float v[4], mx = 0.0f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {  // R <= 128
      const int r = lane + 32 * q;
      v[q] = 0.0f;
      if (r < rank) {
#pragma unroll
        for (int s = 0; s < kMaxSlices; ++s)
          if (s < p.slices) v[q] += ld_cluster(sums + (t * p.Rp + r) * 4, s);
      }
      mx = fmaxf(mx, fabsf(v[q]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    // 2^e brings the largest into [2^9, 2^10); |e| <= 126 keeps both powers normal
    int e = mx > 0.0f ? 9 - ilogbf(mx) : 0;
    e = min(max(e, -126), 126);
    const float up = __int_as_float((127 + e) << 23), down = __int_as_float((127 - e) << 23);
    if (lane == 0) p.fs[t0 + t] = down * __ldg(p.scale + a);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = lane + 32 * q;
      if (r < p.Rk) {
        const float w = v[q] * up;
        const __half h = __float2half_rn(w);
        p.uh[(t0 + t) * p.Rk + r] = h;
        p.ul[(t0 + t) * p.Rk + r] = __float2half_rn(w - __half2float(h));
      }
    }
  }
  if (p.slices > 1) cluster_sync();  // the others may still read this CTA's sums
}

__device__ __forceinline__ uint4 ld_cg16(const __half *p) {
  return __ldcg(reinterpret_cast<const uint4 *>(p));
}

// y + f c of a row's 8 outputs (row k of the products' two), rounded once.
__device__ __forceinline__ uint4 add_rows(uint4 y, float f, const float (&c)[4][4], int k) {
  uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 yy = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
    const __half2 h = __floats2half2_rn(fmaf(f, c[j][k], yy.x), fmaf(f, c[j][2 + k], yy.y));
    w[j] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// RC: 32-rank groups of B_a that a thread holds at a time; NN: 8-row column
// tiles at a time.
template <bool VEC, int RC, int NN>
__global__ void __launch_bounds__(32 * kUpWarps, lora_up_ctas(RC, NN))
    lora_up_kernel(const LoraParams p) {
  // [2][rows][pitch]: the parts of u, rows padded against bank conflicts
  extern __shared__ __align__(16) uint8_t sm[];
  const int pitch = p.Rk + 8;
  int64_t *y_at = reinterpret_cast<int64_t *>(sm), *out_at = y_at + kMaxRows;  // rows' offsets
  float *fs = reinterpret_cast<float *>(out_at + kMaxRows);
  __half *uh = reinterpret_cast<__half *>(fs + kMaxRows);
  __half *ul = uh + p.rows_up * pitch;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tig = lane & 3;
  const int64_t t0 = (int64_t)blockIdx.x * p.rows_up;
  const int rows = (int)min((int64_t)p.rows_up, p.T - t0);
  const Runs runs(p, t0, rows);
  if (threadIdx.x < rows) {
    y_at[threadIdx.x] = runs.row * p.ldy;
    out_at[threadIdx.x] = runs.row * p.ldo;
  }
  __syncthreads();
  const uint4 z = make_uint4(0, 0, 0, 0);
  bool ready = false;  // u is in shared memory
  for (int i0 = (blockIdx.y * kUpWarps + warp) * kOut; !ready || i0 < p.N;
       i0 += gridDim.y * kUpWarps * kOut) {
    const int i = i0 + g * 8;               // this thread's 8 outputs
    const bool all = VEC && i0 + kOut <= p.N;  // all of the warp's exist
    // y of the next step on its way to the L2 (calls of more rows 50.0 -> 48.5 us;
    // few rows have few steps, and 32 of them took 10.7 -> 11.1)
    if (const int next = i0 + gridDim.y * kUpWarps * kOut; NN == 2 && next < p.N && lane < rows)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.y + y_at[lane] + next));
    for (int at = 0, end; at < rows; at = end) {
      const int a = runs.run(at, end);
      const int rank = a < 0 ? 0 : rank_of(p, a);
      const __half *B = p.b + (a < 0 ? 0 : a) * p.b_adapter + (int64_t)i * p.b_row + 8 * tig;
      uint4 bv[RC][4][2];
      auto load_b = [&](int r0) {
#pragma unroll
        for (int q = 0; q < RC; ++q) {
          const int r = r0 + 32 * q;
          const __half *row = B + r;
          if (all && (rank & 7) == 0) {
            const bool on = r + 8 * tig < rank;
#pragma unroll
            for (int j = 0; j < 8; ++j, row += p.b_row)
              bv[q][j >> 1][j & 1] = on ? __ldg(reinterpret_cast<const uint4 *>(row)) : z;
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j, row += p.b_row)
              bv[q][j >> 1][j & 1] = i + j < p.N ? load8<VEC>(row, 0, rank - r - 8 * tig) : z;
          }
        }
      };
      // rows 2 tig + {0, 1} of a column tile
      auto load_y = [&](int n0, uint4 (&yv)[NN][2]) {
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = n0 + 8 * n + 2 * tig + k;
            yv[n][k] = z;
            if (t < end) {
              const __half *src = p.y + y_at[t] + i;
              yv[n][k] = all ? __ldg(reinterpret_cast<const uint4 *>(src))
                             : load8<VEC>(src, 0, p.N - i);
            }
          }
      };
      uint4 yv[NN][2];
      load_y(at, yv);
      if (rank > 0) load_b(0);
      if (!ready) {  // u comes from the launch before
        ready = true;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const int per = p.Rk / 8;  // 16-byte pieces a row
        for (int e = threadIdx.x; e < rows * per; e += 32 * kUpWarps) {
          const int t = e / per, c = (e - t * per) * 8;
          const int64_t src = (t0 + t) * p.Rk + c;
          *reinterpret_cast<uint4 *>(uh + t * pitch + c) = ld_cg16(p.uh + src);
          *reinterpret_cast<uint4 *>(ul + t * pitch + c) = ld_cg16(p.ul + src);
        }
        if (threadIdx.x < rows) fs[threadIdx.x] = __ldcg(p.fs + t0 + threadIdx.x);
        __syncthreads();
      }
      // Whole tiles of rows and outputs, whose ranks are in registers: no bounds.
      int n0 = at;
      if (all && rank > 0 && rank <= 32 * RC) {
        const __half *u = uh + (at + g) * pitch + 8 * tig;
        const float *f = fs + at + 2 * tig;
        for (; n0 + 8 * NN <= end; n0 += 8 * NN, u += 8 * NN * pitch, f += 8 * NN) {
          float c[NN][4][4];
#pragma unroll
          for (int q = 0; q < RC; ++q) {
            if (q > 0 && 32 * q >= rank) break;
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              const uint4 hv = *reinterpret_cast<const uint4 *>(u + 8 * n * pitch + 32 * q);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 b0 = bv[q][j][0], b1 = bv[q][j][1];
                if (q == 0) mma16816_first(c[n][j], b0.x, b1.x, b0.y, b1.y, hv.x, hv.y);
                else mma16816(c[n][j], b0.x, b1.x, b0.y, b1.y, hv.x, hv.y);
                mma16816(c[n][j], b0.z, b1.z, b0.w, b1.w, hv.z, hv.w);
              }
              const uint4 lv = *reinterpret_cast<const uint4 *>(u + 8 * n * pitch + 32 * q +
                                                                p.rows_up * pitch);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 b0 = bv[q][j][0], b1 = bv[q][j][1];
                mma16816(c[n][j], b0.x, b1.x, b0.y, b1.y, lv.x, lv.y);
                mma16816(c[n][j], b0.z, b1.z, b0.w, b1.w, lv.z, lv.w);
              }
            }
          }
          uint4 o[NN][2];
#pragma unroll
          for (int n = 0; n < NN; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) o[n][k] = add_rows(yv[n][k], f[8 * n + k], c[n], k);
          if (n0 + 8 * NN < end) load_y(n0 + 8 * NN, yv);
#pragma unroll
          for (int n = 0; n < NN; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              *reinterpret_cast<uint4 *>(p.out + out_at[n0 + 8 * n + 2 * tig + k] + i) = o[n][k];
        }
      }
      for (; n0 < end; n0 += 8 * NN) {
        float c[NN][4][4];
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) c[n][j][q] = 0.0f;
        for (int r0 = 0; r0 < rank; r0 += 32 * RC) {
          if (rank > 32 * RC && (r0 > 0 || n0 > at)) load_b(r0);
#pragma unroll
          for (int q = 0; q < RC; ++q) {
            if (r0 + 32 * q >= rank) break;
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              if (n > 0 && n0 + 8 * n >= end) break;
              // columns past the run repeat its last row and are not stored
              const int u = min(n0 + 8 * n + g, end - 1) * pitch + r0 + 32 * q + 8 * tig;
              const uint4 hv = *reinterpret_cast<const uint4 *>(uh + u);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 b0 = bv[q][j][0], b1 = bv[q][j][1];
                mma16816(c[n][j], b0.x, b1.x, b0.y, b1.y, hv.x, hv.y);
                mma16816(c[n][j], b0.z, b1.z, b0.w, b1.w, hv.z, hv.w);
              }
              const uint4 lv = *reinterpret_cast<const uint4 *>(ul + u);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 b0 = bv[q][j][0], b1 = bv[q][j][1];
                mma16816(c[n][j], b0.x, b1.x, b0.y, b1.y, lv.x, lv.y);
                mma16816(c[n][j], b0.z, b1.z, b0.w, b1.w, lv.z, lv.w);
              }
            }
          }
        }
        uint4 o[NN][2];
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            o[n][k] = yv[n][k];
            if (a >= 0)
              o[n][k] = add_rows(yv[n][k], fs[min(n0 + 8 * n + 2 * tig + k, rows - 1)], c[n], k);
          }
        if (n0 + 8 * NN < end) load_y(n0 + 8 * NN, yv);
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = n0 + 8 * n + 2 * tig + k;
            if (t >= end) continue;
            __half *dst = p.out + out_at[t] + i;
            if (all) {
              *reinterpret_cast<uint4 *>(dst) = o[n][k];
            } else {
              const uint32_t w[4] = {o[n][k].x, o[n][k].y, o[n][k].z, o[n][k].w};
              for (int q = 0; q < 8 && i + q < p.N; ++q)
                dst[q] = __ushort_as_half((unsigned short)(w[q >> 1] >> (16 * (q & 1))));
            }
          }
      }
    }
  }
}

bool rows16(const void *p, int64_t ld) { return ((uintptr_t)p & 15u) == 0 && ld % 8 == 0; }

template <bool VEC, int NT>
cudaError_t launch_down(const LoraParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3((unsigned)((p.T + p.rows_down - 1) / p.rows_down), (unsigned)p.slices);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)kWarps * p.rows_down * p.Rp * sizeof(float);
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = (unsigned)p.slices;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.order ? 2 : 1;  // it waits itself for the rows' order
  const cudaError_t e = allow_smem<lora_down_kernel<VEC, NT>>(cfg.dynamicSmemBytes);
  return e != cudaSuccess ? e : cudaLaunchKernelEx(&cfg, lora_down_kernel<VEC, NT>, p);
}

template <bool VEC, int RC, int NN>
cudaError_t launch_up(const LoraParams &p, int ctas_n, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  cfg.gridDim = dim3((unsigned)((p.T + p.rows_up - 1) / p.rows_up), (unsigned)ctas_n);
  cfg.blockDim = dim3(32 * kUpWarps);
  cfg.dynamicSmemBytes = kMaxRows * (2 * sizeof(int64_t) + sizeof(float)) +
                         (size_t)p.rows_up * 2 * (p.Rk + 8) * sizeof(__half);
  cfg.stream = s;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, lora_up_kernel<VEC, RC, NN>, p);
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t, int64_t R) {
  const int64_t Rk = (R + 31) / 32 * 32, rows = T > 0 ? T : 1;
  return (size_t)(rows * Rk) * 2 * sizeof(__half) + (size_t)rows * (sizeof(int2) + sizeof(float));
}

qz_status launch_lora(const qz_lora_adapters &ad, const int32_t *index, int64_t T, const __half *x,
                      int64_t ldx, const __half *y, int64_t ldy, __half *out, int64_t ldo,
                      void *workspace, cudaStream_t s) {
  DeviceInfo di;
  const qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  const LoraPlan plan = lora_plan(T, ad.K, ad.N, ad.R, di.sms);
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
  p.Rp = plan.Rp;
  p.Rk = plan.Rk;
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
  p.uh = static_cast<__half *>(workspace);
  p.ul = p.uh + T * p.Rk;
  p.order = reinterpret_cast<int2 *>(p.ul + T * p.Rk);
  p.fs = reinterpret_cast<float *>(p.order + T);
  if (T < kOrderRows || ad.n_adapters < 2) p.order = nullptr;
  p.slices = plan.slices;
  p.k_slice = plan.k_slice;
  p.rows_down = plan.rows_down;
  p.rows_up = plan.rows_up;
  const int n = plan.along_n;
  const bool va = rows16(p.a, p.a_row) && p.a_adapter % 8 == 0 && rows16(x, ldx) && p.K % 8 == 0;
  const bool vb =
      rows16(p.b, p.b_row) && p.b_adapter % 8 == 0 && rows16(y, ldy) && rows16(out, ldo);

  cudaError_t e;
  if (p.order) {
    lora_order_kernel<<<(unsigned)((T + kSegment - 1) / kSegment), 1024, 0, s>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return cuda_status(e);
  }
  if (p.rows_down <= 8)
    e = va ? launch_down<true, 1>(p, s) : launch_down<false, 1>(p, s);
  else
    e = va ? launch_down<true, 4>(p, s) : launch_down<false, 4>(p, s);
  if (e != cudaSuccess) return cuda_status(e);
  // B_a of up to 64 ranks stays in registers for a run's rows
  if (p.rows_up <= 8)
    e = p.R <= 32 ? (vb ? launch_up<true, 1, 1>(p, n, s) : launch_up<false, 1, 1>(p, n, s))
                  : (vb ? launch_up<true, 2, 1>(p, n, s) : launch_up<false, 2, 1>(p, n, s));
  else
    e = p.R <= 32 ? (vb ? launch_up<true, 1, 2>(p, n, s) : launch_up<false, 1, 2>(p, n, s))
                  : (vb ? launch_up<true, 2, 2>(p, n, s) : launch_up<false, 2, 2>(p, n, s));
  return cuda_status(e);
}

qz_status read_lora_error(int *code, int clear) {
  return read_error_word(g_lora_error, code, clear);
}

}  // namespace qz
