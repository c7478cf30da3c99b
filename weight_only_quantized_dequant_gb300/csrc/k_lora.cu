// Low-rank adapters beside a shared projection: out = y + s_a B_a (A_a x).
//
// Two launches: u = A_a x per row (one warp per (row, r)), then the rows of
// B_a against u (one thread per output).  u is fp32 in the workspace.
#include "qz_internal.cuh"

namespace qz {
namespace {

__device__ int g_lora_error = 0;

constexpr int kWarps = 4;

struct LoraParams {
  qz_lora_adapters ad;
  const int32_t *index;
  int64_t T;
  const __half *x, *y;
  __half *out;
  int64_t ldx, ldy, ldo;
  float *u;  // [T][R]
};

__device__ __forceinline__ int adapter_of(const LoraParams &p, int64_t t) {
  const int a = __ldg(p.index + t);
  return a >= 0 && a < p.ad.n_adapters ? a : -1;
}
__device__ __forceinline__ int rank_of(const LoraParams &p, int a) {
  return p.ad.rank ? min(max(__ldg(p.ad.rank + a), 0), (int)p.ad.R) : (int)p.ad.R;
}

__global__ void __launch_bounds__(32 * kWarps) lora_down_kernel(const LoraParams p) {
  const int64_t t = blockIdx.x;
  const int r = blockIdx.y * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= p.ad.R) return;
  const int raw = __ldg(p.index + t), a = adapter_of(p, t);
  if (a < 0) {
    if (raw != -1 && lane == 0) atomicOr(&g_lora_error, 4);
    return;
  }
  float u = 0.0f;
  if (r < rank_of(p, a)) {
    const __half *A = reinterpret_cast<const __half *>(p.ad.a) + a * p.ad.a_adapter + r * p.ad.a_row;
    for (int64_t j = lane; j < p.ad.K; j += 32)
      u = fmaf(__half2float(A[j]), __half2float(p.x[t * p.ldx + j]), u);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) u += __shfl_xor_sync(0xffffffffu, u, s);
  if (lane == 0) p.u[t * p.ad.R + r] = u;
}

__global__ void __launch_bounds__(128) lora_up_kernel(const LoraParams p) {
  const int64_t t = blockIdx.x, i = (int64_t)blockIdx.y * 128 + threadIdx.x;
  if (i >= p.ad.N) return;
  const int a = adapter_of(p, t);
  float v = __half2float(p.y[t * p.ldy + i]);
  if (a >= 0) {
    const __half *B = reinterpret_cast<const __half *>(p.ad.b) + a * p.ad.b_adapter + i * p.ad.b_row;
    float d = 0.0f;
    const int n = rank_of(p, a);
    for (int r = 0; r < n; ++r) d = fmaf(__half2float(B[r]), p.u[t * p.ad.R + r], d);
    v = fmaf(__ldg(p.ad.scale + a), d, v);
  }
  p.out[t * p.ldo + i] = __float2half_rn(v);
}

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t, int64_t R) {
  return (size_t)((T > 0 ? T : 1) * R) * sizeof(float);
}

qz_status launch_lora(const qz_lora_adapters &ad, const int32_t *index, int64_t T, const __half *x,
                      int64_t ldx, const __half *y, int64_t ldy, __half *out, int64_t ldo,
                      void *workspace, cudaStream_t s) {
  const LoraParams p = {ad, index, T, x, y, out, ldx, ldy, ldo, static_cast<float *>(workspace)};
  lora_down_kernel<<<dim3((unsigned)T, (unsigned)((ad.R + kWarps - 1) / kWarps)), 32 * kWarps, 0,
                     s>>>(p);
  lora_up_kernel<<<dim3((unsigned)T, (unsigned)((ad.N + 127) / 128)), 128, 0, s>>>(p);
  return launch_status();
}

qz_status read_lora_error(int *code, int clear) {
  return read_error_word(g_lora_error, code, clear);
}

}  // namespace qz
