// The attention kernel on the 5th-generation tensor cores, over a paged cache of
// fp16 rows (k_attn.cu) or of INT8 rows (k_attn8_tc.cu, Q8 below).
#pragma once

#include <cfloat>
#include <cmath>
#include <cstring>

#include "attn_plan.cuh"

namespace qz {
namespace {

constexpr int kSoftmaxWarps = 8;       // two warpgroups
// With few rows only softmax warps 0 and 4 have any, both on the SM's first
// scheduler: the MMA and load warps sit on others.
constexpr int kQWarp = 8, kMmaWarp = 10, kLoadWarp = 11;  // 8 and 9: queries
constexpr int kThreads = 384;          // the third warpgroup: queries (2), MMA, keys and values
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // of 168 a thread at launch
static_assert(8 * kSoftmaxRegs + 4 * kOtherRegs <= 12 * 168, "register split");
constexpr int kBars = 4096;             // barriers and exchange rows at the start of shared memory
constexpr int kOutBytes = 32 * 64;     // per softmax warp: 32 rows x 32 outputs on their way out
constexpr int kHead = kBars + 8 * kOutBytes;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr int kScaleBlocks = 8;        // INT8 rows: key blocks whose scales are kept
// What is kept of them: factors of the logits and weights [2][kN], bounds of the former
// [4][2], and the fp16 parts of the values' [kN].
constexpr int kScaleSet = 2 * kN * 4 + 32 + kN * 2;
constexpr int kScaleBytes = (kScaleBlocks * kScaleSet + 1023) / 1024 * 1024;
constexpr float kLift = 7.0f;          // log2 of the weight at m
static_assert(kLag + kLift < 16.0f - 0.1f, "weights are fp16 (INT8 rows: times at most 17/16)");

template <int D, int NQ, bool Q8>
struct Cfg {
  // A slot's codes arrive in its upper half, where a thread turns a row into fp16 in place:
  // the row's last 128 bytes are its own codes' (D 64: behind the slot's fp16 rows).
  static constexpr int kCodes = D == 64 ? kN * D * 2 : kN * D;
  static constexpr int kM = 128 * NQ;                  // rows of a tile
  static constexpr int kStage = kN * D * 2 + (Q8 && D == 64 ? kN * D : 0);  // a K or V block
  static constexpr int kQ = kM * D * 2;
  static constexpr int kNS = D == 256 ? 2 : D == 64 ? (Q8 ? 6 : 8) : NQ == 2 ? 4 : 5;
  // a block's scales are there until no warp reads them any more: its K slot is filled again
  // when the softmax of the block NS / 2 - 2 before is over
  static_assert(kNS / 2 + 2 <= kScaleBlocks, "scales");
  static constexpr int kFirst = kHead + (Q8 ? kScaleBytes : 0);
  static constexpr int kSmem = kFirst + kQ + kNS * kStage + 1024;
  static constexpr int kNC = NQ == 2 ? 128 : 64;       // key columns per softmax thread
  static constexpr int kDC = NQ == 2 ? D : D / 2;      // output columns per softmax thread
  static constexpr int kPart = 32 * (kDC + 2);         // floats of one warp's partial
};

struct AttnParams : PlanParams, CapParams, ScaleParams {
  CUtensorMap kmap, vmap;  // [page][head][slot][D], box 64 (128 codes) x min(page, 128) rows
  CUtensorMap qmap;        // [token][head][D], box 64 x G heads x tokens of half a tile
  int q_boxes;             // queries come by qmap
  const __half *q;
  __half *out;
  int64_t q_token, q_head, o_token, o_head;
  float c;              // logit units to log2: |scale| log2(e), or log2(e) with a cap
  uint32_t keep, flip;  // queries are read as (bits & keep) ^ flip: signs turned when scale < 0,
                        // zeros when scale = 0 (c stays positive: masked logits are -inf)
  unsigned *cnt;        // [kMaxCtas][8] arrivals per cut tile (by its first CTA) and warp
  float *part;          // [kMaxCtas][2][8] partials
};

// ------------------------------------------------------------ PTX pieces --
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Four steps of 16 along K: D (tensor memory) (+)= A (shared) B (shared), both
// K-major in 64-column groups, so a step is 32 bytes (2 in descriptor units).
// Descriptors come as their low words (the address field cannot carry: shared
// memory lies below 256 KB) and a common high word: the issuing thread's few
// instructions per product are what a product of this size leaves time for.
__device__ __forceinline__ void mma4_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                        uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 x, y;\n\t.reg .b32 u, v;\n\t"
      "setp.ne.b32 p0, %5, 0;\n\tsetp.eq.b32 p1, %5, %5;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p0;\n\t"
      "add.u32 u, %1, 2;\n\tadd.u32 v, %2, 2;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p1;\n\t"
      "add.u32 u, %1, 4;\n\tadd.u32 v, %2, 4;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p1;\n\t"
      "add.u32 u, %1, 6;\n\tadd.u32 v, %2, 6;\n\tmov.b64 x, {u, %3};\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p1;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// Four steps of 16 keys: D (tensor memory) (+)= A (tensor memory, 8 columns a
// step) B (shared, N-major: 16 rows of 128 bytes a step).
__device__ __forceinline__ void mma4_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi,
                                        uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p0, p1;\n\t.reg .b64 y;\n\t.reg .b32 u, v;\n\t"
      "setp.ne.b32 p0, %5, 0;\n\tsetp.eq.b32 p1, %5, %5;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p0;\n\t"
      "add.u32 u, %1, 8;\n\tadd.u32 v, %2, 128;\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, p1;\n\t"
      "add.u32 u, %1, 16;\n\tadd.u32 v, %2, 256;\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, p1;\n\t"
      "add.u32 u, %1, 24;\n\tadd.u32 v, %2, 384;\n\tmov.b64 y, {v, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [u], y, %4, p1;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
// 32 consecutive 32-bit columns of this thread's lane, without waiting.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Shared-memory operand of 128-byte-swizzled rows of 64 fp16 (8-row groups
// 1024 bytes apart): low word of its descriptor; mn: bytes between 64-column
// groups of an N-major operand (unused when K-major).
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t addr, uint32_t mn) {
  return addr >> 4 | (mn >> 4) << 16;
}
// stride, version, 128-byte swizzle
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;
// A value that every lane holds, as one the compiler knows to be uniform.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
// kind::f16, A = B = f16, D = f32; A K-major, B K-major or N-major.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_n_major) {
  return (1u << 4) | (b_n_major ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------------------- kernel --
// CAP: 0 none, 1 of up to kShortCap, 2 of any size.  Q8: a cache of INT8 rows, which the
// query warps turn into fp16 before they are multiplied (see turn_rows).
template <int D, int NQ, int CAP, bool Q8>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NQ, Q8>;
  constexpr int kM = C::kM, NS = C::kNS, NC = C::kNC, DC = C::kDC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(base);
  uint64_t *kv_full = bars, *kv_empty = bars + kMaxStages;
  uint64_t *s_full = kv_empty + kMaxStages, *p_full = s_full + 2, *o_done = p_full + 2;
  uint64_t *p_half = o_done + 2;  // NQ = 2: the first 64 keys' weights
  uint64_t *q_full = p_half + 2, *xbar = q_full + 1;  // xbar: one per 32-row quarter
  uint64_t *seg_full = xbar + 4, *seg_empty = seg_full + kSegs, *q_empty = seg_empty + kSegs;
  uint64_t *drained = q_empty + 1;  // the products of a CTA that gave up
  uint64_t *kv_ready = drained + 1;  // Q8: a slot's codes are fp16
  uint64_t *half_done = kv_ready + kMaxStages;  // Q8: a stage's product of the first 64 keys
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(half_done + 2);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
  // Copies that the load warp has issued, tiles that the query warps have
  uint32_t *issued = reinterpret_cast<uint32_t *>(abort_flag + 1);  // [kLoadWarp - kQWarp + 1]
  Seg *seg_sm = reinterpret_cast<Seg *>(base + 512);         // [kSegs]
  float *xch = reinterpret_cast<float *>(base + 1024);       // [2][8 warps][32]
  float *scale_sm = reinterpret_cast<float *>(base + kHead);  // [kScaleBlocks][K, V][kN]
  float2 *bound_sm = reinterpret_cast<float2 *>(scale_sm + kScaleBlocks * 2 * kN);  // [..][4]
  __half *part_sm = reinterpret_cast<__half *>(bound_sm + kScaleBlocks * 4);  // [kScaleBlocks][kN]
  uint8_t *q_sm = base + C::kFirst, *kv_sm = q_sm + C::kQ;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&kv_full[i]), Q8 && !p.runs ? 33 : 1);
      mbar_init(smem_u32(&kv_ready[i]), 2);
      mbar_init(smem_u32(&kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), NQ == 2 ? 4 : 8);
      mbar_init(smem_u32(&o_done[i]), 1);
      mbar_init(smem_u32(&p_half[i]), 4);
      mbar_init(smem_u32(&half_done[i]), 1);
    }
    mbar_init(smem_u32(q_full), 2);
    mbar_init(smem_u32(q_empty), 1);
    mbar_init(smem_u32(drained), 1);
    for (int i = 0; i < 4; ++i) mbar_init(smem_u32(&xbar[i]), 2);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_u32(&seg_full[i]), 1);
      mbar_init(smem_u32(&seg_empty[i]), kSoftmaxWarps + 3);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }

  Walker<kM> w;
  w.u = w.u_end = 0;
  if (warp == kLoadWarp) {  // one load's latency either way, few instructions for small batches
    if (p.s.n_seqs <= 32)
      w.template start<1>(p);
    else
      w.template start<8>(p);
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot;  // S of stage or buffer i at 128 i, O at 256 (+ D for stage 1)

  // The n-th announced tile (every warp but the one that announces).
  auto read_seg = [&](uint32_t n, Seg &g) {
    if (!mbar_wait(smem_u32(&seg_full[n % kSegs]), (n / kSegs) & 1, abort_flag)) return false;
    const uint4 *src = reinterpret_cast<const uint4 *>(&seg_sm[n % kSegs]);
    uint4 *dst = reinterpret_cast<uint4 *>(&g);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = src[i];
    return true;
  };
  auto free_seg = [&](uint32_t n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&seg_empty[n % kSegs]));
  };

  // n / G for n < G + 256: (n + 1/2) / G stays further from every whole number
  // than fp32 rounding can move it.
  auto row_token = [&](int n) { return (int)(((float)n + 0.5f) * p.inv_g); };

  // Half of a tile's queries, from token tok on, by TMA (one lane).
  auto copy_queries = [&](const Seg &g, int half, int tok) {
    asm volatile(
        "{\n\t.reg .b64 t;\n\t"
        "mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(smem_u32(q_full)),
        "r"((uint32_t)(kM / 2 * D * 2))
        : "memory");
    const uint32_t dst = smem_u32(q_sm) + (NQ == 2 ? half * (128 * D * 2) : half * 64 * 128);
#pragma unroll
    for (int d = 0; d < D / 64; ++d)
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
          "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst + d * 16384),
          "l"(reinterpret_cast<uint64_t>(&p.qmap)), "r"(d * 64), "r"(g.head * p.G), "r"(tok),
          "r"(smem_u32(q_full))
          : "memory");
  };

  if (warp < kSoftmaxWarps) {
    // ------------------------------------------------------------ softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    const int wg = warp >> 2, quarter = warp & 3;
    const int my_row = (NQ == 2 ? wg * 128 : 0) + quarter * 32 + lane;  // of the tile
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const int col0 = NQ == 2 ? 0 : wg * NC;    // first key column of this thread
    const int out0 = NQ == 2 ? 0 : wg * DC;    // first output column
    const uint32_t o_tm = tmem + lane_base + 256 + (NQ == 2 ? wg * D : out0);
    uint32_t blocks = 0;   // key blocks so far (NQ = 2: of this stage)
    uint32_t ends = 0;     // segments finished (NQ = 2: of this stage)
    uint32_t swaps = 0;    // exchanges with the other warpgroup
    uint32_t scales = 0;   // Q8: key blocks of the tiles so far
    // Q8: logits get their keys' factors (and c with them) where they become weights, and
    // the running maximum is held against a bound of theirs
    constexpr bool kBound = Q8 && CAP == 0;
    // Q8: a thread's 128 columns in two passes, each with a maximum of its own, since the
    // factors that it reads leave no registers for all of them
    constexpr int kParts = Q8 && NQ == 2 ? 2 : 1, NP = NC / kParts;
    const float c = kBound ? 1.0f : p.c;  // of m and the logits
    bool ok = true;
    // The other warpgroup's value of this row (NQ = 1).
    auto exchange = [&](float v, float *other) -> bool {
      float *x = xch + (swaps & 1) * 256;
      x[warp * 32 + lane] = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&xbar[quarter]));
      if (!mbar_wait(smem_u32(&xbar[quarter]), swaps & 1, abort_flag)) return false;
      *other = x[(warp ^ 4) * 32 + lane];
      ++swaps;
      return true;
    };
    uint32_t n_seg = 0;    // tiles read so far
    // Four 16-byte pieces of this lane's row, out through shared memory so that
    // a store covers 64 contiguous bytes of 8 rows: dst[i] is where piece
    // lane % 4 of row 8 i + lane / 4 goes (null: nowhere).
    const uint32_t stage_sm = smem_u32(base) + kBars + warp * kOutBytes;
    auto store_rows = [&](const uint32_t (&v)[16], char *const (&dst)[4], int offset) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                         stage_sm + lane * 64 + ((c ^ ((lane >> 1) & 3)) << 4)),
                     "r"(v[4 * c]), "r"(v[4 * c + 1]), "r"(v[4 * c + 2]), "r"(v[4 * c + 3])
                     : "memory");
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        uint4 o;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                     : "r"(stage_sm + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4)));
        if (dst[i]) *reinterpret_cast<uint4 *>(dst[i] + offset) = o;
      }
      __syncwarp();
    };
    while (ok) {
      Seg g;
      if (!(ok = read_seg(n_seg, g))) break;
      free_seg(n_seg++);
      if (g.rows == 0) break;
      const int warp_row = my_row - lane;
      const int live_rows = min(max(g.rows - warp_row, 0), 32);  // of this warp
      // rows past the tile's end repeat its last row's limits
      const int pos = g.pos + row_token(g.rem + min(my_row, g.rows - 1));
      const int hi = pos + 1, lo = first_key(p, pos);
      float m = -INFINITY, l = 0.0f;
      const int nb = g.b1 - g.b0;
      const uint32_t scale0 = scales;
      scales += nb;
      const bool active = nb > 0 && (NQ == 1 || wg == 0 || g.rows > 128);
      // whole blocks of this range need no mask in this warp
      const int see_lo = __reduce_max_sync(0xffffffffu, lo);
      const int see_hi = __reduce_min_sync(0xffffffffu, hi);
      // NQ = 1: the previous block's product is complete.  Every live warp sees
      // each of them before it lets the next one start: a wait tells a
      // barrier's phases apart by parity alone.
      auto last_product = [&](int b) {
        return b == g.b0 || mbar_wait(smem_u32(&o_done[0]), (blocks - 1) & 1, abort_flag);
      };
      for (int b = g.b0; active && b < g.b1; ++b, ++blocks) {
        const int buf = NQ == 2 ? wg : (int)(blocks & 1);
        const uint32_t ph = NQ == 2 ? blocks & 1 : (blocks >> 1) & 1;
        if (!(ok = mbar_wait(smem_u32(&s_full[buf]), ph, abort_flag))) break;
        if (live_rows == 0) {  // nothing of this warp is stored
          if (lane == 0) {
            if (NQ == 2) mbar_arrive(smem_u32(&p_half[buf]));
            mbar_arrive(smem_u32(&p_full[buf]));
          }
          continue;
        }
        fence_after();
        const uint32_t s_tm = tmem + lane_base + 128 * buf;
        const uint32_t set = (scale0 + b - g.b0) % kScaleBlocks;
#pragma unroll 1
        for (int part = 0; part < kParts; ++part) {
          const int col = col0 + part * NP;  // first key column of this pass
          float s[NP];
#pragma unroll
          for (int k = 0; k < NP / 32; ++k)
            tmem_ld32(s_tm + col + 32 * k, reinterpret_cast<uint32_t *>(s) + 32 * k);
          const float *kf = scale_sm + set * (2 * kN) + col, *vf = kf + kN;
          const float2 *bf = bound_sm + set * 4 + col / 32;
          tmem_ld_wait();
          if (Q8 && CAP) {
#pragma unroll
            for (int k = 0; k < NP; k += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(kf + k);
              s[k] *= f.x, s[k + 1] *= f.y, s[k + 2] *= f.z, s[k + 3] *= f.w;
            }
          }
          if (CAP) {
#pragma unroll
            for (int k = 0; k < NP; ++k) s[k] = CAP == 1 ? cap_far(p, s[k]) : cap_any(p, s[k]);
          }
          // keys [k_lo, k_hi) of this row; a block that no bound cuts needs neither
          if (see_hi - b * kN < col + NP) {  // (the block's end may pass 32 bits)
            const int k_hi = hi - b * kN - col;
#pragma unroll
            for (int k = 0; k < NP; ++k) s[k] = k < k_hi ? s[k] : -INFINITY;
          }
          if (b * kN + col < see_lo) {
            const int k_lo = lo - b * kN - col;
#pragma unroll
            for (int k = 0; k < NP; ++k) s[k] = k >= k_lo ? s[k] : -INFINITY;
          }
          float mb;
          if (kBound) {
            // No logit is above this.  (A masked group times a bound of 0 is NaN, and not taken.)
            mb = -INFINITY;
#pragma unroll
            for (int h = 0; h < NP / 32; ++h) {
              float a = s[32 * h], c = s[32 * h + 1];
#pragma unroll
              for (int k = 2; k < 30; k += 4) {
                a = max3(a, s[32 * h + k], s[32 * h + k + 1]);
                c = max3(c, s[32 * h + k + 2], s[32 * h + k + 3]);
              }
              a = max3(a, s[32 * h + 30], s[32 * h + 31]);
              a = fmaxf(a, c);
              const float2 f = bf[h];
              mb = fmaxf(mb, a * (a > 0.0f ? f.x : f.y));
            }
          } else {
            float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int k = 4; k < NP - 4; k += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[k + 2 * e], s[k + 2 * e + 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[NP - 4 + e]);
            mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          }
          if (NQ == 1) {
            float other;
            if (!(ok = exchange(mb, &other))) break;
            mb = fmaxf(mb, other);
          }
          // move the maximum where it lags too far, and rescale what was summed
          const bool move = (mb - m) * c > kLag || (m == -INFINITY && mb > -INFINITY);
          if (__any_sync(0xffffffffu, move)) {
            if (kBound) {  // the largest logit itself
              mb = -INFINITY;
#pragma unroll
              for (int k = 0; k < NP; k += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(kf + k);
                mb = max3(mb, s[k] * f.x, s[k + 1] * f.y);
                mb = max3(mb, s[k + 2] * f.z, s[k + 3] * f.w);
              }
              if (NQ == 1) {
                float other;
                if (!(ok = exchange(mb, &other))) break;
                mb = fmaxf(mb, other);
              }
            }
            // (kBound: every row of the warp moves, so that the next one comes later)
            const float mn = kBound ? fmaxf(m, mb) : move ? mb : m;
            const float f = m == -INFINITY ? (mn > -INFINITY ? 0.0f : 1.0f) : ex2((m - mn) * c);
            m = mn;
            l *= f;
            if ((b > g.b0 || part > 0) && (!kBound || __any_sync(0xffffffffu, f != 1.0f))) {
              // NQ = 2: this stage's earlier products precede the S just read, but for that of
              // this block's first keys
              if (NQ == 1 && !(ok = last_product(b))) break;
              if (part > 0 && !(ok = mbar_wait(smem_u32(&half_done[wg]), ph, abort_flag))) break;
              fence_after();
#pragma unroll 1
              for (int k = 0; k < DC; k += 32) {
                uint32_t o[32];
                tmem_ld32(o_tm + k, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st32(o_tm + k, o);
              }
            }
          }
          const float mc = m == -INFINITY ? 0.0f : m * c - kLift;
          const float2 mc2 = make_float2(-mc, -mc);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
          for (int h = 0; h < NP / 32; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const int at = 32 * h + 2 * k;
              float4 kc = make_float4(c, c, c, c), vc;
              if (kBound) kc = *reinterpret_cast<const float4 *>(kf + at);
              if (Q8) vc = *reinterpret_cast<const float4 *>(vf + at);
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float2 e = fma2(make_float2(s[at + 2 * j], s[at + 2 * j + 1]),
                                j ? make_float2(kc.z, kc.w) : make_float2(kc.x, kc.y), mc2);
                e.x = ex2(e.x);
                e.y = ex2(e.y);
                sum[j] = add2(sum[j], e);
                if (Q8) e = mul2(e, j ? make_float2(vc.z, vc.w) : make_float2(vc.x, vc.y));
                pk[k + j] = f2h(e.x, e.y);
              }
            }
            tmem_st16(s_tm + col / 2 + 16 * h, pk);
            if (NQ == 2 && kParts == 1 && h == 1) {  // the product starts on these
              tmem_st_wait();
              fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&p_half[buf]));
            }
          }
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          if (NQ == 1 && !(ok = last_product(b))) break;
          tmem_st_wait();
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&(part == kParts - 1 ? p_full : p_half)[buf]));
        }
        if (!ok) break;
      }
      if (!ok) break;
      // ---- the tile's rows, or this CTA's part of them
      if (live_rows == 0) {
        if (active) ++ends;
        continue;
      }
      auto out_at = [&](int r) {  // where a row's outputs go
        const int n = g.rem + r, i = row_token(n);
        return (int64_t)(g.tok + i) * p.o_token + (int64_t)(g.head * p.G + n - i * p.G) * p.o_head +
               out0;
      };
      auto part_of = [&](int cta, int slot) {
        return p.part + (int64_t)((cta * 2 + slot) * kSoftmaxWarps + warp) * C::kPart;
      };
      float *mine_part = part_of(blockIdx.x, g.slot);
      char *dst[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        dst[i] = g.slot < 0 ? reinterpret_cast<char *>(p.out + out_at(warp_row + r))
                            : reinterpret_cast<char *>(mine_part + 64 + r * DC);
        dst[i] = r < live_rows ? dst[i] + (lane & 3) * 16 : nullptr;
      }
      if (active) {
        const uint32_t ph = NQ == 2 ? ends & 1 : (blocks - 1) & 1;
        if (!(ok = mbar_wait(smem_u32(&o_done[NQ == 2 ? wg : 0]), ph, abort_flag))) break;
        ++ends;
        fence_after();
        if (NQ == 1) {
          float other;
          if (!(ok = exchange(l, &other))) break;
          l = wg == 0 ? l + other : other + l;
        }
      }
      if (g.slot < 0) {
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll 1
        for (int k = 0; k < DC; k += 32) {
          uint32_t o[32], v[16];
          if (active) {
            tmem_ld32(o_tm + k, o);
            tmem_ld_wait();
          }
#pragma unroll
          for (int e = 0; e < 16; ++e)
            v[e] = active ? f2h(__uint_as_float(o[2 * e]) * inv,
                                __uint_as_float(o[2 * e + 1]) * inv)
                          : 0u;
          store_rows(v, dst, k * 2);
        }
        continue;
      }
      // ---- cut between CTAs: leave the partial, merge if last
      mine_part[lane] = l > 0.0f ? (m == -INFINITY ? 0.0f : m * c) : -INFINITY;
      mine_part[32 + lane] = l;
#pragma unroll 1
      for (int k = 0; k < DC; k += 32) {
        uint32_t o[32];
        tmem_ld32(o_tm + k, o);
        tmem_ld_wait();
        uint32_t v[16];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = o[16 * h + e];
          store_rows(v, dst, (k + 16 * h) * 4);
        }
      }
      __threadfence();
      __syncwarp();
      unsigned arrived = 0;
      if (lane == 0) arrived = atomicAdd(&p.cnt[g.c_lo * kSoftmaxWarps + warp], 1u);
      arrived = __shfl_sync(0xffffffffu, arrived, 0);
      if ((int)arrived != g.parts - 1) continue;
      __threadfence();
      auto part_at = [&](int k) { return part_of(g.c_lo + k, k == 0 ? g.first_slot : 0); };
      float M = -INFINITY, L = 0.0f;
      for (int k0 = 0; k0 < g.parts; k0 += 8) {
        float mk[8], lk[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float *pp = part_at(min(k0 + k, g.parts - 1));
          mk[k] = k0 + k < g.parts ? __ldcg(pp + lane) : -INFINITY;
          lk[k] = __ldcg(pp + 32 + lane);
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < 8; ++k) mn = fmaxf(mn, mk[k]);
        const float z = mn == -INFINITY ? 0.0f : mn;
        L *= ex2(M - z);
#pragma unroll
        for (int k = 0; k < 8; ++k) L = fmaf(lk[k], ex2(mk[k] - z), L);
        M = mn;
      }
      const float Mz = M == -INFINITY ? 0.0f : M;
      const float inv = L > 0.0f ? 1.0f / L : 0.0f;
      // lanes share the rows' float4 columns, 4 each; 4 partials in flight
      constexpr int F4 = DC / 4, E = 4, U = 4;
      const int items = live_rows * F4;
      const int64_t row_at = out_at(warp_row + lane);
      for (int i0 = 0; i0 < items; i0 += 32 * E) {
        float4 acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int k0 = 0; k0 < g.parts; k0 += U) {
          float4 v[U][E];
          float mk[U];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const bool on = k0 + k < g.parts;
            const float *pp = part_at(min(k0 + k, g.parts - 1));
            mk[k] = on ? __ldcg(pp + lane) : -INFINITY;
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const int it = i0 + e * 32 + lane;
              v[k][e] = on && it < items ? __ldcg(reinterpret_cast<const float4 *>(pp + 64) + it)
                                         : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
          }
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const float wgt = ex2(mk[k] - Mz);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float f = __shfl_sync(0xffffffffu, wgt, min((i0 + e * 32 + lane) / F4, 31));
              acc[e].x = fmaf(v[k][e].x, f, acc[e].x);
              acc[e].y = fmaf(v[k][e].y, f, acc[e].y);
              acc[e].z = fmaf(v[k][e].z, f, acc[e].z);
              acc[e].w = fmaf(v[k][e].w, f, acc[e].w);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int it = i0 + e * 32 + lane, row = min(it / F4, 31);
          const float f = __shfl_sync(0xffffffffu, inv, row);
          const int64_t at = __shfl_sync(0xffffffffu, row_at, row);
          if (it < items)
            *reinterpret_cast<uint2 *>(p.out + at + it % F4 * 4) =
                make_uint2(f2h(acc[e].x * f, acc[e].y * f), f2h(acc[e].z * f, acc[e].w * f));
        }
      }
      if (lane == 0) p.cnt[g.c_lo * kSoftmaxWarps + warp] = 0;
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------------- MMA --
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    constexpr uint32_t id_qk = idesc(128, kN, false), id_pv = idesc(128, D, true);
    uint32_t ring = 0, blocks = 0, segs = 0, n_stage[2] = {0, 0};
    bool ok = true;
    auto slot_addr = [&](uint32_t r) { return smem_u32(kv_sm) + (r % NS) * C::kStage; };
    auto wait_slot = [&](uint32_t r) {
      return mbar_wait(smem_u32(&(Q8 ? kv_ready : kv_full)[r % NS]), (r / NS) & 1, abort_flag);
    };
    const uint32_t tm = uniform(tmem), q_lo = uniform(sdesc_lo(smem_u32(q_sm), 16));
    // (whole warp) S = Q K^T of a stage into S buffer buf
    auto qk = [&](int stage, int buf, uint32_t r, bool free_slot, bool free_q) {
      const uint32_t b = uniform(sdesc_lo(slot_addr(r), 16));
      const uint32_t a = q_lo + stage * (128 * D * 2 / 16), d = tm + uniform(128 * buf);
      const uint32_t done = uniform(smem_u32(&s_full[buf])), qe = uniform(smem_u32(q_empty));
      const uint32_t empty = uniform(smem_u32(&kv_empty[r % NS]));
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 64; ++k)  // 64 columns: 16 KB
          mma4_ss(d, a + k * 1024, b + k * 1024, kDescHi, id_qk, k > 0);
        mma_commit(done);
        if (free_slot) mma_commit(empty);
        if (free_q) mma_commit(qe);
      }
    };
    // (whole warp) O (+)= P V: keys 64 half.. of S buffer buf
    auto pv = [&](int buf, int half, uint32_t o_col, uint32_t r, bool acc, bool free_slot,
                  uint64_t *done) {
      const uint32_t b = uniform(sdesc_lo(slot_addr(r), 16384) + half * 512);
      const uint32_t a = tm + uniform(128 * buf + 32 * half), d = tm + uniform(o_col);
      const uint32_t empty = uniform(smem_u32(&kv_empty[r % NS]));
      const uint32_t bar = done ? uniform(smem_u32(done)) : 0;
      if (elect_one()) {
        mma4_ts(d, a, b, kDescHi, id_pv, acc || half);
        if (free_slot) mma_commit(empty);
        if (bar) mma_commit(bar);
      }
    };
    // Rows of a V block that no query of the tile sees may hold anything, and
    // a zero weight times NaN is NaN: they become zeros.  (Codes are all finite.)
    auto clean = [&](uint32_t r, int b, const Seg &t) {
      if (Q8) return;
      const int lo = t.lo - b * kN, hi = t.hi - b * kN;
      if (lo <= 0 && hi >= kN) return;
      uint8_t *v = kv_sm + (r % NS) * C::kStage;
      for (int i = lane; i < kN * D / 8; i += 32) {  // 16-byte chunks; 8 per row and 64 columns
        const int row = (i >> 3) & (kN - 1);
        if (row < lo || row >= hi) reinterpret_cast<uint4 *>(v)[i] = make_uint4(0, 0, 0, 0);
      }
      fence_async_smem();
      __syncwarp();
    };
    uint32_t n_seg = 0;
    while (ok) {
      Seg g;
      if (!(ok = read_seg(n_seg, g))) break;
      free_seg(n_seg++);
      if (g.rows == 0) break;
      const int nb = g.b1 - g.b0;
      if (nb == 0) continue;
      if (!(ok = mbar_wait(smem_u32(q_full), segs & 1, abort_flag))) break;
      ++segs;
      fence_after();
      if (NQ == 1) {
        for (int j = 0; j <= nb; ++j) {
          if (j < nb) {
            if (!(ok = wait_slot(ring))) break;
            qk(0, (blocks + j) & 1, ring, true, j == nb - 1);
            ++ring;
          }
          if (j > 0) {
            const uint32_t c = blocks + j - 1;
            if (!(ok = wait_slot(ring))) break;
            clean(ring, g.b0 + j - 1, g);
            if (!(ok = mbar_wait(smem_u32(&p_full[c & 1]), (c >> 1) & 1, abort_flag))) break;
            fence_after();
            pv(c & 1, 0, 256, ring, j > 1, false, nullptr);
            pv(c & 1, 1, 256, ring, true, true, &o_done[0]);
            ++ring;
          }
          __syncwarp();
        }
        blocks += nb;
      } else {
        const int stages = g.rows > 128 ? 2 : 1;
        if (!(ok = wait_slot(ring))) break;
        for (int t = 0; t < stages; ++t)
          qk(t, t, ring, t == stages - 1, nb == 1 && t == stages - 1);
        ++ring;
        for (int j = 0; j < nb; ++j) {
          const uint32_t v = ring, kn = ring + 1;
          const bool more = j + 1 < nb;
          if (!(ok = wait_slot(v))) break;
          clean(v, g.b0 + j, g);
          for (int t = 0; t < stages; ++t) {
            if (!(ok = mbar_wait(smem_u32(&p_half[t]), n_stage[t] & 1, abort_flag))) break;
            fence_after();
            pv(t, 0, 256 + t * D, v, j > 0, false, Q8 ? &half_done[t] : nullptr);
            if (!(ok = mbar_wait(smem_u32(&p_full[t]), n_stage[t] & 1, abort_flag))) break;
            fence_after();
            ++n_stage[t];
            pv(t, 1, 256 + t * D, v, true, t == stages - 1, more ? nullptr : &o_done[t]);
            if (more) {
              if (t == 0 && !(ok = wait_slot(kn))) break;
              qk(t, t, kn, t == stages - 1, j + 2 == nb && t == stages - 1);
            }
            __syncwarp();
          }
          if (!ok) break;
          ring += more ? 2 : 1;
        }
      }
    }
  } else if (warp < kQWarp + 2) {
    // ------------------------------------------------------------ queries --
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    // A tile's queries, half of the rows a warp.  Where a group of heads divides
    // them they are a box of the query tensor; else (and for a negative or zero
    // scale, which the copy cannot apply) they are laid row by row as TMA with the
    // 128-byte swizzle would, rows past the tile as zeros.
    constexpr int CPR = D / 8, RPP = 32 / CPR;  // 16-byte chunks a row, rows per pass
    constexpr int PASSES = kM / 2 / RPP;
    const int c = lane % CPR;
    auto tile_row = [&](int k) { return (warp - kQWarp) * (kM / 2) + k * RPP + lane / CPR; };
    auto place = [&](int r) {
      return smem_u32(q_sm) + (r >> 7) * (128 * D * 2) + (c >> 3) * 16384 + (r & 127) * 128 +
             (((c & 7) ^ (r & 7)) << 4);
    };
    // Visits this lane's chunk of its rows in order: f(row, source).
    auto each_row = [&](const Seg &g, auto f) {
      const int r0 = tile_row(0), n = g.rem + r0, i = row_token(n);
      int head = n - i * p.G;
      const __half *src = p.q + (int64_t)(g.tok + i) * p.q_token +
                          (int64_t)(g.head * p.G + head) * p.q_head + c * 8;
      const int toks = row_token(RPP), heads = RPP - toks * p.G;  // RPP rows further on
      const int64_t wrap = p.q_token - p.G * p.q_head;
      const int64_t step = toks * p.q_token + heads * p.q_head;
#pragma unroll 8
      for (int k = 0; k < PASSES; ++k) {
        f(r0 + k * RPP, src);
        src += step;
        head += heads;
        if (head >= p.G) {
          head -= p.G;
          src += wrap;
        }
      }
    };
    // Q8: a tile's blocks of keys and values, half of the rows a warp and a row a lane.  A
    // scale is s r with s of 4 bits, so that s times a code is exact in fp16, and r within
    // 1/16 of 1, which stays in fp32: r (and c, without a cap) multiplies the logit, or the
    // weight.  Keys' s are in units of the largest of 32 keys (2^e, which their r has), not
    // below 2^-21 of it: r is below 15/16 for smaller keys, so that no key's scale depends on
    // its neighbours, and the bound of a group that has one is 0 where its products are
    // negative.  Values' s are fp16 as they are, from 2^-21 to 512, and r likewise.
    // A byte under the bits of 1024 is 1024 + code + 128 once its sign is turned.
    constexpr int kChunks = D == 64 ? 4 : 8;
    uint32_t ring = 0, scales = 0, values = 0, segs = 0;
    auto four_bits = [](float x) {
      return __uint_as_float((__float_as_uint(x) + 0x00080000u) & 0xfff00000u);
    };
    auto turn_rows = [&](const Seg &g) -> bool {
      const int n = 2 * (g.b1 - g.b0);
      for (int i = 0; i < n; ++i, ++ring) {
        const int slot = ring % NS;
        if (!mbar_wait(smem_u32(&kv_full[slot]), (ring / NS) & 1, abort_flag)) return false;
        // keys and values in the order of the load warp
        const bool keys = NQ == 2 ? !(i & 1) : i == 0 || ((i & 1) && i < n - 1);
        const uint32_t set = (keys ? scales++ : values++) % kScaleBlocks;
        const uint32_t at = smem_u32(kv_sm) + slot * C::kStage;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          const int group = (warp - kQWarp) * 2 + half, row = group * 32 + lane;
          __half s;
          bool large = false;  // 1152 s is beyond fp16
          if (keys) {
            float *k = scale_sm + set * (2 * kN) + row, *v = k + kN;
            // (of keys that no row sees, and of missing pages, zeros)
            const int at_key = (g.b0 + (NQ == 2 ? i / 2 : (i + 1) / 2)) * kN;
            const bool seen = row < g.hi - at_key && row >= g.lo - at_key;
            const float ks = seen ? *k : 0.0f, y = seen ? *v : 0.0f;
            // (a key that is not finite has no part in its neighbours' unit)
            const uint32_t bits = __float_as_uint(ks);
            const uint32_t top = __reduce_max_sync(0xffffffffu, bits < 0x7f800000u ? bits : 0u);
            const int e = min(max((int)(top >> 23) - 127, -100), 126);
            const float x = ks * __uint_as_float((uint32_t)(127 - e) << 23);
            const float unit = __uint_as_float((uint32_t)(127 + e) << 23) * (CAP ? 1.0f : p.c);
            // (nor a factor that is not)
            const bool whole = !(x > 0.0f && x < 4.0f);
            const float part = fmaxf(four_bits(x), 0x1p-21f);
            s = __float2half_rn(whole ? x : part);
            // (approximate reciprocals, 2^-23: these two warps are what a block waits for; 4 x 64
            // tokens over up to 24000 keys 190 us, with correctly rounded ones 198)
            // (a factor of 0, of tiny keys and scales, would make a NaN of a masked logit)
            *k = fmaxf((whole ? 1.0f : x * rcp(part)) * unit, 0x1p-126f);
            const bool small = __any_sync(0xffffffffu, x > 0.0f && x < 0x1p-21f);
            if (lane == 0)
              bound_sm[set * 4 + group] =
                  make_float2(1.0625f * unit, small ? 0.0f : 0.9375f * unit);
            const float w = fminf(fmaxf(four_bits(y), 0x1p-21f), 512.0f);
            part_sm[set * kN + row] = __float2half_rn(w);
            *v = y * rcp(w);
          } else {
            s = part_sm[set * kN + row];
            large = __any_sync(0xffffffffu, __half2float(s) > 32.0f);
          }
          const __half2 s2 = __half2half2(s), off = __hmul2(s2, __float2half2_rn(-1152.0f));
          const uint32_t raw = at + C::kCodes + row * (D == 64 ? 64 : 128);
          const uint32_t turn = D == 64 ? (row >> 1) & 3 : row & 7;
          auto scaled = [&](uint32_t biased, uint32_t sel) -> uint32_t {
            const uint32_t b = __byte_perm(biased, 0x64646464u, sel);
            const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&b), s2, off);
            return *reinterpret_cast<const uint32_t *>(&r);
          };
          auto scaled_large = [&](uint32_t biased, uint32_t sel) -> uint32_t {
            const uint32_t b = code_pair(biased, sel);
            const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&b), s2);
            return *reinterpret_cast<const uint32_t *>(&r);
          };
#pragma unroll
          for (int h = 0; h < (D + 127) / 128; ++h) {
            uint4 codes[kChunks];
#pragma unroll
            for (int k = 0; k < kChunks; ++k)
              asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                           : "=r"(codes[k].x), "=r"(codes[k].y), "=r"(codes[k].z),
                             "=r"(codes[k].w)
                           : "r"(raw + h * (kN * 128) + ((k ^ turn) << 4))
                           : "memory");
            auto store = [&](auto f) {
#pragma unroll
              for (int k = 0; k < kChunks; ++k) {
                const uint32_t w[4] = {codes[k].x, codes[k].y, codes[k].z, codes[k].w};
                const uint32_t dst = at + (2 * h + (k >> 2)) * (kN * 128) + row * 128;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const uint32_t a = w[2 * j] ^ 0x80808080u, b = w[2 * j + 1] ^ 0x80808080u;
                  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(
                                   dst + (((2 * (k & 3) + j) ^ (row & 7)) << 4)),
                               "r"(f(a, 0x4140)), "r"(f(a, 0x4342)), "r"(f(b, 0x4140)),
                               "r"(f(b, 0x4342))
                               : "memory");
                }
              }
            };
            if (large)
              store(scaled_large);
            else
              store(scaled);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&kv_ready[slot]));
        if (p.q_boxes && i == 0) {  // the tile before has its last logits about now
          if (segs > 0 && !mbar_wait(smem_u32(q_empty), (segs - 1) & 1, abort_flag)) return false;
          const int half = warp - kQWarp;
          if (lane == 0) copy_queries(g, half, g.tok + half * (kM / 2) / p.G);
          __syncwarp();
          ++segs;
        }
      }
      return true;
    };
    uint32_t n_seg = 0;
    for (;;) {
      Seg g;
      if (!read_seg(n_seg, g)) break;
      free_seg(n_seg++);
      if (g.rows == 0) break;
      if (g.b1 <= g.b0) continue;
      if (Q8 && p.q_boxes) {  // queries come behind the first keys
        if (!turn_rows(g)) break;
        continue;
      }
      if (p.q_boxes) {
        // Rows past the tile are whatever follows (or zeros past the last token):
        // they are computed and not stored.
        const int half = warp - kQWarp, tok = g.tok + half * (kM / 2) / p.G;
        if (segs > 0) {
          if (lane == 0)
#pragma unroll
            for (int d = 0; d < D / 64; ++d)
              asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(
                               reinterpret_cast<uint64_t>(&p.qmap)),
                           "r"(d * 64), "r"(g.head * p.G), "r"(tok)
                           : "memory");
          __syncwarp();
          if (!mbar_wait(smem_u32(q_empty), (segs - 1) & 1, abort_flag)) break;
        }
        if (lane == 0) copy_queries(g, half, tok);
        __syncwarp();
        ++segs;
        continue;
      }
      if (segs > 0) {
        // while the tile before still reads its own, bring these as far as L2
        if (c % 8 == 0)
          each_row(g, [&](int r, const __half *src) {
            if (r < g.rows) asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
          });
        __syncwarp();
        if (!mbar_wait(smem_u32(q_empty), (segs - 1) & 1, abort_flag)) break;
      }
      each_row(g, [&](int r, const __half *src) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(place(r)),
                     "l"(r < g.rows ? src : p.q), "r"(r < g.rows ? 16 : 0)
                     : "memory");
      });
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (p.flip != 0 || p.keep != ~0u) {  // a negative or zero scale
        for (int k = 0; k < PASSES; ++k) {
          const uint32_t at = place(tile_row(k));
          uint32_t v[4];
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                       : "r"(at));
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at),
                       "r"((v[0] & p.keep) ^ p.flip), "r"((v[1] & p.keep) ^ p.flip),
                       "r"((v[2] & p.keep) ^ p.flip), "r"((v[3] & p.keep) ^ p.flip)
                       : "memory");
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(q_full));
      ++segs;
      if (Q8 && !turn_rows(g)) break;
    }
    if (lane == 0) issued[warp - kQWarp] = p.q_boxes ? segs : 0;
  } else {
    // --------------------------------------------------------------- load --
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    uint32_t ring = 0;
    bool ok = true;
    const int ppb = p.page_size >= kN ? 1 : kN >> p.page_shift;  // pages per block
    const int box_rows = min(p.page_size, kN);
    // Page ids, 32 entries of the table at a time and one batch ahead, an entry a
    // lane (-1: none of its slots is needed).
    int batch = 0, ids = -1, ids_ahead = -1;  // first entry of ids; ids; the next 32
    auto fetch = [&](const Seg &g, int first) -> int {
      const int pi = first + lane;
      const int64_t key = (int64_t)pi << p.page_shift;
      if (key >= g.hi || key + p.page_size <= g.lo) return -1;
      const int id = pi < p.s.ld_table ? __ldg(p.s.table + (int64_t)g.seq * p.s.ld_table + pi) : -2;
      return id == -1 ? -2 : id;
    };
    // Lane i's page of block b; outside the pool: an id outside the map, so that
    // the copy fills zeros.
    auto page_of = [&](const Seg &g, int b) -> int {
      const int pi = (int)(((int64_t)b * kN + lane * box_rows) >> p.page_shift);
      if (__shfl_sync(0xffffffffu, pi, ppb - 1) >= batch + 32) {
        batch += 32;
        ids = ids_ahead;
        ids_ahead = fetch(g, batch + 32);
      }
      const int id = __shfl_sync(0xffffffffu, ids, pi - batch);
      if (lane >= ppb || id == -1) return -1;
      if (id < 0 || id >= p.n_pages) {
        atomicOr(&g_attn_error, 4);
        return INT32_MAX;
      }
      return id;
    };
    // (Q8: the scales of the block's keys and values come with its keys)
    uint32_t scales = 0;
    auto issue = [&](bool keys, const Seg &g, int b, int page) -> bool {
      const CUtensorMap *map = keys ? &p.kmap : &p.vmap;
      const int slot = ring % NS;
      if (ring >= NS &&
          !mbar_wait(smem_u32(&kv_empty[slot]), (ring / NS - 1) & 1, abort_flag))
        return false;
      const uint32_t bar = smem_u32(&kv_full[slot]);
      const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
      const uint32_t bytes = __popc(live) * box_rows * D * (Q8 ? 1 : 2);
      float *sc = scale_sm + (scales % kScaleBlocks) * (2 * kN);
      uint32_t runs = 0;
      if (Q8 && keys) {
        runs = 2 * scale_runs(p, page);
        scale_zeros(p, sc, page);
        scale_zeros(p, sc + kN, page);
        __syncwarp();
      }
      if (lane == 0)
        asm volatile(
            "{\n\t.reg .b64 t;\n\t"
            "mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(bar),
            "r"(bytes + runs)
            : "memory");
      __syncwarp();
      if (page >= 0) {
        constexpr int kRow = Q8 && D == 64 ? 64 : 128;  // bytes
        constexpr int kCols = Q8 ? kRow : 64;
        const int at = p.page_size > kN ? (b * kN) & (p.page_size - 1) : 0;
        const uint32_t dst = smem_u32(kv_sm) + slot * C::kStage + (Q8 ? C::kCodes : 0) +
                             lane * box_rows * kRow;
#pragma unroll
        for (int d = 0; d < D / kCols; ++d)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst + d * 16384),
              "l"(reinterpret_cast<uint64_t>(map)), "r"(d * kCols), "r"(at), "r"(g.head),
              "r"(page), "r"(bar)
              : "memory");
      }
      if (Q8 && keys) {
        ++scales;
        scale_copy(p, p.ks, p.ks_page, p.ks_head, p.ks_token, sc, g, b, page, bar);
        scale_copy(p, p.vs, p.vs_page, p.vs_head, p.vs_token, sc + kN, g, b, page, bar);
      }
      if (Q8 && !p.runs)
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar)
                     : "memory");
      __syncwarp();
      ++ring;
      return true;
    };
    // The next tile is announced before a tile's loads, so that its queries come
    // to L2 early, but for the CTA's first tile, whose own loads come first.
    uint32_t n_seg = 0;
    auto announce = [&](const Seg &g) -> bool {
      const uint32_t at = n_seg % kSegs;
      if (n_seg >= kSegs &&
          !mbar_wait(smem_u32(&seg_empty[at]), (n_seg / kSegs - 1) & 1, abort_flag))
        return false;
      if (lane == 0) {
        seg_sm[at] = g;
        mbar_arrive(smem_u32(&seg_full[at]));
      }
      __syncwarp();
      ++n_seg;
      return true;
    };
    Seg next = w.next(p);
    ok = announce(next);
    while (ok && next.rows > 0) {
      const Seg g = next;
      const int nb = g.b1 - g.b0;
      if (nb > 0) {
        batch = (int)(((int64_t)g.b0 * kN) >> p.page_shift);
        ids = fetch(g, batch);
        ids_ahead = fetch(g, batch + 32);
      }
      int prev = -1;
      if (n_seg > 1) ok = announce(next = w.next(p));
      for (int j = 0; ok && j < max(nb, 1); ++j) {
        const int b = g.b0 + j;
        if (nb > 0) {
          const int page = page_of(g, b);
          ok = issue(true, g, b, page);
          if (NQ == 1) {  // K0, K1, V0, K2, V1, ..., the order in which they are used
            if (ok && j > 0) ok = issue(false, g, b - 1, prev);
            if (ok && j == nb - 1) ok = issue(false, g, b, page);
          } else if (ok) {
            ok = issue(false, g, b, page);
          }
          prev = page;
        }
        if (ok && j == 0 && n_seg == 1) ok = announce(next = w.next(p));
      }
    }
    if (lane == 0) issued[kLoadWarp - kQWarp] = ring;
    if (Q8) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (*(volatile int *)abort_flag) {  // (of the whole CTA: every warp has stopped)
    const unsigned long long until = gtimer() + kWaitNs;
    if (warp == kLoadWarp) {
      const uint32_t n = issued[kLoadWarp - kQWarp];
      for (uint32_t r = n - min(n, (uint32_t)NS); r < n; ++r)
        mbar_drain(smem_u32(&kv_full[r % NS]), (r / NS) & 1, until);
    } else if (warp == kMmaWarp) {
      if (elect_one()) mma_commit(smem_u32(drained));
      __syncwarp();
      mbar_drain(smem_u32(drained), 0, until);
    } else if (warp >= kQWarp && warp < kMmaWarp && issued[warp - kQWarp] > 0) {
      mbar_drain(smem_u32(q_full), (issued[warp - kQWarp] - 1) & 1, until);
    }
    fence_before();
    __syncthreads();
    fence_after();
  }
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols)
                 : "memory");
}
// The queries as [token][head][64-column group of D]; false: not such a box.
bool query_map(CUtensorMap *map, const __half *q, int64_t T, int64_t H, int D, int64_t token,
               int64_t head, int G, int rows) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn || G > rows || rows % G) return false;
  // a dimension of one element has no stride of its own
  if (H == 1) head = D;
  if (T == 1) token = H * D;
  const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t stride[2] = {(cuuint64_t)head * 2, (cuuint64_t)token * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(rows / G)};
  const cuuint32_t estride[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(q), dim, stride, box,
            estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// What the launches over either cache have in common.
void set_call(AttnParams *p, const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
              int hkv, const SeqView &sv, float scale, float softcap, int64_t window, __half *out,
              int64_t o_token, int64_t o_head, void *workspace) {
  p->q = q;
  p->out = out;
  p->q_token = q_token;
  p->q_head = q_head;
  p->o_token = o_token;
  p->o_head = o_head;
  set_heads(p, hq, hkv);
  p->keep = scale == 0.0f ? 0u : ~0u;
  p->flip = scale < 0.0f ? 0x80008000u : 0u;
  p->c = set_logits(p, scale, softcap);
  p->window = window > INT32_MAX ? 0 : (int)window;  // longer than any cache: none
  p->s = sv;
  p->cnt = static_cast<unsigned *>(workspace);
  p->part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + QZ_ATTENTION_SYNC_BYTES);
}

template <int D, int NQ, int CAP, bool Q8>
qz_status launch(const AttnParams &p, int sms, cudaStream_t s) {
  using C = Cfg<D, NQ, Q8>;
  const cudaError_t e = allow_smem<attn_kernel<D, NQ, CAP, Q8>>(C::kSmem);
  if (e != cudaSuccess) return cuda_status(e);
  attn_kernel<D, NQ, CAP, Q8><<<sms < kMaxCtas ? sms : kMaxCtas, kThreads, C::kSmem, s>>>(p);
  return launch_status();
}

template <int D, int NQ, bool Q8>
qz_status launch_cap(const AttnParams &p, int sms, cudaStream_t s) {
  if (p.cap == 0.0f) return launch<D, NQ, 0, Q8>(p, sms, s);
  return p.cap <= kShortCap ? launch<D, NQ, 1, Q8>(p, sms, s) : launch<D, NQ, 2, Q8>(p, sms, s);
}

}  // namespace
}  // namespace qz
