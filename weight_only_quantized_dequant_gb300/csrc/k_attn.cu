// Attention of a step's new tokens over the paged cache, on the 5th-generation
// tensor cores.
//
// For one KV head the queries of a sequence are packed row r = token * G +
// head-in-group (G = heads / KV heads), so that a decode step still multiplies
// a matrix and every row of a tile shares its keys:
//   S = Q K^T,  P = e^{x - m},  O += P V,  out = O / l,
// with the running maximum m and sum l of every row (one pass over the keys).
//
//  * Tiles of 128 rows (a "stage") by blocks of 128 keys.  S (fp32) and O (fp32)
//    lie in tensor memory; P overwrites S as fp16 and is the next product's A
//    operand there.  K and V blocks arrive by TMA, page by page, with the
//    128-byte swizzle the MMA reads; V is the N-major B operand as it lies.
//  * Two layouts.  NQ = 2: a tile has 256 rows, each of two warpgroups owns 128
//    of them (one row a thread), and one's softmax runs under the other's MMAs.
//    NQ = 1: 128 rows, S double-buffered over the key blocks; the two
//    warpgroups take 64 key columns of every row each and exchange row maxima
//    through shared memory.  NQ = 1 serves head size 256 (whose O fills half of
//    tensor memory) and calls that bring at most 128 rows a
//    sequence on average (decode, HBM-bound: the padded MMA rows cost nothing there).
//  * m moves only when it would grow by more than 2^8: O is rescaled a few times per
//    row, not per block.  Weights (and with them l and O, whose quotient does not change)
//    are 2^7 e^{x - m}: below 2^15, within fp16, and down to 2^-32 of the largest in the
//    product, so that many small ones together are not lost beside it.
//  * Work units are (tile, key block); every CTA (one per SM) takes an even,
//    contiguous range of all units, which its load warp finds from the lengths
//    on the device and announces tile by tile, so ragged batches and single long
//    contexts fill the GPU alike.  A tile cut between CTAs leaves fp32 partials
//    in the workspace; the last warp to arrive for its 32 rows merges them in
//    CTA order (results repeat).
//
// Measured (by GPU).  32 single tokens over contexts up to 16384, 64 heads, 8
// KV heads of 128: 205-208 us, 6.6 TB/s of keys and values, the rate of a plain copy.
// Four packed prompts up to 4096, 32 heads: 323-345 us, 990-1058 TFLOP/s; four
// chunks of 64 tokens over 24000, 64 heads on 8: 112 us, 925 TFLOP/s.  A block of
// a 256-row tile takes about 3200 SM clocks: 2048 are the MMAs (64 each), the
// rest is the chain of one stage (softmax 1550, its two products 1024 + 500 to
// completion and back) that the other stage's turn does not cover.  A tile's end
// (last product, rows out, next tile's first block) costs about 6000 clocks more.
// Small calls: about 10 us, half of it before the first S (lengths, first page,
// first block), where code and data are read for the first time.
#include <cuda.h>

#include <cfloat>
#include <cmath>
#include <cstring>
#include <mutex>

#include "seq_batch.cuh"

namespace qz {
namespace {

__device__ int g_attn_error = 0;

constexpr int kN = 128;                // keys per block
constexpr int kSoftmaxWarps = 8;       // two warpgroups
// With few rows only softmax warps 0 and 4 have any, both on the SM's first
// scheduler: the MMA and load warps sit on others.
constexpr int kQWarp = 8, kMmaWarp = 10, kLoadWarp = 11;  // 8 and 9: queries
constexpr int kThreads = 384;          // the third warpgroup: queries (2), MMA, keys and values
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;  // of 168 a thread at launch
static_assert(8 * kSoftmaxRegs + 4 * kOtherRegs <= 12 * 168, "register split");
constexpr int kMaxCtas = 160;          // grid cap (partial slots in the workspace)
constexpr int kBars = 4096;             // barriers and exchange rows at the start of shared memory
constexpr int kOutBytes = 32 * 64;     // per softmax warp: 32 rows x 32 outputs on their way out
constexpr int kHead = kBars + 8 * kOutBytes;
constexpr int kMaxStages = 8;
constexpr uint32_t kTmemCols = 512;
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s per wait
constexpr float kLag = 8.0f;           // log2 of how far a key may exceed m
constexpr float kLift = 7.0f;          // log2 of the weight at m
// Caps up to here come from 1 - 2 / (1 + e^2t) alone: off by 2^-22 of the cap, 1.5e-5 in a
// logit, a sixteenth of the weights' rounding.  Four prompts of up to 4096 take 327 us
// without a cap, 634 with one of these and 948 with the form for any cap; 32 decode tokens
// over 16384 207, 261 and 353.
constexpr float kShortCap = 64.0f;
static_assert(kLag + kLift < 16.0f, "weights are fp16");
constexpr float kLog2e = 1.4426950408889634f;
// Units per CTA at least.  One token over 199 keys takes 11.3 us with 1, 10.2 with 3
// and 13.6 with 6; over 1000 keys 13.2, 15.0 and 19.5.
constexpr int kMinUnits = 3;
// Time to merge one partial, in key blocks: 8 tokens (64 rows) over 30000 keys of one KV
// head take 51 us when all SMs share the tile, 34 with this, 31 with 0.5, which costs
// one token over 4096 keys 15.1 -> 17.0 us.
constexpr float kMergeUnits = 0.2f;
// A tile's fixed time, in key blocks.  256 rows: four prompts of up to 4096 take 343
// us with none, 326 with 1, 317 with 2; 128 rows: one token over 199 keys takes 15.1
// us with none, 10.2 with 1, 11.0 with 2.
template <int kM>
constexpr int kTileUnits = kM / 128;
constexpr int kSegs = 4;               // tiles announced ahead

template <int D, int NQ>
struct Cfg {
  static constexpr int kM = 128 * NQ;                  // rows of a tile
  static constexpr int kStage = kN * D * 2;            // bytes of a K or V block
  static constexpr int kQ = kM * D * 2;
  static constexpr int kNS = D == 256 ? 2 : D == 64 ? 8 : NQ == 2 ? 4 : 5;
  static constexpr int kSmem = kHead + kQ + kNS * kStage + 1024;
  static constexpr int kNC = NQ == 2 ? 128 : 64;       // key columns per softmax thread
  static constexpr int kDC = NQ == 2 ? D : D / 2;      // output columns per softmax thread
  static constexpr int kPart = 32 * (kDC + 2);         // floats of one warp's partial
};

struct AttnParams {
  CUtensorMap kmap, vmap;  // [page][head][slot][D], box 64 x min(page, 128) rows
  CUtensorMap qmap;        // [token][head][D], box 64 x G heads x tokens of half a tile
  int q_boxes;             // queries come by qmap
  const __half *q;
  __half *out;
  int64_t q_token, q_head, o_token, o_head;
  int G;                // query heads per KV head
  float inv_g;          // 1 / G
  uint64_t magic_g;     // ceil(2^64 / G), 0 for G = 1
  int hkv, n_pages, page_size, page_shift;
  float c;              // logit units to log2: |scale| log2(e), or log2(e) with a cap
  float cap, cap_in;    // softcap, and |scale| / softcap * 2 log2(e)
  float mag, cap_t;     // |scale|, and |scale| / softcap
  uint32_t keep, flip;  // queries are read as (bits & keep) ^ flip: signs turned when scale < 0,
                        // zeros when scale = 0 (c stays positive: masked logits are -inf)
  int window;           // 0: none
  SeqView s;
  unsigned *cnt;        // [kMaxCtas][8] arrivals per cut tile (by its first CTA) and warp
  float *part;          // [kMaxCtas][2][8] partials
};

// ------------------------------------------------------------ PTX pieces --
__device__ __forceinline__ uint32_t smem_u32(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ unsigned long long gtimer() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait for the phase of the given parity; false (and error 1) if it does not
// complete within kWaitNs or another wait of the CTA gave up.
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, int *abort_flag) {
  const unsigned long long t0 = gtimer();
  for (;;) {
    if (mbar_try(bar, parity)) return true;
    if (*(volatile int *)abort_flag) return false;
    if (gtimer() - t0 > kWaitNs) {
      atomicOr(&g_attn_error, 1);
      *(volatile int *)abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, int *abort_flag) {
  const bool ok = mbar_try(bar, parity) || mbar_wait_slow(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, ok);
}
// The same at the end of a CTA that gave up, until `until`: copies and products in flight
// have to be over before its memory goes.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity,
                                           unsigned long long until) {
  while (!mbar_try(bar, parity))
    if (gtimer() > until) return;
}
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.shared::cta.b64 st, [%0];\n\t}" ::"r"(bar)
      : "memory");
}
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
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two fp32 operations per instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 z, {%6, %7};\n\tfma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
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

// c ? a : b, both formed: a branch for each of a thread's 128 logits costs more.
__device__ __forceinline__ float pick(bool c, float a, float b) {
  float d;
  asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\tselp.f32 %0, %1, %2, p;\n\t}"
      : "=f"(d)
      : "f"(a), "f"(b), "r"((uint32_t)c));
  return d;
}
// cap tanh(t) of a product s = q . k, t = s |scale| / cap: tanh(t) = 1 - 2 / (1 + e^2t),
// which cancels for small t.
__device__ __forceinline__ float cap_far(const AttnParams &p, float s) {
  return p.cap * (1.0f - 2.0f * rcp(1.0f + ex2(s * p.cap_in)));
}
// The same for any cap: below 1/4 by the series t - t^3/3 + 2t^5/15 - 17t^7/315 + 62t^9/2835,
// whose next term is below 2^-26 of the first there.
__device__ __forceinline__ float cap_any(const AttnParams &p, float s) {
  const float t = s * p.cap_t, u = t * t, x = s * p.mag;
  float g = fmaf(u, 62.0f / 2835.0f, -17.0f / 315.0f);
  g = fmaf(u, g, 2.0f / 15.0f);
  g = fmaf(u, g, -1.0f / 3.0f);
  return pick(fabsf(t) < 0.25f, fmaf(x * u, g, x), cap_far(p, s));
}

// --------------------------------------------------------------- schedule --
// n / G for 0 <= n < 2^31, G <= 2^16: the excess of ceil(2^64 / G) over 2^64 / G
// adds less than n / 2^64 < 1 / G.
__device__ __forceinline__ int div_g(const AttnParams &p, int n) {
  return p.magic_g ? (int)__umul64hi((uint64_t)(uint32_t)n, p.magic_g) : n;
}
// Non-negative quotient; the 64-bit division costs several times the 32-bit one.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
  return a / b;
}

// A sequence, and its row tiles per KV head.
struct Seq {
  int i, tok0, q, kv;  // index, first token, new tokens, tokens held
  int rows, nt;        // q * G, row tiles
};

template <int kM>
__device__ __forceinline__ Seq load_seq(const AttnParams &p, int i) {
  Seq s;
  s.i = i;
  const int T = (int)p.s.n_tokens;
  const int a = max(__ldg(p.s.cu_q + i), 0), b = min(__ldg(p.s.cu_q + i + 1), T);
  s.tok0 = a;
  s.q = max(b - a, 0);
  s.kv = max(__ldg(p.s.kv_len + i), 0);
  s.rows = s.q * p.G;
  s.nt = (s.rows + kM - 1) / kM;
  return s;
}

// The first key that the row at position pos sees (pos - window + 1 would leave
// 32 bits for a long window before the first position).
__device__ __forceinline__ int first_key(const AttnParams &p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// Keys [lo, hi) that any row of row tile rt sees, and the blocks that hold them.
struct Range {
  int lo, hi, b0, nb;
};
template <int kM>
__device__ __forceinline__ Range tile_range(const AttnParams &p, const Seq &s, int rt) {
  Range r;
  const int first = s.kv - s.q;  // position of the first new token
  const int last = min((rt + 1) * kM, s.rows) - 1;
  r.hi = max(first + div_g(p, last) + 1, 0);
  r.lo = first_key(p, first + div_g(p, rt * kM));
  r.b0 = r.lo / kN;
  r.nb = r.hi > r.lo ? (r.hi - 1) / kN + 1 - r.b0 : 0;
  return r;
}

// Units of a tile: its key blocks (one if it sees no key), and before them the
// time that a tile costs whatever its length, in blocks.
template <int kM>
__device__ __forceinline__ int tile_units(const Range &r) {
  return kTileUnits<kM> + max(r.nb, 1);
}

// Units of one KV head of each lane's sequence (whole warp): long sequences'
// tiles are counted by all lanes together.
template <int kM>
__device__ __forceinline__ int64_t head_units(const AttnParams &p, const Seq &s) {
  constexpr int kOwn = 4;
  const int lane = threadIdx.x & 31;
  int64_t n = 0;
  for (int rt = 0; rt < min(s.nt, kOwn); ++rt) n += tile_units<kM>(tile_range<kM>(p, s, rt));
  for (unsigned m = __ballot_sync(0xffffffffu, s.nt > kOwn); m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    Seq t;
    t.q = __shfl_sync(0xffffffffu, s.q, src);
    t.kv = __shfl_sync(0xffffffffu, s.kv, src);
    t.rows = __shfl_sync(0xffffffffu, s.rows, src);
    t.nt = __shfl_sync(0xffffffffu, s.nt, src);
    int64_t v = 0;
    for (int rt = kOwn + lane; rt < t.nt; rt += 32) v += tile_units<kM>(tile_range<kM>(p, t, rt));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == src) n += v;
  }
  return n;
}

// What one CTA does of one tile, as the load warp tells the others.
struct __align__(16) Seg {
  int rows;            // rows of the tile (0: the CTA has no more tiles)
  int b0, b1;          // its key blocks [b0, b1) of this CTA; none if the tile sees no key
  int head;            // KV head
  int tok, rem, pos;   // token of row 0, row 0's place among that token's heads, its position
  int lo, hi;          // keys [lo, hi) that any row sees
  int slot;            // -1: all of the tile; else the CTA's partial slot
  int c_lo, parts;     // cut tile: first CTA, and how many share it
  int first_slot;      // cut tile: the first CTA's partial slot (the others': 0)
  int seq;             // sequence
  int pad[2];
};
static_assert(sizeof(Seg) == 64, "four 16-byte reads");

// Walks a CTA's unit range tile by tile (load warp only).  Units are counted
// from the CTA's first.
template <int kM>
struct Walker {
  int u, u_end, first;  // next unit, end, first unit of the current tile
  int seq, head, rt;
  int64_t u_begin, each;  // the CTA's first unit; units per CTA, and one more for the first `more`
  int more;
  __device__ __forceinline__ int64_t begin_of(int cta) const { return each * cta + min(cta, more); }
  __device__ __forceinline__ int owner(int64_t unit) const {
    const int64_t big = (each + 1) * more;
    return unit < big ? (int)div64(unit, each + 1) : more + (int)div64(unit - big, each);
  }
  template <int kPer>
  __device__ __forceinline__ bool start(const AttnParams &p);
  __device__ __forceinline__ Seg next(const AttnParams &p) {
    Seg g;
    g.rows = 0;
    while (u < u_end) {
      Seq s = load_seq<kM>(p, seq);
      while (rt >= s.nt) {  // sequences without new tokens have no tiles
        rt = 0;
        if (s.nt == 0 || ++head == p.hkv) {
          head = 0;
          s = load_seq<kM>(p, ++seq);
        }
      }
      const Range r = tile_range<kM>(p, s, rt);
      const int units = tile_units<kM>(r), tile_first = first;
      const int a = max(u - first - kTileUnits<kM>, 0);                 // of its blocks
      const int b = min(u_end - first, units) - kTileUnits<kM>;
      g.slot = u == 0 ? 0 : 1;
      g.head = head;
      g.seq = seq;
      const int row0 = rt * kM;
      const bool done = u_end - first >= units;
      u = first + min(u_end - first, units);
      if (done) {
        first += units;
        ++rt;
      }
      if (b <= a) continue;  // only the fixed part of the tile's time falls to this CTA
      const int i0 = div_g(p, row0);
      g.rows = min(s.rows - row0, kM);
      g.tok = s.tok0 + i0;
      g.rem = row0 - i0 * p.G;
      g.pos = s.kv - s.q + i0;
      g.lo = r.lo;
      g.hi = r.hi;
      g.b0 = r.b0 + a;
      g.b1 = r.nb == 0 ? g.b0 : r.b0 + b;
      g.c_lo = g.parts = g.first_slot = 0;
      if (a == 0 && done) {
        g.slot = -1;
      } else {
        g.c_lo = owner(u_begin + tile_first + kTileUnits<kM>);
        g.parts = owner(u_begin + tile_first + units - 1) - g.c_lo + 1;
        if (g.parts == 1) g.slot = -1;
        g.first_slot = begin_of(g.c_lo) >= u_begin + tile_first ? 0 : 1;
      }
      break;
    }
    return g;
  }
};

// Inclusive sum over the lanes.
__device__ __forceinline__ int64_t warp_scan(int64_t v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// This CTA's range of the units of all sequences, and the tile that holds its
// first one (whole warp; kPer sequences a lane at a time).  False: no units.
template <int kM>
template <int kPer>
__device__ __forceinline__ bool Walker<kM>::start(const AttnParams &p) {
  const int lane = threadIdx.x & 31, S = p.s.n_seqs;
  int64_t h[kPer];  // units per head of this lane's sequences
  int64_t tiles = 0;  // of this lane's sequences
  auto count = [&](int i0) {
    Seq s[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {  // all loads ahead of their uses
      const int i = i0 + lane * kPer + k;
      s[k] = load_seq<kM>(p, min(i, S - 1));
      if (i >= S) s[k].nt = 0;
    }
    int64_t n = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      n += h[k] = head_units<kM>(p, s[k]);
      tiles += s[k].nt;
    }
    return warp_scan(n * p.hkv);
  };
  int64_t total = 0, incl = 0;
  for (int i0 = 0; i0 < S; i0 += 32 * kPer) {
    incl = count(i0);
    total += __shfl_sync(0xffffffffu, incl, 31);
  }
  // A tile cut in n leaves n partials for one CTA to merge, about kMergeUnits of
  // a block's time each, so a tile of U units is best cut in sqrt(U / kMergeUnits).
  tiles = __shfl_sync(0xffffffffu, warp_scan(tiles), 31) * p.hkv;
  const float cuts = (float)tiles * sqrtf((float)total / ((float)tiles * kMergeUnits));
  const int ctas = (int)min(min((int64_t)gridDim.x, div64(total + kMinUnits - 1, kMinUnits)),
                            (int64_t)ceilf(fmaxf(cuts, 1.0f)));
  if ((int)blockIdx.x >= ctas) return false;
  each = div64(total, ctas);
  more = (int)(total - each * ctas);
  u_begin = begin_of(blockIdx.x);
  u = 0;
  u_end = (int)(begin_of(blockIdx.x + 1) - u_begin);
  int64_t before = 0;
  for (int i0 = 0;; i0 += 32 * kPer) {
    if (S > 32 * kPer) incl = count(i0);
    const unsigned m = __ballot_sync(0xffffffffu, before + incl > u_begin);
    if (m == 0) {
      before += __shfl_sync(0xffffffffu, incl, 31);
      continue;
    }
    const int src = __ffs(m) - 1;
    int64_t at = before + incl, hs = 0;
    int i = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) at -= h[k] * p.hkv;  // units before this lane's sequences
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (hs == 0 && u_begin < at + h[k] * p.hkv) {
        hs = h[k];
        i = i0 + lane * kPer + k;
      } else if (hs == 0) {
        at += h[k] * p.hkv;
      }
    }
    seq = __shfl_sync(0xffffffffu, i, src);
    at = __shfl_sync(0xffffffffu, at, src);
    hs = __shfl_sync(0xffffffffu, hs, src);
    head = (int)div64(u_begin - at, hs);
    at += head * hs;
    const Seq s = load_seq<kM>(p, seq);
    for (rt = 0;; rt += 32) {
      const int n = rt + lane < s.nt ? tile_units<kM>(tile_range<kM>(p, s, rt + lane)) : 0;
      const int64_t in = warp_scan(n);
      const unsigned t = __ballot_sync(0xffffffffu, at + in > u_begin);
      if (t == 0) {
        at += __shfl_sync(0xffffffffu, in, 31);
        continue;
      }
      const int l = __ffs(t) - 1;
      first = (int)(at + __shfl_sync(0xffffffffu, in - n, l) - u_begin);
      rt += l;
      return true;
    }
  }
}

// ---------------------------------------------------------------- kernel --
// CAP: 0 none, 1 of up to kShortCap, 2 of any size.
template <int D, int NQ, int CAP>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ AttnParams p) {
  using C = Cfg<D, NQ>;
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
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drained + 1);
  int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);
  // Copies that the load warp has issued, tiles that the query warps have
  uint32_t *issued = reinterpret_cast<uint32_t *>(abort_flag + 1);  // [kLoadWarp - kQWarp + 1]
  Seg *seg_sm = reinterpret_cast<Seg *>(base + 512);         // [kSegs]
  float *xch = reinterpret_cast<float *>(base + 1024);       // [2][8 warps][32]
  uint8_t *q_sm = base + kHead, *kv_sm = q_sm + C::kQ;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&kv_full[i]), 1);
      mbar_init(smem_u32(&kv_empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&p_full[i]), NQ == 2 ? 4 : 8);
      mbar_init(smem_u32(&o_done[i]), 1);
      mbar_init(smem_u32(&p_half[i]), 4);
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
        float s[NC];
#pragma unroll
        for (int k = 0; k < NC / 32; ++k)
          tmem_ld32(s_tm + col0 + 32 * k, reinterpret_cast<uint32_t *>(s) + 32 * k);
        tmem_ld_wait();
        if (CAP) {
#pragma unroll
          for (int k = 0; k < NC; ++k) s[k] = CAP == 1 ? cap_far(p, s[k]) : cap_any(p, s[k]);
        }
        // keys [k_lo, k_hi) of this row; a block that no bound cuts needs neither
        if (see_hi - b * kN < col0 + NC) {  // (the block's end may pass 32 bits)
          const int k_hi = hi - b * kN - col0;
#pragma unroll
          for (int k = 0; k < NC; ++k) s[k] = k < k_hi ? s[k] : -INFINITY;
        }
        if (b * kN + col0 < see_lo) {
          const int k_lo = lo - b * kN - col0;
#pragma unroll
          for (int k = 0; k < NC; ++k) s[k] = k >= k_lo ? s[k] : -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int k = 4; k < NC - 4; k += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[k + 2 * e], s[k + 2 * e + 1]);
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], s[NC - 4 + e]);
        float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (NQ == 1) {
          float other;
          if (!(ok = exchange(mb, &other))) break;
          mb = fmaxf(mb, other);
        }
        // move the maximum where it lags too far, and rescale what was summed
        const bool move = (mb - m) * p.c > kLag || (m == -INFINITY && mb > -INFINITY);
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? mb : m;
          const float f = m == -INFINITY ? (move ? 0.0f : 1.0f) : ex2((m - mn) * p.c);
          m = mn;
          l *= f;
          if (b > g.b0) {
            // NQ = 2: this stage's earlier products precede the S just read
            if (NQ == 1 && !(ok = last_product(b))) break;
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
        const float mc = m == -INFINITY ? 0.0f : m * p.c - kLift;
        const float2 c2 = make_float2(p.c, p.c), mc2 = make_float2(-mc, -mc);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
        for (int h = 0; h < NC / 32; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float2 e = fma2(make_float2(s[32 * h + 2 * k], s[32 * h + 2 * k + 1]), c2, mc2);
            e.x = ex2(e.x);
            e.y = ex2(e.y);
            sum[k & 1] = add2(sum[k & 1], e);
            pk[k] = f2h(e.x, e.y);
          }
          tmem_st16(s_tm + col0 / 2 + 16 * h, pk);
          if (NQ == 2 && h == 1) {  // the product starts on these
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
        if (lane == 0) mbar_arrive(smem_u32(&p_full[buf]));
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
      mine_part[lane] = l > 0.0f ? (m == -INFINITY ? 0.0f : m * p.c) : -INFINITY;
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
      return mbar_wait(smem_u32(&kv_full[r % NS]), (r / NS) & 1, abort_flag);
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
    // a zero weight times NaN is NaN: they become zeros.
    auto clean = [&](uint32_t r, int b, const Seg &t) {
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
            pv(t, 0, 256 + t * D, v, j > 0, false, nullptr);
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
    uint32_t n_seg = 0, segs = 0;
    for (;;) {
      Seg g;
      if (!read_seg(n_seg, g)) break;
      free_seg(n_seg++);
      if (g.rows == 0) break;
      if (g.b1 <= g.b0) continue;
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
        if (lane == 0) {
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
        }
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
    auto issue = [&](const CUtensorMap *map, const Seg &g, int b, int page) -> bool {
      const int slot = ring % NS;
      if (ring >= NS &&
          !mbar_wait(smem_u32(&kv_empty[slot]), (ring / NS - 1) & 1, abort_flag))
        return false;
      const uint32_t bar = smem_u32(&kv_full[slot]);
      const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
      if (lane == 0)
        asm volatile(
            "{\n\t.reg .b64 t;\n\t"
            "mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(bar),
            "r"((uint32_t)(__popc(live) * box_rows * D * 2))
            : "memory");
      __syncwarp();
      if (page >= 0) {
        const int at = p.page_size > kN ? (b * kN) & (p.page_size - 1) : 0;
        const uint32_t dst = smem_u32(kv_sm) + slot * C::kStage + lane * box_rows * 128;
#pragma unroll
        for (int d = 0; d < D / 64; ++d)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst + d * 16384),
              "l"(reinterpret_cast<uint64_t>(map)), "r"(d * 64), "r"(at), "r"(g.head), "r"(page),
              "r"(bar)
              : "memory");
      }
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
          ok = issue(&p.kmap, g, b, page);
          if (NQ == 1) {  // K0, K1, V0, K2, V1, ..., the order in which they are used
            if (ok && j > 0) ok = issue(&p.vmap, g, b - 1, prev);
            if (ok && j == nb - 1) ok = issue(&p.vmap, g, b, page);
          } else if (ok) {
            ok = issue(&p.vmap, g, b, page);
          }
          prev = page;
        }
        if (ok && j == 0 && n_seg == 1) ok = announce(next = w.next(p));
      }
    }
    if (lane == 0) issued[kLoadWarp - kQWarp] = ring;
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
    } else if (warp >= kQWarp && issued[warp - kQWarp] > 0) {
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

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point.
EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  });
  return fn;
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

// The pool as [page][head][slot][64-column group of D], boxes of one page's
// (at most 128) slots by 64 columns.
qz_status pool_map(CUtensorMap *map, const __half *base, const PagedView &c, int64_t token,
                   int64_t head, int64_t page) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return QZ_ERR_CUDA;
  // a dimension of one element has no stride of its own
  if (c.hkv == 1) head = token;
  if (c.n_pages == 1) page = token;
  const cuuint64_t dim[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page_size, (cuuint64_t)c.hkv,
                             (cuuint64_t)c.n_pages};
  const cuuint64_t stride[3] = {(cuuint64_t)token * 2, (cuuint64_t)head * 2, (cuuint64_t)page * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)(c.page_size < kN ? c.page_size : kN), 1, 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<__half *>(base), dim, stride, box,
         estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? QZ_OK : QZ_ERR_UNSUPPORTED;
}

template <int D, int NQ, int CAP>
qz_status launch(const AttnParams &p, int sms, cudaStream_t s) {
  using C = Cfg<D, NQ>;
  const cudaError_t e = allow_smem<attn_kernel<D, NQ, CAP>>(C::kSmem);
  if (e != cudaSuccess) return cuda_status(e);
  attn_kernel<D, NQ, CAP><<<sms < kMaxCtas ? sms : kMaxCtas, kThreads, C::kSmem, s>>>(p);
  return launch_status();
}

template <int D, int NQ>
qz_status launch_cap(const AttnParams &p, int sms, cudaStream_t s) {
  if (p.cap == 0.0f) return launch<D, NQ, 0>(p, sms, s);
  return p.cap <= kShortCap ? launch<D, NQ, 1>(p, sms, s) : launch<D, NQ, 2>(p, sms, s);
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t D) {
  const int64_t part = 32 * ((D == 256 ? 128 : D) + 2);  // the larger of the two layouts
  return QZ_ATTENTION_SYNC_BYTES + (size_t)kMaxCtas * 2 * kSoftmaxWarps * part * sizeof(float);
}
static_assert(kMaxCtas * kSoftmaxWarps * sizeof(unsigned) <= QZ_ATTENTION_SYNC_BYTES, "counters");

qz_status launch_attention(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                           const PagedView &c, const SeqView &sv, float scale, float softcap,
                           int64_t window, __half *out, int64_t o_token, int64_t o_head,
                           void *workspace, cudaStream_t s) {
  DeviceInfo di;
  qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  st = pool_map(&p.kmap, c.k, c, c.k_token, c.k_head, c.k_page);
  if (st == QZ_OK) st = pool_map(&p.vmap, c.v, c, c.v_token, c.v_head, c.v_page);
  if (st != QZ_OK) return st;
  p.q = q;
  p.out = out;
  p.q_token = q_token;
  p.q_head = q_head;
  p.o_token = o_token;
  p.o_head = o_head;
  p.G = (int)(hq / c.hkv);
  p.inv_g = 1.0f / (float)p.G;
  p.magic_g = p.G > 1 ? ~(uint64_t)0 / (uint64_t)p.G + 1 : 0;
  p.hkv = c.hkv;
  p.n_pages = c.n_pages;
  p.page_size = c.page_size;
  p.page_shift = c.page_shift;
  const float mag = scale == 0.0f ? 1.0f : fabsf(scale);
  p.keep = scale == 0.0f ? 0u : ~0u;
  p.flip = scale < 0.0f ? 0x80008000u : 0u;
  p.c = (softcap > 0.0f ? 1.0f : mag) * kLog2e;
  p.cap = softcap;
  // (finite for the smallest caps: a logit of 0 stays 0, the others reach the cap all the same)
  p.mag = mag;
  p.cap_t = softcap > 0.0f ? fminf(mag / softcap, FLT_MAX) : 0.0f;
  p.cap_in = fminf(p.cap_t * 2.0f * kLog2e, FLT_MAX);
  p.window = window > INT32_MAX ? 0 : (int)window;  // longer than any cache: none
  p.s = sv;
  p.cnt = static_cast<unsigned *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + QZ_ATTENTION_SYNC_BYTES);
  // Two stages of rows pay once a sequence fills the second one: 4 x 64 tokens
  // over 24000 keys, 64 heads on 8, take 111 us with two and 144 with one, four
  // prompts of up to 4096 326 and 381; 8 x 16 tokens over 4000 36.2 with one, 39.7
  // with two, 64 single tokens, 32 heads, 97 and 125.  Short prompts, whose tiles
  // are few, would gain with one (6 of up to 300: 26.8 -> 24.8), but the lengths
  // are known on the device only.  So the rows are the average: a prompt beside many
  // single tokens (one of 4096 and 63 of 1, a KV head a head) has one stage.
  const bool two = c.D < 256 && sv.n_tokens * p.G > (int64_t)128 * sv.n_seqs;
  p.q_boxes = scale > 0.0f && query_map(&p.qmap, q, sv.n_tokens, hq, c.D, q_token, q_head, p.G,
                                        two ? 128 : 64);
  if (c.D == 256) return launch_cap<256, 1>(p, di.sms, s);
  if (c.D == 128) return two ? launch_cap<128, 2>(p, di.sms, s) : launch_cap<128, 1>(p, di.sms, s);
  return two ? launch_cap<64, 2>(p, di.sms, s) : launch_cap<64, 1>(p, di.sms, s);
}

qz_status read_attn_error(int *code, int clear) {
  return read_error_word(g_attn_error, code, clear);
}

}  // namespace qz
