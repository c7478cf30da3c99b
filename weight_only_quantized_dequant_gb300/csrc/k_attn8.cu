// Attention of a step's new tokens over the paged cache of INT8 rows, for steps
// that bring few rows to a KV head (decode and drafts).
//
// For one KV head the queries of a sequence are packed row r = token * G +
// head-in-group; a tile has 8 of them (16: NB = 2), and
//   x_j = scale ks_j (q . kc_j),  out = sum_j e^{x_j} vs_j vc_j / sum_j e^{x_j}
// over the codes kc, vc and the scales ks, vs of the keys.  Codes are exact in fp16
// (a byte under the bits of 1024, less 1152, is the code), so they enter the
// products as they are: ks_j multiplies the logit, vs_j the weight, both in fp32.
//
//  * HBM bounds a decode step: a token and head is 2 (D + 4) bytes, 11 clocks of an
//    SM's share at D 128.  The warp's matrix instruction takes 8 clocks an SM whatever
//    its operands hold, so the rows are its narrow side (8 columns): S^T = K Q^T and
//    O^T = V^T P^T, a key 1/8 of two instructions a step of 16 columns, 8 clocks.
//    With the rows as its 16-row operand a key took 16 (32 tokens over 16384 keys, 64
//    heads on 8: 212 us).
//  * A block of 128 keys comes by TMA, page by page, with the swizzle under which the
//    fragments' 16-byte reads do not conflict; each of eight warps has 16 of the keys to
//    itself, converts their codes, and has a running maximum, sum and output of its own,
//    so nothing is exchanged before the tile's end.
//  * The order of D in a product is free as long as both operands have it: a thread's
//    16 bytes of a key are four steps of the first product, and of a value eight rows
//    of the second's tiles, so that both come as whole 16-byte reads.
//  * Weights are rounded to fp16 once, with vs_j in them: 2^6 e^{x - m} vs_j 2^-E,
//    where m lags the maximum by up to 2^8 and 2^E the largest vs by up to 2.  Their sum
//    is of the rounded ones: where a few keys have most of a row's weight the rounding
//    cancels (8 tokens over 8000 random keys: 2.3e-4 of the output against 2.9e-4 with the
//    sum of the others; the output's own rounding is 2.1e-4).
//    A pair of tiles of 16 rows a sequence (drafts) is still faster than one tile of the
//    other kernel.
//  * Measured: 32 tokens over up to 16384 keys, 64 heads on 8, D 128, 124 us, 5.7 TB/s (the
//    fp16 kernel 207 over its rows); D 64, 32 on 8, 86; 8 over 8192, D 256, cap and window, 34;
//    one token over 200 keys 8.2, which is the launch, the plan and one chain of loads.
//  * The split of (tile, key block) units between CTAs is that of the fp16 kernel.
#include <cstring>

#include "attn_plan.cuh"

namespace qz {
namespace {

constexpr float kLift8 = 6.0f;        // log2 of the weight at m
static_assert(kLift8 + kLag + 1.0f < 16.0f, "weights are fp16");
constexpr int kHead8 = 4096;          // barriers, announced tiles, row maxima and sums

template <int D, int NB>
struct Cfg8 {
  static constexpr int kM = 8 * NB;                 // rows of a tile
  // Warps that multiply: 8, each with 16 of a block's keys, or two such groups that take
  // blocks in turn.  32 tokens over 16384 keys: D 64, 32 heads on 8, 99 us with one group and
  // 86 with two (a warp's chain of loads, conversions and products is longer than its bytes
  // take), D 128, 64 on 8, 124 and 138 (96 registers a thread).
  static constexpr int kGroups = NB == 1 && D == 64 ? 2 : 1;
  static constexpr int kWarps = 8 * kGroups;
  // and a warpgroup that loads
  static constexpr int kThreads = kWarps * 32 + 128;
  static constexpr int kLaunchRegs = kGroups == 2 ? 96 : 168;  // a thread
  static constexpr int kMathRegs = kGroups == 2 ? 104 : 216;
  static constexpr int kOtherRegs = kGroups == 2 ? 64 : 72;
  static_assert(kWarps * kMathRegs + 4 * kOtherRegs <= (kWarps + 4) * kLaunchRegs, "registers");
  static constexpr int kRow = D < 128 ? D : 128;    // bytes of a swizzled row
  static constexpr int kStage = kN * D;             // bytes of a K or V block
  static constexpr int kNS = 131072 / kStage;       // K and V slots: 16, 8, 4
  static constexpr int kSteps = D / 16;             // of the first product
  static constexpr int kBuf = kWarps * kM * kRow * 4;  // warps' outputs, 128 columns at a time
  static constexpr int kQ = D == 256 && NB == 2 ? kSteps * 512 : 0;  // queries by step
  static constexpr int kSmem = 1024 + kHead8 + kNS * kN * 4 + kNS * kStage + kBuf + kQ;
  static constexpr int kPart = kM * (D + 2);        // floats of a partial
};

struct Attn8Params : PlanParams, CapParams, ScaleParams {
  CUtensorMap kmap, vmap;  // [page][head][slot][D] bytes, box 128 (64) x min(page, 128)
  const __half *q;
  __half *out;
  int64_t q_token, q_head, o_token, o_head;
  float c;       // logit units to log2 of what the product and ks give
  float sign;    // of the scale (0: no logits)
  unsigned *cnt; // [kMaxCtas] arrivals per cut tile, by its first CTA
  float *part;   // [kMaxCtas][2] partials
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of fp16, two of a row a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float lds32f(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}

template <int D, int NB, int CAP>
__global__ void __launch_bounds__(Cfg8<D, NB>::kThreads, 1)
    attn8_kernel(const __grid_constant__ Attn8Params p) {
  using C = Cfg8<D, NB>;
  constexpr int kWarps = C::kWarps, kLoadWarp = kWarps, GR = C::kGroups;
  constexpr int kM = C::kM, NS = C::kNS, KS = C::kSteps, MT = D / 16;
  constexpr bool kQinSm = C::kQ > 0;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t *kv_sm = base;
  uint8_t *buf_sm = kv_sm + NS * C::kStage;
  uint8_t *q_sm = buf_sm + C::kBuf;
  float *scale_sm = reinterpret_cast<float *>(q_sm + C::kQ);  // [NS][kN]
  uint8_t *head = reinterpret_cast<uint8_t *>(scale_sm + NS * kN);
  uint64_t *kv_full = reinterpret_cast<uint64_t *>(head), *kv_empty = kv_full + 16;
  uint64_t *seg_full = kv_empty + 16, *seg_empty = seg_full + kSegs;
  uint64_t *met = seg_empty + kSegs;  // the eight warps of a tile
  int *abort_flag = reinterpret_cast<int *>(met + 1);
  unsigned *arrived_sm = reinterpret_cast<unsigned *>(abort_flag + 1);
  Seg *seg_sm = reinterpret_cast<Seg *>(head + 512);           // [kSegs]
  float2 *ml_sm = reinterpret_cast<float2 *>(head + 1024);     // [2][kWarps][kM] maximum and sum

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(&kv_full[i]), p.runs ? 1 : 33);
      mbar_init(smem_u32(&kv_empty[i]), 8);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(smem_u32(&seg_full[i]), 1);
      mbar_init(smem_u32(&seg_empty[i]), kWarps + 3);
    }
    mbar_init(smem_u32(met), kWarps);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  Walker<kM> w;
  w.u = w.u_end = 0;
  if (warp == kLoadWarp) {
    if (p.s.n_seqs <= 32)
      w.template start<1>(p);
    else
      w.template start<8>(p);
  }
  __syncthreads();
  uint32_t issued = 0;  // blocks up to the last that this warp loaded of

  // The n-th announced tile (every warp but the one that announces).
  auto read_seg = [&](uint32_t n, Seg &s) -> bool {
    if (!mbar_wait(smem_u32(&seg_full[n % kSegs]), (n / kSegs) & 1, abort_flag)) return false;
    const uint4 *src = reinterpret_cast<const uint4 *>(&seg_sm[n % kSegs]);
    uint4 *dst = reinterpret_cast<uint4 *>(&s);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = src[i];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&seg_empty[n % kSegs]));
    return true;
  };

  if (warp < kWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMathRegs));
    const int g = lane >> 2, t = lane & 3;
    const int own = warp & 7, group = warp >> 3;  // place in the group
    // n / G for n < G + 256 (see the fp16 kernel)
    auto row_token = [&](int n) { return (int)(((float)n + 0.5f) * p.inv_g); };
    const uint32_t kv0 = smem_u32(kv_sm), sc0 = smem_u32(scale_sm) + own * 64;
    // this thread's 16 bytes of a key: rows g and g + 8 of the warp's 16, chunks 2 t and 2 t + 1
    // (of 8; D 64: t of 4); of a value: rows 2 t + {0, 1, 8, 9}, chunk g (D 64: half of g / 2)
    const int krow = own * 16 + g;
    const uint32_t k_at = krow * C::kRow;
    const uint32_t k_sw = D == 64 ? (t ^ ((krow >> 1) & 3)) << 4 : ((2 * t) ^ (krow & 7)) << 4;
    uint32_t v_at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = own * 16 + 2 * t + (i & 1) + (i >> 1) * 8;
      v_at[i] = r * C::kRow + (D == 64 ? (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8
                                       : (g ^ (r & 7)) << 4);
    }
    // where a row's float4 piece lies in its line of the buffer: 8 lanes with the same piece
    // of two rows' worth of chunks store to different banks
    auto place = [](int row, int piece) {
      const int u = (row >> 1) & 3;
      return piece ^ (D == 64 ? (u & 1) | (u >> 1) << 2 : u);
    };
    uint32_t n_seg = 0, ring = 0, n_met = 0;
    bool ok = true;
    // All eight warps have come here; false if one gave up.
    auto meet = [&]() -> bool {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(met));
      return ok = mbar_wait(smem_u32(met), n_met++ & 1, abort_flag);
    };
    // Queries of a tile: row 8 b + g as an operand (past the tile's end: its last row's).  Step
    // i of the first product has columns 4 i .. 4 i + 3 of this thread's D / 4 (of each 128: D
    // 256).
    uint32_t qb[kQinSm ? 1 : NB][kQinSm ? 1 : KS][2];
    auto query_row = [&](const Seg &s, int b) -> const __half * {
      const int n = s.rem + min(8 * b + g, s.rows - 1), k = row_token(n);
      return p.q + (int64_t)(s.tok + k) * p.q_token +
             (int64_t)(s.head * p.G + n - k * p.G) * p.q_head;
    };
    auto load_queries = [&](const Seg &s) {
      if constexpr (!kQinSm) {
        if (s.rows == 0) return;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const __half *row = query_row(s, b);
#pragma unroll
          for (int i = 0; i < KS; i += 2) {
            const int d = D == 256 ? (i >> 3) * 128 + 32 * t + 4 * (i & 7) : t * (D / 4) + 4 * i;
            const uint4 a = *reinterpret_cast<const uint4 *>(row + d);
            qb[b][i][0] = a.x, qb[b][i][1] = a.y;
            qb[b][i + 1][0] = a.z, qb[b][i + 1][1] = a.w;
          }
        }
      }
    };
    Seg s, next;
    bool taken = false;  // the next tile is read, its queries on their way
    auto take = [&] {
      taken = true;
      ok = read_seg(n_seg++, next);
      if (ok) load_queries(next);
    };
    auto advance = [&] {
      if (!taken) take();
      taken = false;
      s = next;
    };
    for (advance(); ok && s.rows > 0; advance()) {
      const int par = n_seg & 1;
      // rows 8 b + 2 t and 2 t + 1 of the logits
      int hi[NB][2], lo[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int pos = s.pos + row_token(s.rem + min(8 * b + 2 * t + e, s.rows - 1));
          hi[b][e] = pos + 1;
          lo[b][e] = first_key(p, pos);
        }
      }
      int see_lo = max(lo[0][0], lo[NB - 1][1]), see_hi = min(hi[0][0], hi[NB - 1][1]);
      see_lo = __reduce_max_sync(0xffffffffu, see_lo);
      see_hi = __reduce_min_sync(0xffffffffu, see_hi);
      if (kQinSm) {
        const __half *q0 = query_row(s, 0), *q1 = query_row(s, NB - 1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = warp * 2 + k, d = (i >> 3) * 128 + 32 * t + 4 * (i & 7);
          const uint2 a = *reinterpret_cast<const uint2 *>(q0 + d);
          const uint2 c = *reinterpret_cast<const uint2 *>(q1 + d);
          *reinterpret_cast<uint4 *>(q_sm + i * 512 + lane * 16) = make_uint4(a.x, a.y, c.x, c.y);
        }
        if (!meet()) break;
      }
      float o[MT][NB][4];
      float m[NB][2], l[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        m[b][0] = m[b][1] = -INFINITY;
        l[b][0] = l[b][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < MT; ++i) o[i][b][0] = o[i][b][1] = o[i][b][2] = o[i][b][3] = 0.0f;
      }
      float e_pos = exp2f(-40.0f), e_neg = exp2f(40.0f);  // 2^E and 2^-E
      const uint32_t ring0 = ring;
      ring += 2 * (s.b1 - s.b0);
      for (int blk = s.b0 + group; blk < s.b1; blk += GR) {
        const uint32_t at0 = ring0 + 2 * (blk - s.b0);  // of the K slot; the V slot follows
        const uint32_t ks = at0 % NS, vs = ks + 1;
        if (!(ok = mbar_wait(smem_u32(&kv_full[ks]), (at0 / NS) & 1, abort_flag))) break;
        const int key0 = own * 16;  // of the block
        // (the block's end may pass 32 bits)
        const bool none = s.hi - blk * kN <= key0 || (int64_t)blk * kN + key0 + 16 <= s.lo;
        float x[NB][4];  // keys g (0, 1) and g + 8 (2, 3) of rows 2 t and 2 t + 1
        if (!none) {
          float sa[NB][4], sb[NB][4];
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) sa[b][j] = sb[b][j] = 0.0f;
          const uint32_t kb = kv0 + ks * C::kStage + k_at;
#pragma unroll
          for (int h = 0; h < KS / 4; ++h) {  // 16 bytes of a key, four steps
            const uint32_t at = kb + (h >> 1) * (kN * 128) + (k_sw ^ ((h & 1) << 4));
            const uint4 k0 = lds128(at), k1 = lds128(at + 8 * C::kRow);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u0 = w0[i] ^ 0x80808080u, u1 = w1[i] ^ 0x80808080u;
              const uint32_t a[4] = {code_pair(u0, 0x4140), code_pair(u1, 0x4140),
                                     code_pair(u0, 0x4342), code_pair(u1, 0x4342)};
              uint32_t q[4];
              if (kQinSm) {
                const uint4 v = lds128(smem_u32(q_sm) + (4 * h + i) * 512 + lane * 16);
                q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
              }
#pragma unroll
              for (int b = 0; b < NB; ++b)
                mma16816(i & 1 ? sb[b] : sa[b], a,
                         kQinSm ? q[2 * b] : qb[kQinSm ? 0 : b][kQinSm ? 0 : 4 * h + i][0],
                         kQinSm ? q[2 * b + 1] : qb[kQinSm ? 0 : b][kQinSm ? 0 : 4 * h + i][1]);
            }
          }
          const float f0 = lds32f(sc0 + ks * (kN * 4) + g * 4) * p.sign;
          const float f1 = lds32f(sc0 + ks * (kN * 4) + 32 + g * 4) * p.sign;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float v = (sa[b][j] + sb[b][j]) * (j < 2 ? f0 : f1);
              x[b][j] = (CAP == 0 ? v : CAP == 1 ? cap_far(p, v) : cap_any(p, v)) * p.c;
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&kv_empty[ks]));
        if (!(ok = mbar_wait(smem_u32(&kv_full[vs]), (at0 / NS) & 1, abort_flag))) break;
        if (!none) {
          const int k0 = key0 + g;  // keys k0 and k0 + 8 of the block
          if (see_hi - blk * kN < key0 + 16) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (k0 + 4 * (j & 2) >= hi[b][j & 1] - blk * kN) x[b][j] = -INFINITY;
          }
          if (key0 < see_lo - blk * kN) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (k0 + 4 * (j & 2) < lo[b][j & 1] - blk * kN) x[b][j] = -INFINITY;
          }
          float v0 = lds32f(sc0 + vs * (kN * 4) + g * 4);
          float v1 = lds32f(sc0 + vs * (kN * 4) + 32 + g * 4);
          if (s.hi - blk * kN < key0 + 16 || s.lo - blk * kN > key0) {
            // scales of keys that no row sees may be anything
            auto seen = [&](int k) { return k < s.hi - blk * kN && k >= s.lo - blk * kN; };
            v0 = seen(k0) ? v0 : 0.0f;
            v1 = seen(k0 + 8) ? v1 : 0.0f;
          }
          bool move = fmaxf(v0, v1) * e_neg > 2.0f;
#pragma unroll
          for (int b = 0; b < NB; ++b)
            move |= fmaxf(x[b][0], x[b][2]) > m[b][0] + kLag ||
                    fmaxf(x[b][1], x[b][3]) > m[b][1] + kLag;
          if (__any_sync(0xffffffffu, move)) {
            float sv = fmaxf(v0, v1);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) sv = fmaxf(sv, __shfl_xor_sync(0xffffffffu, sv, d));
            const float e = fmaxf(e_pos, __uint_as_float(__float_as_uint(sv) & 0x7f800000u));
            const float fe = e_pos * (1.0f / e);
            e_pos = e;
            e_neg = 1.0f / e;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float mn = fmaxf(x[b][i], x[b][i + 2]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1)
                  mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
                mn = fmaxf(mn, m[b][i]);
                const float f = m[b][i] == -INFINITY ? 0.0f : ex2(m[b][i] - mn);
                m[b][i] = mn;
                l[b][i] *= f;
#pragma unroll
                for (int k = 0; k < MT; ++k) {
                  o[k][b][i] *= f * fe;
                  o[k][b][i + 2] *= f * fe;
                }
              }
          }
          const float n0 = v0 * e_neg, n1 = v1 * e_neg, i0 = rcp(n0), i1 = rcp(n1);
          // a weight as its product has it: what rounding did to a row's largest few is in
          // its sum too (not below fp16's normal numbers, which small scales lead to)
          auto summed = [](float w, float r, float inv) { return r >= 0x1p-14f ? r * inv : w; };
          uint32_t pb[NB][2];
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const float z0 = m[b][0] == -INFINITY ? 0.0f : kLift8 - m[b][0];
            const float z1 = m[b][1] == -INFINITY ? 0.0f : kLift8 - m[b][1];
            const float a0 = ex2(x[b][0] + z0), a1 = ex2(x[b][1] + z1);
            const float b0 = ex2(x[b][2] + z0), b1 = ex2(x[b][3] + z1);
            const uint32_t pa = f2h(a0 * n0, a1 * n0), pc = f2h(b0 * n1, b1 * n1);
            const float2 ra = h2f(pa), rc = h2f(pc);
            l[b][0] += summed(a0, ra.x, i0) + summed(b0, rc.x, i1);
            l[b][1] += summed(a1, ra.y, i0) + summed(b1, rc.y, i1);
            pb[b][0] = transpose8(pa);
            pb[b][1] = transpose8(pc);
          }
          const uint32_t vbase = kv0 + vs * C::kStage;
#pragma unroll
          for (int h = 0; h < (D + 127) / 128; ++h) {
            uint32_t r[4][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (D == 64) {
                const uint2 v = lds64(vbase + v_at[i]);
                r[i][0] = v.x, r[i][1] = v.y;
              } else {
                const uint4 v = lds128(vbase + h * (kN * 128) + v_at[i]);
                r[i][0] = v.x, r[i][1] = v.y, r[i][2] = v.z, r[i][3] = v.w;
              }
            }
#pragma unroll
            for (int c = 0; c < (D == 64 ? 2 : 4); ++c) {
              uint32_t u[4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // two keys' codes side by side, column by column
                const uint32_t ka = r[2 * i][c] ^ 0x80808080u, kb = r[2 * i + 1][c] ^ 0x80808080u;
                u[i] = __byte_perm(ka, kb, 0x5140);
                u[2 + i] = __byte_perm(ka, kb, 0x7362);
              }
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a[4] = {code_pair(u[2 * j], 0x4140), code_pair(u[2 * j], 0x4342),
                                       code_pair(u[2 * j + 1], 0x4140),
                                       code_pair(u[2 * j + 1], 0x4342)};
#pragma unroll
                for (int b = 0; b < NB; ++b)
                  mma16816(o[h * 8 + 2 * c + j][b], a, pb[b][0], pb[b][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&kv_empty[vs]));
      }
      if (!ok) break;
      // the next tile's queries arrive behind this one's end (64 single tokens over up to 500
      // keys, 32 heads: 69.4 us when they were loaded after it, 65.0)
      const bool known = mbar_try(smem_u32(&seg_full[n_seg % kSegs]), (n_seg / kSegs) & 1);
      if (__all_sync(0xffffffffu, known)) take();
      if (!ok) break;
      // ---- the warps' parts of the tile together
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[b][i] += __shfl_xor_sync(0xffffffffu, l[b][i], d);
          if (g == 0)
            ml_sm[(par * kWarps + warp) * kM + 8 * b + 2 * t + i] = make_float2(m[b][i], l[b][i]);
        }
      if (!meet()) break;
      // (a warp's own factor)
      float f[NB][2];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float M = -INFINITY;
#pragma unroll
          for (int k = 0; k < kWarps; ++k)
            M = fmaxf(M, ml_sm[(par * kWarps + k) * kM + 8 * b + 2 * t + i].x);
          f[b][i] = m[b][i] == -INFINITY ? 0.0f : ex2(m[b][i] - M) * e_pos;
        }
      float *mine = p.part + (int64_t)(blockIdx.x * 2 + max(s.slot, 0)) * C::kPart;
      auto out_at = [&](int r) {
        const int n = s.rem + r, k = row_token(n);
        return (int64_t)(s.tok + k) * p.o_token + (int64_t)(s.head * p.G + n - k * p.G) * p.o_head;
      };
      float *buf = reinterpret_cast<float *>(buf_sm);
      constexpr int F4 = C::kRow / 4;  // float4 pieces of a row of the buffer
#pragma unroll
      for (int h = 0; h < (D + 127) / 128; ++h) {
        if (h > 0 && ok) meet();
        if (!ok) break;
        // a thread's F4 / 2 columns of a row are contiguous: two of each tile
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < F4 / 8; ++k) {
              const int row = 8 * b + 2 * t + i, n = h * 8 + 2 * k;
              if (row >= s.rows) continue;
              *reinterpret_cast<float4 *>(
                  buf + ((warp * kM + row) * F4 + place(row, (F4 / 8) * g + k)) * 4) =
                  make_float4(o[n][b][i] * f[b][i], o[n][b][i + 2] * f[b][i],
                              o[n + 1][b][i] * f[b][i], o[n + 1][b][i + 2] * f[b][i]);
            }
        if (!meet()) break;
        for (int it = tid; it < s.rows * F4; it += kWarps * 32) {
          const int r = it / F4, q4 = it % F4, at = place(r, q4);
          float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          float M = -INFINITY, L = 0.0f;
#pragma unroll
          for (int k2 = 0; k2 < kWarps; ++k2) {
            const float4 v =
                *reinterpret_cast<const float4 *>(buf + ((k2 * kM + r) * F4 + at) * 4);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
            M = fmaxf(M, ml_sm[(par * kWarps + k2) * kM + r].x);
          }
#pragma unroll
          for (int k2 = 0; k2 < kWarps; ++k2) {
            const float2 v = ml_sm[(par * kWarps + k2) * kM + r];
            if (v.x > -INFINITY) L = fmaf(v.y, ex2(v.x - M), L);
          }
          if (s.slot < 0) {
            const float inv = L > 0.0f ? 1.0f / L : 0.0f;
            *reinterpret_cast<uint2 *>(p.out + out_at(r) + h * 128 + q4 * 4) =
                make_uint2(f2h(a.x * inv, a.y * inv), f2h(a.z * inv, a.w * inv));
          } else {
            *reinterpret_cast<float4 *>(mine + 2 * kM + r * D + h * 128 + q4 * 4) = a;
            if (q4 == 0 && h == 0) {
              mine[r] = M;
              mine[kM + r] = L;
            }
          }
        }
      }
      if (!ok) break;
      if (s.slot < 0) continue;
      // ---- cut between CTAs: the last to arrive merges, in CTA order
      __threadfence();
      if (!meet()) break;
      if (tid == 0) *arrived_sm = atomicAdd(&p.cnt[s.c_lo], 1u);
      if (!meet()) break;
      const bool last = (int)*arrived_sm == s.parts - 1;
      if (last) {
        __threadfence();
        auto part_at = [&](int k) {
          return p.part + (int64_t)((s.c_lo + k) * 2 + (k == 0 ? s.first_slot : 0)) * C::kPart;
        };
        for (int it = tid; it < s.rows * (D / 4); it += kWarps * 32) {
          const int r = it / (D / 4), q4 = it % (D / 4);
          float M = -INFINITY, L = 0.0f;
          float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          constexpr int U = 8;
          for (int k0 = 0; k0 < s.parts; k0 += U) {
            float mk[U], lk[U];
            float4 v[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const float *pp = part_at(min(k0 + k, s.parts - 1));
              mk[k] = k0 + k < s.parts ? __ldcg(pp + r) : -INFINITY;
              lk[k] = __ldcg(pp + kM + r);
              v[k] = __ldcg(reinterpret_cast<const float4 *>(pp + 2 * kM + r * D) + q4);
            }
            float mn = M;
#pragma unroll
            for (int k = 0; k < U; ++k) mn = fmaxf(mn, mk[k]);
            // (-inf: rows that saw no key, or a NaN in every logit, which goes on as 0 * NaN)
            const float z = mn == -INFINITY ? 0.0f : mn;
            const float f0 = ex2(M - z);
            L *= f0;
            a.x *= f0, a.y *= f0, a.z *= f0, a.w *= f0;
#pragma unroll
            for (int k = 0; k < U; ++k) {
              const float fk = ex2(mk[k] - z);
              L = fmaf(lk[k], fk, L);
              a.x = fmaf(v[k].x, fk, a.x), a.y = fmaf(v[k].y, fk, a.y);
              a.z = fmaf(v[k].z, fk, a.z), a.w = fmaf(v[k].w, fk, a.w);
            }
            M = mn;
          }
          const float inv = L > 0.0f ? 1.0f / L : 0.0f;
          *reinterpret_cast<uint2 *>(p.out + out_at(r) + q4 * 4) =
              make_uint2(f2h(a.x * inv, a.y * inv), f2h(a.z * inv, a.w * inv));
        }
        if (tid == 0) p.cnt[s.c_lo] = 0;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kOtherRegs));
  }
  if (warp >= kLoadWarp) {
    // --------------------------------------------------------------- load --
    // Four warps: keys and values, of every other block each.  (One warp's chain of waits,
    // pages and copies takes 2600 clocks a block, twice what HBM leaves it.)
    const bool keys = ((warp - kLoadWarp) & 1) == 0;
    const uint32_t turn = (uint32_t)(warp - kLoadWarp) >> 1;
    const CUtensorMap *map = keys ? &p.kmap : &p.vmap;
    const float *scales = keys ? p.ks : p.vs;
    const int64_t sc_page = keys ? p.ks_page : p.vs_page, sc_head = keys ? p.ks_head : p.vs_head;
    const int64_t sc_token = keys ? p.ks_token : p.vs_token;
    bool ok = true;
    const int ppb = p.page_size >= kN ? 1 : kN >> p.page_shift;  // pages per block
    const int box_rows = min(p.page_size, kN);
    int batch = 0, ids = -1, ids_ahead = -1;  // as in the fp16 kernel
    auto fetch = [&](const Seg &g, int first) -> int {
      const int pi = first + lane;
      const int64_t key = (int64_t)pi << p.page_shift;
      if (key >= g.hi || key + p.page_size <= g.lo) return -1;
      const int id = pi < p.s.ld_table ? __ldg(p.s.table + (int64_t)g.seq * p.s.ld_table + pi) : -2;
      return id == -1 ? -2 : id;
    };
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
    // Keys or values of block b, the n-th of the CTA.
    auto issue = [&](const Seg &g, int b, uint32_t n, int page) -> bool {
      const uint32_t fill = 2 * n + (keys ? 0 : 1);
      const int slot = fill % NS;
      if (fill >= NS && !mbar_wait(smem_u32(&kv_empty[slot]), (fill / NS - 1) & 1, abort_flag))
        return false;
      const uint32_t bar = smem_u32(&kv_full[slot]);
      const unsigned live = __ballot_sync(0xffffffffu, page >= 0);
      float *sc = scale_sm + slot * kN;
      const uint32_t bytes = __popc(live) * box_rows * D + scale_runs(p, page);
      scale_zeros(p, sc, page);
      __syncwarp();
      if (lane == 0)
        asm volatile(
            "{\n\t.reg .b64 t;\n\t"
            "mbarrier.arrive.expect_tx.shared::cta.b64 t, [%0], %1;\n\t}" ::"r"(bar),
            "r"(bytes)
            : "memory");
      __syncwarp();
      if (page >= 0) {
        const int at = p.page_size > kN ? (b * kN) & (p.page_size - 1) : 0;
        const uint32_t dst = smem_u32(kv_sm) + slot * C::kStage + lane * box_rows * C::kRow;
#pragma unroll
        for (int d = 0; d < (D + 127) / 128; ++d)
          asm volatile(
              "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes "
              "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst + d * (kN * 128)),
              "l"(reinterpret_cast<uint64_t>(map)), "r"(d * 128), "r"(at), "r"(g.head), "r"(page),
              "r"(bar)
              : "memory");
      }
      scale_copy(p, scales, sc_page, sc_head, sc_token, sc, g, b, page, bar);
      if (!p.runs)
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar)
                     : "memory");
      __syncwarp();
      issued = n + 1;
      return true;
    };
    uint32_t n_seg = 0, first = 0;  // tiles; blocks of those before
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
      return true;
    };
    while (ok) {
      Seg g;
      if (warp == kLoadWarp) {
        g = w.next(p);
        ok = announce(g);
      } else {
        ok = read_seg(n_seg, g);
      }
      ++n_seg;
      if (!ok || g.rows == 0) break;
      const int nb = g.b1 - g.b0, skip = (int)((first ^ turn) & 1);
      if (skip < nb) {
        batch = (int)(((int64_t)(g.b0 + skip) * kN) >> p.page_shift);
        ids = fetch(g, batch);
        ids_ahead = fetch(g, batch + 32);
      }
      for (int j = skip; ok && j < nb; j += 2)
        ok = issue(g, g.b0 + j, first + j, page_of(g, g.b0 + j));
      first += nb;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __syncthreads();
  if (*(volatile int *)abort_flag && warp >= kLoadWarp) {  // copies in flight end before the CTA
    const unsigned long long until = gtimer() + kWaitNs;
    for (uint32_t k = 0; k < NS / 4 && issued > 2 * k; ++k) {
      const uint32_t fill = 2 * (issued - 1 - 2 * k) + ((warp - kLoadWarp) & 1);
      mbar_drain(smem_u32(&kv_full[fill % NS]), (fill / NS) & 1, until);
    }
  }
}

template <int D, int NB, int CAP>
qz_status launch(const Attn8Params &p, int sms, cudaStream_t s) {
  using C = Cfg8<D, NB>;
  const cudaError_t e = allow_smem<attn8_kernel<D, NB, CAP>>(C::kSmem);
  if (e != cudaSuccess) return cuda_status(e);
  attn8_kernel<D, NB, CAP><<<sms < kMaxCtas ? sms : kMaxCtas, C::kThreads, C::kSmem, s>>>(p);
  return launch_status();
}

template <int D, int NB>
qz_status launch_cap(const Attn8Params &p, int sms, cudaStream_t s) {
  if (p.cap == 0.0f) return launch<D, NB, 0>(p, sms, s);
  return p.cap <= kShortCap ? launch<D, NB, 1>(p, sms, s) : launch<D, NB, 2>(p, sms, s);
}

template <int D>
qz_status launch_rows(const Attn8Params &p, bool one, int sms, cudaStream_t s) {
  return one ? launch_cap<D, 1>(p, sms, s) : launch_cap<D, 2>(p, sms, s);
}

}  // namespace

qz_status launch_attention_int8(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                                const PagedInt8View &c, const SeqView &sv, float scale,
                                float softcap, int64_t window, __half *out, int64_t o_token,
                                int64_t o_head, void *workspace, cudaStream_t s) {
  const int64_t rows = sv.n_tokens * (hq / c.hkv);  // of a KV head, of all sequences
  // Two tiles of 16 rows read a sequence's keys twice, from L2 the second time, and still take
  // less than one tile of the other kernel: 16 sequences of 32 rows over 8000 keys, 8 heads, D
  // 64, 128, 256: 89, 129, 220 us here and 127, 152, 231 there; three tiles 127, 184, 319 and
  // 129, 157, 233 (of prompts of 24 tokens, 64 of them at D 128, two take 55 and 44).  Only
  // the mean is known here, of all sequences, those without new tokens too, and a step of
  // very uneven ones may lose by it: 255 single tokens over 4000 keys beside a chunk of 2048
  // take 1.35 ms here and 2.47 there, but over 500 beside a chunk over 16384 2.16 and 0.92.
  if (rows > (int64_t)32 * sv.n_seqs)
    return launch_attention_int8_tc(q, hq, q_token, q_head, c, sv, scale, softcap, window, out,
                                    o_token, o_head, workspace, s);
  DeviceInfo di;
  qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  Attn8Params p;
  memset(&p, 0, sizeof(p));
  st = code_map(&p.kmap, c.k, c, c.k_token, c.k_head, c.k_page);
  if (st == QZ_OK) st = code_map(&p.vmap, c.v, c, c.v_token, c.v_head, c.v_page);
  if (st != QZ_OK) return st;
  set_scales(&p, c);
  p.q = q;
  p.out = out;
  p.q_token = q_token;
  p.q_head = q_head;
  p.o_token = o_token;
  p.o_head = o_head;
  set_heads(&p, hq, c.hkv);
  p.sign = scale == 0.0f ? 0.0f : scale < 0.0f ? -1.0f : 1.0f;
  p.c = set_logits(&p, scale, softcap);
  p.window = window > INT32_MAX ? 0 : (int)window;  // longer than any cache: none
  p.s = sv;
  p.cnt = static_cast<unsigned *>(workspace);
  p.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + QZ_ATTENTION_SYNC_BYTES);
  const bool one = rows <= (int64_t)8 * sv.n_seqs;
  if (c.D == 256) return launch_rows<256>(p, one, di.sms, s);
  return c.D == 128 ? launch_rows<128>(p, one, di.sms, s) : launch_rows<64>(p, one, di.sms, s);
}

qz_status read_attn8_error(int *code, int clear) {
  return read_error_word(g_attn_error, code, clear);
}

}  // namespace qz
