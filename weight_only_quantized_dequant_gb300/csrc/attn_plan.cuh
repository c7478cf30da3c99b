// What the attention kernels over the paged caches share: the split of a call's
// work between CTAs, found on the device from the sequences' lengths, barriers
// with bounded waits, and the logits' cap.
#pragma once

#include <cuda.h>

#include <cfloat>
#include <cmath>
#include <mutex>

#include "seq_batch.cuh"

namespace qz {
namespace {

__device__ int g_attn_error = 0;  // (of each translation unit)

constexpr int kN = 128;                // keys per block
constexpr int kMaxCtas = 160;          // grid cap (partial slots in the workspace)
constexpr unsigned long long kWaitNs = 2000000000ull;  // 2 s per wait
constexpr float kLag = 8.0f;           // log2 of how far a key may exceed m
// Caps up to here come from 1 - 2 / (1 + e^2t) alone: off by 2^-22 of the cap, 1.5e-5 in a
// logit, a sixteenth of the weights' rounding.  Four prompts of up to 4096 take 327 us
// without a cap, 634 with one of these and 948 with the form for any cap; 32 decode tokens
// over 16384 207, 261 and 353.
constexpr float kShortCap = 64.0f;
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
constexpr int kTileUnits = (kM + 127) / 128;
constexpr int kSegs = 4;               // tiles announced ahead

// A call's sequences and heads.
struct PlanParams {
  SeqView s;
  int G;             // query heads per KV head
  float inv_g;       // 1 / G
  uint64_t magic_g;  // ceil(2^64 / G), 0 for G = 1
  int hkv;
  int window;        // 0: none
};
inline void set_heads(PlanParams *p, int64_t hq, int hkv) {
  p->G = (int)(hq / hkv);
  p->inv_g = 1.0f / (float)p->G;
  p->magic_g = p->G > 1 ? ~(uint64_t)0 / (uint64_t)p->G + 1 : 0;
  p->hkv = hkv;
}

// The logits' cap: softcap, and the factors of a product s = q . k.
struct CapParams {
  float cap, cap_in;  // softcap, and |scale| / softcap * 2 log2(e)
  float mag, cap_t;   // |scale|, and |scale| / softcap
};
// Sets them; returns what turns logits into powers of two: |scale| log2(e) of a product,
// log2(e) of a capped logit.
inline float set_logits(CapParams *p, float scale, float softcap) {
  const float mag = scale == 0.0f ? 1.0f : fabsf(scale);
  p->cap = softcap;
  // (finite for the smallest caps: a logit of 0 stays 0, the others reach the cap all the same)
  p->mag = mag;
  p->cap_t = softcap > 0.0f ? fminf(mag / softcap, FLT_MAX) : 0.0f;
  p->cap_in = fminf(p->cap_t * 2.0f * kLog2e, FLT_MAX);
  return (softcap > 0.0f ? 1.0f : mag) * kLog2e;
}

// The pages of a cache, and the scales of an INT8 cache (strides in floats).
struct ScaleParams {
  int n_pages, page_size, page_shift;
  int runs;  // a page's scales are contiguous, and its and its heads' places 16-byte aligned
  const float *ks, *vs;
  int64_t ks_page, ks_head, ks_token, vs_page, vs_head, vs_token;
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
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
// Two bytes of codes + 128 (chosen by sel, under the bits of 1024) as fp16 codes.
__device__ __forceinline__ uint32_t code_pair(uint32_t biased, uint32_t sel) {
  const uint32_t v = __byte_perm(biased, 0x64646464u, sel);
  const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&v),
                            __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t *>(&r);
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
__device__ __forceinline__ float cap_far(const CapParams &p, float s) {
  return p.cap * (1.0f - 2.0f * rcp(1.0f + ex2(s * p.cap_in)));
}
// The same for any cap: below 1/4 by the series t - t^3/3 + 2t^5/15 - 17t^7/315 + 62t^9/2835,
// whose next term is below 2^-26 of the first there.
__device__ __forceinline__ float cap_any(const CapParams &p, float s) {
  const float t = s * p.cap_t, u = t * t, x = s * p.mag;
  float g = fmaf(u, 62.0f / 2835.0f, -17.0f / 315.0f);
  g = fmaf(u, g, 2.0f / 15.0f);
  g = fmaf(u, g, -1.0f / 3.0f);
  return pick(fabsf(t) < 0.25f, fmaf(x * u, g, x), cap_far(p, s));
}

// --------------------------------------------------------------- schedule --
// n / G for 0 <= n < 2^31, G <= 2^16: the excess of ceil(2^64 / G) over 2^64 / G
// adds less than n / 2^64 < 1 / G.
__device__ __forceinline__ int div_g(const PlanParams &p, int n) {
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
__device__ __forceinline__ Seq load_seq(const PlanParams &p, int i) {
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
__device__ __forceinline__ int first_key(const PlanParams &p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// Keys [lo, hi) that any row of row tile rt sees, and the blocks that hold them.
struct Range {
  int lo, hi, b0, nb;
};
template <int kM>
__device__ __forceinline__ Range tile_range(const PlanParams &p, const Seq &s, int rt) {
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
__device__ __forceinline__ int64_t head_units(const PlanParams &p, const Seq &s) {
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
  __device__ __forceinline__ bool start(const PlanParams &p);
  __device__ __forceinline__ Seg next(const PlanParams &p) {
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

// The scales of a block's 128 rows of an INT8 cache to dst (whole warp; lane i has the
// block's i-th page, INT32_MAX where the pool has no such page, negative where no row is
// needed).  Where a page's scales are whole 16-byte pieces (p.runs) each page is one bulk
// copy, `scale_runs` bytes in all for the barrier, and `scale_zeros` comes before the
// barrier's arrival; else four a lane by copies that the caller lets arrive there, zeros
// where no row of the tile sees the key or it has no page.
__device__ __forceinline__ bool in_pool(const ScaleParams &p, int page) {
  return page >= 0 && page < p.n_pages;
}
__device__ __forceinline__ uint32_t scale_runs(const ScaleParams &p, int page) {
  return p.runs ? __popc(__ballot_sync(0xffffffffu, in_pool(p, page))) * min(p.page_size, kN) * 4
                : 0;
}
__device__ __forceinline__ void scale_zeros(const ScaleParams &p, float *dst, int page) {
  const int n = min(p.page_size, kN), lane = threadIdx.x & 31;
  if (p.runs && page >= p.n_pages) {
    for (int i = 0; i < n; ++i) dst[lane * n + i] = 0.0f;
    // (a later block's bulk copy goes over them)
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
}
__device__ __forceinline__ void scale_copy(const ScaleParams &p, const float *sc, int64_t sc_page,
                                           int64_t sc_head, int64_t sc_token, float *dst,
                                           const Seg &g, int b, int page, uint32_t bar) {
  const int lane = threadIdx.x & 31;
  if (p.runs) {
    const int n = min(p.page_size, kN);
    if (in_pool(p, page)) {
      const float *src = sc + page * sc_page + g.head * sc_head + ((b * kN) & (p.page_size - 1));
      asm volatile(
          "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
          ::"r"(smem_u32(dst + lane * n)), "l"(src), "r"(n * 4), "r"(bar)
          : "memory");
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = lane + 32 * i;
    const int64_t key = (int64_t)b * kN + k;
    const int pg = __shfl_sync(0xffffffffu, page, k >> min(p.page_shift, 7));
    const bool use = in_pool(p, pg) && key >= g.lo && key < g.hi;
    const float *src =
        use ? sc + pg * sc_page + g.head * sc_head + (key & (p.page_size - 1)) * sc_token : sc;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst + k)), "l"(src),
                 "r"(use ? 4 : 0)
                 : "memory");
  }
}

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
__device__ __forceinline__ bool Walker<kM>::start(const PlanParams &p) {
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

// The pool's codes as [page][head][slot][D], boxes of one page's (at most 128) slots by
// 128 bytes (64).
qz_status code_map(CUtensorMap *map, const int8_t *base, const PagedInt8View &c, int64_t token,
                   int64_t head, int64_t page) {
  EncodeTiledFn fn = encode_tiled();
  if (!fn) return QZ_ERR_CUDA;
  // a dimension of one element has no stride of its own
  if (c.hkv == 1) head = token;
  if (c.n_pages == 1) page = token;
  const cuuint64_t dim[4] = {(cuuint64_t)c.D, (cuuint64_t)c.page_size, (cuuint64_t)c.hkv,
                             (cuuint64_t)c.n_pages};
  const cuuint64_t stride[3] = {(cuuint64_t)token, (cuuint64_t)head, (cuuint64_t)page};
  const cuuint32_t box[4] = {(cuuint32_t)(c.D < 128 ? c.D : 128),
                             (cuuint32_t)(c.page_size < kN ? c.page_size : kN), 1, 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<int8_t *>(base), dim, stride, box,
         estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
         c.D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? QZ_OK : QZ_ERR_UNSUPPORTED;
}

// The pages and scales of a call.
void set_scales(ScaleParams *p, const PagedInt8View &c) {
  p->ks = c.ks;
  p->vs = c.vs;
  p->ks_page = c.ks_page, p->ks_head = c.ks_head, p->ks_token = c.ks_token;
  p->vs_page = c.vs_page, p->vs_head = c.vs_head, p->vs_token = c.vs_token;
  p->n_pages = c.n_pages;
  p->page_size = c.page_size;
  p->page_shift = c.page_shift;
  // (head and page strides count where there are several)
  p->runs = c.ks_token == 1 && c.vs_token == 1 &&
            (((uintptr_t)c.ks | (uintptr_t)c.vs) & 15u) == 0 &&
            (c.hkv == 1 || (c.ks_head | c.vs_head) % 4 == 0) &&
            (c.n_pages == 1 || (c.ks_page | c.vs_page) % 4 == 0);
}

}  // namespace
}  // namespace qz
