// How a call of the low-rank adapters is cut into CTAs.  Host arithmetic only.
#pragma once

#include <cstdint>

namespace qz {

constexpr int kLoraWarps = 8;                      // of the down product's CTAs
constexpr int kLoraUpWarps = 4;
constexpr int kLoraSub = 64;                       // k per warp and step
constexpr int kLoraSlice = kLoraSub * kLoraWarps;  // k per CTA and step
constexpr int kLoraMaxRows = 32;                   // rows of a CTA (a lane each in the search for runs)
constexpr int kLoraOut = 64;                       // outputs per warp and step
// Rows x padded rank of a CTA of the down product: 96 KB of sums.  1500 rows of 8 adapters in
// runs of 300, 4096 x 11008, rank 96: 32 rows a CTA take 78.4 us and 16 79.3 (64 KB); rank 112,
// where 32 rows need 112 KB and leave the L1 too little beside a second CTA: 106.8 and 90.1.
constexpr int kLoraRowRanks = 3072;
constexpr int kLoraMaxSlices = 8;                  // CTAs of a cluster, which split K

// CTAs per SM that the registers of a variant of the up product allow.
constexpr int lora_up_ctas(int rc, int nn) {
  return rc * nn == 1 ? 6 : rc * nn == 2 ? 4 : 3;
}

struct LoraPlan {
  int Rp, Rk;     // ranks rounded up to 16 and 32
  int slices;     // of K: CTAs of a cluster
  int k_slice;    // k per CTA (a multiple of kLoraSlice)
  int rows_down, rows_up;
  int along_n;    // CTAs of the up product along the outputs
};

// The smallest power of two from v on, or the largest that hi allows.
inline int lora_pow2(int64_t v, int hi) {
  int r = 1;
  while (r < v && 2 * r <= hi) r *= 2;
  return r;
}

inline LoraPlan lora_plan(int64_t T, int64_t K, int64_t N, int64_t R, int sms) {
  LoraPlan p;
  p.Rp = (int)((R + 15) / 16 * 16);
  p.Rk = (int)((R + 31) / 32 * 32);
  // Slices of K: as many as there are steps of kLoraSlice, at most kLoraMaxSlices.
  const int64_t steps = (K + kLoraSlice - 1) / kLoraSlice;
  p.slices = (int)(steps < kLoraMaxSlices ? steps : kLoraMaxSlices);
  p.k_slice = (int)((steps + p.slices - 1) / p.slices) * kLoraSlice;
  p.slices = (int)((K + p.k_slice - 1) / p.k_slice);
  // Rows per CTA: one while the GPU holds all of the down product's CTAs at once
  // (2 per SM; a decode step's adapters are read by the whole GPU together), more
  // as calls grow, so that a run's adapter is read by fewer CTAs; the up product
  // likewise at 4 per SM.  64 rows of 16 adapters in turn, 4096 x 4096: 12.4 us,
  // with one row a CTA 14.2; 256 of 16: 13.7, with half as many rows a CTA 20.2.
  // Twice as many help grouped rows and cost scattered ones (256 rows of as many
  // adapters: 35.7 -> 39.8 in the down product, 48.5 in the up product).
  const int64_t want = (int64_t)sms * 2;
  const int cap = kLoraRowRanks / p.Rp < kLoraMaxRows ? kLoraRowRanks / p.Rp : kLoraMaxRows;
  p.rows_down = lora_pow2((T * p.slices + want - 1) / want, cap);
  const int64_t per = kLoraOut * kLoraUpWarps, chunks = (N + per - 1) / per;
  p.rows_up = lora_pow2((T * chunks + 2 * want - 1) / (2 * want), kLoraMaxRows);
  // CTAs along N: as many as the GPU holds at once beside those along the rows
  // (a CTA that has its rows' u goes on to further outputs; a second wave of
  // CTAs would cost as much as the first).
  const int64_t tiles = (T + p.rows_up - 1) / p.rows_up;
  const int64_t slots = (int64_t)sms * lora_up_ctas(R <= 32 ? 1 : 2, p.rows_up <= 8 ? 1 : 2);
  const int64_t fit = slots / tiles > 1 ? slots / tiles : 1;
  p.along_n = (int)(chunks < fit ? chunks : fit);
  return p;
}

}  // namespace qz
