// Device view of a step's sequences and of the paged cache, shared by the
// kernels that write and read it.
#pragma once

#include "qz_internal.cuh"

namespace qz {

struct PagedView {
  __half *k, *v;
  int n_pages, page_size, page_shift, hkv, D;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;
};

// The same with rows of INT8 codes and one fp32 scale a row.
struct PagedInt8View {
  int8_t *k, *v;
  float *ks, *vs;
  int n_pages, page_size, page_shift, hkv, D;
  int64_t k_page, k_head, k_token, v_page, v_head, v_token;          // codes
  int64_t ks_page, ks_head, ks_token, vs_page, vs_head, vs_token;    // scales
};

struct SeqView {
  int n_seqs;
  int64_t n_tokens;
  const int32_t *cu_q, *kv_len, *table;
  int64_t ld_table;
};

// The sequence that token t belongs to, or -1: every lane of a warp calls it
// with the same t; 32 boundaries per load, so 1024 sequences take two.
__device__ __forceinline__ int seq_of_token(const SeqView &s, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = s.n_seqs;  // the answer i is the last of [lo, hi) with cu_q[i] <= t
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const bool below = at < hi && (int64_t)__ldg(s.cu_q + at) <= t;
    const int n = __popc(__ballot_sync(0xffffffffu, below));
    if (n == 0) return -1;  // before the first sequence
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  const bool in = lo < s.n_seqs && (int64_t)__ldg(s.cu_q + lo) <= t &&
                  t < (int64_t)__ldg(s.cu_q + lo + 1);
  return in ? lo : -1;
}

}  // namespace qz
