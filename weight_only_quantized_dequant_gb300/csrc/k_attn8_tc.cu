// Attention over the paged cache of INT8 rows on the 5th-generation tensor cores: the
// kernel over fp16 rows (attn_tc.cuh) for steps that bring more rows to a KV head than two
// of the narrow tiles (chunks and prompts).
//
// Codes arrive by TMA in half of a slot; the two warps that bring the queries turn them into
// fp16 where they lie, so that the products, their order and the softmax are the fp16
// kernel's.  A scale is split: four bits of it multiply the codes, which is exact in fp16 (7 +
// 4 bits), and the rest multiplies, in fp32, the logit (keys) or the weight (values).  Whole
// scales in the fp16 rows would save the softmax a multiplication or two and cost a rounding
// of every key and value, twice the plain form's error.
//
// Measured (64 heads on 8, D 128): 4 x 64 tokens over up to 24000 keys 190 us, 545 TFLOP/s;
// four prompts of up to 2048 (32 heads) 228 (fp16 rows: 114 and 121).  The difference is the
// codes' way through the registers of two warps (a few instructions more there show in the
// whole) and, in the softmax, two factors a key from shared memory, which every lane of a
// row's warp reads.
#include "attn_tc.cuh"

namespace qz {

qz_status launch_attention_int8_tc(const __half *q, int64_t hq, int64_t q_token, int64_t q_head,
                                   const PagedInt8View &c, const SeqView &sv, float scale,
                                   float softcap, int64_t window, __half *out, int64_t o_token,
                                   int64_t o_head, void *workspace, cudaStream_t s) {
  DeviceInfo di;
  qz_status st = device_info(&di);
  if (st != QZ_OK) return st;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  st = code_map(&p.kmap, c.k, c, c.k_token, c.k_head, c.k_page);
  if (st == QZ_OK) st = code_map(&p.vmap, c.v, c, c.v_token, c.v_head, c.v_page);
  if (st != QZ_OK) return st;
  set_scales(&p, c);
  set_call(&p, q, hq, q_token, q_head, c.hkv, sv, scale, softcap, window, out, o_token, o_head,
           workspace);
  // (as over fp16 rows)
  const bool two = c.D < 256 && sv.n_tokens * p.G > (int64_t)128 * sv.n_seqs;
  p.q_boxes = scale > 0.0f && query_map(&p.qmap, q, sv.n_tokens, hq, c.D, q_token, q_head, p.G,
                                        two ? 128 : 64);
  if (c.D == 256) return launch_cap<256, 1, true>(p, di.sms, s);
  if (c.D == 128)
    return two ? launch_cap<128, 2, true>(p, di.sms, s) : launch_cap<128, 1, true>(p, di.sms, s);
  return two ? launch_cap<64, 2, true>(p, di.sms, s) : launch_cap<64, 1, true>(p, di.sms, s);
}

qz_status read_attn8_tc_error(int *code, int clear) {
  return read_error_word(g_attn_error, code, clear);
}

}  // namespace qz
