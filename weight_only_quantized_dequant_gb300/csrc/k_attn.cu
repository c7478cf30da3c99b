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
#include "attn_tc.cuh"

namespace qz {
namespace {

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
  p.n_pages = c.n_pages;
  p.page_size = c.page_size;
  p.page_shift = c.page_shift;
  set_call(&p, q, hq, q_token, q_head, c.hkv, sv, scale, softcap, window, out, o_token, o_head,
           workspace);
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
  if (c.D == 256) return launch_cap<256, 1, false>(p, di.sms, s);
  if (c.D == 128)
    return two ? launch_cap<128, 2, false>(p, di.sms, s) : launch_cap<128, 1, false>(p, di.sms, s);
  return two ? launch_cap<64, 2, false>(p, di.sms, s) : launch_cap<64, 1, false>(p, di.sms, s);
}

qz_status read_attn_error(int *code, int clear) {
  return read_error_word(g_attn_error, code, clear);
}

}  // namespace qz
