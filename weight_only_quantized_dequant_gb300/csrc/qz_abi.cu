// extern "C" entry points of libqz: argument validation, then one launcher.
// Validation never touches the GPU, so an invalid call enqueues nothing.
#include <mutex>

#include <cstring>

#include "qz_internal.cuh"
#include "seq_batch.cuh"

namespace qz {

static thread_local int g_last_cuda_error = 0;
static thread_local int g_overlap = 0;

int overlap_enabled() { return g_overlap; }

qz_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return QZ_OK;
  g_last_cuda_error = (int)e;
  return QZ_ERR_CUDA;
}

qz_status device_info(DeviceInfo *out) {
  constexpr int kMaxDev = 64;
  static DeviceInfo cache[kMaxDev];
  static std::once_flag once[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_status(e);
  if (dev < 0 || dev >= kMaxDev) return QZ_ERR_UNSUPPORTED;
  cudaError_t err = cudaSuccess;
  std::call_once(once[dev], [&] {
    DeviceInfo d;
    err = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess)
      err = cudaDeviceGetAttribute(&d.max_smem_optin,
                                   cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    cache[dev] = d;
  });
  if (err != cudaSuccess) return cuda_status(err);
  if (cache[dev].sms <= 0) return QZ_ERR_CUDA;
  *out = cache[dev];
  return QZ_OK;
}

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// Shared checks of a matrix argument: non-null, 16-B aligned, rows of
// ld*elem bytes that are a multiple of 16, ld >= cols.
qz_status check_mat(const void *p, int64_t rows, int64_t cols, int64_t ld, int elem) {
  if (!p || rows < 1 || cols < 1 || ld < cols) return QZ_ERR_INVALID_ARG;
  if (!aligned16(p) || (ld * elem) % 16 != 0) return QZ_ERR_ALIGNMENT;
  return QZ_OK;
}

#define QZ_TRY(expr)               \
  do {                             \
    qz_status _st = (expr);        \
    if (_st != QZ_OK) return _st;  \
  } while (0)

constexpr int64_t kMaxGemvK = 57344;

qz_status check_int8_weight(const qz_int8_weight *w) {
  if (!w) return QZ_ERR_INVALID_ARG;
  QZ_TRY(check_mat(w->q, w->N, w->K, w->ldq, 1));
  if (!w->scale) return QZ_ERR_INVALID_ARG;
  if (w->K > kMaxGemvK || w->N > ((int64_t)1 << 30)) return QZ_ERR_UNSUPPORTED;
  return QZ_OK;
}

qz_status check_int4o_weight(const qz_int4o_weight *w) {
  if (!w) return QZ_ERR_INVALID_ARG;
  if (w->N < 1 || w->K < 1 || w->n_out < 0 || w->n_out > w->K) return QZ_ERR_INVALID_ARG;
  const int64_t kb = w->K - w->n_out;
  if (!w->perm || !w->scale) return QZ_ERR_INVALID_ARG;
  if (w->n_out > 0 && !w->w_out) return QZ_ERR_INVALID_ARG;
  if (kb > 0 && !w->q4) return QZ_ERR_INVALID_ARG;
  if (w->ld_out < w->n_out || w->ld_q4 < (kb + 1) / 2) return QZ_ERR_INVALID_ARG;
  if (w->ld_out % 8 || w->ld_q4 % 16) return QZ_ERR_ALIGNMENT;
  if ((w->w_out && !aligned16(w->w_out)) || (w->q4 && !aligned16(w->q4)) ||
      !aligned16(w->scale) || !aligned16(w->perm))
    return QZ_ERR_ALIGNMENT;
  if (w->K > kMaxGemvK || w->N > ((int64_t)1 << 30)) return QZ_ERR_UNSUPPORTED;
  return QZ_OK;
}

// Activation/output vectors are read and written one element at a time, so
// they only need the 2-byte alignment of fp16.
qz_status check_vec(const void *x, int64_t B, int64_t len, int64_t ld) {
  if (!x || B < 1 || len < 1 || (B > 1 && ld < len)) return QZ_ERR_INVALID_ARG;
  if ((uintptr_t)x & 1u) return QZ_ERR_ALIGNMENT;
  return QZ_OK;
}

// Fill the per-matrix part of the launch for INT8.
void fill_int8(GemvParams &p, const qz_int8_weight *ws, int n) {
  p.perm = nullptr;
  p.K = (int)ws[0].K;
  p.n_out = 0;
  p.kb = p.K;
  p.cpr = (int)((ws[0].K + 15) / 16);
  p.ocpr = 0;
  p.n_mats = n;
  int64_t rows = 0;
  for (int m = 0; m < QZ_MAX_GROUP; ++m) {
    if (m < n) {
      rows += ws[m].N;
      p.codes[m] = reinterpret_cast<const uint8_t *>(ws[m].q);
      p.ld_codes[m] = ws[m].ldq;
      p.scale[m] = ws[m].scale;
    } else {
      p.codes[m] = nullptr;
      p.ld_codes[m] = 0;
      p.scale[m] = nullptr;
    }
    p.w_out[m] = nullptr;
    p.ld_out[m] = 0;
    p.row_end[m] = rows;
    p.y[m] = nullptr;
  }
  p.total_rows = rows;
}

void fill_int4o(GemvParams &p, const qz_int4o_weight *ws, int n) {
  p.perm = ws[0].perm;
  p.K = (int)ws[0].K;
  p.n_out = (int)ws[0].n_out;
  p.kb = p.K - p.n_out;
  p.cpr = (int)(((p.kb + 1) / 2 + 15) / 16);
  p.ocpr = (p.n_out + 7) / 8;
  p.n_mats = n;
  int64_t rows = 0;
  for (int m = 0; m < QZ_MAX_GROUP; ++m) {
    if (m < n) {
      rows += ws[m].N;
      p.codes[m] = ws[m].q4;
      p.ld_codes[m] = ws[m].ld_q4;
      p.w_out[m] = reinterpret_cast<const __half *>(ws[m].w_out);
      p.ld_out[m] = ws[m].ld_out;
      p.scale[m] = ws[m].scale;
    } else {
      p.codes[m] = nullptr;
      p.ld_codes[m] = 0;
      p.w_out[m] = nullptr;
      p.ld_out[m] = 0;
      p.scale[m] = nullptr;
    }
    p.row_end[m] = rows;
    p.y[m] = nullptr;
  }
  p.total_rows = rows;
}

qz_status gemm_common(bool int4, GemvParams &p, int64_t B, const qz_half *X, int64_t ldx,
                      qz_half *const *Ys, const int64_t *ldys, int n, void *ws, size_t ws_bytes,
                      cudaStream_t s) {
  p.x = reinterpret_cast<const __half *>(X);
  p.overlap = overlap_enabled();
  p.ldx = B > 1 ? ldx : 0;
  for (int m = 0; m < QZ_MAX_GROUP; ++m) p.ldy[m] = (B > 1 && m < n) ? ldys[m] : 0;
  for (int m = 0; m < n; ++m) p.y[m] = reinterpret_cast<__half *>(Ys[m]);
  DeviceInfo di;
  QZ_TRY(device_info(&di));
  // a workspace, when given, is checked whatever path the call then takes
  if (ws) {
    if (ws_bytes < tc_workspace_bytes(int4, B, p.K, p.n_out)) return QZ_ERR_INVALID_ARG;
    if ((uintptr_t)ws & 15u) return QZ_ERR_ALIGNMENT;
  }
  // Batch 1 runs on the CUDA-core GEMV (one fp32 FMA per weight keeps pace
  // with HBM at one input row); batches 2..8 on the warp-MMA GEMV, where the
  // CUDA cores would need one FMA per weight and input row.  Either takes
  // the call when its staged inputs fit in shared memory; larger batches are
  // dense enough for the tcgen05 GEMM, which also takes the small batches at
  // the few K too large to stage (its inputs stream in tiles).
  if (B == 1 && gemv_smem_bytes(int4, 1, p) <= (size_t)di.max_smem_optin)
    return launch_gemv(int4, 1, p, s);
  if (B <= kMvMaxBatch && mv_fits(int4, (int)B, p)) return launch_mv(int4, (int)B, p, s);
  if (B <= 4 && gemv_smem_bytes(int4, (int)B, p) <= (size_t)di.max_smem_optin)
    return launch_gemv(int4, (int)B, p, s);
  int64_t rows[QZ_MAX_GROUP];
  for (int m = 0; m < QZ_MAX_GROUP; ++m)
    rows[m] = m < n ? p.row_end[m] - (m ? p.row_end[m - 1] : 0) : 0;
  return launch_tc(int4, (int)B, p, rows, ws, ws_bytes, s);
}

template <typename W, typename Fill, typename Check>
qz_status sequence_common(bool int4, const W *ws, const int *counts, int n,
                          const qz_half *const *x, qz_half *const *ys, uint32_t *sync,
                          cudaStream_t s, Fill fill, Check check) {
  if (!ws || !counts || !x || !ys || !sync || n < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_SEQ) return QZ_ERR_UNSUPPORTED;
  if (((uintptr_t)sync & 3u) != 0) return QZ_ERR_ALIGNMENT;
  SeqParams sp;
  memset(&sp, 0, sizeof(sp));
  int off = 0;
  for (int k = 0; k < n; ++k) {
    const int c = counts[k];
    if (c < 1) return QZ_ERR_INVALID_ARG;
    if (c > QZ_MAX_GROUP) return QZ_ERR_UNSUPPORTED;
    for (int m = 0; m < c; ++m) {
      QZ_TRY(check(ws[off + m], ws[off]));
      QZ_TRY(check_vec(ys[off + m], 1, ws[off + m].N, 0));
    }
    QZ_TRY(check_vec(x[k], 1, ws[off].K, 0));
    GemvParams &p = sp.t[k];
    fill(p, ws + off, c);
    p.x = reinterpret_cast<const __half *>(x[k]);
    p.ldx = 0;
    p.overlap = overlap_enabled();
    for (int m = 0; m < QZ_MAX_GROUP; ++m) p.ldy[m] = 0;
    for (int m = 0; m < c; ++m) p.y[m] = reinterpret_cast<__half *>(ys[off + m]);
    off += c;
  }
  sp.n = n;
  sp.sync = reinterpret_cast<unsigned int *>(sync);
  return launch_gemv_seq(int4, sp, s);
}
// The address under which the device reads a weight buffer in place: device
// memory, or host memory that is pinned and mapped (unified addressing).
// Pageable or unknown memory is refused, so nothing is launched on it.
qz_status device_view(const void *ptr, const void **dev) {
  if (!ptr) {
    *dev = nullptr;
    return QZ_OK;
  }
  cudaPointerAttributes a;
  const cudaError_t e = cudaPointerGetAttributes(&a, ptr);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return QZ_ERR_INVALID_ARG;
  }
  if (a.type == cudaMemoryTypeUnregistered || !a.devicePointer) return QZ_ERR_INVALID_ARG;
  *dev = a.devicePointer;
  return QZ_OK;
}

template <typename T>
qz_status device_view_t(T *&ptr) {
  const void *d = nullptr;
  QZ_TRY(device_view(ptr, &d));
  ptr = reinterpret_cast<T *>(const_cast<void *>(d));
  return QZ_OK;
}

// Rows of 16-byte vectors that are `strides` halves apart.
qz_status check_rows16(const void *p, int64_t s0, int64_t s1) {
  if (!p || s0 < 0 || s1 < 0) return QZ_ERR_INVALID_ARG;
  if (!aligned16(p) || s0 % 8 || s1 % 8) return QZ_ERR_ALIGNMENT;
  return QZ_OK;
}

constexpr int64_t kMaxTokens = (int64_t)1 << 24;  // grid and index limits of the layer kernels
constexpr int64_t kMaxSeqs = (int64_t)1 << 20;

qz_status paged_view(const qz_kv_cache *c, PagedView *v) {
  if (!c || !c->k || !c->v || c->n_pages < 1 || c->n_kv_heads < 1) return QZ_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->page_size < 1) return QZ_ERR_INVALID_ARG;
  for (const int64_t s : {c->k_page, c->k_head, c->k_token, c->v_page, c->v_head, c->v_token}) {
    if (s < 0) return QZ_ERR_INVALID_ARG;
    if (s % 8) return QZ_ERR_ALIGNMENT;
  }
  if (!aligned16(c->k) || !aligned16(c->v)) return QZ_ERR_ALIGNMENT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QZ_ERR_UNSUPPORTED;
  const int64_t ps = c->page_size;
  if (ps < 8 || ps > 256 || (ps & (ps - 1))) return QZ_ERR_UNSUPPORTED;
  if (c->n_pages > INT32_MAX || c->n_kv_heads > 4096) return QZ_ERR_UNSUPPORTED;
  *v = {reinterpret_cast<__half *>(c->k), reinterpret_cast<__half *>(c->v), (int)c->n_pages,
        (int)ps, __builtin_ctz((unsigned)ps), (int)c->n_kv_heads, (int)c->head_dim, c->k_page,
        c->k_head, c->k_token, c->v_page, c->v_head, c->v_token};
  return QZ_OK;
}

qz_status paged_int8_view(const qz_kv_cache_int8 *c, PagedInt8View *v) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || c->n_pages < 1 || c->n_kv_heads < 1)
    return QZ_ERR_INVALID_ARG;
  if (c->head_dim < 1 || c->page_size < 1) return QZ_ERR_INVALID_ARG;
  for (const int64_t s : {c->k_page, c->k_head, c->k_token, c->v_page, c->v_head, c->v_token}) {
    if (s < 0) return QZ_ERR_INVALID_ARG;
    if (s % 16) return QZ_ERR_ALIGNMENT;
  }
  for (const int64_t s :
       {c->ks_page, c->ks_head, c->ks_token, c->vs_page, c->vs_head, c->vs_token})
    if (s < 0) return QZ_ERR_INVALID_ARG;
  if (!aligned16(c->k) || !aligned16(c->v)) return QZ_ERR_ALIGNMENT;
  if (((uintptr_t)c->k_scale | (uintptr_t)c->v_scale) & 3u) return QZ_ERR_ALIGNMENT;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QZ_ERR_UNSUPPORTED;
  const int64_t ps = c->page_size;
  if (ps < 8 || ps > 256 || (ps & (ps - 1))) return QZ_ERR_UNSUPPORTED;
  if (c->n_pages > INT32_MAX || c->n_kv_heads > 4096) return QZ_ERR_UNSUPPORTED;
  *v = {c->k,       c->v,       c->k_scale,  c->v_scale, (int)c->n_pages, (int)ps,
        __builtin_ctz((unsigned)ps), (int)c->n_kv_heads, (int)c->head_dim,
        c->k_page,  c->k_head,  c->k_token,  c->v_page,  c->v_head,       c->v_token,
        c->ks_page, c->ks_head, c->ks_token, c->vs_page, c->vs_head,      c->vs_token};
  return QZ_OK;
}

qz_status seq_view(const qz_seq_batch *b, SeqView *v) {
  if (!b || b->n_seqs < 0 || b->n_tokens < 0 || b->ld_table < 0) return QZ_ERR_INVALID_ARG;
  if (b->n_tokens > 0 && b->n_seqs > 0) {
    if (!b->cu_q || !b->kv_len || !b->page_table) return QZ_ERR_INVALID_ARG;
    if (((uintptr_t)b->cu_q | (uintptr_t)b->kv_len | (uintptr_t)b->page_table) & 3u)
      return QZ_ERR_ALIGNMENT;
  }
  if (b->n_seqs > kMaxSeqs || b->n_tokens > kMaxTokens || b->ld_table > INT32_MAX)
    return QZ_ERR_UNSUPPORTED;
  *v = {(int)b->n_seqs, b->n_tokens, b->cu_q, b->kv_len, b->page_table, b->ld_table};
  return QZ_OK;
}

// Shared checks of the two appends; *run: whether there is anything to do.
qz_status check_append(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                       const qz_half *k, int64_t k_token, int64_t k_head, const qz_half *v,
                       int64_t v_token, int64_t v_head, const float *rope, int64_t rope_len,
                       const SeqView &b, const qz_half *q_out, int64_t qo_token, int64_t qo_head,
                       bool *run) {
  *run = false;
  if (rope && rope_len < 0) return QZ_ERR_INVALID_ARG;
  if (rope && !aligned16(rope)) return QZ_ERR_ALIGNMENT;
  if (q_out && !q) return QZ_ERR_INVALID_ARG;
  if (rope && q && !q_out) return QZ_ERR_INVALID_ARG;
  if (q_out && (n_heads < 1 || n_heads > 65536)) return QZ_ERR_INVALID_ARG;
  if (b.n_tokens == 0 || b.n_seqs == 0) return QZ_OK;
  QZ_TRY(check_rows16(k, k_token, k_head));
  QZ_TRY(check_rows16(v, v_token, v_head));
  if (q_out) {
    QZ_TRY(check_rows16(q, q_token, q_head));
    QZ_TRY(check_rows16(q_out, qo_token, qo_head));
  }
  *run = true;
  return QZ_OK;
}

// Shared checks of the two attentions.
qz_status check_attention(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                          int hkv, int D, const SeqView &b, float scale, float softcap,
                          int64_t window, const qz_half *out, int64_t o_token, int64_t o_head,
                          const void *workspace, size_t workspace_bytes, bool *run) {
  *run = false;
  if (n_heads < 1 || n_heads % hkv || window < 0 || !(softcap >= 0.0f) ||
      !(scale - scale == 0.0f) || !(softcap - softcap == 0.0f))
    return QZ_ERR_INVALID_ARG;
  if (n_heads > 65536 || b.n_tokens * n_heads > INT32_MAX) return QZ_ERR_UNSUPPORTED;
  if (b.n_tokens == 0 || b.n_seqs == 0) return QZ_OK;
  QZ_TRY(check_rows16(q, q_token, q_head));
  QZ_TRY(check_rows16(out, o_token, o_head));
  if (!workspace ||
      workspace_bytes < attention_workspace_bytes(b.n_tokens, b.n_seqs, n_heads, hkv, D))
    return QZ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return QZ_ERR_ALIGNMENT;
  *run = true;
  return QZ_OK;
}

// Shared checks of the two norms; rows need only the alignment of fp16.
qz_status check_norm(const qz_half *x, int64_t ldx, const qz_half *r, int64_t ldr,
                     const qz_half *w, float bias, float eps, int64_t T, int64_t K,
                     const qz_half *sum, int64_t lds) {
  if (T < 0 || K < 1 || !(eps >= 0.0f) || bias != bias) return QZ_ERR_INVALID_ARG;
  if (K > kMaxGemvK || T > kMaxTokens) return QZ_ERR_UNSUPPORTED;
  if (T == 0) return QZ_OK;
  QZ_TRY(check_vec(x, T, K, ldx));
  QZ_TRY(check_vec(w, 1, K, 0));
  if (r) QZ_TRY(check_vec(r, T, K, ldr));
  if (sum) QZ_TRY(check_vec(sum, T, K, lds));
  return QZ_OK;
}

// Batch-1 grouped product with the weights read in place (zero-copy).
qz_status mapped_common(bool int4, GemvParams &p, const qz_half *x, qz_half *const *ys, int n,
                        cudaStream_t s) {
  p.x = reinterpret_cast<const __half *>(x);
  p.overlap = overlap_enabled();
  p.ldx = 0;
  for (int m = 0; m < QZ_MAX_GROUP; ++m) p.ldy[m] = 0;
  for (int m = 0; m < n; ++m) p.y[m] = reinterpret_cast<__half *>(ys[m]);
  DeviceInfo di;
  QZ_TRY(device_info(&di));
  if (gemv_mapped_smem_bytes(int4, p) > (size_t)di.max_smem_optin) return QZ_ERR_UNSUPPORTED;
  return launch_gemv_mapped(int4, p, s);
}

}  // namespace
}  // namespace qz

using namespace qz;

extern "C" {

const char *qz_status_string(qz_status st) {
  switch (st) {
    case QZ_OK: return "QZ_OK";
    case QZ_ERR_INVALID_ARG: return "QZ_ERR_INVALID_ARG";
    case QZ_ERR_ALIGNMENT: return "QZ_ERR_ALIGNMENT";
    case QZ_ERR_UNSUPPORTED: return "QZ_ERR_UNSUPPORTED";
    case QZ_ERR_CUDA: return "QZ_ERR_CUDA";
    case QZ_ERR_IO: return "QZ_ERR_IO";
    case QZ_ERR_DATA: return "QZ_ERR_DATA";
  }
  return "QZ_ERR_UNKNOWN";
}

int qz_version(void) { return 1 * 10000 + 0 * 100 + 0; }

int qz_last_cuda_error(void) { return g_last_cuda_error; }

qz_status qz_set_overlap(int enable) {
  if (enable != 0 && enable != 1) return QZ_ERR_INVALID_ARG;
  g_overlap = enable;
  return QZ_OK;
}

int qz_get_overlap(void) { return g_overlap; }

qz_status qz_device_error(int *code, int clear) {
  if (!code || (clear != 0 && clear != 1)) return QZ_ERR_INVALID_ARG;
  int a = 0, b = 0, c = 0, d = 0;
  QZ_TRY(read_device_error(&a, clear));
  QZ_TRY(read_gemv_error(&b, clear));
  QZ_TRY(read_embed_error(&c, clear));
  QZ_TRY(read_mv_error(&d, clear));
  int e = 0, f = 0, g = 0;
  QZ_TRY(read_rope_error(&e, clear));
  QZ_TRY(read_attn_error(&f, clear));
  QZ_TRY(read_lora_error(&g, clear));
  int h = 0, i = 0, j = 0;
  QZ_TRY(read_cache8_error(&h, clear));
  QZ_TRY(read_attn8_error(&i, clear));
  QZ_TRY(read_attn8_tc_error(&j, clear));
  *code = a | b | c | d | e | f | g | h | i | j;
  return QZ_OK;
}

// ------------------------------------------------------------------ INT8 --
qz_status qz_quantize_int8(const qz_half *W, int64_t N, int64_t K, int64_t ldw, int8_t *q,
                           int64_t ldq, float *scale, qz_stream s) {
  QZ_TRY(check_mat(W, N, K, ldw, 2));
  QZ_TRY(check_mat(q, N, K, ldq, 1));
  if (!scale) return QZ_ERR_INVALID_ARG;
  if (((uintptr_t)scale & 3u) != 0) return QZ_ERR_ALIGNMENT;
  return launch_quantize_int8(reinterpret_cast<const __half *>(W), N, K, ldw, q, ldq, scale,
                              (cudaStream_t)s);
}

qz_status qz_gemv_int8(const qz_int8_weight *w, const qz_half *x, qz_half *y, qz_stream s) {
  return qz_gemm_int8(w, 1, x, 0, y, 0, nullptr, 0, s);
}

qz_status qz_gemm_int8(const qz_int8_weight *w, int64_t B, const qz_half *X, int64_t ldx,
                       qz_half *Y, int64_t ldy, void *workspace, size_t workspace_bytes,
                       qz_stream s) {
  QZ_TRY(check_int8_weight(w));
  if (B < 1) return QZ_ERR_INVALID_ARG;
  if (B > QZ_MAX_BATCH) return QZ_ERR_UNSUPPORTED;
  QZ_TRY(check_vec(X, B, w->K, ldx));
  QZ_TRY(check_vec(Y, B, w->N, ldy));
  GemvParams p;
  fill_int8(p, w, 1);
  qz_half *ys[1] = {Y};
  return gemm_common(false, p, B, X, ldx, ys, &ldy, 1, workspace, workspace_bytes,
                     (cudaStream_t)s);
}

qz_status qz_embed_int8(const qz_int8_weight *table, const int32_t *tokens, int64_t B,
                        qz_half *out, int64_t ldo, qz_stream s) {
  if (!table || B < 0) return QZ_ERR_INVALID_ARG;
  QZ_TRY(check_mat(table->q, table->N, table->K, table->ldq, 1));
  if (!table->scale) return QZ_ERR_INVALID_ARG;
  if (B == 0) return QZ_OK;
  if (!tokens) return QZ_ERR_INVALID_ARG;
  if (((uintptr_t)tokens & 3u) != 0) return QZ_ERR_ALIGNMENT;
  QZ_TRY(check_mat(out, B, table->K, ldo, 2));
  return launch_embed_int8(table->q, table->ldq, table->scale, table->N, table->K, tokens, B,
                           reinterpret_cast<__half *>(out), ldo, (cudaStream_t)s);
}

qz_status qz_gemv_int8_grouped(const qz_int8_weight *ws, int n, const qz_half *x,
                               qz_half *const *ys, qz_stream s) {
  if (!ws || !ys || n < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP) return QZ_ERR_UNSUPPORTED;
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int8_weight(&ws[m]));
    if (ws[m].K != ws[0].K) return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(ys[m], 1, ws[m].N, 0));
  }
  QZ_TRY(check_vec(x, 1, ws[0].K, 0));
  GemvParams p;
  fill_int8(p, ws, n);
  return gemm_common(false, p, 1, x, 0, ys, nullptr, n, nullptr, 0, (cudaStream_t)s);
}

qz_status qz_gemm_int8_grouped(const qz_int8_weight *ws, int n, int64_t B, const qz_half *X,
                               int64_t ldx, qz_half *const *Ys, const int64_t *ldys,
                               void *workspace, size_t workspace_bytes, qz_stream s) {
  if (!ws || !Ys || !ldys || n < 1 || B < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP || B > QZ_MAX_BATCH) return QZ_ERR_UNSUPPORTED;
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int8_weight(&ws[m]));
    if (ws[m].K != ws[0].K) return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(Ys[m], B, ws[m].N, ldys[m]));
  }
  QZ_TRY(check_vec(X, B, ws[0].K, ldx));
  GemvParams p;
  fill_int8(p, ws, n);
  return gemm_common(false, p, B, X, ldx, Ys, ldys, n, workspace, workspace_bytes,
                     (cudaStream_t)s);
}

size_t qz_gemm_workspace_bytes(int64_t B, int64_t K, int64_t n_out) {
  if (B < 1 || B > QZ_MAX_BATCH || K < 1 || n_out < 0 || n_out > K) return 0;
  // n_out = 0 gives the INT8 size (ceil(K/64) tiles of the gathered input)
  return tc_workspace_bytes(true, B, K, n_out);
}

// ------------------------------------------------------------------ INT4 --
qz_status qz_int4o_layout(int64_t N, int64_t K, int64_t n_out, int64_t *ld_out,
                          int64_t *ld_q4) {
  if (N < 1 || K < 1 || n_out < 0 || n_out > K || !ld_out || !ld_q4) return QZ_ERR_INVALID_ARG;
  const int64_t kb = K - n_out;
  *ld_out = (n_out + 7) / 8 * 8;
  *ld_q4 = ((kb + 1) / 2 + 15) / 16 * 16;
  return QZ_OK;
}

qz_status qz_saliency_accumulate(const qz_half *W, int64_t N, int64_t K, int64_t ldw,
                                 int64_t *colsum, qz_stream s) {
  QZ_TRY(check_mat(W, N, K, ldw, 2));
  if (!colsum) return QZ_ERR_INVALID_ARG;
  if (((uintptr_t)colsum & 7u) != 0) return QZ_ERR_ALIGNMENT;
  if (N > (int64_t)65535 * 256) return QZ_ERR_UNSUPPORTED;
  return launch_saliency(reinterpret_cast<const __half *>(W), N, K, ldw, colsum,
                         (cudaStream_t)s);
}

qz_status qz_select_outliers(const int64_t *colsum, const float *x_profile, int64_t K,
                             int64_t n_out, int32_t *perm, qz_stream s) {
  if (!colsum || !x_profile || !perm || K < 1 || n_out < 0 || n_out > K)
    return QZ_ERR_INVALID_ARG;
  if (((uintptr_t)colsum & 7u) || ((uintptr_t)x_profile & 3u) || ((uintptr_t)perm & 3u))
    return QZ_ERR_ALIGNMENT;
  if (K > ((int64_t)1 << 20)) return QZ_ERR_UNSUPPORTED;
  return launch_select(colsum, x_profile, K, n_out, perm, (cudaStream_t)s);
}

qz_status qz_check_perm(const int32_t *perm, int64_t K, int32_t *flag, qz_stream s) {
  if (!perm || !flag || K < 1) return QZ_ERR_INVALID_ARG;
  if (((uintptr_t)perm & 3u) || ((uintptr_t)flag & 3u)) return QZ_ERR_ALIGNMENT;
  if (K > ((int64_t)1 << 20)) return QZ_ERR_UNSUPPORTED;
  return launch_check_perm(perm, K, flag, (cudaStream_t)s);
}

qz_status qz_quantize_int4_outlier(const qz_half *W, int64_t ldw, const int32_t *perm,
                                   int64_t N, int64_t K, int64_t n_out, qz_half *w_out,
                                   int64_t ld_out, uint8_t *q4, int64_t ld_q4, float *scale,
                                   qz_stream s) {
  QZ_TRY(check_mat(W, N, K, ldw, 2));
  if (!perm || !scale || n_out < 0 || n_out > K) return QZ_ERR_INVALID_ARG;
  const int64_t kb = K - n_out;
  if ((n_out > 0 && !w_out) || (kb > 0 && !q4)) return QZ_ERR_INVALID_ARG;
  if (ld_out < n_out || ld_q4 < (kb + 1) / 2) return QZ_ERR_INVALID_ARG;
  if (ld_out % 8 || ld_q4 % 16 || (w_out && !aligned16(w_out)) || (q4 && !aligned16(q4)) ||
      ((uintptr_t)perm & 3u) || ((uintptr_t)scale & 3u))
    return QZ_ERR_ALIGNMENT;
  if ((ld_out > 0 && !w_out) || (ld_q4 > 0 && !q4)) return QZ_ERR_INVALID_ARG;
  if (K > ((int64_t)1 << 17)) return QZ_ERR_UNSUPPORTED;
  return launch_quantize_int4o(reinterpret_cast<const __half *>(W), ldw, perm, N, K, n_out,
                               reinterpret_cast<__half *>(w_out), ld_out, q4, ld_q4, scale,
                               (cudaStream_t)s);
}

qz_status qz_gemv_int4_outlier(const qz_int4o_weight *w, const qz_half *x, qz_half *y,
                               qz_stream s) {
  return qz_gemm_int4_outlier(w, 1, x, 0, y, 0, nullptr, 0, s);
}

qz_status qz_gemm_int4_outlier(const qz_int4o_weight *w, int64_t B, const qz_half *X,
                               int64_t ldx, qz_half *Y, int64_t ldy, void *workspace,
                               size_t workspace_bytes, qz_stream s) {
  QZ_TRY(check_int4o_weight(w));
  if (B < 1) return QZ_ERR_INVALID_ARG;
  if (B > QZ_MAX_BATCH) return QZ_ERR_UNSUPPORTED;
  QZ_TRY(check_vec(X, B, w->K, ldx));
  QZ_TRY(check_vec(Y, B, w->N, ldy));
  GemvParams p;
  fill_int4o(p, w, 1);
  qz_half *ys[1] = {Y};
  return gemm_common(true, p, B, X, ldx, ys, &ldy, 1, workspace, workspace_bytes,
                     (cudaStream_t)s);
}

qz_status qz_gemm_int4_outlier_grouped(const qz_int4o_weight *ws, int n, int64_t B,
                                       const qz_half *X, int64_t ldx, qz_half *const *Ys,
                                       const int64_t *ldys, void *workspace,
                                       size_t workspace_bytes, qz_stream s) {
  if (!ws || !Ys || !ldys || n < 1 || B < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP || B > QZ_MAX_BATCH) return QZ_ERR_UNSUPPORTED;
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int4o_weight(&ws[m]));
    if (ws[m].K != ws[0].K || ws[m].n_out != ws[0].n_out || ws[m].perm != ws[0].perm)
      return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(Ys[m], B, ws[m].N, ldys[m]));
  }
  QZ_TRY(check_vec(X, B, ws[0].K, ldx));
  GemvParams p;
  fill_int4o(p, ws, n);
  return gemm_common(true, p, B, X, ldx, Ys, ldys, n, workspace, workspace_bytes,
                     (cudaStream_t)s);
}

qz_status qz_gemv_int8_grouped_mapped(const qz_int8_weight *ws, int n, const qz_half *x,
                                      qz_half *const *ys, qz_stream s) {
  if (!ws || !ys || n < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP) return QZ_ERR_UNSUPPORTED;
  qz_int8_weight v[QZ_MAX_GROUP];
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int8_weight(&ws[m]));
    if (ws[m].K != ws[0].K) return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(ys[m], 1, ws[m].N, 0));
    v[m] = ws[m];
    QZ_TRY(device_view_t(v[m].q));
    QZ_TRY(device_view_t(v[m].scale));
  }
  QZ_TRY(check_vec(x, 1, ws[0].K, 0));
  GemvParams p;
  fill_int8(p, v, n);
  return mapped_common(false, p, x, ys, n, (cudaStream_t)s);
}

qz_status qz_gemv_int4_outlier_grouped_mapped(const qz_int4o_weight *ws, int n,
                                              const qz_half *x, qz_half *const *ys,
                                              qz_stream s) {
  if (!ws || !ys || n < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP) return QZ_ERR_UNSUPPORTED;
  qz_int4o_weight v[QZ_MAX_GROUP];
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int4o_weight(&ws[m]));
    if (ws[m].K != ws[0].K || ws[m].n_out != ws[0].n_out || ws[m].perm != ws[0].perm)
      return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(ys[m], 1, ws[m].N, 0));
    v[m] = ws[m];
    QZ_TRY(device_view_t(v[m].perm));
    QZ_TRY(device_view_t(v[m].w_out));
    QZ_TRY(device_view_t(v[m].q4));
    QZ_TRY(device_view_t(v[m].scale));
  }
  QZ_TRY(check_vec(x, 1, ws[0].K, 0));
  GemvParams p;
  fill_int4o(p, v, n);
  return mapped_common(true, p, x, ys, n, (cudaStream_t)s);
}

qz_status qz_gemv_int4_outlier_grouped(const qz_int4o_weight *ws, int n, const qz_half *x,
                                       qz_half *const *ys, qz_stream s) {
  if (!ws || !ys || n < 1) return QZ_ERR_INVALID_ARG;
  if (n > QZ_MAX_GROUP) return QZ_ERR_UNSUPPORTED;
  for (int m = 0; m < n; ++m) {
    QZ_TRY(check_int4o_weight(&ws[m]));
    if (ws[m].K != ws[0].K || ws[m].n_out != ws[0].n_out || ws[m].perm != ws[0].perm)
      return QZ_ERR_INVALID_ARG;
    QZ_TRY(check_vec(ys[m], 1, ws[m].N, 0));
  }
  QZ_TRY(check_vec(x, 1, ws[0].K, 0));
  GemvParams p;
  fill_int4o(p, ws, n);
  return gemm_common(true, p, 1, x, 0, ys, nullptr, n, nullptr, 0, (cudaStream_t)s);
}


qz_status qz_gemv_int8_sequence(const qz_int8_weight *ws, const int *counts, int n,
                                const qz_half *const *x, qz_half *const *ys, uint32_t *sync,
                                qz_stream s) {
  return sequence_common(
      false, ws, counts, n, x, ys, sync, (cudaStream_t)s,
      [](GemvParams &p, const qz_int8_weight *w, int c) { fill_int8(p, w, c); },
      [](const qz_int8_weight &w, const qz_int8_weight &w0) -> qz_status {
        QZ_TRY(check_int8_weight(&w));
        return w.K == w0.K ? QZ_OK : QZ_ERR_INVALID_ARG;
      });
}

qz_status qz_gemv_int4_outlier_sequence(const qz_int4o_weight *ws, const int *counts, int n,
                                        const qz_half *const *x, qz_half *const *ys,
                                        uint32_t *sync, qz_stream s) {
  return sequence_common(
      true, ws, counts, n, x, ys, sync, (cudaStream_t)s,
      [](GemvParams &p, const qz_int4o_weight *w, int c) { fill_int4o(p, w, c); },
      [](const qz_int4o_weight &w, const qz_int4o_weight &w0) -> qz_status {
        QZ_TRY(check_int4o_weight(&w));
        return (w.K == w0.K && w.n_out == w0.n_out && w.perm == w0.perm) ? QZ_OK
                                                                          : QZ_ERR_INVALID_ARG;
      });
}

// ------------------------------------------------------------ layer glue --
qz_status qz_rmsnorm(const qz_half *x, int64_t ldx, const qz_half *residual, int64_t ldr,
                     const qz_half *weight, float w_bias, float eps, int64_t T, int64_t K,
                     qz_half *y, int64_t ldy, qz_half *sum, int64_t lds, qz_stream s) {
  QZ_TRY(check_norm(x, ldx, residual, ldr, weight, w_bias, eps, T, K, sum, lds));
  if (T == 0) return QZ_OK;
  QZ_TRY(check_vec(y, T, K, ldy));
  return launch_rmsnorm(reinterpret_cast<const __half *>(x), ldx,
                        reinterpret_cast<const __half *>(residual), ldr,
                        reinterpret_cast<const __half *>(weight), w_bias, eps, T, K,
                        reinterpret_cast<__half *>(y), ldy, nullptr, 0, nullptr,
                        reinterpret_cast<__half *>(sum), lds, (cudaStream_t)s);
}

qz_status qz_rmsnorm_int8(const qz_half *x, int64_t ldx, const qz_half *residual, int64_t ldr,
                          const qz_half *weight, float w_bias, float eps, int64_t T, int64_t K,
                          int8_t *q, int64_t ldq, float *scale, qz_half *sum, int64_t lds,
                          qz_stream s) {
  QZ_TRY(check_norm(x, ldx, residual, ldr, weight, w_bias, eps, T, K, sum, lds));
  if (T == 0) return QZ_OK;
  if (!q || !scale || (T > 1 && ldq < K)) return QZ_ERR_INVALID_ARG;
  if ((uintptr_t)scale & 3u) return QZ_ERR_ALIGNMENT;
  return launch_rmsnorm(reinterpret_cast<const __half *>(x), ldx,
                        reinterpret_cast<const __half *>(residual), ldr,
                        reinterpret_cast<const __half *>(weight), w_bias, eps, T, K, nullptr, 0, q,
                        ldq, scale, reinterpret_cast<__half *>(sum), lds, (cudaStream_t)s);
}

qz_status qz_rope_append(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                         const qz_half *k, int64_t k_token, int64_t k_head, const qz_half *v,
                         int64_t v_token, int64_t v_head, const float *rope, int64_t rope_len,
                         const qz_kv_cache *cache, const qz_seq_batch *seqs, qz_half *q_out,
                         int64_t qo_token, int64_t qo_head, qz_stream s) {
  PagedView c;
  SeqView b;
  QZ_TRY(paged_view(cache, &c));
  QZ_TRY(seq_view(seqs, &b));
  bool run;
  QZ_TRY(check_append(q, n_heads, q_token, q_head, k, k_token, k_head, v, v_token, v_head, rope,
                      rope_len, b, q_out, qo_token, qo_head, &run));
  if (!run) return QZ_OK;
  return launch_rope_append(
      reinterpret_cast<const __half *>(q), n_heads, q_token, q_head,
      reinterpret_cast<const __half *>(k), k_token, k_head, reinterpret_cast<const __half *>(v),
      v_token, v_head, rope, rope_len, c, b, reinterpret_cast<__half *>(q_out), qo_token, qo_head,
      (cudaStream_t)s);
}

size_t qz_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int64_t n_heads,
                                    int64_t n_kv_heads, int64_t head_dim) {
  if (n_tokens < 0 || n_seqs < 0 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads ||
      n_tokens > kMaxTokens || n_seqs > kMaxSeqs)
    return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return attention_workspace_bytes(n_tokens, n_seqs, n_heads, n_kv_heads, head_dim);
}

qz_status qz_attention_paged(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                             const qz_kv_cache *cache, const qz_seq_batch *seqs, float scale,
                             float softcap, int64_t window, qz_half *out, int64_t o_token,
                             int64_t o_head, void *workspace, size_t workspace_bytes,
                             qz_stream s) {
  PagedView c;
  SeqView b;
  QZ_TRY(paged_view(cache, &c));
  QZ_TRY(seq_view(seqs, &b));
  bool run;
  QZ_TRY(check_attention(q, n_heads, q_token, q_head, c.hkv, c.D, b, scale, softcap, window, out,
                         o_token, o_head, workspace, workspace_bytes, &run));
  if (!run) return QZ_OK;
  return launch_attention(reinterpret_cast<const __half *>(q), n_heads, q_token, q_head, c, b,
                          scale, softcap, window, reinterpret_cast<__half *>(out), o_token, o_head,
                          workspace, (cudaStream_t)s);
}

qz_status qz_rope_append_int8(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                              const qz_half *k, int64_t k_token, int64_t k_head,
                              const qz_half *v, int64_t v_token, int64_t v_head,
                              const float *rope, int64_t rope_len,
                              const qz_kv_cache_int8 *cache, const qz_seq_batch *seqs,
                              qz_half *q_out, int64_t qo_token, int64_t qo_head, qz_stream s) {
  PagedInt8View c;
  SeqView b;
  QZ_TRY(paged_int8_view(cache, &c));
  QZ_TRY(seq_view(seqs, &b));
  bool run;
  QZ_TRY(check_append(q, n_heads, q_token, q_head, k, k_token, k_head, v, v_token, v_head, rope,
                      rope_len, b, q_out, qo_token, qo_head, &run));
  if (!run) return QZ_OK;
  return launch_rope_append_int8(
      reinterpret_cast<const __half *>(q), n_heads, q_token, q_head,
      reinterpret_cast<const __half *>(k), k_token, k_head, reinterpret_cast<const __half *>(v),
      v_token, v_head, rope, rope_len, c, b, reinterpret_cast<__half *>(q_out), qo_token, qo_head,
      (cudaStream_t)s);
}

qz_status qz_cache_read_int8(const qz_kv_cache_int8 *cache, const qz_seq_batch *seqs, qz_half *k,
                             int64_t k_token, int64_t k_head, qz_half *v, int64_t v_token,
                             int64_t v_head, qz_stream s) {
  PagedInt8View c;
  SeqView b;
  QZ_TRY(paged_int8_view(cache, &c));
  QZ_TRY(seq_view(seqs, &b));
  if (b.n_tokens == 0 || b.n_seqs == 0) return QZ_OK;
  QZ_TRY(check_rows16(k, k_token, k_head));
  QZ_TRY(check_rows16(v, v_token, v_head));
  return launch_cache_read_int8(c, b, reinterpret_cast<__half *>(k), k_token, k_head,
                                reinterpret_cast<__half *>(v), v_token, v_head, (cudaStream_t)s);
}

qz_status qz_attention_paged_int8(const qz_half *q, int64_t n_heads, int64_t q_token,
                                  int64_t q_head, const qz_kv_cache_int8 *cache,
                                  const qz_seq_batch *seqs, float scale, float softcap,
                                  int64_t window, qz_half *out, int64_t o_token, int64_t o_head,
                                  void *workspace, size_t workspace_bytes, qz_stream s) {
  PagedInt8View c;
  SeqView b;
  QZ_TRY(paged_int8_view(cache, &c));
  QZ_TRY(seq_view(seqs, &b));
  bool run;
  QZ_TRY(check_attention(q, n_heads, q_token, q_head, c.hkv, c.D, b, scale, softcap, window, out,
                         o_token, o_head, workspace, workspace_bytes, &run));
  if (!run) return QZ_OK;
  return launch_attention_int8(reinterpret_cast<const __half *>(q), n_heads, q_token, q_head, c, b,
                               scale, softcap, window, reinterpret_cast<__half *>(out), o_token,
                               o_head, workspace, (cudaStream_t)s);
}

size_t qz_lora_workspace_bytes(int64_t T, int64_t K, int64_t R) {
  if (T < 0 || T > kMaxTokens || K < 1 || K > ((int64_t)1 << 20) || R < 1 || R > 128) return 0;
  return lora_workspace_bytes(T, K, R);
}

qz_status qz_lora(const qz_lora_adapters *ad, const int32_t *index, int64_t T, const qz_half *x,
                  int64_t ldx, const qz_half *y, int64_t ldy, qz_half *out, int64_t ldo,
                  void *workspace, size_t workspace_bytes, qz_stream s) {
  if (!ad || T < 0 || ad->n_adapters < 0 || ad->R < 1 || ad->K < 1 || ad->N < 1)
    return QZ_ERR_INVALID_ARG;
  if (ad->R > 128 || ad->K > ((int64_t)1 << 20) || ad->N > ((int64_t)1 << 20) || T > kMaxTokens ||
      ad->n_adapters > INT32_MAX)
    return QZ_ERR_UNSUPPORTED;
  if (T == 0) return QZ_OK;
  if (ad->n_adapters > 0) {
    if (!ad->a || !ad->b || !ad->scale || ad->a_row < ad->K || ad->b_row < ad->R ||
        ad->a_adapter < 0 || ad->b_adapter < 0)
      return QZ_ERR_INVALID_ARG;
    if (((uintptr_t)ad->a | (uintptr_t)ad->b) & 1u) return QZ_ERR_ALIGNMENT;
    if (((uintptr_t)ad->scale | (uintptr_t)ad->rank) & 3u) return QZ_ERR_ALIGNMENT;
  }
  if (!index) return QZ_ERR_INVALID_ARG;
  if ((uintptr_t)index & 3u) return QZ_ERR_ALIGNMENT;
  QZ_TRY(check_vec(x, T, ad->K, ldx));
  QZ_TRY(check_vec(y, T, ad->N, ldy));
  QZ_TRY(check_vec(out, T, ad->N, ldo));
  if (!workspace || workspace_bytes < lora_workspace_bytes(T, ad->K, ad->R))
    return QZ_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return QZ_ERR_ALIGNMENT;
  return launch_lora(*ad, index, T, reinterpret_cast<const __half *>(x), T > 1 ? ldx : 0,
                     reinterpret_cast<const __half *>(y), T > 1 ? ldy : 0,
                     reinterpret_cast<__half *>(out), T > 1 ? ldo : 0, workspace, (cudaStream_t)s);
}

qz_status qz_sample(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                    const float *u, const qz_sampling *options, int32_t *token, float *logprob,
                    qz_stream s) {
  if (B < 0 || V < 1 || !options || dtype < QZ_FP16 || dtype > QZ_FP32) return QZ_ERR_INVALID_ARG;
  if (V > QZ_MAX_VOCAB || B > kMaxTokens) return QZ_ERR_UNSUPPORTED;
  if (B == 0) return QZ_OK;
  if (!logits || !u || !token || (B > 1 && ld < V)) return QZ_ERR_INVALID_ARG;
  const qz_sampling &o = *options;
  if ((uintptr_t)logits & (dtype == QZ_FP32 ? 3u : 1u)) return QZ_ERR_ALIGNMENT;
  for (const void *p : {(const void *)u, (const void *)o.temperature, (const void *)o.top_k,
                        (const void *)o.top_p, (const void *)o.min_p, (const void *)token,
                        (const void *)logprob})
    if ((uintptr_t)p & 3u) return QZ_ERR_ALIGNMENT;
  return launch_sample(logits, dtype, B > 1 ? ld : 0, B, V, u, o, token, logprob, (cudaStream_t)s);
}

}  // extern "C"
