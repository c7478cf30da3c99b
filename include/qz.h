/*
 * qz.h - C ABI of libqz: weight-only quantized dequant-GEMV/GEMM for one GB300.
 *
 * The operations follow three web pages about serving a decoder LLM from
 * compressed weights:
 *   [ELG]  "Open Origin - ELG Stream Layer" (INT8 layer paging),
 *   [OTF]  "On-The-Fly Weight Synthesizer (OTF-LLM Engine)" (outlier-aware INT4),
 *   [NTR]  "NTransformer" summary (tiered layer streaming with custom GEMV).
 * Each entry point below names the section of the page that defines it.
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers unless the comment says host.
 *   - The caller allocates and owns every buffer.  The library never allocates
 *     or frees device memory and keeps no pointer to caller memory between
 *     calls (the pager keeps the pointers it is given until it is destroyed).
 *   - fp16 data is passed as qz_half: the bit pattern of an IEEE-754 binary16.
 *   - Matrices are row-major.  ld* is the distance between rows in ELEMENTS
 *     of the array's own type (bytes for int8/uint8 arrays).
 *   - Every call that launches GPU work is asynchronous on the given stream
 *     (NULL = the legacy default stream).  Outputs are valid once the stream
 *     has reached the call.  Calls that overlap on the GPU and write the same
 *     output race.
 *   - Arguments are validated on the host before anything is enqueued: a call
 *     that returns an error has enqueued nothing (QZ_ERR_CUDA excepted: the
 *     launch itself failed, and cudaGetLastError's code is kept in
 *     qz_last_cuda_error(), per host thread).
 *   - Alignment: every device pointer of a MATRIX (W, q, q4, w_out) must be
 *     16-byte aligned and its ld* must make rows 16-byte multiples (ld % 8 == 0
 *     for fp16, ld % 16 == 0 for int8/uint8); activation and output vectors
 *     (x, X, y, Y) need only the 2-byte alignment of fp16, with any ld >= the
 *     row length.  Violations return QZ_ERR_ALIGNMENT.
 *   - Inputs must be finite.  Non-finite weights or profiles give unspecified
 *     (but memory-safe) results.
 *   - No exception, abort or device trap is ever raised by the library.
 */
#ifndef QZ_H
#define QZ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st *qz_stream; /* the same type as cudaStream_t */
typedef uint16_t qz_half;              /* IEEE-754 binary16 bit pattern */

typedef enum {
  QZ_OK = 0,
  QZ_ERR_INVALID_ARG = 1, /* null pointer, negative or inconsistent size */
  QZ_ERR_ALIGNMENT = 2,   /* pointer or leading dimension breaks the 16-B rule */
  QZ_ERR_UNSUPPORTED = 3, /* valid but outside what the kernels handle (see call) */
  QZ_ERR_CUDA = 4,        /* a CUDA launch/enqueue failed; see qz_last_cuda_error */
  QZ_ERR_IO = 5,          /* pager host-side failure (copy enqueue, event) */
  QZ_ERR_DATA = 6         /* data check failed (qz_check_perm) */
} qz_status;

/* Human-readable name of a status; never NULL. */
const char *qz_status_string(qz_status st);
/* Library version as major*10000 + minor*100 + patch. */
int qz_version(void);
/* The cudaError_t of the last QZ_ERR_CUDA returned on this host thread. */
int qz_last_cuda_error(void);

/* Launch overlap for the GEMV/GEMM entry points, per host thread (off by
 * default).  When on, each product kernel is launched with programmatic
 * dependent launch: it may start while the preceding kernel on the stream is
 * still running, starts loading (GEMV: the first ring stage of each warp) or
 * already converts (tensor-core GEMM) the first weight tiles of each CTA, and
 * waits for that kernel (griddepcontrol.wait) before it reads x or writes y.
 * The caller promises that no work still in flight on the stream writes the
 * WEIGHTS of the call (q/q4/w_out/scale/perm); inputs and outputs keep normal
 * stream order.  Returns QZ_ERR_INVALID_ARG unless enable is 0 or 1. */
qz_status qz_set_overlap(int enable);
/* The current host thread's overlap setting (0 or 1). */
int qz_get_overlap(void);

/* The library's device error word, a bit set: 1 if a kernel gave up a
 * bounded wait (its output is then incomplete); 2 if qz_embed_int8 met a
 * token outside its table (that row was written as zeros); 4 if a page, a
 * position or an adapter index lay outside its table (qz_rope_append,
 * qz_attention_paged, their _int8 forms, qz_cache_read_int8, qz_lora; each
 * says what it did then).  0 if none
 * happened since the last clear.  Synchronous (reads device memory);
 * clear = 1 resets it.  Not for use during stream capture. */
qz_status qz_device_error(int *code, int clear);

/* Largest batch the GEMM entry points accept. */
#define QZ_MAX_BATCH 64
/* Largest number of matrices in one grouped launch. */
#define QZ_MAX_GROUP 4
/* Largest number of products in one sequence call (qz_gemv_*_sequence). */
#define QZ_MAX_SEQ 4

/* ======================================================================
 * INT8, one scale per tensor  [ELG "Technical Architecture > INT8
 * Quantization & Direct Mapping": scale = max|W| / 127, q = round(W/scale);
 * "FP16 On-The-Fly GPU Reconstruction": w = q * scale]
 * ====================================================================== */

/* Quantize an fp16 matrix W [N][ldw] to q [N][ldq] int8 and one fp32 scale.
 *   scale = fp32(max |W|) / 127 (IEEE fp32 divide, round to nearest even);
 *   q     = clamp(rint(fp32(W) / scale), -127, 127), rint = half-to-even;
 *   an all-zero W gives scale = 0 and q = 0.
 * Columns K..ldq-1 of q are written as 0.  *scale is used as the running
 * maximum while the call runs, so no other work may read it until the
 * stream has passed this call.  N, K >= 1; ldw >= K; ldq >= K. */
qz_status qz_quantize_int8(const qz_half *W, int64_t N, int64_t K, int64_t ldw,
                           int8_t *q, int64_t ldq, float *scale, qz_stream s);

/* A quantized INT8 matrix as the GEMV calls read it (a host struct holding
 * device pointers).  Bytes q[i][K..ldq) are never used in a product. */
typedef struct {
  const int8_t *q;     /* [N][ldq] codes */
  const float *scale;  /* [1] per-tensor scale */
  int64_t N, K, ldq;
} qz_int8_weight;

/* y[i] = fp16( scale * sum_j q[i][j] * x[j] ), fp32 accumulation, products of
 * the exact integer code with the fp16 input; no fp16 weight is formed.
 * x [K], y [N].  K <= 57344.  The CUDA-core kernel stages the input in
 * shared memory; at the largest K, where it does not fit, the call runs on the
 * tensor-core kernel instead (same result bound). */
qz_status qz_gemv_int8(const qz_int8_weight *w, const qz_half *x, qz_half *y,
                       qz_stream s);

/* Y[b][i] = fp16( scale * sum_j q[i][j] * X[b][j] ) for b < B.
 * X [B][ldx], Y [B][ldy]; 1 <= B <= QZ_MAX_BATCH.  The path depends on the
 * shape, never the result bound: B = 1 as qz_gemv_int8; B = 2..8 on the
 * warp-MMA kernel (mma.sync on the exact codes, fp32 accumulation) when the
 * batch's fp16 inputs and a ring of weight stages fit in shared memory
 * (roughly 2*B*K bytes well under 227 KiB); otherwise, and for B > 8, on
 * the tensor cores (tcgen05, fp16 x fp16 products of the exact codes, fp32
 * accumulation in tensor memory). */
qz_status qz_gemm_int8(const qz_int8_weight *w, int64_t B, const qz_half *X,
                       int64_t ldx, qz_half *Y, int64_t ldy, void *workspace,
                       size_t workspace_bytes, qz_stream s);

/* Device workspace the batched calls use on the tensor-core path: the
 * permuted inputs are gathered once per call into tensor-core tiles there,
 * then streamed into the GEMM by bulk copies; behind them lie the fp32
 * partial sums of output tiles whose K range is cut between SMs (at most two
 * per SM) and their arrival counters, so that every SM gets the same share
 * of the call's work.  B inputs of K channels with n_out outlier channels (0
 * for INT8); 0 for invalid sizes.  Host only; the size does not depend on N
 * or the device.  The workspace argument of qz_gemm_* may be NULL (the
 * tensor-core kernel then gathers its inputs itself and gives each SM whole
 * 128-row tiles only, much more slowly); if given it must be 16-byte aligned
 * and at least this many bytes (checked whatever path the call takes:
 * QZ_ERR_INVALID_ARG if short, QZ_ERR_ALIGNMENT if misaligned, before
 * anything is enqueued), caller-owned, and not used by other work while the
 * call runs.  Only the tensor-core path uses it.  Results with and without a
 * workspace agree within the products' rounding bound, not bit for bit (the
 * fp32 partial sums are added in a different order). */
size_t qz_gemm_workspace_bytes(int64_t B, int64_t K, int64_t n_out);

/* n matrices (1 <= n <= QZ_MAX_GROUP) that read the same input x, in one
 * launch (q/k/v, gate/up).  Each keeps its own scale.  ws: host array of n
 * structs with equal K; ys: host array of n device pointers. */
qz_status qz_gemv_int8_grouped(const qz_int8_weight *ws, int n,
                               const qz_half *x, qz_half *const *ys,
                               qz_stream s);

/* The batched form of qz_gemv_int8_grouped: n matrices (1 <= n <=
 * QZ_MAX_GROUP) of equal K read the same inputs X [B][ldx] in one call, and
 * Ys[m] [B][ldys[m]] receives matrix m's outputs.  Ys and ldys are host
 * arrays of n entries.  Batch limits, the CUDA-core/tensor-core choice and
 * the workspace are those of qz_gemm_int8 (one workspace serves the whole
 * group: qz_gemm_workspace_bytes(B, K, 0)). */
qz_status qz_gemm_int8_grouped(const qz_int8_weight *ws, int n, int64_t B,
                               const qz_half *X, int64_t ldx, qz_half *const *Ys,
                               const int64_t *ldys, void *workspace,
                               size_t workspace_bytes, qz_stream s);

/* Rows of an INT8 vocabulary table (embed_tokens) as fp16 activations
 * [OTF "Architecture & Key Innovations", key innovation 4: vocabulary
 * lookup tables compressed to INT8; ELG "FP16 On-The-Fly GPU
 * Reconstruction": q * scale as fp16]:
 *   out[b][j] = fp16(q[tokens[b]][j] * scale), b < B, j < K,
 * the exact product rounded once to the nearest fp16, ties to even.
 * table: the quantized [V][K] table (V = table->N), as qz_quantize_int8
 * makes it (one scale per tensor); any K.  tokens: device int32 [B], 4-byte
 * aligned.  out: device fp16 [B][ldo], 16-byte aligned, ldo >= K, ldo a
 * multiple of 8.  B >= 0 (B = 0 enqueues nothing).  A token outside [0, V)
 * is not read: its row of out is written as zeros and bit 2 of the device
 * error word (qz_device_error) is set.
 * With tied word embeddings the same table is the output projection
 * (lm_head): qz_gemv_int8(table, h, logits) gives
 * logits[v] = scale * sum_j q[v][j] h[j]. */
qz_status qz_embed_int8(const qz_int8_weight *table, const int32_t *tokens,
                        int64_t B, qz_half *out, int64_t ldo, qz_stream s);

/* ======================================================================
 * Outlier-aware INT4  [OTF "Architecture & Key Innovations": diagram and
 * key innovation 3 (global_perm_idx; top-1% channels by |W| x |X_profile|
 * kept in FP16; background INT4 in [-7,7], zero-point 0, 2:1 uint8 packing;
 * output = outlier product + background product); key innovation 1 (packed
 * weights dequantized in registers, no fp16 weight tensor)]
 *
 * Format of one [N][K] matrix with n_out outlier channels, kb = K - n_out:
 *   perm  int32 [K]          : permuted input t reads x[perm[t]]; t < n_out
 *                              are the outliers (global_perm_idx);
 *   w_out fp16  [N][ld_out]  : w_out[i][t] = W[i][perm[t]], t < n_out;
 *   q4    uint8 [N][ld_q4]   : background code of permuted input n_out + t'
 *                              in byte t'/2, low nibble if t' even, as the
 *                              two's-complement nibble (values -7..7);
 *   scale fp32  [N]          : s_i = fp32(max_t' |W[i][perm[n_out+t']]|) / 7.
 * ld_out = roundup(n_out, 8), ld_q4 = roundup(ceil(kb/2), 16); padding is 0.
 * ====================================================================== */

/* Row strides of the format (host only, no GPU work).  ld_out/ld_q4: host. */
qz_status qz_int4o_layout(int64_t N, int64_t K, int64_t n_out, int64_t *ld_out,
                          int64_t *ld_q4);

/* colsum[j] += sum_i |W[i][j]| * 2^24, exactly, as int64 (every fp16 value
 * is an integer multiple of 2^-24, so the sum is order-independent).  Call it
 * once per matrix that shares the permutation; the caller zeroes colsum. */
qz_status qz_saliency_accumulate(const qz_half *W, int64_t N, int64_t K,
                                 int64_t ldw, int64_t *colsum, qz_stream s);

/* Build global_perm_idx from colsum [K] and the activation profile
 * x_profile [K] (fp32): score_j = fp64(colsum[j]) * fp64(|x_profile[j]|); the
 * n_out channels of highest score (ties: lower j first) come first, in
 * ascending j, then the rest in ascending j.  0 <= n_out <= K <= 2^20.
 * perm [K] int32 is also used as working storage during the call. */
qz_status qz_select_outliers(const int64_t *colsum, const float *x_profile,
                             int64_t K, int64_t n_out, int32_t *perm,
                             qz_stream s);

/* *flag = 0 if perm [K] is a permutation of 0..K-1, 1 if an entry is out of
 * range, 2 if an entry repeats.  K <= 2^20.  The host reads flag after the
 * stream reaches the call; QZ_ERR_DATA is the host's verdict for flag != 0. */
qz_status qz_check_perm(const int32_t *perm, int64_t K, int32_t *flag,
                        qz_stream s);

/* Quantize W [N][ldw] fp16 with the given perm into the format above.
 * w_out may be NULL when n_out == 0.  ld_out/ld_q4 must be at least the
 * values of qz_int4o_layout and keep the 16-B rule; all padding is written
 * as 0.  Each CTA stages one fp16 row of W in shared memory, so K is limited
 * by the device's opt-in shared memory per block: 2 * roundup(K, 8) bytes
 * must fit (K <= 116224 on GB300's 227 KiB); beyond that, and beyond
 * K = 2^17 on any device, the call returns QZ_ERR_UNSUPPORTED. */
qz_status qz_quantize_int4_outlier(const qz_half *W, int64_t ldw,
                                   const int32_t *perm, int64_t N, int64_t K,
                                   int64_t n_out, qz_half *w_out,
                                   int64_t ld_out, uint8_t *q4, int64_t ld_q4,
                                   float *scale, qz_stream s);

/* One quantized INT4-outlier matrix (host struct holding device pointers). */
typedef struct {
  int64_t N, K, n_out, ld_out, ld_q4;
  const int32_t *perm;
  const qz_half *w_out; /* may be NULL when n_out == 0 */
  const uint8_t *q4;
  const float *scale;
} qz_int4o_weight;

/* y[i] = fp16( sum_{t<n_out} w_out[i][t] * x[perm[t]]
 *            + s_i * sum_{t'} q[i][t'] * x[perm[n_out+t']] )
 * fp32 accumulation of exact products; x is gathered through perm into
 * shared memory inside the kernel.  x [K] in ORIGINAL channel order, y [N].
 * K <= 57344. */
qz_status qz_gemv_int4_outlier(const qz_int4o_weight *w, const qz_half *x,
                               qz_half *y, qz_stream s);

/* The same for a batch: X [B][ldx], Y [B][ldy], 1 <= B <= QZ_MAX_BATCH; the
 * same choice of kernels as qz_gemm_int8.  Every kernel keeps the outlier
 * and background products apart and combines them as y = D_out + s_i * D_bg. */
qz_status qz_gemm_int4_outlier(const qz_int4o_weight *w, int64_t B,
                               const qz_half *X, int64_t ldx, qz_half *Y,
                               int64_t ldy, void *workspace,
                               size_t workspace_bytes, qz_stream s);

/* Allocation-free variant of qz_gemm_int4_outlier.  The pages have no
 * counterpart; it exists for callers that cannot allocate device memory at
 * the point of the call (code running during CUDA-graph capture, where
 * cudaMalloc is not allowed; plugins inside a host application that owns the
 * device memory budget; loops that must not touch an allocator after
 * start-up).  Instead of a caller workspace it uses a library-owned static
 * device array of QZ_NOALLOC_SCRATCH_BYTES, which every GPU that loads the
 * library holds until the process exits; it allocates nothing itself.
 * Limit: qz_gemm_workspace_bytes(B, K, n_out) must not exceed
 * QZ_NOALLOC_SCRATCH_BYTES (e.g. B = 64 up to K ~ 48k), else
 * QZ_ERR_UNSUPPORTED.  All calls share the array (it keeps the last call's
 * contents, every call rewrites what it reads): calls that overlap on the
 * GPU, on any stream, race.  The first call on a device looks the array's
 * device address up (cudaGetSymbolAddress) and should come before any stream
 * capture.  Same arguments and result as qz_gemm_int4_outlier otherwise. */
#define QZ_NOALLOC_SCRATCH_BYTES (16u << 20)
qz_status qz_gemm_int4_outlier_noalloc(const qz_int4o_weight *w, int64_t B,
                                       const qz_half *X, int64_t ldx,
                                       qz_half *Y, int64_t ldy, qz_stream s);

/* n matrices sharing one input and one permutation (same perm pointer, K and
 * n_out), one launch.  ws: host array; ys: host array of device pointers. */
qz_status qz_gemv_int4_outlier_grouped(const qz_int4o_weight *ws, int n,
                                       const qz_half *x, qz_half *const *ys,
                                       qz_stream s);

/* The batched form of qz_gemv_int4_outlier_grouped: n matrices sharing K,
 * n_out and perm read X [B][ldx]; Ys[m] [B][ldys[m]] receives matrix m's
 * outputs (host arrays of n entries).  Otherwise as qz_gemm_int4_outlier;
 * one workspace of qz_gemm_workspace_bytes(B, K, n_out) bytes serves the
 * group. */
qz_status qz_gemm_int4_outlier_grouped(const qz_int4o_weight *ws, int n, int64_t B,
                                       const qz_half *X, int64_t ldx,
                                       qz_half *const *Ys, const int64_t *ldys,
                                       void *workspace, size_t workspace_bytes,
                                       qz_stream s);

/* ======================================================================
 * Dependent products in one launch  [no counterpart on the pages: a decoder
 * layer's four products (q,k,v; o; gate,up; down) run back to back, each
 * reading the previous one's result through the layer glue, so one launch
 * per layer replaces four]
 *
 * n batch-1 grouped products (1 <= n <= QZ_MAX_SEQ) run in order in one
 * launch: product k multiplies the next counts[k] matrices of ws (equal K;
 * for INT4 also equal n_out and perm, as in the grouped calls) with x[k] and
 * stores them to the next counts[k] entries of ys.  Product k reads x[k] only
 * after every output of products 0..k-1 has been stored, so x[k] may be one
 * of those outputs.  Results equal the separate grouped calls bit for bit.
 *   ws, ys: host arrays of sum(counts) entries; counts, x: host arrays of n.
 *   sync: device uint32, 4-byte aligned, 0 before the first call; every call
 *   that completes leaves it 0.  Calls that can be in flight at the same time
 *   (for example consecutive calls under qz_set_overlap) need different
 *   words; after a device error (qz_device_error) it must be zeroed again.
 * The launch holds one CTA on every SM and its CTAs wait on one another
 * (bounded in time, reported through qz_device_error), so it must not share
 * the GPU with work that keeps SMs busy indefinitely.
 * ====================================================================== */
qz_status qz_gemv_int8_sequence(const qz_int8_weight *ws, const int *counts, int n,
                                const qz_half *const *x, qz_half *const *ys,
                                uint32_t *sync, qz_stream s);
qz_status qz_gemv_int4_outlier_sequence(const qz_int4o_weight *ws, const int *counts,
                                        int n, const qz_half *const *x,
                                        qz_half *const *ys, uint32_t *sync,
                                        qz_stream s);

/* ======================================================================
 * Zero-copy products  ["Open Origin - ELG Stream Layer", Technical
 * Architecture > INT8 Quantization & Direct Mapping: INT8 tensors kept in a
 * pre-allocated pinned memory pool and reached by zero-copy DMA; "NTransformer"
 * summary, 3-Tier Adaptive Caching, Tier B: layers kept in pinned RAM]
 *
 * The batch-1 grouped products with the weights read in place by the GPU:
 * every weight buffer of ws (codes, scales, and for INT4 outliers and perm)
 * may be pinned host memory mapped into the device's address space
 * (cudaHostAlloc, or cudaHostRegister with cudaHostRegisterMapped; under
 * unified addressing the host pointer is the device pointer) or device
 * memory.  Each call asks the runtime for the device address of every buffer
 * (cudaPointerGetAttributes); pageable or unknown memory gives
 * QZ_ERR_INVALID_ARG and nothing is launched.  x and ys are device memory.
 * Results equal the device-resident calls bit for bit; only the way codes
 * are read differs (plain loads by every lane, over the host link, instead
 * of bulk copies).  The host memory must stay pinned and unchanged until the
 * stream has passed the call.  Same sizes and errors as the grouped calls.
 * ====================================================================== */
qz_status qz_gemv_int8_grouped_mapped(const qz_int8_weight *ws, int n,
                                      const qz_half *x, qz_half *const *ys,
                                      qz_stream s);
qz_status qz_gemv_int4_outlier_grouped_mapped(const qz_int4o_weight *ws, int n,
                                              const qz_half *x,
                                              qz_half *const *ys, qz_stream s);

/* ======================================================================
 * Layer pager  [ELG "Key Features" 2 (prefetch, transfer, reconstruct,
 * purge) and 3 (a second CUDA stream copies layer N+1 while layer N
 * computes); NTR "3-Tier Adaptive Caching", Tier B (pinned RAM, H2D DMA)]
 *
 * Double-buffers packed layers from pinned host memory into two device
 * slots owned by the caller.  acquire(L) makes the compute stream wait until
 * layer L is in its slot and starts the copy of layer L+1 into the other
 * slot (after the compute that last used that slot, recorded by release);
 * release(L) marks the end of the compute work that reads layer L.  Layers
 * must be acquired in order 0, 1, ..., n-1 (then 0 again for the next pass).
 * The "purge" of the page becomes slot reuse: nothing is freed in the loop.
 * ====================================================================== */
typedef struct qz_pager qz_pager;

/* host_layers: host array of n_layers pinned host pointers; bytes: host
 * array of their sizes (each <= slot_bytes, multiple of 16); slot0/slot1:
 * device buffers of slot_bytes each.  The pager creates its own events; it
 * is destroyed with qz_pager_destroy.  *out receives the handle (host). */
qz_status qz_pager_create(const void *const *host_layers, const size_t *bytes,
                          int n_layers, void *slot0, void *slot1,
                          size_t slot_bytes, qz_stream copy_stream,
                          qz_stream compute_stream, qz_pager **out);
/* *dev_ptr (host) receives the device slot that holds `layer`. */
qz_status qz_pager_acquire(qz_pager *p, int layer, const void **dev_ptr);
qz_status qz_pager_release(qz_pager *p, int layer);
/* Waits for the pager's copies to finish, then frees its host state. */
qz_status qz_pager_destroy(qz_pager *p);

/* Host-side fault injection for tests: make the copy enqueue of layer
 * `layer` (at its next prefetch) fail as if cudaMemcpyAsync had failed.
 * The pager then drains its copy stream and acquire returns QZ_ERR_IO.
 * layer = -1 clears the injection.  Touches no GPU state. */
qz_status qz_pager_inject_copy_failure(qz_pager *p, int layer);

/* ======================================================================
 * Layer glue for serving  [the pages name a decoder LLM but define no step
 * between its products; these are the usual definitions of such a layer]
 *
 * Sizes here: T tokens (rows) of a step, packed sequence after sequence.
 * ====================================================================== */

/* Residual addition and root-mean-square normalisation of T rows:
 *   h[t][j] = x[t][j] + residual[t][j]   (h = x when residual is NULL)
 *   y[t][j] = fp16( h[t][j] * rsqrt(mean_j h[t][j]^2 + eps) * (w_bias + weight[j]) )
 * h is held in fp32 (the norm is that of the unrounded sum) and rounded once
 * when stored to sum [T][lds] (NULL: not stored).  weight: fp16 [K]; w_bias is
 * 0, or 1 for models that store w - 1.  sum may be x or residual and y may be x
 * (same pointer and stride: in place).  T >= 0 (0 enqueues nothing), 1 <= K <=
 * 57344, eps >= 0.  2-byte alignment and any stride >= K suffice; rows whose
 * every array is 16-byte aligned with K and strides multiples of 8 are read
 * and written 16 bytes at a time. */
qz_status qz_rmsnorm(const qz_half *x, int64_t ldx, const qz_half *residual, int64_t ldr,
                     const qz_half *weight, float w_bias, float eps, int64_t T, int64_t K,
                     qz_half *y, int64_t ldy, qz_half *sum, int64_t lds, qz_stream s);

/* The same with the normalised rows in INT8, one fp32 scale per row, by the
 * rule of qz_quantize_int8 applied to the unrounded y:
 *   scale[t] = max_j |y[t][j]| / 127;  q = clamp(rint(y / scale), -127, 127);
 * a row of zeros gives scale 0 and codes 0 (whatever eps), a row with a NaN or an
 * infinity in x, residual or weight a scale that is not finite and codes 0.
 * q [T][ldq], ldq >= K (columns K.. are not written), scale [T]. */
qz_status qz_rmsnorm_int8(const qz_half *x, int64_t ldx, const qz_half *residual, int64_t ldr,
                          const qz_half *weight, float w_bias, float eps, int64_t T, int64_t K,
                          int8_t *q, int64_t ldq, float *scale, qz_half *sum, int64_t lds,
                          qz_stream s);

/* A paged key/value cache: a pool of n_pages pages of page_size tokens.  The
 * row of token slot t of page p and KV head h starts at k + p * k_page +
 * h * k_head + t * k_token (strides in halves; v likewise) and holds head_dim
 * contiguous fp16 values.  page_size: 8, 16, 32, 64, 128 or 256.  head_dim:
 * 64, 128 or 256.  k and v 16-byte aligned, strides multiples of 8. */
typedef struct {
  qz_half *k, *v;
  int64_t n_pages, page_size, n_kv_heads, head_dim;
  int64_t k_page, k_head, k_token;
  int64_t v_page, v_head, v_token;
} qz_kv_cache;

/* The sequences of a step (device arrays, read when the call runs).  Sequence
 * i brings the new tokens cu_q[i] .. cu_q[i+1]-1 of the n_tokens packed rows
 * (cu_q non-decreasing, within 0..n_tokens; rows outside every sequence are
 * not written and do not matter) and holds kv_len[i] tokens, the new ones
 * last: its new token j has position kv_len[i] - (cu_q[i+1] - cu_q[i]) + j.
 * Token position p lies in slot p % page_size of page
 * page_table[i * ld_table + p / page_size]. */
typedef struct {
  int64_t n_seqs, n_tokens;
  const int32_t *cu_q;       /* [n_seqs + 1] */
  const int32_t *kv_len;     /* [n_seqs] */
  const int32_t *page_table; /* [n_seqs][ld_table] */
  int64_t ld_table;          /* pages a sequence may have; entries past its last page are not read */
} qz_seq_batch;

/* Rotary position embedding of new queries and keys, and storage of the keys
 * and values into the cache.  With half = head_dim / 2 and row
 * (c_0..c_{half-1}, s_0..s_{half-1}) = rope[position]:
 *   x'[j] = x[j] c_j - x[j + half] s_j,  x'[j + half] = x[j + half] c_j + x[j] s_j,
 * computed in fp32 and rounded once.  q, q_out: [n_tokens][n_heads][head_dim]
 * with strides q_token, q_head (q_out may be q); k, v likewise with
 * n_kv_heads.  rope: fp32 [rope_len][head_dim], or NULL to store the keys as
 * they are (q_out may then be NULL; otherwise q is copied).  q may be NULL with
 * q_out to store keys and values only.  A new token whose position is negative,
 * has no page, or lies beyond rope (its page outside the pool included) is not
 * stored, its q_out row is zeros, and bit 4 of the device error word is set
 * (a negative position, of a sequence that holds fewer tokens than are new,
 * sets no bit).  Two sequences must not share a page that both write.
 * Pointers 16-byte aligned, strides multiples of 8. */
qz_status qz_rope_append(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                         const qz_half *k, int64_t k_token, int64_t k_head, const qz_half *v,
                         int64_t v_token, int64_t v_head, const float *rope, int64_t rope_len,
                         const qz_kv_cache *cache, const qz_seq_batch *seqs, qz_half *q_out,
                         int64_t qo_token, int64_t qo_head, qz_stream s);

/* Attention of the new tokens over the paged cache (which already holds their
 * keys and values).  For query head g, KV head h = g / (n_heads / n_kv_heads)
 * and a new token at position p of its sequence:
 *   x_j = scale * q . k_j;  if softcap > 0: x_j = softcap * tanh(x_j / softcap);
 *   out = sum_j e^{x_j} v_j / sum_j e^{x_j}  over j <= p, j < kv_len and, if
 *   window > 0, j > p - window.
 * One new token per sequence is a decode step; kv_len = number of new tokens
 * is a whole prompt.  A query that sees no key (kv_len 0, or fewer tokens held
 * than new) gives zeros.  Slots that no query of a call sees (past kv_len,
 * before every window, free pages) may hold anything, NaN included; the
 * others must be finite.  A page outside the pool, or beyond ld_table, reads as
 * zeros (keys and values) and sets bit 4 of the device error word.
 * Logits, softmax sums and outputs are held in fp32; the weights e^{x_j - m} are
 * rounded to fp16 where they enter the tensor cores (to 2^-11 of each, or 2^-32 of
 * the largest).  softcap is good to fp32 at any size; up to 64 the capped logit is
 * off by 2^-22 of the cap and is cheaper.  scale: finite.
 * q, out: [n_tokens][n_heads][head_dim] with strides q_token, q_head, o_token,
 * o_head; 16-byte aligned, strides multiples of 8; out must not overlap q.
 * n_tokens * n_heads < 2^31.
 * workspace: qz_attention_workspace_bytes bytes of device memory, 16-byte
 * aligned, the first QZ_ATTENTION_SYNC_BYTES of them zeroed before its first
 * use and left zero by every call that completes (zero them again after device
 * error 1); calls that can be in flight at the same time need different ones.
 * Results repeat bit for bit. */
#define QZ_ATTENTION_SYNC_BYTES 8192
qz_status qz_attention_paged(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                             const qz_kv_cache *cache, const qz_seq_batch *seqs, float scale,
                             float softcap, int64_t window, qz_half *out, int64_t o_token,
                             int64_t o_head, void *workspace, size_t workspace_bytes,
                             qz_stream s);

/* Workspace of qz_attention_paged for up to n_seqs sequences with up to
 * n_tokens new tokens in all; 0 for invalid sizes.  Host only. */
size_t qz_attention_workspace_bytes(int64_t n_tokens, int64_t n_seqs, int64_t n_heads,
                                    int64_t n_kv_heads, int64_t head_dim);

/* A paged key/value cache of INT8 rows: every row (a token slot of a KV head) is
 * head_dim codes and one fp32 scale, and stands for code * scale.  The codes lie
 * as the rows of qz_kv_cache do (strides in bytes, multiples of 16; k and v
 * 16-byte aligned), the scale of token slot t of page p and head h at
 * k_scale + p * ks_page + h * ks_head + t * ks_token (strides in floats; v
 * likewise).  Same page sizes and head sizes. */
typedef struct {
  int8_t *k, *v;
  float *k_scale, *v_scale;
  int64_t n_pages, page_size, n_kv_heads, head_dim;
  int64_t k_page, k_head, k_token;
  int64_t v_page, v_head, v_token;
  int64_t ks_page, ks_head, ks_token;
  int64_t vs_page, vs_head, vs_token;
} qz_kv_cache_int8;

/* qz_rope_append into a cache of INT8 rows.  With y the value, or the rotated key
 * rounded to fp32 (from its exact products), by the rule of qz_quantize_int8:
 *   scale = fp32(max_j |y[j]|) / 127;  code[j] = clamp(rint(y[j] / scale), -127, 127)
 * (IEEE fp32 divisions, ties to even); a row of zeros gives scale 0 and codes 0, a
 * row with a NaN or an infinity a scale that is not finite and codes 0.  q_out,
 * positions, what is not stored, and errors are those of qz_rope_append. */
qz_status qz_rope_append_int8(const qz_half *q, int64_t n_heads, int64_t q_token, int64_t q_head,
                              const qz_half *k, int64_t k_token, int64_t k_head,
                              const qz_half *v, int64_t v_token, int64_t v_head,
                              const float *rope, int64_t rope_len,
                              const qz_kv_cache_int8 *cache, const qz_seq_batch *seqs,
                              qz_half *q_out, int64_t qo_token, int64_t qo_head, qz_stream s);

/* Rows of such a cache as fp16: row t of k and v [n_tokens][n_kv_heads][head_dim]
 * (strides k_token, k_head, ...) is the cache's row of the token that seqs gives
 * row t, fp16(code * scale), the product rounded to fp32 before.  So the sequences
 * of a step give its new tokens, and cu_q with the running sums of kv_len all
 * that is held.  Rows outside every sequence, and tokens of a negative position
 * (which read as zeros), are as in qz_rope_append; a page outside the pool or
 * beyond ld_table reads as zeros and sets bit 4 of the device error word.  k and
 * v 16-byte aligned, strides multiples of 8. */
qz_status qz_cache_read_int8(const qz_kv_cache_int8 *cache, const qz_seq_batch *seqs, qz_half *k,
                             int64_t k_token, int64_t k_head, qz_half *v, int64_t v_token,
                             int64_t v_head, qz_stream s);

/* qz_attention_paged over a cache of INT8 rows: k_j and v_j are the rows' codes
 * times their scales.  Nothing of them is rounded to fewer than 32 bits: codes enter
 * the products as they are, or times four bits of their scales (exact in fp16), and
 * the scales, or the rest of them, multiply logits and weights in fp32.  The
 * weights times that of the values' scales are rounded to fp16 where they enter the
 * tensor cores (to 2^-11 of each, or 2^-30 of the largest that the sequence's new
 * tokens see).  Scales are those of qz_rope_append_int8: not negative, the values' at
 * most 65504 / 127.  A seen row whose scale is not finite makes outputs of its
 * sequence in the step that see it NaN, and may, if it is a value's, those of its
 * other rows.
 * Everything else is as in qz_attention_paged, with the same workspace (which
 * calls of both may share one after the other); codes of slots that no query sees
 * may hold anything, and so may their scales. */
qz_status qz_attention_paged_int8(const qz_half *q, int64_t n_heads, int64_t q_token,
                                  int64_t q_head, const qz_kv_cache_int8 *cache,
                                  const qz_seq_batch *seqs, float scale, float softcap,
                                  int64_t window, qz_half *out, int64_t o_token, int64_t o_head,
                                  void *workspace, size_t workspace_bytes, qz_stream s);

/* Low-rank adapters of many requests beside a shared projection:
 *   out[t][i] = fp16( y[t][i] + scale[a] * sum_{r < rank[a]} B_a[i][r] * u_r ),
 *   u_r = sum_j A_a[r][j] x[t][j],  a = index[t];
 * a row with index -1 has no adapter (out = y).  y: the projection's output
 * [T][ldy] (qz_gemm_* of the same x), out [T][ldo] (may be y).  A_a = a +
 * a * a_adapter, rows a_row apart; B_a = b + a * b_adapter, rows b_row
 * apart (halves).  rank NULL: all R.  1 <= R <= 128, ranks are clamped to 0..R.
 * Sums are fp32; between the two products u is held to 22 bits of its row's
 * largest value (two fp16 parts), at every K.  An index outside
 * -1..n_adapters-1 counts as -1 and sets bit 4 of the device error word.
 * Rows with the same index share reads of their adapter, in calls of fewer than
 * 128 rows when they are neighbours.  2-byte alignment suffices; 16-byte aligned
 * operands with K, R and strides multiples of 8 run fastest.  K, N <= 2^20.
 * workspace: qz_lora_workspace_bytes(T, K, R) bytes, 16-byte aligned (any
 * contents); calls that can be in flight at the same time need different ones. */
typedef struct {
  const qz_half *a, *b;
  const float *scale;  /* [n_adapters] */
  const int32_t *rank; /* [n_adapters] or NULL */
  int64_t n_adapters, R, K, N;
  int64_t a_adapter, a_row, b_adapter, b_row;
} qz_lora_adapters;

qz_status qz_lora(const qz_lora_adapters *ad, const int32_t *index, int64_t T,
                  const qz_half *x, int64_t ldx, const qz_half *y, int64_t ldy, qz_half *out,
                  int64_t ldo, void *workspace, size_t workspace_bytes, qz_stream s);
size_t qz_lora_workspace_bytes(int64_t T, int64_t K, int64_t R);

/* The next tokens of B requests from their logits.  With x = row b of the logits
 * (NaN counts as -inf) and m its largest:
 *   w_i = e^{(x_i - m) / temperature};
 *   top_k: the k tokens of largest logit are kept (1 <= k < V; others keep all);
 *   top_p: of those, the fewest, largest first, whose weights sum to top_p of all
 *     of theirs, one at least (top_p < 1; others keep all);
 *   min_p: of those, the ones with w_i >= min_p (0 < min_p; 1 and above keep the
 *     largest only).
 * Equal logits are taken lowest index first.  token[b] is the first kept i whose
 * running sum of kept weights, by index, exceeds u[b] times their total, and
 * logprob[b] = ln(w_i / total) (logprob may be NULL).  temperature <= 0 takes the
 * largest logit (probability 1).  u outside [0, 1) is taken as the nearest value
 * in it.  A row without any logit above -inf gives token -1 and logprob -inf;
 * logits of +inf share all the weight.
 * Weights are held as integers, 2^45 for the largest (to 2^-28 of each and half a
 * unit; below 2^-46 of the largest they are 0), and summed exactly: results repeat
 * bit for bit and a row's do not depend on the others.
 * logits [B][ld] of the given type, aligned to its size (16-byte aligned rows are
 * read faster), ld >= V.  Options: a device array of B values, or NULL and one
 * value for all rows.  1 <= V <= QZ_MAX_VOCAB, B <= 2^24. */
typedef enum { QZ_FP16 = 0, QZ_BF16 = 1, QZ_FP32 = 2 } qz_dtype;
#define QZ_MAX_VOCAB (1 << 18)
typedef struct {
  const float *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  float temperature_all;
  int32_t top_k_all;
  float top_p_all, min_p_all;
} qz_sampling;
qz_status qz_sample(const void *logits, int dtype, int64_t B, int64_t V, int64_t ld,
                    const float *u, const qz_sampling *options, int32_t *token, float *logprob,
                    qz_stream s);

#ifdef __cplusplus
}
#endif
#endif /* QZ_H */
