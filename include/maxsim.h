/*
 * maxsim.h -- C ABI of libmaxsim.so, late-interaction MaxSim scoring on
 * NVIDIA GB300 (sm_103a).
 *
 * The operator ("TileMaxSim: IO-Aware GPU MaxSim Scoring with Dimension
 * Tiling and Fused Product Quantization", §1; "FLASH-MAXSIM: IO-Aware Fused
 * Kernels for Late-Interaction Scoring", Abstract):
 *
 *     score(Q, D_b) = sum_{i < nq} max_{j < L_b} <q_i, d_j>
 *
 * for a query Q of nq token embeddings and a document D_b of L_b token
 * embeddings, all of dimension d. Inputs are taken as given: the library
 * does not normalise them (the "cosine" of the pages is the dot product of
 * L2-normalised embeddings).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every tensor pointer is a DEVICE pointer owned by the caller, row-major
 *    and contiguous. The library allocates and frees no device memory;
 *    where an operation needs scratch space the caller passes a workspace
 *    sized by the matching *_workspace_size() query.
 *  - Element pointers must be 16-byte aligned (TMA and vector loads).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream). Every call is asynchronous on that stream and returns as soon
 *    as its kernels are enqueued; outputs are valid once the stream reaches
 *    that point.
 *  - Errors: argument problems found on the host return
 *    MAXSIM_ERR_INVALID_ARG or MAXSIM_ERR_UNSUPPORTED before anything is
 *    launched. A failed launch returns MAXSIM_ERR_CUDA. Problems found on
 *    the device (inconsistent CSR offsets or lengths, a pipeline wait that
 *    gave up) cannot be returned by the asynchronous call; the kernel
 *    records them in a per-device status word, treats a bad document as
 *    empty, and maxsim_device_status() reports them. No kernel traps, asserts
 *    or spins without a bound. No C++ exception crosses this ABI.
 *  - Outputs are fp32 (scores, gradients) or int32 (indices). An empty
 *    document (L_b = 0) scores 0.0 and has argmax -1.
 *  - The argmax of query token i in document b is the LOWEST doc-local token
 *    index j attaining the maximum similarity.
 *  - Per-device state: on its first call on a device the library looks up
 *    the device addresses of its own global variables (the status word, the
 *    table of maxsim_score_pq_noalloc) and keeps them for the life of the
 *    process. cudaDeviceReset() invalidates them: do not reset a device
 *    between calls into this library.
 */
#ifndef MAXSIM_H_
#define MAXSIM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum maxsim_status {
    MAXSIM_OK = 0,
    MAXSIM_ERR_INVALID_ARG = 1,  /* NULL/misaligned pointer, negative size, bad lengths/offsets */
    MAXSIM_ERR_UNSUPPORTED = 2,  /* valid arguments the library does not handle (e.g. d % 64 != 0 on the tensor-core path) */
    MAXSIM_ERR_CUDA = 3,         /* a CUDA runtime call or kernel launch failed */
    MAXSIM_ERR_TIMEOUT = 4,      /* a device pipeline wait gave up after its time bound */
    MAXSIM_ERR_WORKSPACE = 5     /* workspace NULL or smaller than the size query returned */
} maxsim_status;

typedef enum maxsim_dtype {
    MAXSIM_BF16 = 0,   /* bf16 in, fp32 accumulate (tcgen05 tensor cores) */
    MAXSIM_FP16 = 1,   /* fp16 in, fp32 accumulate (tcgen05 tensor cores) */
    MAXSIM_FP32 = 2    /* fp32 in, fp32 FFMA on the CUDA cores */
} maxsim_dtype;

/* Bits of the device status word (see maxsim_device_status). */
#define MAXSIM_DEVERR_TIMEOUT    0x1u  /* a pipeline wait exceeded its time bound */
#define MAXSIM_DEVERR_BAD_INPUT  0x2u  /* a document's offsets/length were out of range */

/*
 * maxsim_debug_set_faults -- TEST-ONLY switches of the failure-detection
 * path; not part of the operator, never needed in normal use. Applies to the
 * current device, to every kernel launched after the call returns (the call
 * is synchronous).
 *   flags          MAXSIM_DEBUG_STALL_FWD_LOADER: the loader role of the
 *                  tensor-core forward kernel (maxsim_score / _varlen with
 *                  bf16 or fp16 and queries below 256 tokens) and of the
 *                  attention kernels (maxsim_attention / _backward) issues no copy,
 *                  so the kernel's other roles wait on barriers nothing will
 *                  complete; their bounded waits run out, record
 *                  MAXSIM_DEVERR_TIMEOUT and the kernel exits with no copy or
 *                  MMA in flight (its outputs are then undefined). 0 = off.
 *   wait_limit_ns  bound of every pipeline wait; 0 restores the default (2 s).
 * Call maxsim_debug_set_faults(0, 0) to return to normal operation. Unknown
 * flag bits return MAXSIM_ERR_INVALID_ARG; a failed copy MAXSIM_ERR_CUDA.
 */
#define MAXSIM_DEBUG_STALL_FWD_LOADER 0x1u
maxsim_status maxsim_debug_set_faults(unsigned int flags, uint64_t wait_limit_ns);

/* Library version: major*10000 + minor*100 + patch. */
int maxsim_version(void);

/* Human-readable name of a status code (static string, never NULL). */
const char *maxsim_status_string(maxsim_status status);

/*
 * maxsim_device_status -- synchronises `stream`, then reads and clears the
 * status word of the current device. *flags (may be NULL) receives the
 * MAXSIM_DEVERR_* bits seen since the last call. Returns MAXSIM_ERR_TIMEOUT
 * if the timeout bit was set, else MAXSIM_ERR_INVALID_ARG if the bad-input
 * bit was set, else MAXSIM_OK (or MAXSIM_ERR_CUDA if the stream failed).
 */
maxsim_status maxsim_device_status(void *stream, unsigned int *flags);

/*
 * maxsim_score -- padded layout, one or more queries.
 *
 * Follows TileMaxSim §1 (operator), §2(1) (every document byte streamed
 * from HBM once, the per-query-token maximum kept on chip), §2(2)
 * (dimension tiling: partial dot products over d-chunks are summed before
 * the maximum) and §5 (fixed-Nd padding with a length mask); FLASH-MAXSIM
 * Figure 1 / Algorithm 2 (running maximum from -inf, only the scalar score
 * written back).
 *
 *   Q          [n_queries, nq, d]  dtype
 *   D          [B, nd, d]          dtype; document b's tokens are rows
 *                                  0 .. L_b-1 of D[b]; rows L_b .. nd-1 are
 *                                  never read by the tensor-core path beyond
 *                                  a 32-row granule and never contribute
 *   doc_len    [B] int32 or NULL   L_b (0 <= L_b <= nd); NULL means L_b = nd
 *   out        [n_queries, B] fp32 out[q*B + b] = score(Q[q], D_b)
 *   argmax_out [n_queries, B, nq] int32 or NULL
 *
 * Limits: nq >= 1, n_queries >= 1, nd >= 1, B >= 0 (B = 0 is a no-op).
 * BF16/FP16: d % 64 == 0 and 64 <= d <= 1024. FP32: d % 4 == 0, d <= 1024.
 */
maxsim_status maxsim_score(const void *Q, int n_queries, int nq, int d,
                           const void *D, int64_t B, int nd, const int32_t *doc_len,
                           maxsim_dtype dtype, float *out, int32_t *argmax_out,
                           void *stream);

/*
 * maxsim_length_order -- length-bucketed document order (TileMaxSim §5:
 * fixed-Nd padding wastes token compute on variable-length corpora, and
 * batching documents of similar length recovers the throughput). Writes the
 * permutation order_out[B] that sorts the documents by their number of 8-row
 * granules, ceil(L_b / 8), ascending and stably (equal keys keep index
 * order). It depends only on the lengths: compute it once per corpus and
 * pass it to maxsim_score_ordered for every query.
 *   doc_len    [B] int32, 0 <= L_b <= nd (padded layout), or
 *   offsets    [B+1] int64 (CSR layout; nd ignored, lengths above 8176
 *              tokens share the last bucket) -- exactly one of the two, or
 *              neither (every document has nd tokens: the identity order)
 *   workspace  >= maxsim_length_order_workspace_size(B, nd, csr) bytes,
 *              16-byte aligned (per-warp bucket counts)
 * A length outside [0, nd] (or a decreasing offset) counts as 0 and sets
 * MAXSIM_DEVERR_BAD_INPUT. B <= INT32_MAX.
 */
size_t maxsim_length_order_workspace_size(int64_t B, int nd, int csr);
maxsim_status maxsim_length_order(const int32_t *doc_len, const int64_t *offsets, int64_t B, int nd,
                                  int32_t *order_out, void *workspace, size_t workspace_bytes, void *stream);

/*
 * maxsim_score_ordered -- maxsim_score with the documents walked in the order
 * doc_order (a permutation of [0, B), e.g. from maxsim_length_order), so each
 * thread block scores documents of similar length. Results are written at
 * the documents' own indices and are identical to maxsim_score's: a
 * document's result depends only on its own rows. An entry outside [0, B)
 * is skipped and sets MAXSIM_DEVERR_BAD_INPUT; duplicates leave the missing
 * documents' outputs unwritten. Same arguments and limits as maxsim_score,
 * bf16/fp16 only, and queries shorter than 256 tokens (longer ones, and fp32,
 * return MAXSIM_ERR_UNSUPPORTED).
 */
maxsim_status maxsim_score_ordered(const void *Q, int n_queries, int nq, int d,
                                   const void *D, int64_t B, int nd, const int32_t *doc_len,
                                   const int32_t *doc_order, maxsim_dtype dtype, float *out,
                                   int32_t *argmax_out, void *stream);

/*
 * maxsim_score_varlen -- variable-length, padding-free documents in CSR
 * form (FLASH-MAXSIM, Abstract: variable-length padding-free scoring;
 * TileMaxSim §5: the padding waste it removes).
 *
 *   D_packed   [total_tokens, d] dtype; document b owns rows
 *              offsets[b] .. offsets[b+1]-1
 *   offsets    [B+1] int64, offsets[0] = 0, non-decreasing,
 *              offsets[B] = total_tokens (checked on the device: a document
 *              whose range falls outside [0, total_tokens] is scored as
 *              empty and sets MAXSIM_DEVERR_BAD_INPUT)
 *   out        [n_queries, B] fp32; argmax_out [n_queries, B, nq] int32 or NULL
 *
 * Same dtype and d limits as maxsim_score.
 */
maxsim_status maxsim_score_varlen(const void *Q, int n_queries, int nq, int d,
                                  const void *D_packed, const int64_t *offsets,
                                  int64_t B, int64_t total_tokens,
                                  maxsim_dtype dtype, float *out, int32_t *argmax_out,
                                  void *stream);

/*
 * maxsim_score_pq -- fused product-quantisation scoring (TileMaxSim §2(3)):
 * the per-query table T[i,m,k] = q_i[m*(d/M) .. (m+1)*(d/M)) . C[m,k,:] is
 * built once into the workspace, then each token's similarity is
 * sum_m T[i, m, codes[j,m]] by table lookup; decoded vectors never exist.
 *
 *   Q          [nq, d] fp32
 *   codebooks  [M, K, d/M] fp32 (d % M == 0, K <= 256)
 *   codes      [total_tokens, M] uint8, CSR documents as in maxsim_score_varlen
 *   out        [B] fp32; argmax_out [B, nq] int32 or NULL
 *   workspace  >= maxsim_score_pq_workspace_size(nq, M, K) bytes, 16-byte
 *              aligned; holds the table (groups of 8 query tokens, fp32);
 *              contents on entry are ignored, the call overwrites it.
 *
 * Limits: 1 <= nq <= 1024; M % 4 == 0, 4 <= M <= 64; 1 <= K <= 256;
 * d % M == 0, d <= 1024; one 8-token table group (M * K * 32 bytes) plus
 * 64 KB of code staging must fit in shared memory (M * K <= 5056), else
 * MAXSIM_ERR_UNSUPPORTED. A code >= K is clamped to K-1 and sets
 * MAXSIM_DEVERR_BAD_INPUT. Missing or short workspace: MAXSIM_ERR_WORKSPACE.
 */
size_t maxsim_score_pq_workspace_size(int nq, int M, int K);
maxsim_status maxsim_score_pq(const float *Q, int nq, int d,
                              const float *codebooks, int M, int K,
                              const uint8_t *codes, const int64_t *offsets,
                              int64_t B, int64_t total_tokens,
                              float *out, int32_t *argmax_out,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * maxsim_score_pq_noalloc -- maxsim_score_pq for callers that cannot
 * allocate device memory. The source pages have no counterpart: this is a
 * library convenience, not part of the method.
 *
 * Some callers have no way to hand over a workspace: code that runs where a
 * device allocation is forbidden or unavailable (a host callback, a hook
 * inside another library, a plugin without an allocator). This variant keeps
 * the PQ table in a fixed 1 MiB device array compiled into the library
 * (present on every GPU that loads it, until the process exits) and
 * allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *
 *   Arguments, layouts, results and other limits: as maxsim_score_pq,
 *   without the workspace.
 *   Limit: the table, ceil(nq/8)*8 * M * K * 4 bytes, must fit in 1 MiB
 *   (e.g. nq <= 64 at M = 16, K = 256); larger requests return
 *   MAXSIM_ERR_WORKSPACE before anything is launched.
 *   Set-up: the first call on each device looks up the array's device
 *   address with that device current; make that first call before any
 *   stream capture. A failed lookup returns MAXSIM_ERR_CUDA. The address is
 *   kept until the process exits, so the device must not be reset
 *   (cudaDeviceReset) between calls.
 *   Sharing: every call uses the same array, and it keeps the previous
 *   call's table. Each call rewrites every entry it reads, so no clearing is
 *   needed; but calls whose kernels overlap on the GPU (for example on two
 *   streams) race on the array and give wrong results -- serialise them.
 */
maxsim_status maxsim_score_pq_noalloc(const float *Q, int nq, int d,
                                      const float *codebooks, int M, int K,
                                      const uint8_t *codes, const int64_t *offsets,
                                      int64_t B, int64_t total_tokens,
                                      float *out, int32_t *argmax_out, void *stream);

/*
 * maxsim_score_streamed -- maxsim_score for documents that stay in host
 * memory, e.g. a corpus larger than GPU memory (TileMaxSim deep reading §5
 * names it as an open limitation). Same operator and outputs as
 * maxsim_score; per-document results are identical to scoring the same
 * documents from device memory.
 *   Q            device [n_queries, nq, d] (as maxsim_score)
 *   D_host       HOST [B, nd, d] in dtype; page-locked memory (cudaHostAlloc /
 *                torch pin_memory) lets copies overlap scoring, pageable
 *                memory works but serialises each copy
 *   doc_len_host HOST int32 [B] or NULL (as doc_len of maxsim_score)
 *   out, argmax_out  device, as maxsim_score
 *   workspace    device, 16-byte aligned, >= the size returned below
 *   chunk_docs   documents per chunk (>= 1); two chunks of device buffers
 *                alternate: the copy of chunk k + 1 (on a library-owned
 *                copy stream) runs while chunk k is scored on `stream`.
 * Returns after enqueueing; D_host, doc_len_host and the workspace must
 * stay valid and unchanged until `stream` has completed. Errors as
 * maxsim_score; a short workspace returns MAXSIM_ERR_WORKSPACE. On any other
 * error return, the copies the call had queued have finished (the call waits
 * for them), though kernels already queued on `stream` may still run.
 */
size_t maxsim_score_streamed_workspace_size(int n_queries, int nq, int nd, int d, maxsim_dtype dtype,
                                            int64_t chunk_docs);
maxsim_status maxsim_score_streamed(const void *Q, int n_queries, int nq, int d, const void *D_host,
                                    int64_t B, int nd, const int32_t *doc_len_host, maxsim_dtype dtype,
                                    float *out, int32_t *argmax_out, void *workspace,
                                    size_t workspace_bytes, int64_t chunk_docs, void *stream);

/*
 * maxsim_score_i8 -- INT8 x INT8 scoring (FLASH-MAXSIM, Abstract) with
 * per-token symmetric scales:
 *   dot(i,j) = sum_k Q[i,k] * D[j,k]        exact int32
 *   sim(i,j) = (float)dot(i,j) * d_scale[j] one fp32 multiply
 *   m_i      = max_j sim(i,j)
 *   out[b]   = sum_i q_scale[i] * m_i       fp32
 *
 *   Q [nq, d] int8, q_scale [nq] fp32 (> 0)
 *   D [total_tokens, d] int8, d_scale [total_tokens] fp32 (> 0); CSR as above
 *   out [B] fp32; maxv_out [B, nq] fp32 (m_i), maxdot_out [B, nq] int32
 *   (dot at the argmax), argmax_out [B, nq] int32 -- each of the last three
 *   may be NULL.
 *
 * sm_103a has no tcgen05 8-bit integer MMA. For nq <= 32 and d <= 192 the
 * int8 operands are converted to fp16 on chip and multiplied on tcgen05:
 * int8 values and products are exact in fp16 and the partial sums (|.| <=
 * 2^22) in the fp32 accumulator, so the dots are exact. Other shapes run on
 * the warp-level IMMA path (mma.sync m16n8k32 s8).
 *
 * Limits: 1 <= nq <= 256; d in {64, 128, 192, 256, 384, 512, 768, 1024}
 * (so |dot| < 2^24 and (float)dot is exact); Q and D 16-byte aligned.
 */
maxsim_status maxsim_score_i8(const int8_t *Q, const float *q_scale, int nq, int d,
                              const int8_t *D, const float *d_scale,
                              const int64_t *offsets, int64_t B, int64_t total_tokens,
                              float *out, float *maxv_out, int32_t *maxdot_out,
                              int32_t *argmax_out, void *stream);

/*
 * maxsim_backward -- gradients through the forward argmax (FLASH-MAXSIM,
 * Abstract: the backward pass reuses the forward argmax, with an
 * inverse-grid CSR construction and an atomic-free, destination-owned
 * gradient reduction). With loss = sum_{q,b} dS[q,b] * score[q,b] and
 * a = argmax[q,b,i]:
 *   dQ[q,i,:] = sum_b dS[q,b] * D[b, a, :]
 *   dD[b,j,:] = sum_q dS[q,b] * sum_{i : a = j} Q[q,i,:]
 * Each output row is written by exactly one thread block (no atomics); for
 * dD every document's argmax entries are grouped by token (a counting sort
 * on chip: the inverse CSR) before the sums.
 *
 *   Q [n_queries, nq, d], D [B, nd, d] (dtype BF16 or FP16), doc_len as in
 *   maxsim_score; argmax [n_queries, B, nq] int32 from maxsim_score
 *   (-1 = empty document); dS [n_queries, B] fp32.
 *   dQ [n_queries, nq, d] fp32 and dD [B, nd, d] fp32 are fully written
 *   (rows no argmax points at are 0).
 *   workspace >= maxsim_backward_workspace_size(...) bytes (see below).
 *
 * Limits: d % 64 == 0, d <= 1024; n_queries * nq <= 65536; the per-document
 * sort must fit in shared memory: about (10 * nd + 2 * n_queries * nq) * 2
 * bytes <= ~227 KB (e.g. nd <= 8192 with n_queries * nq = 16384). FP32 inputs
 * return MAXSIM_ERR_UNSUPPORTED. An argmax entry outside [0, L_b) (or -1 for
 * a non-empty document) is skipped and sets MAXSIM_DEVERR_BAD_INPUT.
 * The inverse CSR lives in shared memory, one document at a time. For
 * B >= 2048 the dQ sweep is split into up to 8 document ranges whose
 * partial sums go to the workspace (maxsim_backward_workspace_size bytes,
 * 16-byte aligned; 0 bytes -- NULL allowed -- for smaller B) and are added
 * in range order, so results do not depend on scheduling. A missing or
 * short workspace returns MAXSIM_ERR_WORKSPACE.
 */
size_t maxsim_backward_workspace_size(int n_queries, int nq, int d, int64_t B, int nd);
maxsim_status maxsim_backward(const void *Q, int n_queries, int nq, int d,
                              const void *D, int64_t B, int nd, const int32_t *doc_len,
                              maxsim_dtype dtype, const int32_t *argmax, const float *dS,
                              float *dQ, float *dD,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * maxsim_backward_dq -- the dQ half of maxsim_backward alone, for training
 * with a frozen document side (pre-encoded documents: no dD is wanted).
 * Same formula, arguments, limits, workspace and errors as maxsim_backward,
 * without Q (dQ does not depend on it) and without dD. Runs the same kernels
 * as the dQ half of maxsim_backward, so dQ is identical to that call's.
 */
maxsim_status maxsim_backward_dq(int n_queries, int nq, int d,
                                 const void *D, int64_t B, int nd, const int32_t *doc_len,
                                 maxsim_dtype dtype, const int32_t *argmax, const float *dS,
                                 float *dQ, void *workspace, size_t workspace_bytes, void *stream);

/*
 * maxsim_backward_dd -- the dD half of maxsim_backward alone (the inverse-grid
 * CSR and the destination-owned dD rows), for training with a frozen query
 * side. Same formula, arguments, limits and errors as maxsim_backward,
 * without D (dD does not depend on it), dQ and the workspace (dD needs none).
 * dD is identical to that of maxsim_backward.
 */
maxsim_status maxsim_backward_dd(const void *Q, int n_queries, int nq, int d,
                                 int64_t B, int nd, const int32_t *doc_len,
                                 maxsim_dtype dtype, const int32_t *argmax, const float *dS,
                                 float *dD, void *stream);

/*
 * Operators of the token encoder whose embeddings MaxSim scores. They work on
 * the CSR layout of maxsim_score_varlen: T packed tokens, document b owning
 * tokens offsets[b] .. offsets[b+1]-1 (offsets[0] = 0, offsets[B] = T, int64).
 * A padded batch [B, nd] is the same with offsets[b] = b * nd.
 *
 * maxsim_heads is a [T, heads, d] view of device memory with d contiguous
 * elements and any token and head strides (in elements), so that q, k and v may
 * lie side by side in one projection's output. The struct itself is on the
 * host. In a view that is written no two rows may share an element (one of its
 * strides steps over all that the other one reaches, and both are at least d);
 * others return MAXSIM_ERR_INVALID_ARG.
 */
typedef struct maxsim_heads {
    void *data;
    int64_t token_stride;
    int64_t head_stride;
} maxsim_heads;

/*
 * maxsim_rotary_frequencies -- the table of maxsim_rotary, on the HOST (no
 * device call): freq_host[i], i < rot_dim / 2, is the turn of pair i from one
 * position to the next, in units of 2^-64 of a whole turn.
 *   theta_i = base^(-2i / rot_dim) radians, and with a factor s:
 *   NONE    theta_i
 *   LINEAR  theta_i / s (positions are interpolated)
 *   NTK     theta_i with base * s^(rot_dim / (rot_dim - 2))
 *   YARN    theta_i for pairs that turn more than 32 times within
 *           original_length positions, theta_i / s for those that turn less
 *           than once, and between them theta_i (1 - c) + theta_i / s c with c
 *           linear in the pair's number i: 0 at the number (a real one, rounded
 *           down) that turns 32 times, 1 at the one (rounded up) that turns
 *           once. Checkpoints that were extended this way want this ramp; the
 *           one of "YaRN: Efficient Context Window Extension of Large Language
 *           Models", 3.2, is linear in the number of turns instead.
 * *amplitude receives 1, or 0.1 ln s + 1 for YARN (that paper's 3.4).
 * rot_dim even and >= 2 (>= 4 for NTK), base > 1, s >= 1, original_length >= 1
 * for YARN; otherwise MAXSIM_ERR_INVALID_ARG.
 */
typedef enum maxsim_rotary_scaling {
    MAXSIM_ROTARY_NONE = 0,
    MAXSIM_ROTARY_LINEAR = 1,
    MAXSIM_ROTARY_NTK = 2,
    MAXSIM_ROTARY_YARN = 3
} maxsim_rotary_scaling;
maxsim_status maxsim_rotary_frequencies(int rot_dim, double base, maxsim_rotary_scaling scaling,
                                        double factor, int64_t original_length,
                                        uint64_t *freq_host, float *amplitude);

/*
 * maxsim_rotary -- turns pair i of every head of token t by
 * position(t) * freq[i]:
 *   y1 = amplitude * (x1 cos - x2 sin),  y2 = amplitude * (x2 cos + x1 sin)
 * with (x1, x2) = (x[i], x[i + rot_dim/2]), or (x[2i], x[2i+1]) when
 * `interleaved` is not 0. Dimensions rot_dim .. d-1 are copied. `inverse` not
 * 0 turns the other way: the gradient of the call with the same arguments.
 *
 *   x, out     [T, heads, d] views, dtype BF16, FP16 or FP32, aligned to their
 *              elements; out may be x (same strides), and may not overlap it
 *              otherwise
 *   freq       [rot_dim / 2] uint64, device
 *   offsets    [B+1] int64: positions count from each document's start; a
 *              token outside every document, or in one with inconsistent
 *              offsets, has position 0 and sets MAXSIM_DEVERR_BAD_INPUT
 *   positions  [T] int32: positions as given (not with offsets). With neither,
 *              token t has position t.
 *
 * Arithmetic is fp32, rounded once. The angle is made in 64-bit integers from
 * the position, so it is as exact at position 10^6 as at 1.
 * Limits: rot_dim even, 2 <= rot_dim <= d, d <= 4096, T < 2^31, heads <= 65535.
 */
maxsim_status maxsim_rotary(const maxsim_heads *x, int64_t T, int heads, int d, int rot_dim,
                            const uint64_t *freq, const int64_t *offsets, int64_t B,
                            const int32_t *positions, int interleaved, float amplitude, int inverse,
                            maxsim_dtype dtype, const maxsim_heads *out, void *stream);

/*
 * maxsim_attention -- softmax attention within each packed document.
 * With i and j counted within document b, and z over the keys that row i sees:
 *   s_ij = scale * <q_i, k_j>
 *   c_ij = cap * tanh(s_ij / cap) if cap > 0, else s_ij
 *   z_ij = c_ij - slopes[h] * |i - j|   (slopes NULL: 0)
 *   lse_i = ln(sum_j exp z_ij),  out_i = sum_j exp(z_ij - lse_i) v_j
 * Row i sees key j if j < key_len[b] (NULL: the document's length) and
 *   FULL     always
 *   CAUSAL   j <= i
 *   PREFIX   j <= i or j < prefix_len[b]
 * Every token is a row, those at or past key_len[b] too (a query's mask
 * tokens). A row that sees nothing (key_len[b] = 0) has out 0 and lse
 * -infinity.
 * Query head h reads key-value head h / (heads / kv_heads).
 *
 *   q, out     [T, heads, d] views; k, v [T, kv_heads, d] views
 *   lse        [heads, T] fp32, or NULL; maxsim_attention_backward needs it
 *
 * Scores, softmax statistics and sums are fp32 on tensor-core products of the
 * inputs; the weights are rounded to the inputs' type for their product with
 * v. A capped score is within 2^-22 of the cap for caps up to 128, within 2^-20 of
 * itself for greater ones. Keys at or past key_len[b], and other documents, never reach a row, even
 * if they hold NaN or infinity. (A key that is hidden from a row only by the
 * order of tokens has weight 0 there, so its v must be finite.)
 *
 * Limits: dtype BF16 or FP16 (FP32 returns MAXSIM_ERR_UNSUPPORTED); d a
 * multiple of 8, 8 <= d <= 128; heads a multiple of kv_heads, heads <= 65535;
 * T < 2^31 - 256; B < 2^31, and not 0 unless T is; scale, and a cap > 0, from 2^-60 to 2^60; all views 16-byte aligned with strides that are
 * multiples of 8 elements, positive and below 2^39. out may overlap no input.
 * Inconsistent offsets, a key_len outside [0, length] (clamped) or a negative
 * prefix_len (taken as 0) set MAXSIM_DEVERR_BAD_INPUT; a document whose offsets
 * leave [0, T], or with a decrease at its start or end, is skipped. Rows outside every document are not
 * written.
 */
typedef enum maxsim_mask {
    MAXSIM_MASK_FULL = 0,
    MAXSIM_MASK_CAUSAL = 1,
    MAXSIM_MASK_PREFIX = 2
} maxsim_mask;

typedef struct maxsim_attention_spec {
    int64_t T, B;
    int32_t heads, kv_heads, d;
    maxsim_dtype dtype;
    maxsim_mask mask;
    float scale;
    float cap;                  /* <= 0: scores are not capped */
    const int64_t *offsets;     /* [B+1], device */
    const int32_t *key_len;     /* [B], device, or NULL */
    const int32_t *prefix_len;  /* [B], device; PREFIX only */
    const float *slopes;        /* [heads], device, or NULL */
} maxsim_attention_spec;

maxsim_status maxsim_attention(const maxsim_attention_spec *spec, const maxsim_heads *q, const maxsim_heads *k,
                               const maxsim_heads *v, const maxsim_heads *out, float *lse, void *stream);

/*
 * maxsim_attention_backward -- gradients of maxsim_attention, from its out
 * and lse and the gradient dO of out:
 *   dV_j = sum_i p_ij dO_i,  dP_ij = <dO_i, v_j>,  p_ij = exp(z_ij - lse_i)
 *   dS_ij = p_ij (dP_ij - <dO_i, out_i>) (1 - (c_ij / cap)^2) scale
 *   dQ_i = sum_j dS_ij k_j,  dK_j = sum_i dS_ij q_i
 * dK and dV of a key-value head are the sums over its query heads. dQ, dK and
 * dV [T, heads or kv_heads, d] have the inputs' dtype and are written once by
 * the block that owns the row: no atomics, results do not depend on
 * scheduling. Rows that see nothing and hidden keys have gradient 0. Slopes
 * are constants.
 * lse and out have to be those of this call's keys alone: the rounding of
 * <dO_i, out_i> is mended by sum_j p_ij = 1 and sum_j p_ij dP_ij = <dO_i, out_i>,
 * so an lse merged over shards of the keys gives wrong dQ and dK.
 * dO, q, k and v must be finite where a row and a key that only the order of
 * tokens hides from one another lie in one document.
 * Sums are fp32; p and dS are rounded to the inputs' type for their products. In
 * FP16 both are held times a power of two that suits the document's largest dO
 * and v, so that neither small gradients nor long documents lose bits; p_ij
 * (dP_ij - <dO_i, out_i>) must stay below 65504 in size.
 * Limits as in maxsim_attention, for dO and the gradients too; heads / kv_heads
 * times a document's length below about 10^8 (the block that owns 128 keys walks
 * over that many rows, and waits are bounded by 2 s). workspace: at least
 * maxsim_attention_backward_workspace_size(spec) bytes, 16-byte aligned.
 */
size_t maxsim_attention_backward_workspace_size(const maxsim_attention_spec *spec);
maxsim_status maxsim_attention_backward(const maxsim_attention_spec *spec, const maxsim_heads *dO,
                                        const maxsim_heads *q, const maxsim_heads *k, const maxsim_heads *v,
                                        const maxsim_heads *out, const float *lse, const maxsim_heads *dq,
                                        const maxsim_heads *dk, const maxsim_heads *dv, void *workspace,
                                        size_t workspace_bytes, void *stream);

/*
 * maxsim_clip_grad_norm -- the global 2-norm of many gradient tensors, and
 * their clipping:
 *   norm = sqrt(sum of all squares),  out = grad * min(1, max_norm / (norm + 1e-6))
 * The four arrays are on the HOST and are read before the call returns;
 * grads[i] and outs[i] are device pointers to sizes[i] contiguous elements of
 * dtypes[i] (a maxsim_dtype; types may be mixed), aligned to their elements.
 * outs[i] may be grads[i] (in place), and overlaps no other tensor otherwise. An
 * outs[i] that lies differently from grads[i] against 16-byte boundaries is
 * written element by element (twice the time for a whole encoder's gradients).
 * *norm (device, fp32) receives the norm before clipping. Squares are added in
 * fp32 within a thread's part of a 32 KB chunk and in fp64 beyond, in an order that depends
 * only on the sizes; values whose squares leave fp32's range are added in fp64.
 * A NaN makes norm and all outputs NaN; an infinity makes norm infinite, itself
 * NaN and every finite element 0.
 * workspace: at least maxsim_clip_grad_norm_workspace_size(n_tensors) bytes,
 * 16-byte aligned. n_tensors may be 0 (norm 0).
 */
size_t maxsim_clip_grad_norm_workspace_size(int n_tensors);
maxsim_status maxsim_clip_grad_norm(const void *const *grads, void *const *outs, const int64_t *sizes,
                                    const int32_t *dtypes, int n_tensors, float max_norm, float *norm,
                                    void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* MAXSIM_H_ */
