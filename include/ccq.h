/*
 * ccq.h -- C ABI of the MI355X (gfx950) Curvature-Conditioned Query read step.
 *
 * The method (gist.science summary of arXiv 2606.01294, "不要阅读一切：一种基于曲率条件
 * 的线性注意力查询", §2 "理论推导", "机制" and "集成"):
 *   keys are unit vectors; the running, undecayed key statistics give
 *     mu_t = (1/t) sum_{j<=t} k_j,  Cbar_t = (1/t) sum_{j<=t} k_j k_j^T,
 *     Sigma_t = Cbar_t - mu_t mu_t^T;
 *   the gate is lambda_t = sigmoid(w_lambda . q_t + b_lambda) (one scalar per token and head);
 *   the cleaned query is q_clean = q_t - lambda_t Sigma_t q_t;
 *   the write rule is left as it is, and the read is o_t = S_t q_clean with S_t the
 *   state after token t's write.
 * Write rules (named by the pages, standard definitions):
 *   CCQ_RULE_GLA : S_t = S_{t-1} diag(alpha_t) + v_t k_t^T,  alpha_t = exp(log_alpha_t) per key channel;
 *   CCQ_RULE_GDN : S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T, scalar alpha_t, beta_t.
 *
 * Statistic state.  The pages keep one extra d_k x d_k matrix and one d_k vector per head
 * (summary §2 "机制").  This library stores them as SUMS: C = sum k k^T, ksum = sum k, plus
 * the token count n, and applies 1/n per token.
 *
 * Conventions for every entry point
 *   - All pointers are DEVICE pointers owned by the caller; the library allocates no memory,
 *     keeps no pointer after it returns and holds no global mutable state.  Calls are
 *     reentrant.  The one exception is ccq_fwd_chunked_noalloc, whose workspace is a device
 *     array the library holds (see there).
 *   - Work is enqueued on `hip_stream` (a hipStream_t; NULL = the default stream) without any
 *     host synchronisation.  The caller keeps buffers alive until the stream has passed the
 *     call.
 *   - Every pointer must be 16-byte aligned.  Tensors are dense, row-major, in the shapes
 *     given below.
 *   - Argument errors return a negative ccq_status BEFORE anything is enqueued.  A failed
 *     launch returns CCQ_ERR_LAUNCH.  Faults inside a kernel surface at the caller's next
 *     synchronisation; the library does not hide them.
 *   - Keys must be L2-normalised (unit keys are the precondition of the eigenvalue bound
 *     eig(I - lambda Sigma) in [1 - lambda, 1], 10100.com write-up, section "方法解析"): either
 *     by the caller, or by the library when CCQ_FLAG_NORMALIZE_KEYS is set.
 *   - Supported shapes: d_k == d_v, d in {64, 128} for CCQ_DTYPE_BF16, d == 64 for
 *     CCQ_DTYPE_F32; chunk == 64 (or 0, meaning 64).  Anything else is CCQ_ERR_UNSUPPORTED.
 */
#ifndef CCQ_H_
#define CCQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CCQ_OK = 0,
  CCQ_ERR_INVALID_ARG = -1,  /* null required pointer, non-positive size, bad enum, partial carry */
  CCQ_ERR_UNSUPPORTED = -2,  /* valid request this build has no kernel for (d, dtype, chunk)    */
  CCQ_ERR_MISALIGNED = -3,   /* a pointer is not 16-byte aligned                                 */
  CCQ_ERR_LAUNCH = -4,       /* the HIP runtime refused a launch                                 */
  CCQ_ERR_WORKSPACE = -5     /* workspace missing or smaller than ccq_fwd_workspace_bytes()      */
} ccq_status;

typedef enum { CCQ_RULE_GLA = 0, CCQ_RULE_GDN = 1 } ccq_rule;

/* Storage dtype of q, k, v, log_alpha, beta and o.  The carry is always fp32. */
typedef enum { CCQ_DTYPE_F32 = 0, CCQ_DTYPE_BF16 = 1 } ccq_dtype;

/* Option bits (ccq_fwd_params.flags, ccq_decode_step's flags).
 * CCQ_FLAG_NORMALIZE_KEYS: the library scales every key to unit L2 norm, k / max(|k|, 1e-12)
 * computed in fp32 from the stored key, before any use (statistics, gate, read and write).
 * Without it keys are used as given and must already be unit vectors.
 * CCQ_FLAG_PACKED_COV: the second-moment sum C, which is symmetric, is passed as its upper
 * triangle only: d_k (d_k + 1) / 2 fp32 entries per head, row by row (C[0][0..d_k-1],
 * C[1][1..d_k-1], ..., C[d_k-1][d_k-1]), so entry C[i][j], i <= j, sits at index
 * i d_k - i (i - 1) / 2 + (j - i).  It applies to C0 and C_out of ccq_fwd_chunked and to C
 * of ccq_decode_step, whose per-head stride becomes d_k (d_k + 1) / 2.  The statistics
 * are the extra state the method keeps per head (summary §2 "机制"); the 10100.com
 * write-up's section "代价与边界" names that state's memory as the method's inference cost,
 * and the packed form moves about half of C's bytes in a decode step. */
typedef enum { CCQ_FLAG_NORMALIZE_KEYS = 1, CCQ_FLAG_PACKED_COV = 2 } ccq_flag;

/* Arguments of ccq_fwd_chunked.  Zero-initialise, then fill in. */
typedef struct {
  int32_t rule;   /* ccq_rule  */
  int32_t dtype;  /* ccq_dtype */
  int32_t B, H, T;
  int32_t d_k, d_v;
  int32_t chunk;     /* 64, or 0 for the default (64)                                         */
  int32_t segments;  /* sequence segments per (b, h) chain processed in parallel; 0 = choose  */

  const void *q;         /* [B, H, T, d_k] dtype                                               */
  const void *k;         /* [B, H, T, d_k] dtype, unit rows                                    */
  const void *v;         /* [B, H, T, d_v] dtype                                               */
  const void *log_alpha; /* GLA: [B, H, T, d_k]; GDN: [B, H, T]; dtype; log of the decay       */
  const void *beta;      /* GDN: [B, H, T] dtype in (0, 1); GLA: must be NULL                  */
  const float *w_lambda; /* [H, d_k] fp32 gate weights                                          */
  const float *b_lambda; /* [H] fp32 gate bias (-INFINITY switches the cleaning off exactly)    */

  /* Carry in: all four NULL (start from zeros, n0 = 0) or all four set. */
  const float *S0;       /* [B, H, d_v, d_k]                                                    */
  const float *C0;       /* [B, H, d_k, d_k]  sum of k k^T  ([B, H, d_k (d_k+1)/2] packed)      */
  const float *ksum0;    /* [B, H, d_k]       sum of k                                          */
  const int64_t *n0;     /* [B, H]            token count                                       */

  void *o;               /* [B, H, T, d_v] dtype, written                                       */

  /* Carry out: all four NULL (not wanted) or all four set.  May alias or overlap the carry in:
   * with more than one segment the call then first copies the carry in (and n0) into the
   * workspace, which ccq_fwd_workspace_bytes always leaves room for, and reads only the copy. */
  float *S_out;
  float *C_out;          /* same layout as C0                                                    */
  float *ksum_out;
  int64_t *n_out;

  void *workspace;        /* device scratch of at least ccq_fwd_workspace_bytes(p) bytes, or  */
  size_t workspace_bytes; /* NULL / 0 when that function returns 0                            */

  /* Optional per-kernel timing: NULL, or an array of 4 caller-created hipEvent_t that are
   * recorded on hip_stream before the segment-summary kernel, after it, after the carry scan
   * and after the main kernel.  With one segment the first three are recorded together,
   * just before the main kernel.  A failed record returns CCQ_ERR_LAUNCH. */
  void *const *phase_events;

  int32_t flags;          /* ccq_flag bits; unknown bits are CCQ_ERR_INVALID_ARG            */

  /* Optional (training): NULL, or ccq_chunk_carry_bytes(dtype, B, H, T, d_k) bytes of device
   * memory that receive the carry at the start of every 64-token chunk c of every chain
   * i = b H + h, for a later ccq_bwd_chunked of the same inputs (its chunk_carry): S_c then C_c,
   * each [d][d] row-major in dtype, at element offset (i NC + c) 2 d^2 (NC = ceil(T / 64); C full,
   * whatever the flags say about the carry in and out), followed by the key sums m_c, [d] fp32
   * each, at float offset (i NC + c) d of the region after all of them.  The chunk carries are
   * those of the keys as used (normalised in the kernel if the flag asks for it).  16-byte
   * aligned (else CCQ_ERR_MISALIGNED). */
  void *chunk_carry;
} ccq_fwd_params;

/* Bytes of the chunk-carry buffer of ccq_fwd_params.chunk_carry / ccq_bwd_params.chunk_carry for
 * these sizes (0 for an unsupported dtype, non-positive sizes or d_k != d_v shapes the chunked
 * calls reject): B H ceil(T / 64) (2 d^2 sizeof(dtype) + 4 d). */
size_t ccq_chunk_carry_bytes(int32_t dtype, int32_t B, int32_t H, int32_t T, int32_t d);

/*
 * Chunked prefill of one CCQ layer: o for every token and, optionally, the final carry.
 * The result is the per-token recurrence above evaluated exactly (up to rounding) with
 * chunks of 64 tokens; the statistics are carried chunk by chunk exactly as the backbone's
 * state is (summary §2 "机制").  A call with a carry in continues the sequence
 * the carry came from.  T need not be a multiple of 64.
 * Precondition (GLA): the call cuts its T tokens into chunks of 64 counted from its own first
 * token (tokens 64c .. 64c + 63).  Within every chunk the decay is factored with the chunk's
 * start as reference, so for every key channel the sum of log_alpha over a whole chunk
 * (equivalently, since log_alpha <= 0, from the chunk's first token to any later token of it)
 * must stay above -80: an average log decay above -1.25 per token (alpha > 0.29).  Beyond it
 * e^{-B} overflows in fp32 and o and the carry are not finite; nothing checks this.
 * Gated DeltaNet has no such limit.  Returns a ccq_status.
 */
int ccq_fwd_chunked(const ccq_fwd_params *p, void *hip_stream);

/* Bytes of device workspace ccq_fwd_chunked needs for these arguments (0 if none).  Depends
 * only on rule, dtype, B, H, T, d_k, d_v, chunk and segments.  Returns 0 for invalid p too. */
size_t ccq_fwd_workspace_bytes(const ccq_fwd_params *p);

/* Size of the device array ccq_fwd_chunked_noalloc takes its workspace from: 64 MiB. */
#define CCQ_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * ccq_fwd_chunked for callers that cannot allocate device memory: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.  It computes exactly what
 * ccq_fwd_chunked computes, with the same kernels, but calls no allocating routine and takes no
 * workspace: p->workspace and p->workspace_bytes are ignored, and the workspace is a
 * CCQ_NOALLOC_SCRATCH_BYTES device array inside the library.  Each device the library runs on
 * holds its own copy of that array from the first such call on it until the process ends.
 * Segments: with p->segments == 0 the library's own choice, made longer (fewer per chain) until
 * its workspace fits the array; a p->segments whose workspace (ccq_fwd_workspace_bytes) exceeds
 * CCQ_NOALLOC_SCRATCH_BYTES returns CCQ_ERR_WORKSPACE before anything is enqueued.  Every call
 * on a device shares that device's array and leaves its contents behind (no call needs it to
 * start at zero): calls that can overlap on one device -- on different streams, or from
 * different threads -- race on it and must be serialised by the caller.  The first call on a
 * device looks the array up (hipGetSymbolAddress) with that device current; a failed lookup
 * returns CCQ_ERR_LAUNCH.  Other arguments, errors and semantics as ccq_fwd_chunked.
 */
int ccq_fwd_chunked_noalloc(const ccq_fwd_params *p, void *hip_stream);

/*
 * One decode step for N sequences x H heads, state updated in place:
 *   n += 1; C += k k^T; ksum += k; Sigma q = C q / n - ksum (ksum . q) / n^2;
 *   q_clean = q - lambda Sigma q; write rule; o = S q_clean.
 * q, k: [N, H, d_k] dtype; v: [N, H, d_v] dtype; log_alpha: GLA [N, H, d_k] / GDN [N, H];
 * beta: GDN [N, H] (GLA: NULL); w_lambda [H, d_k], b_lambda [H] fp32;
 * S [N, H, d_v, d_k], C [N, H, d_k, d_k] (with CCQ_FLAG_PACKED_COV: [N, H, d_k (d_k+1)/2]),
 * ksum [N, H, d_k] fp32 and n [N, H] int64 are read and written in place; o [N, H, d_v]
 * dtype is written.  flags: ccq_flag bits; unknown bits are CCQ_ERR_INVALID_ARG.
 * Returns a ccq_status.
 */
int ccq_decode_step(int32_t rule, int32_t dtype, int32_t N, int32_t H, int32_t d_k, int32_t d_v,
                    const void *q, const void *k, const void *v, const void *log_alpha,
                    const void *beta, const float *w_lambda, const float *b_lambda, float *S,
                    float *C, float *ksum, int64_t *n, void *o, int32_t flags, void *hip_stream);

/*
 * Key-covariance subspace diagnostic (the geometric check of the 10100.com write-up, section
 * "记忆体检": Δμ, how much less needle keys than distractor keys align with the top-16
 * eigen-subspace of the key covariance; negative means the needle lies off the high-variance
 * directions).  Per (b, h):
 *   Sigma = C / n - mu mu^T with mu = ksum / n (the statistics of the read step; C, ksum, n as
 *           carried by ccq_fwd_chunked / ccq_decode_step; n <= 0 gives Sigma = 0),
 *   eigvals [B, H, d_k]    : the eigenvalues of Sigma, descending,
 *   basis   [B, H, r, d_k] : the top-r unit eigenvectors as rows, each with its largest-
 *                            magnitude entry positive (the lowest index among equal ones),
 *   align   [B, H, T]      : a_t = |basis k_t|^2 / |k_t|^2 for every key k_t of k
 *                            ([B, H, T, d_k] dtype; a_t = 0 for a zero key),
 *   delta_mu [B, H]        : mean a_t over tokens with needle[b][h][t] != 0 minus the mean over
 *                            the others (NaN when either set is empty); needle [B, H, T] uint8,
 *   iters   [B, H] int32   : bisection work of the head: the multisection rounds of its d_k
 *                            eigenvalues, summed (0 for Sigma = 0; optional, may be NULL).
 * needle and delta_mu are both NULL (no Δμ) or both set; iters may be NULL; every other
 * pointer is required.
 * flags: CCQ_FLAG_PACKED_COV (C packed as for the other entry points); other bits are
 * CCQ_ERR_INVALID_ARG.  1 <= r <= min(32, d_k); d_k in {64, 128}; B * H <= 65535; dtype as for
 * the other entry points.  The eigen-decomposition runs in fp32: Householder tridiagonalisation,
 * bisection on Sturm counts for the eigenvalues (to about 1e-6 of the largest), inverse
 * iteration with Gram-Schmidt for the eigenvectors (orthonormal to about 1e-6); the subspace, and with it a_t, is well defined when eigenvalue r
 * exceeds eigenvalue r + 1.  Returns a ccq_status.
 */
int ccq_key_subspace(int32_t dtype, int32_t B, int32_t H, int32_t T, int32_t d_k, int32_t r,
                     const float *C, const float *ksum, const int64_t *n, const void *k,
                     const uint8_t *needle, float *eigvals, float *basis, float *align,
                     float *delta_mu, int32_t *iters, int32_t flags, void *hip_stream);

/*
 * Backward of one step of the recurrence (the adjoint of ccq_decode_step), for training: the
 * pages train CCQ models from scratch (10100.com write-up, section "方法解析" point 3).  For N
 * sequences x H heads, given the carry BEFORE the step (S, C, ksum, n: as ccq_decode_step reads
 * them, full-matrix C), the token (q, k, v, log_alpha, beta), the gate parameters, the output
 * gradient d_o [N, H, d_v] fp32 and the adjoint of the carry AFTER the step (dS [N, H, d_v, d_k],
 * dC [N, H, d_k, d_k], dksum [N, H, d_k], fp32; zeros after the last token), it
 *   - overwrites dS, dC, dksum in place with the adjoint of the carry BEFORE the step (dC is
 *     the adjoint of C as a general matrix; only its symmetric part acts on keys),
 *   - writes the fp32 gradients dq, dk [N, H, d_k], dv [N, H, d_v], dlog_alpha (GLA [N, H, d_k],
 *     GDN [N, H]), dbeta (GDN [N, H]; GLA: NULL), and per-sequence gate-parameter gradients
 *     dw_lambda [N, H, d_k] and db_lambda [N, H] (the gradient of the shared [H, d_k] / [H]
 *     parameters is their sum over sequences and steps).
 * Running it over the tokens of a sequence in reverse order, each time from that token's carry
 * before the step, gives the gradients of the whole recurrence (backpropagation through time).
 * Inputs are used as given (flags must be 0: no in-kernel key normalisation, full C).
 * d_k == d_v == 128; dtype is that of q, k, v, log_alpha, beta.  Returns a ccq_status.
 */
int ccq_step_backward(int32_t rule, int32_t dtype, int32_t N, int32_t H, int32_t d_k, int32_t d_v,
                      const void *q, const void *k, const void *v, const void *log_alpha,
                      const void *beta, const float *w_lambda, const float *b_lambda,
                      const float *S, const float *C, const float *ksum, const int64_t *n,
                      const float *d_o, float *dS, float *dC, float *dksum, float *dq, float *dk,
                      float *dv, float *dlog_alpha, float *dbeta, float *dw_lambda,
                      float *db_lambda, int32_t flags, void *hip_stream);

/* Static description of a status code (never NULL). */
const char *ccq_status_string(int32_t status);

/* ABI version of this header: 11. */
int32_t ccq_abi_version(void);

/* Arguments of ccq_bwd_chunked.  Zero-initialise, then fill in. */
typedef struct {
  int32_t rule;   /* ccq_rule: CCQ_RULE_GLA or CCQ_RULE_GDN                                      */
  int32_t dtype;  /* ccq_dtype of q, k, v, log_alpha and d_o                                       */
  int32_t B, H, T;
  int32_t d_k, d_v;
  int32_t chunk;  /* 64, or 0 for the default (64)                                                 */

  /* The forward's inputs, exactly as given to ccq_fwd_chunked (unit keys, no flags); log_alpha is
   * [B, H, T, d_k] for GLA and [B, H, T] for Gated DeltaNet (whose beta comes at the end). */
  const void *q, *k, *v, *log_alpha; /* [B, H, T, d] dtype                                         */
  const float *w_lambda;             /* [H, d_k]                                                    */
  const float *b_lambda;             /* [H]                                                         */
  const float *S0, *C0, *ksum0;      /* carry in: all four NULL (zeros) or all four set (full C)    */
  const int64_t *n0;

  const void *d_o;                   /* [B, H, T, d_v] dtype: gradient of the loss w.r.t. o          */
  /* Adjoint of the carry out (gradient of the loss w.r.t. S_T, C_T, ksum_T): all NULL (zero) or
   * all set; [B, H, d_v, d_k], [B, H, d_k, d_k] (as a general matrix), [B, H, d_k] fp32. */
  const float *dS_T, *dC_T, *dksum_T;

  /* Gradients, fp32, written: */
  float *dq, *dk;        /* [B, H, T, d_k]                                                          */
  float *dv;             /* [B, H, T, d_v]                                                          */
  float *dlog_alpha;     /* [B, H, T, d_k] (GLA) or [B, H, T] (Gated DeltaNet)                      */
  float *dw_lambda;      /* [B, H, d_k] per sequence: the [H, d_k] parameter's gradient is their sum */
  float *db_lambda;      /* [B, H]      per sequence                                                */
  float *dS0, *dC0, *dksum0; /* adjoint of the carry in: all NULL (not wanted) or all set          */

  void *workspace;        /* at least ccq_bwd_workspace_bytes(p) bytes of device memory             */
  size_t workspace_bytes;
  /* Optional per-pass timing: NULL, or 5 caller-created hipEvent_t recorded before the chunk
   * carries, after them, after pass A, after the reverse scan and after pass B. */
  void *const *phase_events;
  int32_t flags;          /* must be 0                                                               */
  /* Gated DeltaNet only (both NULL for GLA): the forward's beta [B, H, T] (dtype) and its
   * gradient dbeta [B, H, T] (fp32, written). */
  const void *beta;
  float *dbeta;
  /* Optional: NULL (the backward recomputes the forward carry at every chunk start), or the
   * chunk_carry buffer a ccq_fwd_chunked call with the same inputs and carry in filled (layout
   * there); the backward then reads the chunk carries from it and skips their recomputation
   * (the segment summary, scan and chunk walk).  Results agree with the recomputing path up to
   * rounding.  16-byte aligned (else CCQ_ERR_MISALIGNED). */
  const void *chunk_carry;
} ccq_bwd_params;

/*
 * Chunked backward of ccq_fwd_chunked, on either write rule (training; the pages train CCQ models
 * on both backbones from scratch, 10100.com write-up, section "方法解析" point 3, gist.science
 * summary §4): for the loss
 *   L = <d_o, o> + <dS_T, S_T> + <dC_T, C_T> + <dksum_T, ksum_T>
 * of the forward with the same inputs and carry in, it writes dL/dq, dL/dk, dL/dv,
 * dL/dlog_alpha (and dL/dbeta for Gated DeltaNet), the per-sequence gate-parameter gradients and,
 * when asked for, the adjoint of the carry in.  The forward carry at every 64-token chunk start is
 * recomputed, or read from the forward's chunk_carry when given, and each chunk's gradients follow from it and the
 * adjoint carried back from later chunks: for GLA through the diagonal decay, for Gated DeltaNet
 * through the transpose of each chunk's d_k x d_k state transition.  Results equal
 * backpropagation through the per-token recurrence up to rounding; the forward's precondition on
 * the GLA log decay applies.
 * Supported: d_k == d_v, d in {64, 128} for CCQ_DTYPE_BF16, d == 64 for CCQ_DTYPE_F32,
 * flags == 0; B * H <= 65535; B * H * ceil(T / 64) < 2^31.  beta and dbeta are set for Gated
 * DeltaNet and NULL for GLA (else CCQ_ERR_INVALID_ARG).  Returns a ccq_status.
 */
int ccq_bwd_chunked(const ccq_bwd_params *p, void *hip_stream);

/* Bytes of device workspace ccq_bwd_chunked needs (0 for invalid p).  Depends only on rule,
 * dtype, B, H, T and d_k: per (b, h) and 64-token chunk, the carry and the carried-back adjoints
 * and fp32 [64, d_k] tiles (GLA: also the forward carry update, 0.36 MB per chunk at d_k = 128,
 * bf16; Gated DeltaNet: also the chunk's 64 x 64 triangular inverse, 0.21 MB per chunk), plus for
 * Gated DeltaNet the prefill's segment slots. */
size_t ccq_bwd_workspace_bytes(const ccq_bwd_params *p);

/* ------------------------------------------------------------------------------------------
 * Operators around the read step.  They keep the conventions above (device pointers, nothing
 * allocated, errors before anything is enqueued, 16-byte aligned pointers, work on hip_stream
 * alone), with these differences: where a tensor has strides they are given in elements, the
 * last dimension is always dense, and a stride whose bytes are not a multiple of 16 is
 * CCQ_ERR_MISALIGNED (the logits of ccq_beam_select may start a row anywhere).  Buffers that are
 * written must not overlap any other buffer of the call, except where an entry says so
 * (CCQ_ERR_INVALID_ARG where the library sees it).  A workspace holds nothing between calls, but
 * two calls that can run at the same time need one each: so do two captured graphs that can.
 * ------------------------------------------------------------------------------------------ */

/* Norm of a query or key row x of d entries: y = x r w with the optional weight w and
 *   CCQ_NORM_NONE: r = 1;
 *   CCQ_NORM_RMS : r = 1 / sqrt(mean(x^2) + eps);
 *   CCQ_NORM_L2  : r = 1 / max(|x|, 1e-12), the unit keys the read step asks for (the norm of
 *                  CCQ_FLAG_NORMALIZE_KEYS). */
typedef enum { CCQ_NORM_NONE = 0, CCQ_NORM_RMS = 1, CCQ_NORM_L2 = 2 } ccq_norm;

/* Arguments of ccq_qk_norm_rope.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of q, k, q_out, k_out                                    */
  int32_t B, T, H_q, H_k, d; /* H_k divides H_q if expand_keys; d in {64, 128}; H_q or H_k may be 0 */
  int32_t q_norm, k_norm;    /* ccq_norm                                                           */
  int32_t rot;               /* leading entries of a row that are rotated: 0 .. d, a multiple of 16 */
  int32_t interleaved;       /* 0: entry i turns with entry i + rot / 2; 1: entry 2 i with 2 i + 1  */
  int32_t expand_keys;       /* 1: k_out has H_q heads, head h holding key head h / (H_q / H_k)     */
  float eps;                 /* of CCQ_NORM_RMS, >= 0                                               */
  const void *q;             /* [B, T, H_q, d], strides below; NULL when H_q == 0                   */
  const void *k;             /* [B, T, H_k, d], strides below; NULL when H_k == 0                   */
  int64_t q_stride_b, q_stride_t, q_stride_h; /* >= 0: part of a packed projection, for instance   */
  int64_t k_stride_b, k_stride_t, k_stride_h;
  const int64_t *positions;  /* [B, T], or NULL: token t stands at position0 + t                    */
  int64_t position0;
  const float *inv_freq;     /* [rot / 2] angle per position of every pair; NULL when rot == 0      */
  const float *q_weight;     /* [d] or NULL (ones)                                                  */
  const float *k_weight;     /* [d] or NULL (ones)                                                  */
  void *q_out;               /* [B, H_q, T, d], written; may not be q                               */
  void *k_out;               /* [B, H_k, T, d], or [B, H_q, T, d] with expand_keys, written         */
} ccq_qk_params;

/*
 * Queries and keys of a projection, made ready for the read step in one pass: every head's row is
 * normalised, weighted, rotated by its position (rotary embedding; the angle position * inv_freq
 * is formed and reduced in 64 bits, to within 2^-51 of itself, then turned in 32: positions of
 * 10^8 lose nothing that fp32 holds) and stored head-major as
 * ccq_fwd_chunked ([B, H, T, d]) and ccq_decode_step (T = 1: [N, H, d]) read it.  A rotation keeps
 * lengths, so keys under CCQ_NORM_L2 without a weight are unit keys.  The arithmetic is fp32; the
 * result is rounded once.  Either side may be absent (H_q == 0 or H_k == 0).  A value row is
 * laid out the same way by CCQ_NORM_NONE and rot == 0.  At most 4,096 heads a side and fewer than
 * 2^28 tokens B T at d = 128, 2^29 at d = 64; 2^30 in the gradient (CCQ_ERR_UNSUPPORTED beyond, and
 * for other d or rot).  Returns a ccq_status.
 */
int ccq_qk_norm_rope(const ccq_qk_params *p, void *hip_stream);

/* Arguments of ccq_qk_norm_rope_backward.  Zero-initialise, then fill in. */
typedef struct {
  ccq_qk_params fwd;         /* the forward's arguments; q_out and k_out are not used              */
  const float *dq_out;       /* [B, H_q, T, d] fp32: gradient of q_out, as ccq_bwd_chunked leaves it */
  const float *dk_out;       /* fp32, the shape of k_out                                            */
  void *dq;                  /* [B, T, H_q, d] dtype, strides below, written                        */
  void *dk;                  /* [B, T, H_k, d] dtype, strides below, written: summed over shared heads */
  int64_t dq_stride_b, dq_stride_t, dq_stride_h; /* no two rows may overlap, of dk's either          */
  int64_t dk_stride_b, dk_stride_t, dk_stride_h;
  float *dq_weight;          /* [d] fp32, written (set if and only if q_weight is)                  */
  float *dk_weight;          /* [d] fp32, written (set if and only if k_weight is)                  */
  void *workspace;           /* ccq_qk_backward_workspace_bytes(p) bytes, or NULL when that is 0    */
  size_t workspace_bytes;
} ccq_qk_bwd_params;

/* Gradient of ccq_qk_norm_rope: dq, dk and the weights' gradients, summed over B, T and heads in
 * a fixed order (two calls give the same bits).  Where an L2 norm is at its floor the norm is a
 * constant.  Returns a ccq_status. */
int ccq_qk_norm_rope_backward(const ccq_qk_bwd_params *p, void *hip_stream);
/* Bytes of device workspace that call needs: 0 without weights and for invalid p. */
size_t ccq_qk_backward_workspace_bytes(const ccq_qk_bwd_params *p);

/* Arguments of ccq_scan.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of x, log_alpha and y                                     */
  int32_t B, T, D;           /* D a multiple of 8                                                   */
  int32_t complement;        /* 1: the input is scaled by 1 - alpha                                 */
  const void *x;             /* [B, T, D], strides below                                            */
  const void *log_alpha;     /* [B, T, D], strides below; -INFINITY starts the channel anew          */
  int64_t x_stride_b, x_stride_t;   /* >= 0                                                         */
  int64_t la_stride_b, la_stride_t; /* >= 0                                                         */
  const int32_t *lengths;    /* [B] tokens of each sequence (taken into 0 .. T), or NULL: T each     */
  const float *h0;           /* [B, D] state before the first token, or NULL: zeros                 */
  void *y;                   /* [B, T, D] dtype, written: h_t; rows at t >= length are left as they were */
  float *h_out;              /* [B, D] state after the last token, or NULL; may be h0 itself        */
  float *chunk_carry;        /* NULL, or [B, ceil(T / 64), D] fp32: the state before every 64-token
                                chunk that starts inside the sequence, for ccq_scan_backward         */
  void *workspace;           /* ccq_scan_workspace_bytes(p) bytes, or NULL when that is 0            */
  size_t workspace_bytes;
} ccq_scan_params;

/*
 * Gated linear recurrence, channel by channel:
 *   h_t = alpha_t h_{t-1} + s_t x_t,  alpha_t = exp(log_alpha_t),  s_t = 1 or 1 - alpha_t,  y_t = h_t.
 * The state is fp32 throughout and a call continues where h0 left off, so T = 1 with h_out == h0
 * is the serving step.  Where alpha_t is 0 the old state is dropped, whatever it holds (an
 * infinity or NaN before it does not pass); alpha_t is 0 for log_alpha_t below about -87.  (With
 * the complement scale an infinite input may give NaN instead of itself.)  Gates above 1 are taken
 * as they are, and a state of 0 stays 0 behind any number of them; growth of another state, and of
 * the gradient that reaches a token from behind, is told as long as the product of consecutive
 * gates stays below 2^128.  Rows behind a sequence's length are neither read into a result nor
 * written.  Long sequences are cut along T and the pieces joined in a fixed order: two calls give
 * the same bits.  D <= 2^24, B T <= 2^30, B D < 2^31, and
 * for T > 8 fewer than 2^23 workgroups, which B ceil(T / 64) ceil(D / 128) < 2^23 always keeps to
 * (CCQ_ERR_UNSUPPORTED beyond; the gradient alike).  Returns a ccq_status.
 */
int ccq_scan(const ccq_scan_params *p, void *hip_stream);
/* Bytes of device workspace ccq_scan needs (0 if none and for invalid p): depends on dtype, B, T, D. */
size_t ccq_scan_workspace_bytes(const ccq_scan_params *p);

/* Arguments of ccq_scan_backward.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of x, log_alpha, dy, dx and dlog_alpha                    */
  int32_t B, T, D;
  int32_t complement;
  const void *x, *log_alpha; /* the forward's inputs, strides below                                 */
  const void *dy;            /* [B, T, D] gradient of y, strides below                              */
  int64_t x_stride_b, x_stride_t, la_stride_b, la_stride_t, dy_stride_b, dy_stride_t; /* >= 0        */
  const int32_t *lengths;    /* the forward's                                                       */
  const float *h0;           /* the forward's                                                       */
  const float *dh_out;       /* [B, D] gradient of h_out, or NULL: zeros                            */
  const float *chunk_carry;  /* the forward's, or NULL: recomputed (T <= 64: h0 is all there is)    */
  void *dx, *dlog_alpha;     /* [B, T, D] dtype, written; zeros at t >= length                      */
  float *dh0;                /* [B, D], written, or NULL; may be dh_out itself                      */
  void *workspace;           /* ccq_scan_backward_workspace_bytes(p) bytes, or NULL when that is 0   */
  size_t workspace_bytes;
} ccq_scan_bwd_params;

/* Gradient of ccq_scan: with the adjoint a_t = dy_t + alpha_{t+1} a_{t+1} (dh_out behind the last
 * token), dx_t = s_t a_t, dlog_alpha_t = alpha_t a_t (h_{t-1} - [complement] x_t) and
 * dh0 = alpha_0 a_0.  States and adjoints are fp32; the states come from chunk_carry and the
 * inputs, not from the rounded y.  Where alpha_t is 0 both products are 0.  Returns a
 * ccq_status. */
int ccq_scan_backward(const ccq_scan_bwd_params *p, void *hip_stream);
size_t ccq_scan_backward_workspace_bytes(const ccq_scan_bwd_params *p);

/* Arguments of ccq_beam_select.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of logits                                                 */
  int32_t N, K, V, M;        /* requests, beams of each, vocabulary, picks: K <= 64, M <= min(64, K V),
                                K V < 2^31, K ceil(V / 16384) <= 4096 and N K < 2^24                */
  const void *logits;        /* [N, K, V], a row every logits_stride elements                        */
  int64_t logits_stride;     /* >= V                                                                 */
  const float *scores;       /* [N, K] log-probability of every beam so far                          */
  const uint8_t *finished;   /* [N, K], non-zero: the beam is complete; or NULL: none is             */
  int32_t pad_token;         /* 0 .. V - 1: the one token a finished beam goes on with               */
  int32_t *token, *parent;   /* [N, M] written: the picks' tokens and the beams they continue        */
  float *score;              /* [N, M] written: their scores                                         */
  void *workspace;           /* ccq_beam_select_workspace_bytes(p) bytes                             */
  size_t workspace_bytes;
} ccq_beam_params;

/*
 * One selection step of beam search.  Continuing beam k with token v scores
 *   scores[k] + logits[k][v] - log sum_u exp logits[k][u],
 * and a finished beam goes on with pad_token alone, at its old score (every other token: -inf).
 * For each request the M best of the K V continuations, best first; equal ones in order of beam,
 * then token.  A NaN logit counts as -inf and +inf as the largest finite number; a beam whose
 * score is -inf or NaN, finished or not, has only continuations at -inf, and so has a row of -inf.
 * The normaliser is formed so that scores of different beams compare as they would in 64 bits (its
 * terms near the top in 64 bits, the tail in 32 with sums in 64, all from their distance to the top:
 * masks of any finite size and logits far from zero take nothing from it).  Beside a logit, or at a
 * score, so large that 64 bits no longer tell a beam's other continuations apart, it is not told
 * which of those are picked.  Returns a ccq_status.
 */
int ccq_beam_select(const ccq_beam_params *p, void *hip_stream);
size_t ccq_beam_select_workspace_bytes(const ccq_beam_params *p);

/* Most states of one ccq_beam_reorder. */
#define CCQ_MAX_REORDER_STATES 16

/*
 * Moves carried states to the beams that continue them, in place: for every state s, request i
 * and beam j, row (i K + j) of states[s] becomes what row (i K + parent[i][j]) was.  A row is
 * row_bytes[s] bytes, a multiple of 4: S, C, ksum and n of a decode step with N K sequences, h of
 * ccq_scan, or anything else kept per beam.  parent is [N, K]; a parent outside 0 .. K - 1 leaves
 * its beam as it is.  1 <= K <= 64, N K <= 2^24, rows of at most 2^36 bytes, and N times the pieces
 * of 4,096 bytes that the states' rows make (1,024 bytes where K > 16 or a row is no multiple of 16)
 * below 2^24 (CCQ_ERR_UNSUPPORTED beyond).  1 <= n_states <= CCQ_MAX_REORDER_STATES; states and
 * row_bytes are host arrays, read before the call returns.  Rows that stay are neither read nor
 * written.  Returns a ccq_status.
 */
int ccq_beam_reorder(int32_t n_states, void *const *states, const size_t *row_bytes, int32_t N, int32_t K,
                     const int32_t *parent, void *hip_stream);

/* Arguments of ccq_linear_attn.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of q, k, v and o                                          */
  int32_t gate_dtype;        /* ccq_dtype of log_alpha                                              */
  int32_t B, T;              /* sequences, and the most tokens of one                               */
  int32_t H, H_q, H_k, H_v;  /* heads of o; H_q, H_k and H_v divide H: head h reads query head
                                h / (H / H_q), and key and value heads alike                        */
  int32_t d_k, d_v;          /* each 64 or 128                                                      */
  float scale;               /* of the outputs; finite                                              */
  const void *q, *k, *v;     /* [B, T, H_q | H_k | H_v, d_k | d_k | d_v], strides below             */
  int64_t q_stride_b, q_stride_t, q_stride_h; /* >= 0                                               */
  int64_t k_stride_b, k_stride_t, k_stride_h;
  int64_t v_stride_b, v_stride_t, v_stride_h;
  const void *log_alpha;     /* [B, T, H], strides below, any (0: a gate for each head, say), starting anywhere; or NULL: no decay */
  int64_t la_stride_b, la_stride_t, la_stride_h; /* >= 0                                            */
  const int32_t *lengths;    /* [B] tokens of each sequence (taken into 0 .. T), or NULL            */
  const int32_t *offsets;    /* [B + 1], or NULL.  Packed sequences: the tensors have one row for each of
                                `rows` tokens, sequence b those from offsets[b] to offsets[b + 1] - 1 (the
                                first T of them, if there are more), never falling; strides over b are
                                not read.  Not with lengths                                         */
  int64_t rows;              /* with offsets: rows of the packed tensors; else 0                    */
  const float *S0;           /* [B, H, d_v, d_k] state before the first token, or NULL: zeros       */
  void *o;                   /* [B, T, H, d_v] dtype, strides below, written; rows of no token are left as they were */
  int64_t o_stride_b, o_stride_t, o_stride_h; /* no two rows may overlap                            */
  float *S_out;              /* [B, H, d_v, d_k] state after the last token, or NULL; may be S0 itself */
  void *workspace;           /* ccq_linear_attn_workspace_bytes(p) bytes, or NULL when that is 0    */
  size_t workspace_bytes;
} ccq_linear_attn_params;

/*
 * Linear attention with one decay for each head (and token):
 *   S_t = alpha_t S_{t-1} + v_t k_t^T,  alpha_t = exp(log_alpha_t),  o_t = scale S_t q_t,
 * the write rule of the read step with a scalar in the place of the decay per key channel, and no
 * cleaning of the query.  A prompt is worked on in chunks of 64 tokens; T = 1 with S_out == S0 is the
 * serving step.  The state is fp32 throughout.  Where the inputs have 16 bits and T > 8, a chunk's scores
 * and the state are rounded to 16 bits once on the way to o.  Gates are taken as they are, above 1 too, as
 * long as the product of consecutive gates, and S q with the state before a chunk, stay inside the range of
 * fp32; where alpha_t is 0 (below 2^-126, log_alpha_t below about -87.3365) the state before token t is dropped,
 * whatever it holds and whatever entered it.  An input that is infinite or NaN may reach the outputs of all tokens of its 64-token chunk, earlier ones
 * too, and beyond it what the formula says; what stands in rows of no token reaches nothing.
 * Long sequences with few heads are cut along T and the pieces joined in a fixed order: two calls give
 * the same bits.  B H <= 2^20, B T <= 2^30, rows < 2^31, strides over tokens below 2^24
 * (CCQ_ERR_UNSUPPORTED beyond, and for other d).  Returns a ccq_status.
 */
int ccq_linear_attn(const ccq_linear_attn_params *p, void *hip_stream);
/* Bytes of device workspace that call needs (0 if none, so for T = 1, and for invalid p): depends on the sizes alone. */
size_t ccq_linear_attn_workspace_bytes(const ccq_linear_attn_params *p);

/* Arguments of ccq_linear_attn_backward.  Zero-initialise, then fill in. */
typedef struct {
  ccq_linear_attn_params fwd; /* the forward's arguments; o, S_out and its workspace are not used   */
  int32_t grad_dtype;        /* ccq_dtype of dq, dk and dv: CCQ_DTYPE_F32, or that of q             */
  const void *d_o;           /* [B, T, H, d_v] dtype: gradient of o, strides below                  */
  int64_t do_stride_b, do_stride_t, do_stride_h; /* >= 0                                            */
  const float *dS_out;       /* [B, H, d_v, d_k] gradient of S_out, or NULL: zeros                  */
  void *dq, *dk, *dv;        /* grad_dtype, the shapes of q, k and v, strides below, written: summed over
                                the heads that share a row; zeros in rows of no token: at t >= length,
                                before, between and behind packed sequences, past the first T of one */
  int64_t dq_stride_b, dq_stride_t, dq_stride_h; /* no two rows may overlap                         */
  int64_t dk_stride_b, dk_stride_t, dk_stride_h;
  int64_t dv_stride_b, dv_stride_t, dv_stride_h;
  void *dlog_alpha;          /* [B, T, H] (packed: [rows, H]) gate_dtype, dense, written, or NULL: one entry
                                for each token whatever the strides of log_alpha: a gate that tokens
                                share has their sum as its gradient; zeros in rows of no token       */
  float *dS0;                /* [B, H, d_v, d_k], written, or NULL                                  */
  void *workspace;           /* ccq_linear_attn_backward_workspace_bytes(p) bytes                   */
  size_t workspace_bytes;
} ccq_linear_attn_bwd_params;

/* Gradient of ccq_linear_attn.  With the adjoint A_t = scale d_o_t q_t^T + alpha_{t+1} A_{t+1} (dS_out
 * behind the last token): dq_t = scale S_t^T d_o_t, dk_t = A_t^T v_t, dv_t = A_t k_t,
 * dlog_alpha_t = alpha_t <A_t, S_{t-1}>, which is formed as the sum over i >= t of
 * q_i . dq_i - k_i . dk_i, plus <dS_out, S_out>, or, where an alpha behind t is 0, over the tokens before that
 * one alone; 0 where alpha_t is 0.  What is infinite or NaN in a chunk may so reach the dlog_alpha of earlier
 * chunks too, as far back as the last alpha of 0 before its chunk.  Sums over shared heads go in a
 * fixed order: two calls give the same bits.  Returns a ccq_status. */
int ccq_linear_attn_backward(const ccq_linear_attn_bwd_params *p, void *hip_stream);
size_t ccq_linear_attn_backward_workspace_bytes(const ccq_linear_attn_bwd_params *p);

/* Activations of ccq_group_norm: x, x sigmoid(x), sigmoid(x). */
typedef enum { CCQ_ACT_NONE = 0, CCQ_ACT_SILU = 1, CCQ_ACT_SIGMOID = 2 } ccq_activation;

/* Arguments of ccq_group_norm.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of x, gate and y                                          */
  int32_t B, T, G, d;        /* G groups of d channels a token; d a multiple of 8, at most 1024      */
  int32_t center;            /* 1: the group's mean is taken off first; 0: mean square alone        */
  int32_t activation;        /* ccq_activation                                                      */
  int32_t affine_shared;     /* 1: weight and bias are [d], the same for every group; 0: [G, d]     */
  float eps;                 /* >= 0                                                                */
  const void *x;             /* [B, T, G, d], strides below                                         */
  const void *gate;          /* [B, T, G, d], strides below, or NULL                                */
  int64_t x_stride_b, x_stride_t, x_stride_h;          /* >= 0: over sequences, tokens, groups      */
  int64_t gate_stride_b, gate_stride_t, gate_stride_h; /* >= 0                                      */
  const float *weight;       /* or NULL (ones)                                                      */
  const float *bias;         /* or NULL (zeros)                                                     */
  void *y;                   /* [B, T, G, d] dtype, strides below, written; may be x or gate itself */
  int64_t y_stride_b, y_stride_t, y_stride_h;          /* no two rows may overlap                   */
} ccq_group_norm_params;

/*
 * Group norm of every token by itself, channels last, with an activation: with the mean mu (center) and
 * r = 1 / sqrt(mean((x - mu)^2) + eps) of a group's d channels, z = (x - mu) r weight + bias and
 *   y = act(z)        without a gate,
 *   y = z act(gate)   with one.
 * It takes the heads of a linear-attention or read-step output (head-major through its strides) to the
 * output projection (token-major).  The arithmetic is fp32 (a group's sum of squares must stay inside its range);
 * the result is rounded once.  Fewer than 2^31
 * groups B T G, G < 2^16 (CCQ_ERR_UNSUPPORTED beyond, and for other d).  Returns a ccq_status.
 */
int ccq_group_norm(const ccq_group_norm_params *p, void *hip_stream);

/* Arguments of ccq_group_norm_backward.  Zero-initialise, then fill in. */
typedef struct {
  ccq_group_norm_params fwd; /* the forward's arguments; y is not used                              */
  const void *dy;            /* [B, T, G, d] dtype: gradient of y, strides below                    */
  int64_t dy_stride_b, dy_stride_t, dy_stride_h;       /* >= 0                                      */
  void *dx;                  /* [B, T, G, d] dtype, strides below, written; may be dy itself        */
  int64_t dx_stride_b, dx_stride_t, dx_stride_h;       /* no two rows may overlap                   */
  void *dgate;               /* the same for the gate; set if and only if gate is; may be gate itself */
  int64_t dgate_stride_b, dgate_stride_t, dgate_stride_h;
  float *dweight, *dbias;    /* the shapes of weight and bias, written; each set if and only if that is */
  void *workspace;           /* ccq_group_norm_backward_workspace_bytes(p) bytes, or NULL when that is 0 */
  size_t workspace_bytes;
} ccq_group_norm_bwd_params;

/* Gradient of ccq_group_norm; weight and bias are summed over tokens (and groups that share them) in a
 * fixed order: two calls give the same bits.  Returns a ccq_status. */
int ccq_group_norm_backward(const ccq_group_norm_bwd_params *p, void *hip_stream);
size_t ccq_group_norm_backward_workspace_bytes(const ccq_group_norm_bwd_params *p);

/* Arguments of ccq_logits_adjust.  Zero-initialise, then fill in. */
typedef struct {
  int32_t dtype;             /* ccq_dtype of logits and out                                         */
  int32_t R, V;              /* rows (beams of all requests), vocabulary                            */
  int32_t L;                 /* width of history; 0 with history NULL                               */
  int32_t n_bias;            /* width of the bias lists, 0 .. 1024; 0 with them NULL                */
  const void *logits;        /* [R, V], a row every logits_stride elements, anywhere                */
  int64_t logits_stride;     /* >= V                                                                */
  const int32_t *history;    /* [R, L] tokens seen; one outside 0 .. V - 1 counts for nothing       */
  const int32_t *lengths;    /* [R] tokens in each row's history (taken into 0 .. L), or NULL: L     */
  const int32_t *prompt_lengths; /* [R] how many of them, in front, are the prompt's, or NULL: none  */
  float repetition, presence, frequency; /* the penalties of every row whose list below is NULL      */
  const float *repetition_rows, *presence_rows, *frequency_rows; /* [R], or NULL                     */
  const int32_t *bias_token; /* [R, n_bias]; one outside 0 .. V - 1 counts for nothing              */
  const float *bias_value;   /* [R, n_bias]; a token that stands in the list twice gets both         */
  const uint32_t *allowed;   /* [R, ceil(V / 32)]: token v may follow if bit v % 32 of word v / 32 is set;
                                or NULL: all may                                                     */
  void *out;                 /* [R, V] dtype, a row every out_stride elements, written; may be logits itself,
                                with the same stride                                                 */
  int64_t out_stride;        /* >= V                                                                */
} ccq_logits_adjust_params;

/*
 * Logits made ready for a selection (ccq_beam_select) or for sampling.  For token v of a row, which stands
 * c times in the row's history behind the prompt:
 *   x = logits[v];  if v stands in the history, prompt or not: x = x > 0 ? x / repetition : x repetition;
 *   x = x - frequency c - presence [c > 0] + the sum of v's biases, in the list's order;
 *   out[v] = x if v is allowed, else -INFINITY (whatever x is).
 * The arithmetic is fp32; the result is rounded once; a logit that nothing touches stays as it is, a NaN
 * or infinity too.  repetition must be above 0 (a row's own is taken as it stands).  Every pointer needs the
 * alignment of its elements only, so rows of a larger batch can be given as they are.  V <= 2^24, L <= 2^24,
 * R (V / 4096 + 1) < 2^24 (CCQ_ERR_UNSUPPORTED beyond).  Returns a ccq_status.
 */
int ccq_logits_adjust(const ccq_logits_adjust_params *p, void *hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* CCQ_H_ */
