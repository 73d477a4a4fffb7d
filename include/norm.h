/*
 * norm.h -- C ABI of libnorm: row-wise LayerNorm and RMSNorm on one GB300 GPU
 * (sm_103a): forward, fused residual-add + RMSNorm forward, and the training
 * backward with gamma/beta gradients.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Layout.  A "row tensor" is N rows of H elements, row-major, the last
 *   (normalised) dimension contiguous, consecutive rows `ld` ELEMENTS apart
 *   (ld >= H).  A (B, T, H) tensor is passed as N = B*T rows.  gamma, beta,
 *   dgamma and dbeta have shape (H,) and are indexed by column only.  mean and
 *   rstd have shape (N,), fp32.
 * Memory.  Every pointer is CUDA device memory owned by the caller (any
 *   allocator, e.g. PyTorch's).  The library never allocates, frees or keeps a
 *   pointer after the call returns.  Its only device memory is module-scope:
 *   one error word per device (norm_device_errors) and the fixed workspace of
 *   ln_backward_static_workspace.
 * Streams.  Work is enqueued on `stream` (a cudaStream_t; NULL = the legacy
 *   default stream) and runs asynchronously; the call returns once the work is
 *   enqueued.  Outputs are valid after the stream reaches that point.
 * Dtypes.  `x_dtype` types the row tensors (x, residual, y, h_out, dy, dx);
 *   `w_dtype` types gamma, beta, dgamma, dbeta and must equal x_dtype or be
 *   NORM_F32.  All statistics and arithmetic are fp32; stored values are
 *   rounded to nearest, ties to even (an fp16 value past 65504 rounds to
 *   infinity).
 * eps.  Added INSIDE the square root: rstd = 1/sqrt(var + eps).  eps must be
 *   finite and > 0.
 * Alignment.  Rows whose pointers and strides are 16-byte aligned take the
 *   128-bit vector path; half-precision rows that are 32-byte aligned with H
 *   a multiple of 16 take the faster 256-bit paths; anything else is still
 *   correct (scalar path).
 * Errors.  Arguments are validated on the host before anything is enqueued;
 *   an invalid call returns an error and enqueues nothing.  A failed launch
 *   returns NORM_ERR_CUDA.  No entry point aborts, throws or prints.
 * Threads.  Every entry point is thread-safe.  The host-side library state
 *   is a per-device cache of device attributes (filled once, under a lock),
 *   the kernel-family override of norm_set_kernel_path and the timing event
 *   of norm_set_bwd_split_event (one atomic value each for the whole
 *   process).
 *
 * Sources: "Skill: Write a Triton LayerNorm Kernel", "Skill: Write CUDA
 * LayerNorm Kernel", "Skill: Write a Triton Fused Add+RMSNorm Kernel" and the
 * Fast-LLM pull request "Rewrite Triton normalization backward kernel_1
 * (#499)".  Each declaration names the section it implements.
 */
#ifndef NORM_H_
#define NORM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* norm_stream_t; /* same type as cudaStream_t */

typedef enum {
  NORM_OK = 0,
  NORM_ERR_INVALID_VALUE = 1, /* bad size, stride, eps, null or overlapping pointer */
  NORM_ERR_UNSUPPORTED = 2,   /* dtype combination not provided */
  NORM_ERR_WORKSPACE = 3,     /* backward workspace missing, too small or misaligned */
  NORM_ERR_CUDA = 4           /* a CUDA runtime call or kernel launch failed */
} norm_status;

/* fp32, bfloat16 and IEEE binary16 ("Skill: Write a Triton LayerNorm Kernel",
 * Inputs the agent should gather first, item 3: fp16, bf16 or fp32 inputs,
 * statistics accumulated in fp32). */
typedef enum { NORM_F32 = 0, NORM_BF16 = 1, NORM_F16 = 2 } norm_dtype;

/*
 * LayerNorm forward.  "Skill: Write a Triton LayerNorm Kernel", Required
 * reasoning process steps 1-10; "Skill: Write CUDA LayerNorm Kernel", steps
 * 1-7 (Welford statistics with the parallel merge, eps inside rsqrt):
 *   mean = sum_j x_j / H,  var = sum_j (x_j - mean)^2 / H  (biased),
 *   rstd = 1/sqrt(var + eps),  y_j = (x_j - mean) * rstd * gamma_j + beta_j.
 * x     [N x ldx]  input rows.
 * gamma [H] or NULL (= all ones);  beta [H] or NULL (= all zeros).
 * y     [N x ldy]  output rows.  May be exactly x (same pointer and stride) for
 *                  an in-place call; any other overlap with x is rejected.
 * mean, rstd [N] fp32 or NULL: the statistics saved for the backward.
 * N >= 0, H >= 1.  N == 0 enqueues nothing, and then every row and statistics
 * pointer may be NULL.
 */
norm_status ln_forward(const void* x, int64_t ldx, const void* gamma, const void* beta,
                       void* y, int64_t ldy, float* mean, float* rstd,
                       int64_t N, int64_t H, float eps,
                       norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * RMSNorm forward.  "Skill: Write CUDA LayerNorm Kernel", Kernel design rules
 * (RMSNorm); "Skill: Write a Triton LayerNorm Kernel", step 5:
 *   rstd = 1/sqrt(sum_j x_j^2 / H + eps),  y_j = x_j * rstd * gamma_j.
 * No mean subtraction and no beta.  Arguments as in ln_forward; rstd may be
 * NULL.
 */
norm_status rms_forward(const void* x, int64_t ldx, const void* gamma,
                        void* y, int64_t ldy, float* rstd,
                        int64_t N, int64_t H, float eps,
                        norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * Fused residual add + RMSNorm forward.  "Skill: Write a Triton Fused
 * Add+RMSNorm Kernel", Required reasoning process steps 1-9:
 *   h = x + residual formed in fp32;  h_out = h rounded to x_dtype;
 *   rstd = 1/sqrt(sum_j h_j^2 / H + eps);  y_j = h_j * rstd * gamma_j, with y
 *   computed from the fp32 h, not from the rounded h_out.
 * x [N x ldx], residual [N x ldr]: inputs.
 * h_out [N x ldh]: the summed residual stream.  It may be exactly x or exactly
 *   residual (same pointer and stride: in-place update); any other overlap is
 *   rejected.
 * y [N x ldy]: must not overlap x, residual or h_out.
 * rstd [N] fp32 or NULL (saved for training).
 */
norm_status fused_add_rms_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                  const void* gamma, void* y, int64_t ldy,
                                  void* h_out, int64_t ldh, float* rstd,
                                  int64_t N, int64_t H, float eps,
                                  norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * Bytes of device workspace the backward needs for a row width H on CUDA
 * device `device`: the bounded fp32 partial buffer for dgamma/dbeta of
 * "Rewrite Triton normalization backward kernel_1 (#499)", Summary item 2
 * (a fixed number of partial rows tied to the SM count, independent of N).
 * Returns 0 if H < 1 or the device cannot be queried.
 */
size_t norm_bwd_workspace_bytes(int64_t H, int device);

/*
 * LayerNorm backward.  "Skill: Write CUDA LayerNorm Kernel", step 8, with
 * g_j = dy_j * gamma_j and x_hat_j = (x_j - mean) * rstd:
 *   dx_j     = rstd/H * (H*g_j - sum(g) - x_hat_j * sum(g * x_hat)),
 *   dgamma_j = sum over all N rows of dy_j * x_hat_j,
 *   dbeta_j  = sum over all N rows of dy_j.
 * Rows are grid-strided over a CTA count tied to the SM count; each CTA folds
 * its rows into one fp32 partial row in `workspace`, and a second kernel sums
 * the partials and casts once to w_dtype ("Rewrite Triton normalization
 * backward kernel_1 (#499)", Summary items 1-2).
 * dy [N x lddy], x [N x ldx]: inputs.  mean, rstd [N] fp32: the forward's
 *   saved statistics (required).
 * gamma [H] or NULL (= ones).
 * dx [N x lddx]: output; may be exactly dy (in place); must not overlap x.
 * dgamma, dbeta [H] in w_dtype, or NULL to skip that gradient.  They are
 *   overwritten, not accumulated into.  With N == 0 they are set to zero, the
 *   row and statistics pointers may be NULL and no workspace is needed.
 * workspace: device memory of at least norm_bwd_workspace_bytes(H, device)
 *   bytes, 16-byte aligned; needed only when dgamma or dbeta is non-NULL.  Its
 *   contents need no initialisation and are undefined afterwards.  Calls that
 *   share one workspace must be ordered on the GPU (e.g. one stream).
 */
norm_status ln_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                        const float* mean, const float* rstd, const void* gamma,
                        void* dx, int64_t lddx, void* dgamma, void* dbeta,
                        void* workspace, size_t workspace_bytes,
                        int64_t N, int64_t H,
                        norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * RMSNorm backward (derived from the RMSNorm forward; no page prints it):
 * with g_j = dy_j * gamma_j and x_hat_j = x_j * rstd,
 *   dx_j     = rstd * (g_j - x_hat_j * sum(g * x_hat) / H),
 *   dgamma_j = sum over all N rows of dy_j * x_hat_j.
 * Arguments as in ln_backward, without mean and dbeta.
 */
norm_status rms_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const float* rstd, const void* gamma,
                         void* dx, int64_t lddx, void* dgamma,
                         void* workspace, size_t workspace_bytes,
                         int64_t N, int64_t H,
                         norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * ln_backward for callers that cannot allocate device memory when they call
 * it -- for example a plugin inside a framework that owns all device memory
 * and gives plugins no allocator, or latency-critical code that must not pay
 * for cudaMalloc mid-step.  (The pages have no counterpart: this is an
 * interface convenience, not part of the method.)
 *
 * Same arguments and results as ln_backward, without the workspace: the
 * dgamma/dbeta partial rows go to a scratch array of
 * NORM_STATIC_WORKSPACE_BYTES (64 MiB) compiled into the library, one copy per
 * GPU that loads it, held until the process exits.  Nothing is allocated.
 * - Widths whose partial rows need more than that (when dgamma or dbeta is
 *   requested: norm_bwd_workspace_bytes(H, device) > the limit; H up to about
 *   27000 on a 152-SM GPU), or that the device cannot be asked to size, are
 *   refused with NORM_ERR_WORKSPACE.
 * - Every call looks up the current device's copy of the array
 *   (cudaGetSymbolAddress, a host-side lookup).  Under lazy module loading
 *   (CUDA's default) the 64 MiB are reserved when the library's device code
 *   is first used on a device, which may be this call: make one set-up call
 *   (N == 0 is enough) before any stream capture and before a framework takes
 *   the device's memory.  If that reservation fails the call returns
 *   NORM_ERR_CUDA and norm_last_error() names the failed step.
 * - Every call on a device shares the one array, which keeps the last call's
 *   contents; no part of it needs clearing, as each call writes every partial
 *   value before reading it.  Calls whose GPU work overlaps (other streams,
 *   other host threads) race on the array and must be ordered, e.g. on one
 *   stream.
 */
#define NORM_STATIC_WORKSPACE_BYTES ((size_t)64 << 20)
norm_status ln_backward_static_workspace(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                                         const float* mean, const float* rstd, const void* gamma,
                                         void* dx, int64_t lddx, void* dgamma, void* dbeta,
                                         int64_t N, int64_t H,
                                         norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * LayerNorm backward from the forward's saved output instead of x.
 * "Rewrite Triton normalization backward kernel_1 (#499)", Benchmark harness:
 * the backward reads the output the forward saved.  x_hat is recovered as
 * (y - beta) / gamma and the formulas of ln_backward run on it with the saved
 * rstd ("Skill: Write CUDA LayerNorm Kernel", Required reasoning process
 * step 8).  x and mean are not needed.
 * y [N x ldy]: the forward's output (ln_forward's y, same gamma and beta).
 * rstd [N] fp32: the forward's saved rstd.  gamma, beta [H] or NULL (ones,
 *   zeros).  A column whose gamma is 0 holds no trace of x_hat: its dx and
 *   dgamma come out non-finite (IEEE division by zero); nothing is checked.
 * dx, dgamma, dbeta, workspace: as ln_backward; dx may be exactly dy and must
 *   not overlap y.  x_hat recovered from a rounded y carries that rounding
 *   (2^-9 relative for bf16, 2^-11 for fp16) into dx and dgamma.
 */
norm_status ln_backward_from_output(const void* dy, int64_t lddy, const void* y, int64_t ldy, const float* rstd,
                                    const void* gamma, const void* beta, void* dx, int64_t lddx, void* dgamma,
                                    void* dbeta, void* workspace, size_t workspace_bytes, int64_t N, int64_t H,
                                    norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * RMSNorm backward from the saved output: x_hat = y / gamma, then the
 * formulas of rms_backward with the saved rstd.  Arguments as
 * ln_backward_from_output without beta/dbeta.
 */
norm_status rms_backward_from_output(const void* dy, int64_t lddy, const void* y, int64_t ldy, const float* rstd,
                                     const void* gamma, void* dx, int64_t lddx, void* dgamma, void* workspace,
                                     size_t workspace_bytes, int64_t N, int64_t H, norm_dtype x_dtype,
                                     norm_dtype w_dtype, norm_stream_t stream);

/*
 * Fused residual add + RMSNorm backward.  "Skill: Write a Triton Fused
 * Add+RMSNorm Kernel", Required reasoning process steps 9-10: the backward
 * reads the stored sum h and rstd; the RMSNorm gradient with respect to h,
 *   dL/dh_j = rstd * (g_j - h_hat_j * sum(g * h_hat) / H) + dh_in_j,
 *   with g = dy * gamma and h_hat = h * rstd,
 * is the gradient of both inputs (dh/dx = dh/dresidual = 1).  dh_in is the
 * gradient arriving through the stored h itself (the residual stream's later
 * consumers), added in the same pass, or NULL.  dgamma_j = sum over rows of
 * dy_j * h_hat_j.
 * dy [N x lddy], h [N x ldh] (the forward's h_out), rstd [N] fp32, gamma [H]
 *   or NULL.
 * dx [N x lddx]: dL/dh for x.  May be exactly dy or dh_in (in place); must
 *   not overlap h.
 * dres [N x lddres]: dL/dh again, for the residual input; NULL to write dx
 *   only; exactly dx when x and residual were one tensor, which then
 *   receives the sum 2 * dL/dh.
 * dgamma [H] or NULL; workspace as in rms_backward.
 */
norm_status fused_add_rms_backward(const void* dy, int64_t lddy, const void* h, int64_t ldh,
                                   const float* rstd, const void* gamma,
                                   const void* dh_in, int64_t lddh_in,
                                   void* dx, int64_t lddx, void* dres, int64_t lddres, void* dgamma,
                                   void* workspace, size_t workspace_bytes, int64_t N, int64_t H,
                                   norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * Block join forward: the RMSNorm after a block, its gate, the scaled residual
 * add and the RMSNorm before the next block, in one pass.  (An extension of
 * fused_add_rms_forward; the pages have no counterpart.)
 *   p = x * rstd_post * gamma_post   (NORM_SANDWICH_POST; else p = x),
 *   h = residual_scale * residual + gate * p   formed in fp32; h_out = h
 *       rounded to x_dtype,
 *   y = h * rstd_pre * gamma_pre     (NORM_SANDWICH_PRE), from the fp32 h,
 *   rstd = 1/sqrt(sum_j v_j^2 / H + eps) of x's and of h's rows.
 * x [N x ldx], residual [N x ldr]: inputs.
 * gamma_post, gamma_pre [H] or NULL (ones).
 * gate [gate_rows x ldgate] in gate_dtype (x_dtype or NORM_F32) or NULL (ones):
 *   gate_rows divides N, and gate row k serves rows k*N/gate_rows up to
 *   (k+1)*N/gate_rows (1: one vector for all rows; B: one for each sequence of
 *   a (B, T, H) tensor).
 * h_out [N x ldh]: may be exactly x or exactly residual; any other overlap is
 *   rejected.  y [N x ldy]: must not overlap x, residual or h_out.
 * rstd_post, rstd_pre [N] fp32 or NULL (saved for sandwich_rms_grad).
 * norms: NORM_SANDWICH_POST, NORM_SANDWICH_PRE or both.  The gamma, statistic
 *   and output of a norm that is not taken must be NULL.
 * residual_scale must be finite.
 */
#define NORM_SANDWICH_POST 1u
#define NORM_SANDWICH_PRE 2u
#define NORM_SANDWICH_BOTH 3u
norm_status sandwich_rms(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                         const void* gamma_post, const void* gate, int64_t ldgate, int64_t gate_rows,
                         const void* gamma_pre, void* y, int64_t ldy, void* h_out, int64_t ldh,
                         float* rstd_post, float* rstd_pre, int64_t N, int64_t H, float eps,
                         float residual_scale, unsigned norms, norm_dtype x_dtype, norm_dtype w_dtype,
                         norm_dtype gate_dtype, norm_stream_t stream);

/*
 * Bytes of device workspace sandwich_rms_grad needs for a row width H and a
 * number of gate rows (0 without a gate) on CUDA device `device`; independent
 * of N and, past one, of the number of gate rows.  Returns 0 if an argument is
 * out of range or the device cannot be queried.
 */
size_t sandwich_rms_workspace_bytes(int64_t H, int64_t gate_rows, int device);

/*
 * Gradient of sandwich_rms, from the stored h and the saved statistics.  With
 * h_hat = h * rstd_pre, o_hat = x * rstd_post (x without the norm after the
 * block), g = dy * gamma_pre:
 *   dh   = dh_in + rstd_pre * (g - h_hat * sum(g * h_hat) / H),
 *   dres = residual_scale * dh,
 *   dp   = gate * dh,  q = dp * gamma_post,
 *   dx   = rstd_post * (q - o_hat * sum(q * o_hat) / H)   (dx = dp without it),
 *   dgamma_pre  = sum over rows of dy * h_hat,
 *   dgamma_post = sum over rows of dp * o_hat,
 *   dgate[k]    = sum over gate row k's rows of dh * o_hat * gamma_post.
 * dy [N x lddy] (NULL without NORM_SANDWICH_PRE, as h, gamma_pre, rstd_pre and
 *   dgamma_pre), dh_in [N x lddh_in] or NULL (zeros; required when dy is NULL):
 *   the gradient that arrives through the stored h.
 * dx [N x lddx]: may be exactly dy.  dres [N x lddres]: may be exactly dh_in.
 *   Otherwise neither overlaps an input or the other.
 * dgamma_post, dgamma_pre [H] in w_dtype, dgate [gate_rows x lddgate] in
 *   gate_dtype, or NULL to skip.  Overwritten, not accumulated into; zero with
 *   N == 0.
 * workspace: sandwich_rms_workspace_bytes(H, gate_rows, device) bytes, 16-byte
 *   aligned; needed only when a parameter gradient is.  As in ln_backward, calls
 *   that share it must be ordered.
 * Sums have a fixed order: the same inputs give the same bits.
 */
norm_status sandwich_rms_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* h, int64_t ldh,
                              const float* rstd_post, const float* rstd_pre, const void* gamma_post,
                              const void* gate, int64_t ldgate, int64_t gate_rows, const void* gamma_pre,
                              const void* dh_in, int64_t lddh_in, void* dx, int64_t lddx, void* dres,
                              int64_t lddres, void* dgamma_post, void* dgate, int64_t lddgate, void* dgamma_pre,
                              void* workspace, size_t workspace_bytes, int64_t N, int64_t H, float residual_scale,
                              unsigned norms, norm_dtype x_dtype, norm_dtype w_dtype, norm_dtype gate_dtype,
                              norm_stream_t stream);

/* Type of token ids. */
typedef enum { NORM_I32 = 0, NORM_I64 = 1 } norm_itype;

/*
 * Token lookup: the rows that start a residual stream.  (No counterpart on the
 * pages; embedding_rms is to the first block what fused_add_rms_forward is to
 * the others.)
 *   h_i = scale * table[tokens_i], formed in fp32, rounded to the row dtype;
 *   embedding_rms also y_i = h_i * rstd_i * gamma from the fp32 h_i, with
 *   rstd_i = 1/sqrt(sum_j h_ij^2 / H + eps).
 * table [V x ldt] in the row dtype.  tokens [N], contiguous, of token_type.
 * h [N x ldh], y [N x ldy]: outputs, clear of the inputs and of each other.
 * gamma [H] or NULL (ones).  rstd [N] fp32 or NULL.
 * A token outside [0, V) gives a row of zeros and raises
 * NORM_DEVICE_ERR_BAD_TOKEN.  V and N are at most 2^31 - 2; scale is finite.
 */
norm_status embedding_lookup(const void* table, int64_t ldt, int64_t V, const void* tokens, norm_itype token_type,
                             void* h, int64_t ldh, int64_t N, int64_t H, float scale, norm_dtype dtype,
                             norm_stream_t stream);
norm_status embedding_rms(const void* table, int64_t ldt, int64_t V, const void* tokens, norm_itype token_type,
                          const void* gamma, void* y, int64_t ldy, void* h, int64_t ldh, float* rstd, int64_t N,
                          int64_t H, float eps, float scale, norm_dtype x_dtype, norm_dtype w_dtype,
                          norm_stream_t stream);

/*
 * Bytes of device workspace embedding_grad needs for up to N tokens of H columns
 * (never fewer for more tokens).  Returns 0 if an argument is out of range.
 */
size_t embedding_grad_workspace_bytes(int64_t N, int64_t H);

/*
 * Gradient of the table: dtable[v] = scale * sum of dh_i over the tokens equal
 * to v, in fp32, rounded once; with accumulate != 0 it is added to what dtable
 * holds (only the rows of tokens that occur are then touched), else rows no
 * token names are set to zero.  The tokens are sorted by id (stably, on the
 * GPU), so the sums have a fixed order: the same inputs give the same bits.
 * dh [N x lddh]: the gradient of h.  dtable [V x lddt] in w_dtype (the row
 *   dtype or NORM_F32), clear of the inputs.
 * padding_idx: a token that has no gradient, or -1.  Tokens outside [0, V) are
 *   left out and raise NORM_DEVICE_ERR_BAD_TOKEN.
 * workspace: embedding_grad_workspace_bytes(N, H) bytes (or those of a larger
 *   N), 16-byte aligned; calls that share it must be ordered.
 */
norm_status embedding_grad(const void* dh, int64_t lddh, const void* tokens, norm_itype token_type, void* dtable,
                           int64_t lddt, int64_t V, void* workspace, size_t workspace_bytes, int64_t N, int64_t H,
                           float scale, int64_t padding_idx, int accumulate, norm_dtype x_dtype, norm_dtype w_dtype,
                           norm_stream_t stream);

/*
 * Heads of a projection: a (B, T, H, D) tensor of D contiguous columns a head,
 * by its strides in elements (none negative; that of a dim of one is not
 * looked at).  (B, T, H, D) and (B, H, T, D) layouts, and the queries' or keys'
 * part of a fused projection's output, are such.
 */
typedef struct {
  void* data;
  int64_t batch_stride, token_stride, head_stride;
} norm_heads;

/*
 * Rotation by position.  cos, sin [rows x cos_stride / sin_stride] of columns/2
 * elements in `dtype` (the row dtype or NORM_F32): the angles of position p are
 * in row p.  columns: how many of a head's first columns are rotated, even.
 * Pair i of them is columns (i, i + columns/2), or with interleaved != 0 columns
 * (2i, 2i + 1).  positions: one for each token, by its strides (0: shared), or
 * NULL: token t of each sequence has position t, and T is at most `rows`.
 */
typedef struct {
  const void* cos;
  int64_t cos_stride;
  const void* sin;
  int64_t sin_stride;
  int64_t rows, columns;
  norm_dtype dtype;
  int interleaved;
  const void* positions;
  norm_itype position_type;
  int64_t position_batch_stride, position_token_stride;
} norm_rotation;

/*
 * RMSNorm of each head of queries and keys, and the rotation by their tokens'
 * positions, in one pass (the norm inside an attention block).  For each head x:
 *   n = x * rstd * gamma,  rstd = 1/sqrt(sum_j x_j^2 / D + eps),
 *   y_a = n_a * cos - n_b * sin,  y_b = n_b * cos + n_a * sin  for each rotated
 *   pair (a, b),  y_j = n_j for the other columns; all in fp32, rounded once.
 * q [B, T, q_heads, D], k [B, T, k_heads, D]: either may have no heads (and is
 *   then NULL).  D is at most 512; where a part of a head is rotated in halves,
 *   ceil(columns / 16) + ceil((D - columns) / 16) is at most 32 as well (always so
 *   up to D = 496).  At most 65535 heads a side and 2^31 - 1 tokens.
 * gamma_q, gamma_k [D] or NULL (ones).  rotation: NULL for the norm alone.
 * q_out, k_out: outputs of distinct elements.  Each may be exactly its input (in
 *   place); otherwise they are clear of the inputs and of each other.  Parts of
 *   one fused tensor count as clear where their columns are: queries behind keys,
 *   or a head's query and key side by side.
 * A token whose position is outside the table gives heads of zeros and raises
 * NORM_DEVICE_ERR_BAD_POSITION.
 */
norm_status head_rms_rotary(const norm_heads* q, int64_t q_heads, const norm_heads* k, int64_t k_heads,
                            const void* gamma_q, const void* gamma_k, const norm_heads* q_out, const norm_heads* k_out,
                            const norm_rotation* rotation, int64_t B, int64_t T, int64_t D, float eps,
                            norm_dtype x_dtype, norm_dtype w_dtype, norm_stream_t stream);

/*
 * Bytes of device workspace head_rms_rotary_grad needs for heads of D columns on
 * CUDA device `device`; independent of all else.  Returns 0 if an argument is out
 * of range or the device cannot be queried.
 */
size_t head_rms_rotary_workspace_bytes(int64_t D, int device);

/*
 * Gradient of head_rms_rotary from its inputs (statistics are formed again).  For
 * each head, u the gradient dy turned back by its token's angles:
 *   w  = u * gamma,
 *   dx = rstd * (w - x * rstd^2 * sum(w * x) / D),
 *   dgamma = sum over all tokens and the side's heads of u * x * rstd.
 * dyq, dyk: the outputs' gradients; q, k: the forward's inputs.
 * dq, dk: each may be exactly its dyq or dyk; otherwise clear of the inputs and
 *   of each other, as the forward's outputs.
 * dgamma_q, dgamma_k [D] in w_dtype, or NULL to skip.  Overwritten; zero with no
 *   tokens.  A token with a position outside the table has no gradient.
 * workspace: head_rms_rotary_workspace_bytes(D, device) bytes, 16-byte aligned;
 *   needed only when a dgamma is.  Calls that share it must be ordered.
 * Sums have a fixed order: the same inputs give the same bits.
 */
norm_status head_rms_rotary_grad(const norm_heads* dyq, const norm_heads* q, int64_t q_heads, const norm_heads* dyk,
                                 const norm_heads* k, int64_t k_heads, const void* gamma_q, const void* gamma_k,
                                 const norm_heads* dq, const norm_heads* dk, void* dgamma_q, void* dgamma_k,
                                 const norm_rotation* rotation, void* workspace, size_t workspace_bytes, int64_t B,
                                 int64_t T, int64_t D, float eps, norm_dtype x_dtype, norm_dtype w_dtype,
                                 norm_stream_t stream);

/*
 * Log probabilities of given tokens: the end of a residual stream.  For each row
 * z of V logits, a = scale (> 0; an inverse temperature), m = max_j z_j:
 *   l = log(sum_j exp(a (z_j - m))),  p_j = exp(a (z_j - m) - l),
 *   logprob = a (z_t - m) - l for the row's token t,
 *   entropy = -sum_j p_j log p_j  (a term with p_j = 0 counts as 0),
 *   lse = a m + l,  stats = (m, l), kept apart for token_logprobs_grad,
 *   and the `top` most probable tokens, larger logits first and equal ones by id.
 * logits [N x ldl] in `dtype`.  tokens [N], contiguous, or NULL (no logprob).  A
 *   row whose token is ignore_index (NORM_NO_IGNORE: none is) has logprob 0.  A
 *   token outside [0, V) has so too and raises NORM_DEVICE_ERR_BAD_TOKEN.
 * logprob [N] (with tokens), entropy [N], lse [N], stats [N x 2, 8-byte aligned]:
 *   fp32; entropy, lse and stats may be NULL.  top_logprobs fp32, top_ids int64
 *   [N x top]; top is at most NORM_MAX_TOP, 0 for none (then both NULL).
 * A logit of -inf has probability 0 and is no alternative: where fewer than `top`
 *   are left, the rest is id -1 with log probability -inf (NaN is none either).
 *   A row that is -inf throughout has logprob, lse and stats of -inf and entropy
 *   0.  A row with a NaN or +inf has NaN in all but its maximum and its ids (and
 *   the logprob of 0 of a row without a token, the -inf of an id -1).
 * N is at most 2^28.
 */
#define NORM_MAX_TOP 32
#define NORM_NO_IGNORE INT64_MIN
norm_status token_logprobs(const void* logits, int64_t ldl, const void* tokens, norm_itype token_type, float scale,
                           int64_t ignore_index, float* logprob, float* entropy, float* lse, float* stats,
                           float* top_logprobs, int64_t* top_ids, int64_t top, int64_t N, int64_t V, norm_dtype dtype,
                           norm_stream_t stream);

/*
 * Gradient of the logits from those of token_logprobs' outputs, fp32 [N] or NULL
 * (zeros; not all of them):
 *   dlogits_j = a (dlogprob (1[j = t] - p_j) + dlse p_j - dentropy p_j (log p_j + entropy)).
 * stats [N x 2], entropy [N] (with dentropy): the forward's.  tokens as in the
 *   forward (read only with dlogprob); a row without a token has no dlogprob.
 * dlogits [N x lddl]: may be exactly logits (in place), else clear of it.
 * A row that is -inf throughout has no gradient.  The alternatives have none.
 */
norm_status token_logprobs_grad(const float* dlogprob, const void* logits, int64_t ldl, const void* tokens,
                                norm_itype token_type, const float* stats, const float* entropy, const float* dentropy,
                                const float* dlse, float scale, int64_t ignore_index, void* dlogits, int64_t lddl,
                                int64_t N, int64_t V, norm_dtype dtype, norm_stream_t stream);

/* A static, human-readable name for a status code (never NULL). */
const char* norm_status_str(norm_status status);

/* Version of this ABI: major*10000 + minor*100 + patch. */
int norm_abi_version(void);

/* The CUDA call and error behind the calling thread's most recent
 * NORM_ERR_CUDA ("" if none yet).  Static per-thread storage, never NULL. */
const char* norm_last_error(void);

/*
 * Device-side error bits raised since the last clear, for CUDA device
 * `device`.  Kernels never trap: every wait inside them is bounded (2 s), and a
 * wait that runs out sets NORM_DEVICE_ERR_WAIT_TIMEOUT here and abandons the
 * call's remaining work.  The read is synchronous; call it after the streams
 * that ran the kernels have been synchronised.  clear != 0 resets the bits.
 */
#define NORM_DEVICE_ERR_WAIT_TIMEOUT 1u
#define NORM_DEVICE_ERR_BAD_COPY 2u /* a bulk copy failed its bounds check and was skipped */
#define NORM_DEVICE_ERR_BAD_TOKEN 4u /* a token id outside its table was met (and left out) */
#define NORM_DEVICE_ERR_BAD_POSITION 8u /* a position outside the rotation's table was met (and left out) */
norm_status norm_device_errors(int device, unsigned int* flags, int clear);

/*
 * Self-test of the failure path above: enqueue one small kernel that waits,
 * with the given limit, on a barrier nothing ever signals.  The wait gives up
 * after limit_ns (1 ms .. 2 s, else NORM_ERR_INVALID_VALUE), sets
 * NORM_DEVICE_ERR_WAIT_TIMEOUT on the current device and returns; the CUDA
 * context stays usable.  No data is touched.
 */
norm_status norm_selftest_bounded_wait(unsigned long long limit_ns, norm_stream_t stream);

/*
 * Testing and tuning: the kernel-family policy for every later call in the
 * process.  0 = automatic (the default), 1 = register rows (else the strided
 * loop), 2 = strided loop only, 3 = bulk-copy pipeline first.  A family is
 * used only where the call meets its requirements (alignment, row width);
 * every family computes the same results within rounding.  The block join and
 * the token lookup have two families: 2 is their loop, anything else the
 * automatic choice.  The per-head norm and the log probabilities have one.
 */
norm_status norm_set_kernel_path(int path);

/*
 * Timing: split every later backward call in the process into its two
 * kernels.  The bounded partial reduction of "Rewrite Triton normalization
 * backward kernel_1 (#499)" runs the backward as a main kernel (dx and the
 * per-CTA dgamma/dbeta partial rows) and a second kernel that sums the
 * partials; its Benchmark harness asks for the device time of each.  When
 * `event` (a cudaEvent_t, or NULL to turn the split off) is set, each backward
 * records it on its stream after the main kernel and launches the reduction
 * as an ordinary dependent launch instead of a programmatic one, so events
 * recorded before and after the call bracket the two kernels.  Results are
 * unchanged.  One value for the whole process; for benchmarks, not for
 * concurrent production calls.
 */
norm_status norm_set_bwd_split_event(void* event);

#ifdef __cplusplus
}
#endif

#endif /* NORM_H_ */
