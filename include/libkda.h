/*
 * libkda -- Kimi Delta Attention (KDA) on AMD Instinct MI355X (gfx950).
 *
 * KDA is a delta-rule linear attention with a channel-wise forget gate whose
 * per-head state is a fixed-size dk x dv matrix ("Kimi K3 深度解析", section 3.1;
 * blog.csdn.net article on the Kimi K3 report, section 一.1).  Per head and
 * token t, with state S (dk x dv), gate alpha_t in (0,1]^dk and scalar beta_t:
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *     o_t = S_t^T q_t                  (the output reads the updated state)
 *
 * No output scale and no normaliser is applied: q and k are used as given.
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor pointer is a DEVICE pointer to a contiguous row-major array,
 *    aligned to 16 bytes.  The caller owns all memory; the library allocates
 *    and frees no device memory inside these calls, and synchronises nothing
 *    except in the check mode described below.
 *  - `dtype` gives the element type of q, k, v, log_alpha, beta and o.  States
 *    (S0, S_T, S, S_zero_end, M, S_in, S_start) are always fp32.
 *  - The gate is passed in log space: log_alpha = log(alpha), one value per key
 *    channel, and must lie in [-1, 0]; beta must lie in [0, 1].  The pages
 *    describe the gate as lower-bounded so that long sequences neither overflow
 *    nor underflow (blog.csdn.net article, section 一.1); the kernels rely on
 *    the bound (|cumulative log-decay| <= 64 inside a 64-token chunk).  By
 *    default nothing checks it: a gate below the bound can give inf or NaN
 *    outputs with KDA_OK.  With the "check" option set (below), every call that
 *    takes log_alpha and beta first reduces them on the device, waits for the
 *    answer (it synchronises `stream`), and returns KDA_ERR_PRECONDITION,
 *    launching nothing else, when a value is out of range or not finite.
 *  - Supported head sizes: dk == dv == 64 or 128, for both dtypes.
 *  - Errors: arguments are validated on the host before anything is launched;
 *    on error nothing is written and a status != KDA_OK is returned, with a
 *    description in kda_last_error() (thread-local).  Work is enqueued
 *    asynchronously on `stream`; a launch failure returns KDA_ERR_HIP.
 *  - Calls never abort the process.  The only global state is per device and
 *    created on first use: the compute-unit count, the check flag, and for the
 *    sequence-split prefill a second stream (with two events) per caller
 *    stream, kept for the process lifetime; plus the process-wide options.
 *  - Options (kda_set_option): process-wide tuning and debugging switches,
 *    read from the environment once, at the first call that needs them, and
 *    changed at run time with kda_set_option.  Every choice they make gives the
 *    same result up to rounding.  See kda_set_option for the list.
 */
#ifndef LIBKDA_H
#define LIBKDA_H

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 8

typedef enum {
  KDA_OK = 0,
  KDA_ERR_NULL = 1,         /* a required pointer is NULL                    */
  KDA_ERR_SHAPE = 2,        /* negative size, dk != dv, or size overflow      */
  KDA_ERR_UNSUPPORTED = 3,  /* head size / dtype combination not built        */
  KDA_ERR_ALIGN = 4,        /* a pointer is not 16-byte aligned               */
  KDA_ERR_WORKSPACE = 5,    /* a required workspace is missing or too small   */
  KDA_ERR_PRECONDITION = 6, /* check mode: log_alpha outside [-1, 0] or beta
                               outside [0, 1] (or not finite)                 */
  KDA_ERR_HIP = 7           /* the HIP runtime reported an error              */
} kda_status;

typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/*
 * Chunked prefill of B*H independent heads over T tokens.
 * Evaluates the recurrence above exactly (up to rounding) in 64-token chunks:
 * parallel inside a chunk, sequential across chunks ("Kimi K3 开源日来了",
 * section "FlashKDA").
 *   q, k, log_alpha : [B, H, T, dk]   dtype
 *   v               : [B, H, T, dv]   dtype
 *   beta            : [B, H, T]       dtype, in [0, 1]
 *   S0              : [B, H, dk, dv]  fp32 start states, or NULL for zero
 *   o               : [B, H, T, dv]   dtype, written
 *   S_T             : [B, H, dk, dv]  fp32 end states, written; may alias S0
 *   workspace       : device scratch of workspace_bytes bytes, or NULL
 * Any T >= 0 is accepted (a last partial chunk is masked); T == 0 copies S0
 * (or zeros) to S_T.
 *
 * With few heads and a long sequence, the call can cut every sequence into G
 * segments and apply the context-parallel decomposition of the same section
 * ("针对适配的 Infra", KDA context parallelism) on this GPU (kda_prefill_plan
 * reports the cut).  By default every segment is prefilled at once, segment 0
 * from S0 and the others from zero, outputs included.  A short walk over the
 * first chunks of every later segment's transfer map decides, on the device,
 * whether the map is exactly zero there (it then stays zero).  If so, the
 * segment's outputs past those chunks and its end state are already the true
 * ones up to rounding, and only those first chunks are prefilled again from
 * the segment's true start state (from a merge of the segments' end states
 * and maps).  If not, the segment takes the longer way: its zero-start state
 * and map from the segment pass, then its whole prefill again from its start
 * state.  Option "fixup" 0 selects the earlier pipeline instead: the first T0
 * tokens prefilled directly beside the segment pass over the G - 1 segments
 * after them, the merge, then the prefill of those G segments.
 * The split path needs kda_prefill_workspace_bytes() of workspace (fp32
 * states, 3G - 2 per head, and G - 1 small segment records; 3G - 1 states
 * with fixup 0); with a smaller or NULL workspace the call runs the
 * single-pass path instead.  The workspace is only used by work enqueued by
 * this call; calls on one stream may share it.
 * The segment pass runs on a second stream of the library's own, one per
 * (device, caller stream) pair (created at the first split call on that stream,
 * default priority), forked from and joined back to `stream` with events, so
 * all of the call's work is ordered after earlier work on `stream` and before
 * later work on it, and split calls on different caller streams do not wait for
 * each other.
 */
size_t kda_prefill_workspace_bytes(int B, int H, int T, int dk, int dv, kda_dtype dtype);

kda_status kda_chunk_prefill(const void* q, const void* k, const void* v, const void* log_alpha,
                             const void* beta, const float* S0, void* o, float* S_T, int B, int H,
                             int T, int dk, int dv, kda_dtype dtype, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/*
 * kda_chunk_prefill for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, and harnesses that forbid hipMalloc.
 * Same arguments and results as kda_chunk_prefill without the workspace: the
 * sequence-split path takes its workspace from a scratch array the library
 * holds on each device (64 MiB, a file-scope device array that the device keeps
 * until the process ends), and the call itself allocates nothing.  The split
 * plan of every shape fits it on a 256-CU device with the default options; a
 * plan that needs more (e.g. a large "split" option) returns KDA_ERR_WORKSPACE
 * and launches nothing.  Nothing in the scratch array has to start at any value
 * (every byte the call reads there it has written first), but all calls on one
 * device share it: calls that can overlap on one device (on different streams,
 * or from different threads) race and must not be issued; calls on one stream
 * are ordered and safe.
 */
kda_status kda_chunk_prefill_noalloc(const void* q, const void* k, const void* v, const void* log_alpha,
                                     const void* beta, const float* S0, void* o, float* S_T, int B, int H,
                                     int T, int dk, int dv, kda_dtype dtype, hipStream_t stream);

/*
 * kda_chunk_prefill that also keeps state snapshots for prefix caching.  The
 * KDA state of a request has a fixed size and is stored only at a sparse subset
 * of the 512-token block boundaries that prefix matching uses ("Kimi K3
 * 开源日来了", section "针对适配的 Infra", prefix-cache paragraph); a cache hit
 * then resumes from the longest stored boundary.
 *   snap_interval : tokens between snapshots, a positive multiple of 64 (the
 *                   chunk length; 512 or a multiple of it in the pages' use), or
 *                   0 for none
 *   S_snap        : [B, T / snap_interval, H, dk, dv] fp32 (floor division):
 *                   entry [b, j, h] is head (b, h)'s state after its first
 *                   (j + 1) * snap_interval tokens.  Required (16-byte aligned)
 *                   when that count is nonzero, ignored otherwise; must not
 *                   overlap any other argument.
 * Every other argument, the workspace and the paths taken are as for
 * kda_chunk_prefill, whose outputs this call reproduces bit for bit.
 * Errors: KDA_ERR_SHAPE for a negative interval or one that is not a multiple
 * of 64; the rest as for kda_chunk_prefill.
 */
kda_status kda_chunk_prefill_snap(const void* q, const void* k, const void* v, const void* log_alpha,
                                  const void* beta, const float* S0, void* o, float* S_T,
                                  float* S_snap, int snap_interval, int B, int H, int T, int dk,
                                  int dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                                  hipStream_t stream);

/*
 * The cut kda_chunk_prefill would use for this shape when given
 * kda_prefill_workspace_bytes() of workspace: a first part of *T0 tokens
 * prefilled directly, then *G segments of *Tseg tokens (the last one possibly
 * shorter, ending at T).  *G == 1 (*T0 == 0, *Tseg == T) means the
 * single-pass path.  With the default pipeline *T0 is 0 and segment 0 starts
 * from S0; with option "fixup" 0, *T0 > 0.  T0 and Tseg are multiples of 64
 * on the split path.  Writes nothing else and launches nothing.
 */
kda_status kda_prefill_plan(int B, int H, int T, int dk, int dv, kda_dtype dtype, int* T0, int* G,
                            int* Tseg);

/*
 * Last step of the context-parallel decomposition (same section): every
 * segment, once its true start state is known, runs its own prefill.  Here all
 * G = ceil(T / Tseg) segments of all B*H heads run in one call, segment i
 * covering tokens [i*Tseg, min((i+1)*Tseg, T)) and starting from S_start[i].
 *   q, k, v, log_alpha, beta, o : as for kda_chunk_prefill (T >= 1 tokens)
 *   S_start : [G, B, H, dk, dv] fp32 start states, or NULL for zero
 *   S_T     : [B, H, dk, dv] fp32, written with the end state of the last segment
 * With S_start from kda_segment_transfer + kda_segment_merge this reproduces
 * kda_chunk_prefill over the whole sequence.  Tseg >= 1; S_T must not alias
 * S_start.
 */
kda_status kda_chunk_prefill_segments(const void* q, const void* k, const void* v,
                                      const void* log_alpha, const void* beta, const float* S_start,
                                      void* o, float* S_T, int B, int H, int T, int Tseg, int dk,
                                      int dv, kda_dtype dtype, hipStream_t stream);

/*
 * One decode step for N*H independent heads: applies the recurrence for one
 * token to the fp32 state held in place (the state is the fixed-size per-request
 * KDA cache, "Kimi K3 开源日来了", section "针对适配的 Infra").
 *   q, k, log_alpha : [N, H, dk]      dtype
 *   v               : [N, H, dv]      dtype
 *   beta            : [N, H]          dtype
 *   S               : [N, H, dk, dv]  fp32, read and overwritten
 *   o               : [N, H, dv]      dtype, written
 */
kda_status kda_decode_step(const void* q, const void* k, const void* v, const void* log_alpha,
                           const void* beta, float* S, void* o, int N, int H, int dk, int dv,
                           kda_dtype dtype, hipStream_t stream);

/*
 * Several consecutive tokens per sequence in one pass over the state: the
 * verification step of speculative decoding, for which the K3 report
 * fine-tunes a draft model (blog.csdn.net article on the Kimi K3 report,
 * section 二, deployment-aware training).  Equivalent to ntok calls of
 * kda_decode_step, reading and writing the state once.
 *   q, k, log_alpha : [N, H, ntok, dk]   dtype
 *   v               : [N, H, ntok, dv]   dtype
 *   beta            : [N, H, ntok]       dtype (any element alignment)
 *   S_in            : [N, H, dk, dv]     fp32 state before the tokens
 *   S_out           : [N, H, dk, dv]     fp32, written with the state after all
 *                                        ntok tokens; may alias S_in (in place)
 *   o               : [N, H, ntok, dv]   dtype, written
 *   S_pos           : [N, ntok, H, dk, dv] fp32 or NULL: entry [n, t, h] is the
 *                     state after token t, the rollback point when only tokens
 *                     0..t are accepted; must not overlap any other argument
 * ntok == 0 copies S_in to S_out.  Errors: as for kda_decode_step.
 */
kda_status kda_decode_tokens(const void* q, const void* k, const void* v, const void* log_alpha,
                             const void* beta, const float* S_in, float* S_out, void* o, float* S_pos,
                             int N, int H, int ntok, int dk, int dv, kda_dtype dtype, hipStream_t stream);

/*
 * First half of the context-parallel decomposition ("Kimi K3 开源日来了",
 * section "针对适配的 Infra", KDA Context Parallelism): the sequence of every
 * (b, h), of T = G * Tseg tokens, is cut into G segments; for each segment this
 * computes, independently of the others,
 *   S_zero_end : [G, B, H, dk, dv]  fp32, its end state when started from zero
 *   M          : [G, B, H, dk, dk]  fp32, its transfer map, so that the end
 *                state from any start state X is  M X + S_zero_end.
 *   k, log_alpha : [B, H, T, dk] dtype;  v : [B, H, T, dv];  beta : [B, H, T].
 * Tseg >= 1.  q is not needed.
 */
kda_status kda_segment_transfer(const void* k, const void* v, const void* log_alpha,
                                const void* beta, float* S_zero_end, float* M, int B, int H, int G,
                                int Tseg, int dk, int dv, kda_dtype dtype, hipStream_t stream);

/*
 * Second half: the exchange that recovers each segment's true start state
 * (same section).  Per (b, h), sequentially over segments i = 0..G-1:
 *     S_start[i] = S;   S = M[i] S + S_zero_end[i];       and finally S_T = S,
 * starting from S = S_in (NULL for zero).  All arrays fp32:
 *   S_in [B,H,dk,dv] or NULL; S_zero_end [G,B,H,dk,dv]; M [G,B,H,dk,dk];
 *   S_start [G,B,H,dk,dv] or NULL (not written); S_T [B,H,dk,dv].
 * S_T may alias S_in; it must not alias S_zero_end, M or S_start.
 */
kda_status kda_segment_merge(const float* S_in, const float* S_zero_end, const float* M,
                             float* S_start, float* S_T, int B, int H, int G, int dk, int dv,
                             hipStream_t stream);

/*
 * Gradients of the prefill, for training (the K3 report credits FlashKDA with
 * faster training as well as inference: myzaker "Kimi K3 开源日来了", section
 * "FlashKDA").  For a loss L with dL/do = dO and dL/dS_T = dS_T this computes
 * the gradients with respect to every input of kda_chunk_prefill
 * (reverse-mode chain rule).
 *   q, k, v, log_alpha, beta, S0 : as for kda_chunk_prefill (S0 NULL = zero)
 *   dO   : [B, H, T, dv] dtype, or NULL (= 0)
 *   dS_T : [B, H, dk, dv] fp32, or NULL (= 0)
 *   dq, dk_, dlog_alpha : [B, H, T, dk] dtype;  dv_ : [B, H, T, dv] dtype;
 *   dbeta : [B, H, T] dtype;  dS0 : [B, H, dk, dv] fp32.
 * Each gradient takes the dtype of the input it belongs to (the states' is
 * fp32), as autograd frameworks expect.
 * bf16 inputs run in the chunked form, on the matrix cores (bf16 operands,
 * fp32 accumulation): a forward pass that keeps, for every 64-token chunk, its
 * start state S and Delta; beside it the reverse chain over the chunks
 * (dS' -> dS, which needs no forward state), which keeps dU = Diag(Gam) dS'
 * of every chunk and writes dv_; then every (head, chunk)'s remaining
 * gradients in parallel.  For tokens with beta below 2^-30 the two chains
 * also keep W = V - Kh S, Xbar and the token's row of strict_lower(Kh Kb^T),
 * from which such a token's dbeta is formed.  fp32
 * inputs run the recurrence's token steps backwards in fp32, token by token,
 * one workgroup (or two, each with half of the state's columns) per head.
 * The workspace (device memory, at least kda_backward_workspace_bytes for the
 * same dtype, 16-byte aligned) holds, for bf16, room for those per-chunk
 * values (bf16: S and dS' dk x dv each, W, Delta and Xbar 64 x dv each, the
 * 64 x 64 lower blocks; 117 KiB per chunk-head at d = 128) and one fp32 end
 * state per head; for fp32, a state
 * checkpoint every 64 tokens, the entering
 * states and vectors u = (Diag(alpha) S)^T k of one 64-token interval, per
 * head, and the two halves' row sums.  Its contents on return are undefined.
 * No output may alias an input or the workspace.  The bf16 path forks part of
 * its work to the same per-caller-stream side stream as the sequence-split
 * prefill.  Errors: KDA_ERR_NULL for a missing required pointer,
 * KDA_ERR_WORKSPACE for a missing workspace or one below the required size.
 */
size_t kda_backward_workspace_bytes(int B, int H, int T, int dk, int dv, kda_dtype dtype);
kda_status kda_prefill_backward(const void* q, const void* k, const void* v, const void* log_alpha,
                                const void* beta, const float* S0, const void* dO, const float* dS_T,
                                void* dq, void* dk_, void* dv_, void* dlog_alpha, void* dbeta,
                                float* dS0, int B, int H, int T, int dk, int dv, kda_dtype dtype,
                                void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * ------------------------------------------------------------------------
 * Companion operators.  A layer runs its q, k and v through a short causal
 * convolution before the recurrence; hybrid models interleave KDA layers with
 * scalar-decay (selective state space) layers; and a serving engine keeps the
 * fixed-size states of many prefixes.  The calls below share the conventions at
 * the top of this file except where they say otherwise:
 *  - sequences may be strided: a kda_strides gives the distance in elements
 *    between consecutive batch entries, heads and tokens of a [B, H, T, d]
 *    array whose rows of d elements are contiguous, so that a projection's
 *    token-major output [B, T, H * d] is read in place.  NULL means contiguous
 *    [B, H, T, d].  Rows must start on 16-byte boundaries: strides (of
 *    dimensions larger than 1) are multiples of 16 bytes and not negative, a
 *    token's at most 2^23 elements; those of an output are not 0 and its rows
 *    do not overlap.
 *  - `lens` (NULL: every sequence has T tokens) is a device array of B ints:
 *    sequence b has its first lens[b] tokens (clamped to [0, T]).  The padding
 *    behind them is neither read into the results nor written.
 *  - a workspace belongs to its call until that call's work is done: calls that
 *    can overlap (on several streams, or in graphs replayed at once) take one each.
 * Outputs must not overlap inputs except where stated; one that starts at the same
 * address as an input of q, k, v or x is refused with KDA_ERR_UNSUPPORTED.
 */
typedef struct { long long b, h, t; } kda_strides;

typedef enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1 } kda_activation;

/*
 * Short causal convolution, one filter of K taps (2, 3 or 4) per channel:
 *     e = [state_in; x],  pre[t] = bias + sum_k weight[k] e[t + k],  o[t] = act(pre[t])
 * with act(x) = x or x * sigmoid(x) (SiLU).
 *   x, o       : [B, H, T, d] dtype, strides xs and os; d * sizeof(dtype) a
 *                multiple of 16
 *   weight     : [H, d, K] dtype (any element alignment);  bias : [H, d] or NULL
 *   state_in   : [B, H, K - 1, d] dtype, contiguous: the tokens before the first
 *                one, oldest first; NULL for zeros
 *   state_out  : the same shape, or NULL: the last K - 1 rows of e before token
 *                T (lens[b]), to go on from; must not be state_in
 * T == 0 copies state_in (or zeros) to state_out.
 */
kda_status kda_conv_prefill(const void* x, const kda_strides* xs, const void* weight, const void* bias,
                            const void* state_in, const int* lens, void* o, const kda_strides* os,
                            void* state_out, int B, int H, int T, int d, int K, kda_activation act,
                            kda_dtype dtype, hipStream_t stream);

/*
 * One token of the same convolution for N sequences: x, o [N, H, d] (strides b
 * and h; t is ignored), state [N, H, K - 1, d] read and moved on in place.
 */
kda_status kda_conv_step(const void* x, const kda_strides* xs, void* state, const void* weight,
                         const void* bias, void* o, const kda_strides* os, int N, int H, int d, int K,
                         kda_activation act, kda_dtype dtype, hipStream_t stream);

/*
 * Gradients of kda_conv_prefill (without lens) for dL/do = dO and dL/dstate_out =
 * dstate_out (NULL: zero): dx as x, dweight as weight, dbias as bias (NULL: not
 * written), dstate_in as state_in (NULL: not written), each in dtype; sums over
 * tokens and sequences are held in fp32 and added in a fixed order.  B and T are at
 * least 1 (unless H * d is 0, when there is nothing to do).
 * The workspace (kda_conv_backward_workspace_bytes) holds partial sums.
 */
size_t kda_conv_backward_workspace_bytes(int B, int H, int T, int d, int K, kda_dtype dtype);
kda_status kda_conv_backward(const void* x, const kda_strides* xs, const void* weight, const void* bias,
                             const void* state_in, const void* dO, const kda_strides* dos,
                             const void* dstate_out, void* dx, const kda_strides* dxs, void* dweight,
                             void* dbias, void* dstate_in, int B, int H, int T, int d, int K,
                             kda_activation act, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                             hipStream_t stream);

/*
 * Selective state space scan with one decay per head and token.  Per head, with
 * state S (dk x dv):
 *     S_t = exp(log_alpha_t) S_{t-1} + beta_t k_t v_t^T,   o_t = S_t^T q_t + D v_t
 * In state space terms k and q are B and C, v the input, beta the step size dt,
 * log_alpha = dt * A, and D the skip.
 *   q, k            : [B, G, T, dk] dtype, G dividing H: heads h with the same
 *                     h / (H / G) share them
 *   v, o            : [B, H, T, dv] dtype
 *   log_alpha, beta : [B, H, T] dtype (strides b, h, t in elements, any element
 *                     alignment), log_alpha <= 0 (-inf clears the state), beta
 *                     finite.  Option "check" validates that (padding excepted)
 *                     before launching.
 *   D               : [H] dtype (any element alignment) or NULL (no skip)
 *   S0, S_T         : [B, H, dk, dv] fp32; S0 NULL for zero; S_T may be S0
 * dk and dv are 64 or 128, independently.  T == 0 copies S0 (or zeros) to S_T.
 * bf16 inputs use bf16 matrix products with fp32 accumulation; states are
 * carried in fp32.  An infinity or NaN in q, k or v may also reach the other
 * tokens of its 64-token chunk, or not reach the states behind a decay of zero.
 * Sequences too few to fill the device are cut into segments (each one's
 * zero-start end state, a merge, then every segment from its true start); that
 * needs kda_ssm_prefill_workspace_bytes() of workspace, and with less, or NULL,
 * the call walks each sequence in one piece.
 */
typedef struct { kda_strides q, k, v, log_alpha, beta, o; } kda_ssm_strides;

size_t kda_ssm_prefill_workspace_bytes(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype);
kda_status kda_ssm_prefill(const void* q, const void* k, const void* v, const void* log_alpha,
                           const void* beta, const void* D, const float* S0, const int* lens, void* o,
                           float* S_T, const kda_ssm_strides* strides, int B, int H, int G, int T, int dk,
                           int dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/*
 * One token of the scan for N sequences: q, k [N, G, dk], v, o [N, H, dv],
 * log_alpha, beta [N, H] (any element alignment), all contiguous; S [N, H, dk,
 * dv] fp32 in place.
 */
kda_status kda_ssm_step(const void* q, const void* k, const void* v, const void* log_alpha,
                        const void* beta, const void* D, float* S, void* o, int N, int H, int G, int dk,
                        int dv, kda_dtype dtype, hipStream_t stream);

/*
 * Gradients of kda_ssm_prefill (without lens; padding tokens with beta = 0 and
 * log_alpha = 0 pass the state on) for dL/do = dO and dL/dS_T = dS_T (NULL:
 * zero).  dq, dk_ (summed over a group's heads), dv_, dlog_alpha, dbeta and dD
 * (NULL without D) take their input's shape, in dtype, dS0 fp32 (NULL: not
 * written).  Sums are fp32 in a fixed order.  The strides of dlog_alpha and
 * dbeta are free; B and T are at least 1 (unless H is 0).  A gate of -inf has a
 * dlog_alpha of zero.
 */
typedef struct { kda_strides dO, dq, dk, dv, dlog_alpha, dbeta; } kda_ssm_grad_strides;

size_t kda_ssm_backward_workspace_bytes(int B, int H, int G, int T, int dk, int dv, kda_dtype dtype);
kda_status kda_ssm_backward(const void* q, const void* k, const void* v, const void* log_alpha,
                            const void* beta, const void* D, const float* S0, const void* dO,
                            const float* dS_T, void* dq, void* dk_, void* dv_, void* dlog_alpha,
                            void* dbeta, void* dD, float* dS0, const kda_ssm_strides* strides,
                            const kda_ssm_grad_strides* grad_strides, int B, int H, int G, int T, int dk,
                            int dv, kda_dtype dtype, void* workspace, size_t workspace_bytes,
                            hipStream_t stream);

/*
 * The quantised state cache: KDA or scan states (prefix snapshots, parked
 * requests) in 8 bits.  A row of dv values is cut into blocks of 32 that share a
 * power-of-two scale 2^p, the smallest (at least 2^-126) that brings the block's
 * largest value to at most 127 (int8) or 448 (e4m3), so that only the rounding of
 * each value loses anything: at most 2^(p-1), that is, 1/254 to 1/127 of the
 * block's largest value (int8), or the larger of 2^-4 of the value itself and
 * 2^(p-10) (e4m3).  A value far below its block's largest becomes zero: up to
 * 2^(p-1) (int8) or 2^(p-10) (e4m3, about 2^-18 of the largest).
 *   S      : [n, H, dk, dv] fp32 (S_snap of kda_chunk_prefill_snap as it stands)
 *   slots  : [n] ints on the device, the cache entry of each state.  Store skips
 *            entries outside [0, nslots); of entries that name the same slot
 *            the last one is stored.  Load writes zeros for entries outside.
 *   cache  : [nslots, H, dk, dv] bytes (int8 or OCP e4m3 values)
 *   scales : [nslots, H, dk, dv / 32] bytes: exponent + 127; 255 marks a block
 *            that held an infinity or NaN and reads back as NaN
 * dv is a multiple of 32, n at most 65536.  slots and scales may have any
 * alignment of their elements.
 */
typedef enum { KDA_CACHE_INT8 = 0, KDA_CACHE_E4M3 = 1 } kda_cache_format;

kda_status kda_state_store(const float* S, const int* slots, void* cache, void* scales, int n, int nslots,
                           int H, int dk, int dv, kda_cache_format format, hipStream_t stream);
kda_status kda_state_load(const void* cache, const void* scales, const int* slots, float* S, int n,
                          int nslots, int H, int dk, int dv, kda_cache_format format, hipStream_t stream);

/*
 * Process-wide options.  Each starts from the environment variable of the same
 * name in capitals with a KDA_ prefix (KDA_SPLIT, ...), read once, at the first
 * call that needs the options; kda_set_option changes one for every later call
 * (thread-safe; calls already enqueued are not affected).  value -1 restores the
 * library's default.  Names:
 *   "split"            segments of the sequence-split prefill (after the first
 *                      part with fixup 0; 0 = never split, >= 2 = that many;
 *                      default: chosen from the shape and the compute-unit
 *                      count)
 *   "fixup"            0: the split prefill's earlier pipeline (first part
 *                      beside the segment pass, merge, prefill of every
 *                      segment); default 1 (segments from zero, heads
 *                      corrected)
 *   "head_chunks"      chunks of every segment's map walked before deciding
 *                      whether it has vanished, and prefilled again when it
 *                      has (1..1024; default 4)
 *   "transfer_cost16"  with fixup 0: the first part's length ratio, in 16ths
 *                      (1..64)
 *   "map_skip"         0: the segment pass keeps updating transfer-map columns
 *                      that have become exactly zero (same results bit for bit
 *                      for finite inputs); default 1
 *   "nc"               consumer waves per workgroup of the chunk kernels
 *                      (1, 2, 4, 8 where built; default: chosen from the shape)
 *   "bw_split"         workgroups per head of the backward's chunk kernels (1 or
 *                      2; default: chosen from the shape)
 *   "bw_overlap"       bf16 backward from 16 chunks per head: 1 runs the
 *                      reverse chain in two launches (later half of the
 *                      chunks, then earlier half) and the later half's per-chunk
 *                      gradients beside the earlier half's chain, on the side
 *                      stream; 0 (default) runs the chain whole, then every
 *                      chunk's gradients.  Same results bit for bit
 *   "check"            1: validate log_alpha and beta on the device before every
 *                      call that reads them (see the conventions above; for the
 *                      scan log_alpha <= 0 and beta finite); default 0
 *   "log"              1: print every launch's shape to stderr; default 0
 * kda_set_option returns KDA_ERR_SHAPE for an unknown name or a value the option
 * does not take; kda_get_option writes the value in effect (-1: default).
 */
kda_status kda_set_option(const char* name, long long value);
kda_status kda_get_option(const char* name, long long* value);

/*
 * Profiling only.  In a library built with KDA_PHASE_STAMPS (build.py
 * --stamps, libkda_stamps.so), every later sequence-split prefill records,
 * for each workgroup of its main launch (the prefill of every segment from
 * zero), the shader clock (s_memtime) of every wave at five points of
 * pipeline steps 32 .. 47: the step's start, the end of the elementwise phase
 * (producer waves) or of the chain (consumer waves), after the first barrier,
 * the end of the score tiles, after the second barrier.  With the environment
 * variable KDA_STAMP_TARGET set to "ckpt" or "reverse" when this is called,
 * the bf16 prefill backward's checkpoint pass or its reverse chain (in the
 * reverse chain, step i is chunk nch - 1 - i) records them instead.
 *   stamps : device buffer of count 64-bit entries, indexed
 *            [workgroup][step - 32][wave][point] with 8 wave slots; a
 *            workgroup whose entries do not fit records nothing; NULL (or
 *            count 0) stops recording
 * The regular library returns KDA_ERR_UNSUPPORTED and records nothing.
 */
kda_status kda_debug_phase_stamps(unsigned long long* stamps, size_t count);

/*
 * Profiling only (any build): the duration of the main launch (the prefill of
 * every segment from zero) of sequence-split prefills, timed with HIP events
 * recorded on the caller's stream around that launch, so that the calls
 * themselves are not synchronised.
 *   kda_debug_time_main_launches(count): arms count event pairs (1 .. 256)
 *     for the next count sequence-split prefills on the current device, and
 *     forgets what an earlier arming recorded; 0 disarms.  KDA_ERR_SHAPE for a
 *     count out of range.
 *   kda_debug_main_launch_ms(ms, count, recorded): *recorded = the launches
 *     timed since the arming; waits for them and writes the first
 *     min(count, *recorded) durations in milliseconds to ms (host memory).
 * One caller at a time: calls that overlap on other threads may take each
 * other's pairs.
 */
kda_status kda_debug_time_main_launches(int count);
kda_status kda_debug_main_launch_ms(float* ms, int count, int* recorded);

const char* kda_status_string(kda_status status);
const char* kda_last_error(void);
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LIBKDA_H */
