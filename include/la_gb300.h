/*
 * la_gb300.h -- C ABI of the GB300 (sm_103a) causal linear attention library.
 *
 * What the library computes.  For every (batch b, head h) sequence of L tokens
 * with queries q_t, keys k_t (width d_k) and values v_t (width d_v), a matrix
 * state S in R^{d_k x d_v} evolves as
 *
 *     S_t = a_t S_{t-1} + phi(k_t) v_t^T,        o_t = phi(q_t)^T S_t
 *
 * (update before read; S_{-1} = S0 or zero).  Sources:
 *   - "Linear / Sparse Attention - minimal runnable implementation",
 *     linear_attn_recurrent (the self-inclusive recurrence, S in R^{d_k x d_v})
 *     and linear_attn_chunkwise (the chunk form the prefill kernels evaluate:
 *     inter-chunk read Q_c S, intra-chunk ((Q_c K_c^T) .* tril) V_c with the
 *     diagonal included, then S += K_c^T V_c; a ragged last chunk);
 *   - "CS336 lecture 4, code 1: linear attention",
 *     gated_linear_attention_recurrent (S_t = gamma_t S_{t-1} + k_t v_t^T;
 *     constant gamma is RetNet, input-dependent gamma_t the Mamba-2 gate) and
 *     gated_linear_attention_parallel (decay factors taken in log space);
 *   - "Linear / sparse attention tutorial" section 6.2 (the two-part chunk
 *     computation; gates multiply the state and the in-chunk mask by the
 *     cumulative decay) and section 8.1 (decode keeps only the fixed-size
 *     state);
 *   - "adv13 - Linear Attention / SSM" section 3.2 / 4.2 (phi applied to q
 *     and k, never to v) and Q1 (phi = elu + 1).
 *
 * Conventions for every entry point:
 *   - Pointers to tensors are DEVICE pointers owned by the caller; the library
 *     never frees them and never allocates device memory.  Tensors are dense,
 *     row-major, contiguous, and must start on a 16-byte boundary.
 *   - Calls are asynchronous on the CUDA stream passed as `cuda_stream`
 *     (a cudaStream_t; NULL = the legacy default stream).  The return status
 *     covers argument validation and kernel launch; a device-side timeout of a
 *     bounded wait is reported by la_device_status().
 *   - No call aborts, throws or prints.  On any non-zero status the reason is
 *     available from la_last_error() on the calling thread.
 */
#ifndef LA_GB300_H
#define LA_GB300_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int la_status;

#define LA_OK                 0  /* success */
#define LA_ERR_INVALID_ARG    1  /* bad pointer, size, alignment or enum value */
#define LA_ERR_UNSUPPORTED    2  /* valid request the library has no kernel for */
#define LA_ERR_CUDA           3  /* a CUDA runtime call or launch failed */
#define LA_ERR_DEVICE_TIMEOUT 4  /* a kernel's bounded wait ran out (la_device_status) */

/* Feature map phi applied to q and k. */
#define LA_PHI_IDENTITY 0        /* phi(x) = x ("tutorial" 2.1: RetNet / GLA use phi = id) */
#define LA_PHI_ELU1     1        /* phi(x) = elu(x) + 1 = x + 1 (x > 0), exp(x) (x <= 0) */

/* Element type of q, k, v and of the outputs O / o.  The state is always fp32. */
#define LA_F32  0
#define LA_BF16 1

/* How the per-token decay a_t is given (always in log space, fp32). */
#define LA_DECAY_NONE       0   /* a_t = 1; decay pointer ignored (may be NULL)    */
#define LA_DECAY_HEAD       1   /* decay[h] = log gamma_h, shape [H] (RetNet)      */
#define LA_DECAY_TOKEN      2   /* decay[b,h,t] = log alpha_t, shape [B,H,L]       */
#define LA_DECAY_GATE_LOGIT 3   /* decay[b,h,t] = g_t, alpha_t = exp(-softplus(g_t)),
                                   shape [B,H,L] (Mamba-2-style input gate)       */

/* Select phi for all later calls in this process (atomic; default identity).
 * Returns LA_ERR_INVALID_ARG for an unknown value. */
la_status la_set_feature_map(int phi);

/* The feature map currently selected. */
int la_get_feature_map(void);

/* Bytes of device workspace la_chunk_fwd needs for this problem (0 if none).
 * The workspace holds per-segment partial states when the sequence is split
 * across CTAs; its contents need no initialisation and are not kept. */
size_t la_chunk_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk,
                                    int dtype);

/* Number of kernel launches one la_chunk_fwd call makes for this problem
 * (host-only query; 0 for an empty problem or an unsupported one). */
int la_chunk_fwd_kernel_count(int B, int H, int L, int d_k, int d_v, int chunk, int dtype);

/*
 * Chunkwise-parallel causal linear attention over whole sequences (prefill).
 *
 *   q, k      [B,H,L,d_k]  dtype            (read)
 *   v         [B,H,L,d_v]  dtype            (read)
 *   dtype     LA_F32 or LA_BF16
 *   chunk     chunk size C (tokens per chunk); the result does not depend on
 *             it up to rounding.  The tensor-core path takes C = 64; the
 *             fp32 / general path takes 1 <= C <= 64.
 *   decay_kind / decay   see LA_DECAY_*; decay is fp32 device memory.
 *   S0        [B,H,d_k,d_v] fp32 initial state, or NULL for zero   (read)
 *   O         [B,H,L,d_v]   dtype, every row written                (write)
 *   S_final   [B,H,d_k,d_v] fp32 state after the last token, or NULL
 *             (write; may be the same buffer as S0)
 *   workspace device scratch of at least la_chunk_fwd_workspace_bytes(...)
 *             bytes (may be NULL when that is 0); ws_bytes = its size.
 *
 * Supported: d_k, d_v in {16, 32, 64, 128}; fp32 inputs run the fp32 SIMT
 * kernel, bf16 inputs with d_k = d_v in {64, 128} and C = 64 run the tcgen05
 * tensor-core kernels, other bf16 shapes the SIMT kernel.  L = 0 writes
 * S_final = S0 (or zero).  Errors: LA_ERR_INVALID_ARG (null or misaligned
 * pointer, negative size, unknown enum, workspace too small),
 * LA_ERR_UNSUPPORTED (a d or C outside the list), LA_ERR_CUDA.
 */
la_status la_chunk_fwd(const void *q, const void *k, const void *v, int dtype,
                       int B, int H, int L, int d_k, int d_v, int chunk,
                       int decay_kind, const float *decay,
                       const float *S0, void *O, float *S_final,
                       void *workspace, size_t ws_bytes, void *cuda_stream);

/*
 * One recurrent decode step for B*H sequences, state updated in place:
 *
 *     S <- alpha S + phi(k) v^T ;   o = phi(q)^T S      (update, then read)
 *
 *   q, k       [B,H,d_k] dtype   (read)
 *   v          [B,H,d_v] dtype   (read)
 *   log_alpha  [B,H] fp32 log of the decay, or NULL for alpha = 1  (read)
 *   S          [B,H,d_k,d_v] fp32, read and overwritten             (in/out)
 *   o          [B,H,d_v] dtype                                      (write)
 *
 * Supported: d_k = d_v in {16, 32, 64, 128}.  Errors as for la_chunk_fwd.
 */
la_status la_decode_step(const void *q, const void *k, const void *v, int dtype,
                         int B, int H, int d_k, int d_v,
                         const float *log_alpha, float *S, void *o, void *cuda_stream);

/*
 * The non-causal matrix form, for B*H independent sequences of L tokens:
 *
 *     S = phi(K)^T V  (summed over all L tokens) ;   O = phi(Q) S
 *
 * (page "adv13 - Linear Attention / SSM", section 4.3, linear_attention_matrix;
 * page "CS336 lecture 4, code 1: linear attention", demo_associativity: the
 * order (Q K^T) V = Q (K^T V)).  Every token reads the same state: there is no
 * causal mask, no decay and no initial state.  The feature map is the one set
 * by la_set_feature_map.
 *
 *   q, k       [B,H,L,d] bf16                          (read)
 *   v          [B,H,L,d] bf16                          (read)
 *   O          [B,H,L,d] bf16                          (write)
 *   S          [B,H,d,d] fp32, the state phi(K)^T V, or NULL (write)
 *   workspace  device scratch of la_noncausal_fwd_workspace_bytes(...) bytes
 *
 * All pointers are device pointers owned by the caller, row-major and
 * 16-byte aligned; the call is asynchronous on `cuda_stream`.
 * Supported: bf16 with d_k = d_v = d in {64, 128}.  L = 0 writes S = 0.
 * Errors: LA_ERR_INVALID_ARG (null or misaligned pointer, negative size,
 * workspace too small), LA_ERR_UNSUPPORTED (another dtype or d), LA_ERR_CUDA.
 */
la_status la_noncausal_fwd(const void *q, const void *k, const void *v, int dtype,
                           int B, int H, int L, int d_k, int d_v,
                           void *O, float *S, void *workspace, size_t ws_bytes,
                           void *cuda_stream);
size_t la_noncausal_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v);

/*
 * Three further forms of the recurrence (q, k, v and O in dtype = LA_F32 or
 * LA_BF16; states fp32).  Each runs over whole sequences like la_chunk_fwd,
 * and each is also its own decode step:
 * with L = 1 and the output state aliasing the input state, one call advances
 * every sequence by one token.  phi is the one set by la_set_feature_map.
 * Supported: d_k, d_v in {16, 32, 64, 128}; chunk 1..64 where one is taken
 * (the result does not depend on it up to rounding).  L = 0 passes the
 * initial states through (or zeroes the outputs when none is given).  Errors:
 * LA_ERR_INVALID_ARG (null or misaligned pointer, negative size, unknown
 * enum), LA_ERR_UNSUPPORTED (a d or chunk outside the list), LA_ERR_CUDA.
 * Pointers are device pointers owned by the caller, row-major, 16-byte
 * aligned; the calls are asynchronous on `cuda_stream` and allocate nothing.
 * The per-channel gate and the delta rule run on the CUDA cores in fp32.
 */

/*
 * Normalised linear attention ("Linear / sparse attention tutorial" Q11 and
 * section 2.2): the state carries a key sum z next to S, which decays with S,
 *
 *     S_t = a_t S_{t-1} + phi(k_t) v_t^T,   z_t = a_t z_{t-1} + phi(k_t),
 *     o_t = phi(q_t)^T S_t / (phi(q_t)^T z_t).
 *
 * For bf16 with d_k = d_v = 64 and chunk 64 it is one pass of the tensor-core
 * prefill kernels: a column of ones rides with v, so z travels as one more
 * state column and each row's denominator comes out of the same products as
 * its numerator, and the epilogue divides before it stores O.  Otherwise the
 * numerator runs on the la_chunk_fwd kernels (the tensor-core ones for bf16,
 * d_k = d_v = 128, chunk 64), then a scan of z forms the denominators and
 * divides O in place.  There is no epsilon in the denominator: choose a
 * positive feature map (LA_PHI_ELU1), as the tutorial does, or the quotient
 * may be undefined.
 *
 *   q, k   [B,H,L,d_k] dtype;  v, O [B,H,L,d_v] dtype
 *   decay_kind / decay   as for la_chunk_fwd
 *   S0     [B,H,d_k,d_v] fp32 or NULL (zero);  z0 [B,H,d_k] fp32 or NULL (zero)
 *   S_final, z_final   the states after the last token, or NULL; each may be
 *          the same buffer as S0 / z0.
 *   workspace  device scratch of la_normalised_fwd_workspace_bytes(...) bytes,
 *          or NULL when that is 0 (the one-pass form on a sequence short
 *          enough for one CTA); ws_bytes = its size.  Its contents need no
 *          initialisation and are not kept.
 */
la_status la_normalised_fwd(const void *q, const void *k, const void *v, int dtype,
                            int B, int H, int L, int d_k, int d_v, int chunk,
                            int decay_kind, const float *decay,
                            const float *S0, const float *z0, void *O,
                            float *S_final, float *z_final,
                            void *workspace, size_t ws_bytes, void *cuda_stream);
size_t la_normalised_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk,
                                         int dtype);

/*
 * Per-channel (diagonal) gate, as in GLA ("Linear / sparse attention
 * tutorial" Q21):
 *
 *     S_t = diag(alpha_t) S_{t-1} + phi(k_t) v_t^T,   o_t = phi(q_t)^T S_t,
 *
 * one decay per key channel and token.
 *
 *   log_alpha  [B,H,L,d_k] fp32, log alpha_t[i] (expected <= 0), 16-byte
 *              aligned like the other tensors                      (read)
 *   S0         [B,H,d_k,d_v] fp32 or NULL;  S_final may alias S0.
 *   workspace  device scratch of la_channel_gate_fwd_workspace_bytes(...)
 *              bytes (16-byte aligned), or NULL; ws_bytes = its size.  With it
 *              (bf16, d_k = d_v in {64, 128}, chunk 64, when the query is not
 *              0) each sequence is cut into segments that run side by side: a
 *              state pass over every segment but the last, then the segments'
 *              outputs, each folding in the states of the segments before it.
 *              With NULL each sequence runs in one piece.
 *              A non-NULL workspace smaller than the query or misaligned is
 *              LA_ERR_INVALID_ARG.  Its contents need no initialisation and are
 *              not kept.
 */
la_status la_channel_gate_fwd(const void *q, const void *k, const void *v, int dtype,
                              int B, int H, int L, int d_k, int d_v, int chunk,
                              const float *log_alpha, const float *S0, void *O,
                              float *S_final, void *workspace, size_t ws_bytes,
                              void *cuda_stream);
size_t la_channel_gate_fwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk,
                                           int dtype);

/*
 * The (gated) delta rule ("Linear / Sparse Attention - minimal runnable
 * implementation", delta_rule_recurrent; "Linear / sparse attention tutorial"
 * Q21 for the gate), with the state as [d_k, d_v] like the others:
 *
 *     S_t = alpha_t (S_{t-1} - beta_t k (k^T S_{t-1})) + beta_t k v_t^T,
 *     o_t = phi(q_t)^T S_t,      k = phi(k_t).
 *
 * Keys are used as given (after phi): the rule assumes unit-norm keys, and
 * normalising them is the caller's step.  Runs token by token.
 *
 *   beta       [B,H,L] fp32 write strengths                        (read)
 *   log_alpha  [B,H,L] fp32 log of the gate, or NULL for alpha = 1  (read)
 *   S0         [B,H,d_k,d_v] fp32 or NULL;  S_final may alias S0.
 */
la_status la_delta_fwd(const void *q, const void *k, const void *v, int dtype,
                       int B, int H, int L, int d_k, int d_v,
                       const float *beta, const float *log_alpha,
                       const float *S0, void *O, float *S_final, void *cuda_stream);

/*
 * The operators of a state space block, and the norms around a block.
 *
 * They extend the conventions above in two points.  Activations are token
 * major: [B,L,D] with a row per token, whose rows may lie `*_stride` elements
 * apart (>= the row's width; sequence b starts at row b*L), so that a slice of a wider projection's
 * output is read or written in place.  And a pointer to activations needs no
 * more than its element's alignment (rows that keep 16-byte alignment are
 * read in 16-byte vectors).  Parameters (weights, biases, A, the skip and the
 * norm weights) and recurrent states are fp32, 16-byte aligned.
 *
 *   lengths   int32 [B] device memory, or NULL.  lengths[b] <= L tokens of
 *             sequence b are real (values outside [0, L] count as the nearer
 *             bound).  Rows behind them are neither read nor written, and the
 *             final state is the state after lengths[b] tokens.
 *
 * Outputs may not overlap inputs, parameters and lengths among them, nor a
 * workspace anything, except as stated: a final state may be the buffer of its
 * initial state, so that L = 1 is a decode step in place.
 * Errors: LA_ERR_INVALID_ARG (null, misaligned or overlapping pointer,
 * negative size, stride shorter than a row, unknown enum, workspace too
 * small), LA_ERR_UNSUPPORTED (a size outside the stated range), LA_ERR_CUDA.
 * The calls are asynchronous on `cuda_stream`, allocate nothing, and give the
 * same bits on every run.  They do not depend on la_set_feature_map.
 */
#define LA_ACT_NONE    0         /* act(x) = x                   */
#define LA_ACT_SILU    1         /* act(x) = x / (1 + exp(-x))   */
#define LA_ACT_SIGMOID 2         /* act(x) = 1 / (1 + exp(-x))   */

#define LA_NORM_RMS    0         /* x / sqrt(mean(x^2) + eps)                  */
#define LA_NORM_LAYER  1         /* (x - mean(x)) / sqrt(var(x) + eps)         */

/*
 * Causal depthwise convolution over time, the short mixing step in front of a
 * recurrence:
 *
 *     y[b,t,c] = act(bias[c] + sum_{w < width} weight[c,w] x[b,t-width+1+w,c])
 *
 * where the rows before the first token come from state0.
 *
 *   x, y         [B,L,D] dtype, rows x_stride / y_stride elements apart
 *   weight       [D,width] fp32, width in 2..8; bias [D] fp32 or NULL (zero)
 *   activation   LA_ACT_NONE or LA_ACT_SILU
 *   state0       [B,width-1,D] dtype: the width-1 inputs before the first
 *                token, oldest first; NULL = zero
 *   state_final  [B,width-1,D] dtype: the last width-1 inputs (of state0 and
 *                x together), or NULL; may be state0's buffer
 *
 * Supported: L and D up to 2^30.
 */
la_status la_causal_conv_fwd(const void *x, long long x_stride, int dtype, int B, int L, int D,
                             int width, const float *weight, const float *bias, int activation,
                             const int *lengths, const void *state0, void *y,
                             long long y_stride, void *state_final, void *cuda_stream);

/*
 * Selective state space scan: a diagonal recurrence with its own decay for
 * every (channel, state) pair and token,
 *
 *     delta    = dt[b,t,c] + dt_bias[c], through softplus if dt_softplus
 *     h[c,n]   = exp(delta A[c,n]) h[c,n] + delta B[b,t,g,n] x[b,t,c]
 *     y[b,t,c] = (sum_n C[b,t,g,n] h[c,n] + skip[c] x[b,t,c]) * silu(z[b,t,c])
 *
 * with g = c / (D / groups).  la_chunk_fwd covers the recurrences whose decay
 * one head shares, la_channel_gate_fwd those whose decay the value channels
 * share.
 *
 *   x, dt, y     [B,L,D] dtype, rows *_stride elements apart
 *   z            [B,L,D] dtype gate, or NULL (no gate)
 *   Bm, Cm       [B,L,groups,N] dtype; the groups*N values of a token are
 *                contiguous, tokens b_stride / c_stride elements apart
 *   A            [D,N] fp32 (negative for a decaying state; used as given)
 *   dt_bias      [D] fp32 or NULL (zero);  skip [D] fp32 or NULL (zero)
 *   h0, h_final  [B,D,N] fp32 initial and final state; each may be NULL, and
 *                h_final may be h0's buffer
 *   workspace    device scratch of la_selective_scan_fwd_workspace_bytes(...)
 *                bytes (16-byte aligned), or NULL; ws_bytes = its size.  With
 *                it (when the query is not 0) a long sequence runs as several
 *                segments side by side; with NULL it runs in one piece.  A
 *                non-NULL workspace smaller than the query is
 *                LA_ERR_INVALID_ARG.  Its contents need no initialisation and
 *                are not kept.
 *
 * Supported: N in 1..256, D a multiple of groups, L and D up to 2^30.  With
 * dt_softplus a dt of minus infinity, or of the type's lowest value, is a step
 * of zero: the token keeps the state.  A NaN in x or dt, an infinity in x or an
 * infinite delta makes its channel's outputs and states non-finite from its
 * token on, an infinity possibly as a NaN; other channels are not touched.
 */
la_status la_selective_scan_fwd(const void *x, long long x_stride, const void *dt,
                                long long dt_stride, const void *z, long long z_stride,
                                const void *Bm, long long b_stride, const void *Cm,
                                long long c_stride, int dtype, int B, int L, int D, int N,
                                int groups, const float *A, const float *dt_bias,
                                int dt_softplus, const float *skip, const float *h0,
                                const int *lengths, void *y, long long y_stride,
                                float *h_final, void *workspace, size_t ws_bytes,
                                void *cuda_stream);
size_t la_selective_scan_fwd_workspace_bytes(int B, int L, int D, int N, int groups);

/*
 * Norm and gate of a block's heads, on the way to its output projection:
 *
 *     y[b,t,h*d+i] = norm(x[b,h,t,:])[i] w[i] (+ bias[i]) * act(gate[b,t,h*d+i])
 * or, with gate_first,
 *     y[b,t,h*d+i] = norm(x[b,h,t,:] * act(gate[b,t,h*d:h*d+d]))[i] w[i] (+ bias[i])
 *
 * x is read where it lies: O as la_chunk_fwd and its kin write it
 * ([B,H,L,d]: strides H*L*d, L*d, d) or a token-major [B,L,H*d] (strides
 * L*H*d, d, H*d); y and gate are token major, so the heads move behind the
 * tokens in the same pass.
 *
 *   x            dtype, element (b,h,t,i) at b*x_b_stride + h*x_h_stride +
 *                t*x_t_stride + i (strides >= 0)
 *   gate         [B,L,H*d] dtype, rows gate_stride apart, or NULL (no gate)
 *   weight, bias [weight_heads,d] fp32, weight_heads = 1 (shared by the
 *                heads) or H; each may be NULL (one / zero)
 *   norm         LA_NORM_*;  activation LA_ACT_*;  eps >= 0
 *   y            [B,L,H*d] dtype, rows y_stride apart; may be gate's buffer
 *                when y_stride = gate_stride
 *
 * Supported: d in 1..16384.  Squares are summed in fp32, here and in
 * la_residual_norm_fwd: a row with values above 1e19 gives zeros.
 */
la_status la_gated_norm_fwd(const void *x, long long x_b_stride, long long x_h_stride,
                            long long x_t_stride, const void *gate, long long gate_stride,
                            int dtype, int B, int H, int L, int d, int norm, int activation,
                            int gate_first, const float *weight, const float *bias,
                            int weight_heads, float eps, void *y, long long y_stride,
                            void *cuda_stream);

/*
 * The residual step between two blocks in one pass: the norm after a block,
 * its residual scale, the addition, and the norm before the next block,
 *
 *     u = norm(x) post_weight   (u = x when post_weight is NULL)
 *     r = residual + alpha scale u            (residual NULL: 0; scale NULL: 1)
 *     residual_out = r,   y = norm(r) weight + bias
 *
 * y is formed from r before its rounding to res_dtype.
 *
 *   x, y                    [rows,D] dtype, contiguous; y may be x's buffer
 *   residual, residual_out  [rows,D] res_dtype (dtype or LA_F32), contiguous;
 *                           residual_out may be residual's buffer, or NULL
 *   post_weight, scale, weight, bias   [D] fp32, each may be NULL
 *
 * Supported: D in 1..16384.
 */
la_status la_residual_norm_fwd(const void *x, int dtype, const void *residual, int res_dtype,
                               long long rows, int D, const float *post_weight,
                               const float *scale, float alpha, const float *weight,
                               const float *bias, int norm, float eps, void *y,
                               void *residual_out, void *cuda_stream);

/*
 * The training pass of a layer: positions, and backward passes.
 *
 * The conventions of the state space block's operators hold here too:
 * pointers to activations and their gradients need their element's alignment
 * only, parameters, their gradients, decays and states are fp32 and 16-byte
 * aligned (positions, offsets, lengths and frequencies 4-byte), outputs may
 * not overlap inputs except as stated, and a call gives the same bits on every
 * run.  [B,H,L,d] tensors of the same strides may interleave without sharing an
 * element (the parts of a packed projection, whatever the order of its axes, at
 * full length or a prefix of it); an output of other strides lies in a range of
 * its own.  Nothing of a forward call is kept: a backward call gets what it needs
 * as arguments.
 *
 * A parameter's gradient is a sum over rows; it is formed in fp32 in a fixed
 * order and overwrites its buffer (nothing is accumulated).  Its shares need
 * `workspace`, device scratch of the query's bytes (16-byte aligned); its
 * contents need no initialisation and are not kept.  Gradients that are NULL
 * are not formed, and without any of them the workspace may be NULL.
 */

/* How rotary frequencies are scaled for contexts longer than the trained one. */
#define LA_ROTARY_PLAIN  0  /* f_i = base^(-2 i / rotary_dim)                                */
#define LA_ROTARY_LINEAR 1  /* f_i / factor: positions interpolated                          */
#define LA_ROTARY_NTK    2  /* base * factor^(rotary_dim / (rotary_dim - 2)) as the base     */
#define LA_ROTARY_YARN   3  /* f_i up to pair `low`, f_i / factor from pair `high` on, a blend
                               linear in the pair between them; scale 0.1 ln(factor) + 1     */

/*
 * Rotary frequencies of the pairs, rounded once from 64 bits, into HOST memory:
 * inv_freq[rotary_dim / 2], and `scale` (NULL: not wanted), what la_rotary_fwd
 * takes as its scale.  factor >= 1 (unused by PLAIN); trained_length, fast and
 * slow are used by YARN alone (32 and 1 are customary).  There pair p makes
 * trained_length f_p / 2 pi turns over the trained length; low and high are the
 * pairs of `fast` and of `slow` turns, as checkpoints trained with this scaling have
 * them: p = rotary_dim ln(trained_length / (2 pi turns)) / (2 ln base), low rounded
 * down (and at least 0), high up (at most rotary_dim - 1; where that is not above low,
 * the pairs behind low are scaled in full).  Errors: LA_ERR_INVALID_ARG.  (The pages leave out the rotation of their retention
 * layer, "Linear / sparse attention tutorial" sections 2.4 and 10; these are the
 * operators that bring it.)
 */
la_status la_rotary_frequencies(int rotary_dim, double base, int scaling, double factor,
                                double trained_length, double fast, double slow,
                                float *inv_freq, float *scale);

/*
 * Rotary positions of q and k in one call: the pairs (x_i, x_j) of the first
 * rotary_dim values of every head become
 *
 *     scale * (x_i cos a - x_j sin a, x_i sin a + x_j cos a),   a = position * inv_freq[pair]
 *
 * and the values behind them are copied.  Pair p is (2p, 2p+1) if `interleaved`,
 * else (p, p + rotary_dim / 2).  la_rotary_bwd turns by -a: it takes the
 * gradients of q_out and k_out to those of q and k.  The angle is exact however
 * far the position lies (to position * 2^-64 turns, for frequencies up to 1);
 * sine and cosine are fp32.
 *
 *   q, q_out   dtype, element (b,h,t,i) at b*b_stride + h*h_stride +
 *              t*t_stride + i (strides >= 0): a slice of a projection's
 *              token-major output, or [B,H,L,d] as la_chunk_fwd reads it.
 *              q_out may be q with q's strides (in place).
 *   k, k_out   the same with heads_k heads; both NULL: no k
 *   inv_freq   [rotary_dim / 2] fp32 device memory, radians for each token
 *              (finite; infinities and NaN count as zero)
 *   positions  int32 [B,L], or NULL: token t's position is t
 *   offsets    int32 [B] added to the positions, or NULL (decode: the tokens
 *              that each sequence already has)
 *   lengths    int32 [B], or NULL: tokens from lengths[b] on are neither read
 *              nor written
 *
 * Supported: even rotary_dim in 2..d, d and heads up to 16384, L up to 2^30.
 */
la_status la_rotary_fwd(const void *q, long long q_b_stride, long long q_h_stride,
                        long long q_t_stride, int heads_q, const void *k, long long k_b_stride,
                        long long k_h_stride, long long k_t_stride, int heads_k, int dtype, int B,
                        int L, int d, int rotary_dim, int interleaved, const float *inv_freq,
                        float scale, const int *positions, const int *offsets,
                        const int *lengths, void *q_out, long long qo_b_stride,
                        long long qo_h_stride, long long qo_t_stride, void *k_out,
                        long long ko_b_stride, long long ko_h_stride, long long ko_t_stride,
                        void *cuda_stream);
la_status la_rotary_bwd(const void *dq, long long q_b_stride, long long q_h_stride,
                        long long q_t_stride, int heads_q, const void *dk, long long k_b_stride,
                        long long k_h_stride, long long k_t_stride, int heads_k, int dtype, int B,
                        int L, int d, int rotary_dim, int interleaved, const float *inv_freq,
                        float scale, const int *positions, const int *offsets,
                        const int *lengths, void *dq_out, long long qo_b_stride,
                        long long qo_h_stride, long long qo_t_stride, void *dk_out,
                        long long ko_b_stride, long long ko_h_stride, long long ko_t_stride,
                        void *cuda_stream);

/*
 * Backward pass of la_chunk_fwd, of the same arguments: with S_t = a_t S_{t-1} +
 * phi(k_t) v_t^T, o_t = S_t^T phi(q_t) and G_t the gradient of S_t,
 *
 *     G_t = phi(q_t) do_t^T + a_{t+1} G_{t+1},     dphi(q)_t = S_t do_t,
 *     dphi(k)_t = G_t v_t,   dv_t = G_t^T phi(k_t),   dlog a_t = a_t <G_t, S_{t-1}>,
 *
 * and dq = dphi(q) phi'(q), dk likewise.
 *
 *   q, k, v, chunk, decay_kind, decay, S0   as the forward call had them (the
 *              result does not depend on chunk); phi is the one set by
 *              la_set_feature_map at this call
 *   dO         [B,H,L,d_v] dtype, the gradient of O
 *   dS_final   [B,H,d_k,d_v] fp32, the gradient of S_final, or NULL (zero)
 *   dq, dk, dv dtype, of the shapes of q, k and v
 *   ddecay     fp32 of decay's shape: the gradient of log gamma [H] (summed over
 *              the batch and the tokens), of log alpha or of the gate logit
 *              [B,H,L]; or NULL
 *   dS0        [B,H,d_k,d_v] fp32, the gradient of S0 (given or not), or NULL:
 *              a long sequence's pieces run back to front, each handing its
 *              dS0 on as the dS_final of the one before
 *   workspace  device scratch of la_chunk_bwd_workspace_bytes_for(...) bytes,
 *              which this call needs (with the feature map set now, its decay kind and
 *              whether ddecay and dS0 are wanted), or of la_chunk_bwd_workspace_bytes(...),
 *              enough for any of them
 *
 * With bf16 tensors, dq, dk and dv come from operands rounded once to bf16 (the
 * scores, the states, and the keys and queries times a decay), with fp32 sums and
 * states; phi's values of elu + 1 enter dq and dk with 16 bits.  They are 1.1 to 1.6 times as
 * far off as outputs rounded from fp32 (1.8e-3 to 2.6e-3 of their size, not 1.7e-3).  Where ddecay or dS0 is wanted those that they depend on keep fp32's
 * 24 bits, at about twice the work; with fp32 tensors all do.  ddecay adds up the pairs
 * that a token lies between, so that of a token that nearly resets the state, however
 * small beside its neighbours', is as exact as theirs.  A log decay below -200 counts as a
 * decay of zero.
 *
 * q, k, v, dO, dq, dk, dv and the states are 16-byte aligned, decays 4-byte.
 * Supported: d_k, d_v in {16, 32, 64, 128}, L up to 2^30.  L = 0 passes
 * dS_final through to dS0 (or zeroes it).
 */
la_status la_chunk_bwd(const void *q, const void *k, const void *v, int dtype, int B, int H,
                       int L, int d_k, int d_v, int chunk, int decay_kind, const float *decay,
                       const float *S0, const void *dO, const float *dS_final, void *dq, void *dk,
                       void *dv, float *ddecay, float *dS0, void *workspace, size_t ws_bytes,
                       void *cuda_stream);
size_t la_chunk_bwd_workspace_bytes(int B, int H, int L, int d_k, int d_v, int chunk, int dtype);
size_t la_chunk_bwd_workspace_bytes_for(int B, int H, int L, int d_k, int d_v, int chunk,
                                        int dtype, int decay_kind, int ddecay, int dS0);

/*
 * Backward pass of la_gated_norm_fwd, of the same arguments:
 *
 *   dy         [B,L,H*d] dtype, the gradient of y, rows dy_stride apart
 *   x, gate, weight, bias, weight_heads, norm, activation, gate_first, eps
 *              as the forward call had them
 *   dx         dtype, x's gradient, with strides like x's (its own: [B,H,L,d]
 *              goes to la_chunk_bwd as dO); may be x with x's strides
 *   dgate      [B,L,H*d] dtype, rows dgate_stride apart; given where gate is.
 *              May be gate's or dy's buffer with its stride.
 *   dweight, dbias  [weight_heads,d] fp32, or NULL
 *
 * Supported: d in 1..16384, H up to 65535.
 */
la_status la_gated_norm_bwd(const void *dy, long long dy_stride, const void *x,
                            long long x_b_stride, long long x_h_stride, long long x_t_stride,
                            const void *gate, long long gate_stride, int dtype, int B, int H,
                            int L, int d, int norm, int activation, int gate_first,
                            const float *weight, const float *bias, int weight_heads, float eps,
                            void *dx, long long dx_b_stride, long long dx_h_stride,
                            long long dx_t_stride, void *dgate, long long dgate_stride,
                            float *dweight, float *dbias, void *workspace, size_t ws_bytes,
                            void *cuda_stream);
size_t la_gated_norm_bwd_workspace_bytes(int B, int H, int L, int d, int weight_heads);

/*
 * Backward pass of la_residual_norm_fwd; without residual and post norm it is
 * that of a layer norm (or RMS norm) by itself.
 *
 *   dy            [rows,D] dtype, the gradient of y
 *   r             [rows,D] res_dtype, residual_out as the forward call wrote it
 *   dr            [rows,D] res_dtype, the gradient of residual_out, or NULL (zero)
 *   x             [rows,D] dtype, the forward call's x: needed where post_weight
 *                 or dscale is given, else not read
 *   dx            [rows,D] dtype, x's gradient; may be dy's or x's buffer
 *   dresidual     [rows,D] res_dtype, residual's gradient, or NULL; may be dr's
 *                 buffer
 *   dweight, dbias, dpost_weight, dscale   [D] fp32, each may be NULL
 *
 * Supported: D in 1..16384.
 */
la_status la_residual_norm_bwd(const void *dy, int dtype, const void *r, const void *dr,
                               int res_dtype, const void *x, long long rows, int D,
                               const float *post_weight, const float *scale, float alpha,
                               const float *weight, int norm, float eps, void *dx,
                               void *dresidual, float *dweight, float *dbias,
                               float *dpost_weight, float *dscale, void *workspace,
                               size_t ws_bytes, void *cuda_stream);
size_t la_residual_norm_bwd_workspace_bytes(long long rows, int D);

/*
 * la_chunk_fwd for callers that cannot allocate device memory.  (The pages
 * have no counterpart: this is a deployment variant of la_chunk_fwd.)
 *
 * Some callers cannot call cudaMalloc where they run prefill -- code inside
 * an allocator or memory-pool callback, processes whose device footprint is
 * fixed after start-up, or code that runs while another component holds the
 * allocator.  This entry point takes the same arguments as la_chunk_fwd
 * without the workspace: the segment states live in one static device array
 * of LA_NOALLOC_SCRATCH_BYTES, held on each GPU until the process exits.  It
 * calls no cudaMalloc, cudaFree or other allocating routine.
 *
 *   - When the bytes are reserved: the CUDA runtime loads modules lazily by
 *     default, so the array is placed on a device when it is first looked
 *     up there.  Call la_chunk_fwd_noalloc_prepare() once per device, with
 *     that device current, at start-up (before any stream capture and before
 *     the point where allocation is forbidden).  A device not prepared is
 *     prepared by its first la_chunk_fwd_noalloc call, which may then
 *     reserve the bytes itself.
 *   - The looked-up address is cached per device.  It does not survive
 *     cudaDeviceReset: call la_chunk_fwd_noalloc_prepare() again after one.
 *   - Problems whose workspace (la_chunk_fwd_workspace_bytes) exceeds
 *     LA_NOALLOC_SCRATCH_BYTES are rejected with LA_ERR_UNSUPPORTED before
 *     any device work; la_last_error() names both sizes.
 *   - Every call on a device shares the one array and leaves its contents
 *     behind.  Nothing in it has to start at zero (each call writes every
 *     part it reads before reading it), but calls whose kernels overlap on
 *     the GPU (different streams, or different host threads without
 *     ordering) race on it and give wrong results: order them.
 * Errors: as la_chunk_fwd, plus LA_ERR_UNSUPPORTED for a too-large problem.
 */
#define LA_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
la_status la_chunk_fwd_noalloc(const void *q, const void *k, const void *v, int dtype,
                               int B, int H, int L, int d_k, int d_v, int chunk,
                               int decay_kind, const float *decay,
                               const float *S0, void *O, float *S_final, void *cuda_stream);

/* Look up (again) the static scratch on the current device and cache its
 * address; under lazy module loading this is where the scratch is reserved.
 * LA_OK, or LA_ERR_CUDA with the runtime's message. */
la_status la_chunk_fwd_noalloc_prepare(void);

/* Size in bytes of the static scratch la_chunk_fwd_noalloc uses. */
size_t la_chunk_fwd_noalloc_scratch_bytes(void);

/* Synchronise `cuda_stream`, then report and clear the device error word that
 * kernels set when a bounded wait runs out: LA_OK, LA_ERR_DEVICE_TIMEOUT (the
 * message names the kernel and the wait) or LA_ERR_CUDA. */
la_status la_device_status(void *cuda_stream);

/* Self-test of the timeout path: launches one CTA that waits on an mbarrier
 * nothing ever arrives at, with a spin limit of `spin_limit` polls; the
 * kernel records the timeout, releases what it holds and exits.  Returns the
 * status la_device_status() then reports (LA_ERR_DEVICE_TIMEOUT expected). */
la_status la_selftest_wait_timeout(unsigned int spin_limit, void *cuda_stream);

/* Message for the last non-zero status on this thread ("" if none). */
const char *la_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* LA_GB300_H */
