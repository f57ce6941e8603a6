/*
 * convlower, sequence mixing -- the operators a language model's recurrent
 * mixer needs beside its dense projections (which conv2d_fwd computes as
 * channels-last 1x1 layers):
 *
 *   conv1d_causal_*  a short depthwise causal convolution along each sequence;
 *   delta_rule_*     the gated delta rule, in chunks for prompts and training,
 *                    token by token for generation;
 *   branch_norm_*    the end of a block: norm of the branch, gate, scaled
 *                    residual sum and the next block's norm.
 *
 * Conventions shared by every entry point (beyond those of convlower.h:
 * device pointers, caller-owned buffers that do not overlap, work enqueued on
 * `stream` without a synchronisation, status codes, nothing launched by a
 * call that fails on the host)
 * ---------------------------------------------------------------------------
 * Sequences  Tokens of all sequences lie one after another in one packed
 *   axis of T tokens.  cu_seqlens is a device array of N + 1 int32 values,
 *   cu_seqlens[0] = 0 <= ... <= cu_seqlens[N] = T; sequence n is the tokens
 *   [cu_seqlens[n], cu_seqlens[n+1]), possibly none.  NULL: N sequences of
 *   T / N tokens each (T a multiple of N).  Other values give undefined
 *   results, but no access outside the caller's buffers.
 * Strides    *_stride arguments are in elements, from one token to the next;
 *   the last axis is dense, and the heads of a token lie one after another
 *   (head h at h * head_size).  Buffers without a stride are dense.
 * Dtype      CONV_DTYPE_FP32, _BF16 or _FP16 for every tensor not said to be
 *   fp32.  Sums, states and statistics are fp32; each result is rounded once,
 *   to nearest-even.  The chunked delta rule multiplies operands of 22 bits
 *   (see there).
 */
#ifndef CONVLOWER_MIXER_H
#define CONVLOWER_MIXER_H

#include "convlower.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MIX_ACT_NONE = 0, MIX_ACT_SILU = 1, MIX_ACT_SIGMOID = 2 } mix_act_t;

/* Limits, above which a call returns CONV_ERR_UNSUPPORTED; so do more tokens,
 * rows, requests or channels than one launch has threads for (2^32: some 2^30
 * tokens of a convolution, 2^28 rows of up to 128 16-bit values of a norm). */
#define MIX_CONV1D_MAX_WIDTH 8   /* taps of conv1d_causal_* */
#define MIX_DELTA_MAX_DK 128     /* key head size of delta_rule_* */
#define MIX_DELTA_MAX_DV 256     /* value head size of delta_rule_* */
#define MIX_DELTA_MAX_STRIDE (1 << 22) /* token stride of v, o and d_o of delta_rule_fwd and _bwd, in elements */
#define MIX_NORM_MAX_WIDTH 32768 /* row length of branch_norm_* */

/* ---- causal convolution --------------------------------------------------
 *   z[t,c] = bias[c] + sum_{j < W} w[c,j] * x[t - (W-1) + j, c],  y = act(z)
 * within each sequence; in place of what lies before a sequence's first token
 * stands its state, the W-1 inputs before it ([N][W-1][D], oldest first), or
 * zeros without one.  act: MIX_ACT_NONE or MIX_ACT_SILU.
 *   x [T][D] (x_stride), w [D][W], bias [D] or NULL, state or NULL,
 *   y [T][D], state_out [N][W-1][D] or NULL: the last W-1 inputs of each
 *   sequence, its state included. */
conv_status_t conv1d_causal_fwd(const void *x, int64_t x_stride, const void *w, const void *bias, const void *state,
                                const int32_t *cu_seqlens, void *y, void *state_out, int64_t T, int N, int D, int W,
                                mix_act_t act, conv_dtype_t dtype, conv_stream_t stream);

/* Gradients of conv1d_causal_fwd.  dy [T][D] (dy_stride); dstate_out: the
 * gradient of state_out, or NULL for none.  dx [T][D], dw [D][W], dbias [D]
 * (NULL without a bias), dstate [N][W-1][D] (NULL: not wanted); each is
 * overwritten.  The sums over tokens are added in a fixed order. */
conv_status_t conv1d_causal_bwd_workspace_size(int64_t T, int N, int D, int W, size_t *bytes_out);
conv_status_t conv1d_causal_bwd(const void *dy, int64_t dy_stride, const void *dstate_out, const void *x,
                                int64_t x_stride, const void *w, const void *bias, const void *state,
                                const int32_t *cu_seqlens, void *dx, void *dw, void *dbias, void *dstate, int64_t T,
                                int N, int D, int W, mix_act_t act, conv_dtype_t dtype, conv_stream_t stream,
                                void *workspace, size_t workspace_bytes);

/* One token for each of R requests: x [R][D] (x_stride), y [R][D].  Request r
 * keeps its last W-1 inputs in pool[slots[r]] (pool [P][W-1][D]; slots NULL:
 * r), which is read and moved on by one.  A slot outside [0, P) is a padding
 * request: its y is zero and no state changes.  The slots in use differ. */
conv_status_t conv1d_causal_step(const void *x, int64_t x_stride, const void *w, const void *bias, void *pool,
                                 const int32_t *slots, void *y, int R, int P, int D, int W, mix_act_t act,
                                 conv_dtype_t dtype, conv_stream_t stream);

/* ---- gated delta rule ----------------------------------------------------
 * Per value head a state S [dk][dv] (fp32), and for each token
 *   S <- exp(g) S;  u = beta (v - S'k);  S <- S + k u';  o = scale * S'q
 * with q, k [T][Hk][dk], v, o [T][Hv][dv], g [T][Hv] fp32 (log decay, <= 0;
 * -inf clears the state), beta [T][Hv] (beta_dtype: `dtype` or
 * CONV_DTYPE_FP32).  Value head h reads query/key head h / (Hv / Hk); Hv is a
 * multiple of Hk.  qk_norm: q and k are first divided by
 * sqrt(sum of squares + 1e-6).  state, state_out [N][Hv][dk][dv] fp32, NULL:
 * starts at zero / not wanted.
 *
 * delta_rule_fwd works on chunks of 64 tokens.  saved: NULL, or a buffer of
 * saved_bytes (from the size query) that delta_rule_bwd of the same inputs
 * takes.
 *
 * Digits     The chunked form's products take their operands in two halves, 22
 *   bits: q, k and what is made of them (16-bit q and k are exact), v - S'k, u,
 *   d_o, the state, and the states and gradients that are saved.  They are
 *   added up in fp32, and the state that is carried is fp32.  Float32 results
 *   are off by less than 1e-6 of the norm of a head; a value keeps all 22 bits
 *   while it is not below 2^-17 of the largest of its column in the chunk.
 *   The decays' gradients are sums in which large terms cancel: their error is
 *   relative to the terms.  The token form is fp32 throughout.
 * Infinities and NaN in a token's inputs may reach the chunk's tokens before
 *   it as well; never another sequence, nor, but through q and k, another head. */
conv_status_t delta_rule_fwd_workspace_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                            size_t *bytes_out);
conv_status_t delta_rule_saved_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                    size_t *bytes_out);
conv_status_t delta_rule_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const float *g, const void *beta, const float *state,
                             const int32_t *cu_seqlens, void *o, float *state_out, int64_t T, int N, int Hk, int Hv,
                             int dk, int dv, float scale, int qk_norm, conv_dtype_t dtype, conv_dtype_t beta_dtype,
                             conv_stream_t stream, void *workspace, size_t workspace_bytes, void *saved,
                             size_t saved_bytes);

/* Gradients of delta_rule_fwd.  d_o [T][Hv][dv] (do_stride); dstate_out: the
 * gradient of state_out, or NULL.  dq, dk_out, dv_out, dg (fp32) and dbeta
 * are shaped like q, k, v, g and beta, dense; dstate [N][Hv][dk][dv] fp32 or
 * NULL.  Heads of q and k that several value heads share get the sum, added
 * in a fixed order. */
conv_status_t delta_rule_bwd_workspace_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                            size_t *bytes_out);
conv_status_t delta_rule_bwd(const void *d_o, int64_t do_stride, const float *dstate_out, const void *q,
                             int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             const float *g, const void *beta, const int32_t *cu_seqlens, const void *saved,
                             size_t saved_bytes, void *dq, void *dk_out, void *dv_out, float *dg, void *dbeta,
                             float *dstate, int64_t T, int N, int Hk, int Hv, int dk, int dv, float scale,
                             int qk_norm, conv_dtype_t dtype, conv_dtype_t beta_dtype, conv_stream_t stream,
                             void *workspace, size_t workspace_bytes);

/* L tokens (one, or a few drafted ones) for each of R requests, one after
 * another: q, k, v, g, beta and o as above with T = R * L, request r the
 * tokens [r L, (r+1) L).  Its state is pool[slots[r]] (pool
 * [P][Hv][dk][dv] fp32; slots NULL: r), updated in place.  Slots as for
 * conv1d_causal_step. */
conv_status_t delta_rule_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const float *g, const void *beta, float *pool, const int32_t *slots,
                              void *o, int R, int L, int P, int Hk, int Hv, int dk, int dv, float scale, int qk_norm,
                              conv_dtype_t dtype, conv_dtype_t beta_dtype, conv_stream_t stream);

/* ---- branch norm ---------------------------------------------------------
 *   u = y / sqrt(mean(y^2) + eps) * w_post
 *   r = x + alpha * act(gate) * u
 *   h = r / sqrt(mean(r^2) + eps) * w_next
 * on R rows of D.  x NULL: nothing is added; gate NULL: 1; w_next NULL: no h
 * (h NULL).  gate [G][D] with G = R (one per row), 1 (one for all) or a
 * divisor of R (row i takes gate row i / (R / G)).  stats (fp32 [2][R], NULL:
 * not wanted): 1 / sqrt of both means, for branch_norm_bwd. */
conv_status_t branch_norm_fwd(const void *x, const void *y, const void *w_post, const void *gate, const void *w_next,
                              void *r, void *h, float *stats, int64_t R, int D, int64_t G, float alpha, float eps,
                              mix_act_t act, conv_dtype_t dtype, conv_stream_t stream);

/* Gradients of branch_norm_fwd: dr [R][D] (NULL: zero), dh [R][D] (NULL:
 * zero); dx [R][D], dy [R][D], dw_post [D], dgate [G][D], dw_next [D]; those
 * of absent inputs are NULL.  The sums over rows are added in a fixed order. */
conv_status_t branch_norm_bwd_workspace_size(int64_t R, int D, int64_t G, size_t *bytes_out);
conv_status_t branch_norm_bwd(const void *dr, const void *dh, const void *x, const void *y, const void *w_post,
                              const void *gate, const void *w_next, const float *stats, void *dx, void *dy,
                              void *dw_post, void *dgate, void *dw_next, int64_t R, int D, int64_t G, float alpha,
                              float eps, mix_act_t act, conv_dtype_t dtype, conv_stream_t stream, void *workspace,
                              size_t workspace_bytes);

#ifdef __cplusplus
}
#endif

#endif /* CONVLOWER_MIXER_H */
