/*
 * convlower, feed-forward -- the other half of a language model's block, beside
 * the sequence mixing of convlower_mixer.h:
 *
 *   gated_ffn_*      both projections, the activation and the product in one
 *                    kernel, and its gradients;
 *   gated_ffn8_fwd   the same on 8-bit rows and weights with scales;
 *   gated_ffn_w4_fwd, linear_w4_fwd
 *                    the same, and one projection alone, for a few tokens on
 *                    4-bit weights with group scales;
 *   norm_quant_fwd   residual sum and norm that leave 8-bit rows with scales.
 *
 * The projection back to the model's width is a channels-last 1x1 layer
 * (conv2d_fwd), or linear_w4_fwd.  The conventions of convlower_mixer.h hold:
 * device pointers, caller-owned buffers that do not overlap, work enqueued on
 * `stream` without a synchronisation, status codes, nothing launched by a call
 * that fails on the host; *_stride arguments are in elements from one token to
 * the next, everything without one is dense.  Sums are fp32; each result is
 * rounded once, to nearest-even, but where a function says otherwise.  Any
 * sizes and addresses are taken; rows that lie at multiples of 16 bytes are
 * read fastest.
 */
#ifndef CONVLOWER_FFN_H
#define CONVLOWER_FFN_H

#include "convlower.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The activation of the gate: z, z s(z), s(z), and the tanh form of the
 * Gaussian one, z s(2 sqrt(2/pi) (z + 0.044715 z^3)); s(z) = 1 / (1 + e^-z). */
typedef enum { FFN_ACT_NONE = 0, FFN_ACT_SILU = 1, FFN_ACT_SIGMOID = 2, FFN_ACT_GELU = 3 } ffn_act_t;

/* Limits, above which a call returns CONV_ERR_UNSUPPORTED; so do more rows than
 * one launch has blocks for (products of 4 bits: some 2^20 to 2^22 rows, by what
 * is said there of the weights; the norm: 2^22 of the widest). */
#define FFN_MAX_WIDTH (1 << 20)  /* D, F and strides, in elements */
#define FFN_MAX_NORM_WIDTH 32768 /* row length of norm_quant_fwd */

/* ---- gated feed-forward product ------------------------------------------
 *   g = x w_gate',  u = x w_up',  h = act(g) * u
 * x [T][D] (x_stride), w_gate, w_up [F][D], h [T][F].  dtype: fp32, bf16 or
 * fp16 for all of them.  saved: NULL, or a buffer of the size that the query
 * gives, for gated_ffn_bwd: g and u in fp32. */
conv_status_t gated_ffn_saved_size(int64_t T, int F, size_t *bytes_out);
conv_status_t gated_ffn_fwd(const void *x, int64_t x_stride, const void *w_gate, const void *w_up, void *h, void *saved,
                            size_t saved_bytes, int64_t T, int D, int F, ffn_act_t act, conv_dtype_t dtype,
                            conv_stream_t stream);

/* Gradients of gated_ffn_fwd: dh [T][F] (dh_stride); dx [T][D], dw_gate, dw_up
 * [F][D], each overwritten.  The gradients of g and u are rounded to dtype
 * before the products with the weights and with x (fp16: times a power of two
 * that keeps the largest in range; what is below 2^-38 of it counts as zero).
 * Sums over tokens are added in a fixed order. */
conv_status_t gated_ffn_bwd_workspace_size(int64_t T, int D, int F, conv_dtype_t dtype, size_t *bytes_out);
conv_status_t gated_ffn_bwd(const void *dh, int64_t dh_stride, const void *x, int64_t x_stride, const void *w_gate,
                            const void *w_up, const void *saved, size_t saved_bytes, void *dx, void *dw_gate,
                            void *dw_up, int64_t T, int D, int F, ffn_act_t act, conv_dtype_t dtype,
                            conv_stream_t stream, void *workspace, size_t workspace_bytes);
/* The same for frozen weights or an input without a gradient: dx, or dw_gate
 * and dw_up together, may be NULL, and their product is left out. */
conv_status_t gated_ffn_bwd_some(const void *dh, int64_t dh_stride, const void *x, int64_t x_stride,
                                 const void *w_gate, const void *w_up, const void *saved, size_t saved_bytes, void *dx,
                                 void *dw_gate, void *dw_up, int64_t T, int D, int F, ffn_act_t act,
                                 conv_dtype_t dtype, conv_stream_t stream, void *workspace, size_t workspace_bytes);

/* The product on 8 bits: x [T][D] (x_stride), w_gate and w_up [F][D] are e4m3
 * (CONV_DTYPE_FP8_E4M3); a value stands for itself times its row's scale,
 * x_scale [T], gate_scale [F], up_scale [F] (fp32).  h [T][F]: bf16 or fp16
 * (dtype). */
conv_status_t gated_ffn8_fwd(const void *x, int64_t x_stride, const float *x_scale, const void *w_gate,
                             const float *gate_scale, const void *w_up, const float *up_scale, void *h, int64_t T,
                             int D, int F, ffn_act_t act, conv_dtype_t dtype, conv_stream_t stream);

/* ---- products with 4-bit weights -----------------------------------------
 *   y[r,f] = sum_d x[r,d] scales[f, d / group] (code[f,d] - zeros[f, d / group])
 * x [R][D] (x_stride), D a multiple of 8; w [F][D/2] bytes, at a multiple of 4,
 * each with the codes (0..15) of two neighbours, the earlier one in the low half;
 * scales and zeros [F][ceil(D / group)] in dtype, zeros NULL: 8; group 32, 64 or
 * 128; y [R][F].  Made for a few tokens: each 64 take the weights again (gated
 * groups of 32: each 32; float32, and 16-bit rows at odd multiples of 2 bytes:
 * each 16).  A row of x that holds an infinity or a NaN gives NaN; finite ones do not
 * overflow where y does not, but for bf16 and fp32 zero points past 384. */
conv_status_t linear_w4_fwd(const void *x, int64_t x_stride, const void *w, const void *scales, const void *zeros,
                            void *y, int64_t R, int D, int F, int group, conv_dtype_t dtype, conv_stream_t stream);

/* h = act(g) * u of two such products; zeros for both or for neither. */
conv_status_t gated_ffn_w4_fwd(const void *x, int64_t x_stride, const void *w_gate, const void *gate_scales,
                               const void *gate_zeros, const void *w_up, const void *up_scales, const void *up_zeros,
                               void *h, int64_t R, int D, int F, int group, ffn_act_t act, conv_dtype_t dtype,
                               conv_stream_t stream);

/* ---- norm with an 8-bit result -------------------------------------------
 *   r = x + res,  n = r / sqrt(mean(r^2) + eps) * w
 *   scale = max(max |n|, 2^-100) / 448,  q = e4m3(n / scale)
 * on R rows of D.  res NULL: r = x, and r (the output) must be NULL; otherwise
 * r [R][D], which is x + res rounded, may be NULL if not wanted.  The norm
 * takes the sum before it is rounded.  q [R][D] e4m3, scale [R] fp32.  A row
 * with an infinity or a NaN, or whose squares add up past the largest fp32
 * number, has a NaN scale, and all its q are NaN. */
conv_status_t norm_quant_fwd(const void *x, const void *res, const void *w, void *r, void *q, float *scale, int64_t R,
                             int D, float eps, conv_dtype_t dtype, conv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CONVLOWER_FFN_H */
