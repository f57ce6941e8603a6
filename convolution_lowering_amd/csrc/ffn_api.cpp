// The C ABI of include/convlower_ffn.h: argument checks and launches.  Every
// check is on the host, before the first launch.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int64_t kMaxRows = (1LL << 31) - 1 - 256;

bool ffn_dtype_ok(conv_dtype_t d) { return d == CONV_DTYPE_FP32 || d == CONV_DTYPE_BF16 || d == CONV_DTYPE_FP16; }
size_t bytes_of(conv_dtype_t d) { return d == CONV_DTYPE_FP32 ? 4 : 2; }
bool act_ok(ffn_act_t a) {
    return a == FFN_ACT_NONE || a == FFN_ACT_SILU || a == FFN_ACT_SIGMOID || a == FFN_ACT_GELU;
}
// Whether every pointer of `must` is there and all are aligned to `es` bytes.
bool pointers_ok(std::initializer_list<const void *> must, std::initializer_list<const void *> may, size_t es) {
    for (const void *p : must)
        if (!p || (uintptr_t)p % es) return false;
    for (const void *p : may)
        if ((uintptr_t)p % es) return false;
    return true;
}
conv_status_t hip_status(hipError_t e) {
    return e == hipSuccess ? CONV_OK : e == kTooLarge ? CONV_ERR_UNSUPPORTED : CONV_ERR_HIP;
}

conv_status_t ffn_sizes(int64_t T, int D, int F, ffn_act_t act, int64_t stride) {
    if (T < 0 || D < 1 || F < 1 || !act_ok(act) || stride < D) return CONV_ERR_INVALID_ARG;
    if (T > kMaxRows || D > FFN_MAX_WIDTH || F > FFN_MAX_WIDTH || stride > FFN_MAX_WIDTH) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}
int64_t saved_pitch(int F) { return (F + 3) / 4 * 4; }

// The workspace of the backward pass holds the gradients of g and u, rows of whole
// 128-byte pieces, what fp16 keeps of their range, and then the parts' sums of either
// product.
int padded(int F, conv_dtype_t dtype) {
    const int piece = dtype == CONV_DTYPE_FP32 ? 32 : 64;
    return (F + piece - 1) / piece * piece;
}

size_t dgu_bytes(int64_t T, int F, conv_dtype_t dtype) { return (size_t)T * 2 * (size_t)padded(F, dtype) * bytes_of(dtype); }
size_t range_bytes(conv_dtype_t dtype) { return dtype == CONV_DTYPE_FP16 ? (kFfnRangeAt + kFfnRangeBlocks) * sizeof(float) : 0; }

conv_status_t w4_check(const void *x, int64_t x_stride, const void *y, int64_t R, int D, int F, int group,
                       conv_dtype_t dtype) {
    if (R < 0 || D < 1 || F < 1 || D % 8 || x_stride < D || !ffn_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    if (group != 32 && group != 64 && group != 128) return CONV_ERR_INVALID_ARG;
    if (R > kMaxRows || D > FFN_MAX_WIDTH || F > FFN_MAX_WIDTH || x_stride > FFN_MAX_WIDTH) return CONV_ERR_UNSUPPORTED;
    if (R && !pointers_ok({x, y}, {}, bytes_of(dtype))) return CONV_ERR_INVALID_ARG;
    return CONV_OK;
}
bool w4_weights_ok(const void *w, const void *scales, const void *zeros, conv_dtype_t dtype) {
    return pointers_ok({w}, {}, 4) && pointers_ok({scales}, {zeros}, bytes_of(dtype));
}

}  // namespace

// The time of a product is that of the blocks of one CU, one K tile after another.
// A block's K tile of 128 bytes takes, in microseconds (bf16, all CUs at work; 256 x
// 128 is the tile's rows of a by columns of each half of b):
//   256 x 128  1.15, one block on a CU at a time;
//   256 x 64   0.82;
//   128 x 64   0.62, two at once 1.00;
//   64 x 32    0.42, two 0.56, three 0.94;
//   32 x 32    0.27, two 0.34, three 0.45, four 0.60.
// (forward, 4096 to 10240 features: 512 tokens 80, 108, 101, 149, 198 us in this order, 200
// tokens 74, 55, 66, 72, 99, 128 tokens 71, 51, 46, 60, 67; 2048 to 4096: 400 tokens 38, 28,
// 20, 29, 32, 200 tokens 37, 27, 19, 16, 21, 64 tokens 35, 26, 18, 14, 11.)  float32 tiles
// take what their matrix instructions do, 16 times a 16-bit tile's 16 cycles each.  Rows
// at any address (64 x 32 only) wait for their way through registers: 2.0, two at
// once 2.1, three 2.4 (gradients of 768 tokens, 500 to 800 features: 77 us with the
// times of aligned rows, 42 with these).  A
// product that needs no second matrix (plain) may share its K tiles out to several
// grids, whose float32 sums are written, read and added by one more launch: 4 us and
// 8 bytes a value and grid at 4 TB/s.  (Both gradients' products of 200 tokens, 4096
// wide and 10240: 246 us in one grid of 64 x 32 each, 160 as chosen here.)
static const struct {
    int m, n;
    double at[4];  // of one, two, three, four blocks on a CU
    int most, threads;
} kTiles[] = {{256, 128, {1.15}, 1, 512},
              {256, 64, {0.82}, 1, 512},
              {128, 64, {0.62, 1.00}, 2, 512},
              {64, 32, {0.42, 0.56, 0.94}, 3, 256},
              {32, 32, {0.27, 0.34, 0.45, 0.60}, 4, 256}};
FfnPlan ffn_plan(int64_t M, int N, int K, int value_bytes, bool plain, bool vec, bool a_of_m) {
    const int per = 128 / value_bytes, nk = K ? (K - 1) / per + 1 : 1;
    FfnPlan best{FFN_TILE_64x32, 1};
    double least = 1e300;
    for (int t = vec ? 0 : 3; t < (vec && !a_of_m ? 5 : 4); ++t) {
        const int n = plain ? 2 * kTiles[t].n : kTiles[t].n;
        const double blocks = (double)((M + kTiles[t].m - 1) / kTiles[t].m) * ((N + n - 1) / n);
        for (int s = 1; s <= (plain ? 32 : 1) && (s == 1 || nk / s >= 4); ++s) {
            const double on = std::ceil(blocks * s / 256);  // blocks of a CU
            const int most = kTiles[t].most, rest = (int)std::fmod(on, most);
            static const double kAny[] = {2.0, 2.1, 2.4};
            const double *at = vec ? kTiles[t].at : kAny;
            double tile = (on - rest) / most * at[most - 1] + (rest ? at[rest - 1] : 0.0);
            if (value_bytes == 4 && vec) tile = on * kTiles[t].m * kTiles[t].n * 2 / 65536.0 * 7.2;
            double us = tile * ((nk + s - 1) / s + 2);
            if (s > 1) us += 4 + (double)s * M * ffn_part_pitch(N) * 8 / 4e6;
            if (us < least) least = us, best = {t, s};
        }
    }
    return best;
}

bool ffn_choose(FfnGemmArgs &a, int dtype, bool plain, bool a_of_m, bool b_of_m) {
    const int es = dtype == CONV_DTYPE_FP8_E4M3 ? 1 : (int)bytes_of((conv_dtype_t)dtype), V = 16 / es;
    a.vec = (a_of_m && b_of_m ? 0 : a.K) % V == 0 && (a_of_m ? a.M : 0) % V == 0 && (b_of_m ? a.N : 0) % V == 0 && a.as % V == 0 && a.bs % V == 0;
    for (const void *p : {a.a, a.b0, a.b1}) a.vec = a.vec && (uintptr_t)p % 16 == 0;
    const FfnPlan plan = ffn_plan(a.M, a.N, a.K, es, plain, a.vec, a_of_m);
    a.tile = plan.tile, a.splits = plan.splits;
    const auto &t = kTiles[plan.tile];
    const int n = plain ? 2 * t.n : t.n;
    return grid_fits(((a.M + t.m - 1) / t.m) * ((a.N + n - 1) / n), t.threads, a.splits);
}

hipError_t launch_ffn_gated_f32(const FfnGemmArgs &a, bool saving, hipStream_t st);
hipError_t launch_ffn_gated_bf16(const FfnGemmArgs &a, bool saving, hipStream_t st);
hipError_t launch_ffn_gated_f16(const FfnGemmArgs &a, bool saving, hipStream_t st);
hipError_t launch_ffn_gated_fp8(const FfnGemmArgs &a, int out_dtype, hipStream_t st);
hipError_t launch_ffn_dx_f32(const FfnGemmArgs &a, hipStream_t st);
hipError_t launch_ffn_dw_f32(const FfnGemmArgs &a, hipStream_t st);
hipError_t launch_ffn_dx_bf16(const FfnGemmArgs &a, hipStream_t st);
hipError_t launch_ffn_dw_bf16(const FfnGemmArgs &a, hipStream_t st);
hipError_t launch_ffn_dx_f16(const FfnGemmArgs &a, hipStream_t st);
hipError_t launch_ffn_dw_f16(const FfnGemmArgs &a, hipStream_t st);

hipError_t launch_ffn_gated(const FfnGemmArgs &a, FfnEpilogue e, int dtype, int out_dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP8_E4M3) return launch_ffn_gated_fp8(a, out_dtype, st);
    if (dtype == CONV_DTYPE_FP32) return launch_ffn_gated_f32(a, e == FFN_SAVING, st);
    if (dtype == CONV_DTYPE_FP16) return launch_ffn_gated_f16(a, e == FFN_SAVING, st);
    return launch_ffn_gated_bf16(a, e == FFN_SAVING, st);
}
hipError_t launch_ffn_dx(const FfnGemmArgs &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return launch_ffn_dx_f32(a, st);
    if (dtype == CONV_DTYPE_FP16) return launch_ffn_dx_f16(a, st);
    return launch_ffn_dx_bf16(a, st);
}
hipError_t launch_ffn_dw(const FfnGemmArgs &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return launch_ffn_dw_f32(a, st);
    if (dtype == CONV_DTYPE_FP16) return launch_ffn_dw_f16(a, st);
    return launch_ffn_dw_bf16(a, st);
}

}  // namespace convlower

using namespace convlower;

extern "C" {

conv_status_t gated_ffn_saved_size(int64_t T, int F, size_t *bytes_out) {
    if (!bytes_out || T < 0 || F < 1) return CONV_ERR_INVALID_ARG;
    if (T > kMaxRows || F > FFN_MAX_WIDTH) return CONV_ERR_UNSUPPORTED;
    *bytes_out = (size_t)T * 2 * (size_t)saved_pitch(F) * sizeof(float);
    return CONV_OK;
}

conv_status_t gated_ffn_fwd(const void *x, int64_t x_stride, const void *w_gate, const void *w_up, void *h, void *saved,
                            size_t saved_bytes, int64_t T, int D, int F, ffn_act_t act, conv_dtype_t dtype,
                            conv_stream_t stream) {
    if (!ffn_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    conv_status_t st = ffn_sizes(T, D, F, act, x_stride);
    if (st != CONV_OK) return st;
    size_t keep = 0;
    if ((st = gated_ffn_saved_size(T, F, &keep)) != CONV_OK) return st;
    if (!T) return CONV_OK;
    if (!pointers_ok({x, w_gate, w_up, h}, {}, bytes_of(dtype)) || (uintptr_t)saved % 16) return CONV_ERR_INVALID_ARG;
    if (saved && saved_bytes < keep) return CONV_ERR_WORKSPACE;
    FfnGemmArgs a{};
    a.a = x, a.b0 = w_gate, a.b1 = w_up, a.as = x_stride, a.bs = D, a.M = T, a.N = F, a.K = D, a.act = act, a.out = h;
    a.saved = (float *)saved, a.pitch = saved_pitch(F);
    if (!ffn_choose(a, dtype, false, false, false)) return CONV_ERR_UNSUPPORTED;
    return hip_status(launch_ffn_gated(a, saved ? FFN_SAVING : FFN_GATED, dtype, dtype, (hipStream_t)stream));
}

conv_status_t gated_ffn_bwd_workspace_size(int64_t T, int D, int F, conv_dtype_t dtype, size_t *bytes_out) {
    if (!bytes_out || !ffn_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    const conv_status_t st = ffn_sizes(T, D, F, FFN_ACT_NONE, D);
    if (st != CONV_OK) return st;
    const int es = (int)bytes_of(dtype), Fp = padded(F, dtype);
    size_t part = 0;
    for (int vec = 0; vec < 2; ++vec) {
        const int dx = ffn_plan(T, D, 2 * Fp, es, true, vec, false).splits, dw = ffn_plan(2 * (int64_t)Fp, D, (int)T, es, true, vec, true).splits;
        if (dx > 1) part = std::max(part, (size_t)dx * T * ffn_part_pitch(D) * 4);
        if (dw > 1) part = std::max(part, (size_t)dw * 2 * Fp * ffn_part_pitch(D) * 4);
    }
    *bytes_out = T ? dgu_bytes(T, F, dtype) + range_bytes(dtype) + part : 0;
    return CONV_OK;
}

conv_status_t gated_ffn_bwd_some(const void *dh, int64_t dh_stride, const void *x, int64_t x_stride,
                                 const void *w_gate, const void *w_up, const void *saved, size_t saved_bytes, void *dx,
                                 void *dw_gate, void *dw_up, int64_t T, int D, int F, ffn_act_t act,
                                 conv_dtype_t dtype, conv_stream_t stream, void *workspace, size_t workspace_bytes) {
    if (!ffn_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    conv_status_t st = ffn_sizes(T, D, F, act, x_stride);
    if (st != CONV_OK) return st;
    const size_t es = bytes_of(dtype);
    if (!pointers_ok({w_gate, w_up}, {dh, x, dx, dw_gate, dw_up}, es) || dh_stride < F) return CONV_ERR_INVALID_ARG;
    if ((T && (!dh || !x)) || !dw_gate != !dw_up) return CONV_ERR_INVALID_ARG;
    if (!pointers_ok({}, {saved, workspace}, 16)) return CONV_ERR_INVALID_ARG;
    if (dh_stride > FFN_MAX_WIDTH) return CONV_ERR_UNSUPPORTED;
    size_t need = 0, keep = 0;
    if ((st = gated_ffn_saved_size(T, F, &keep)) != CONV_OK) return st;
    if ((st = gated_ffn_bwd_workspace_size(T, D, F, dtype, &need)) != CONV_OK) return st;
    if (T && (!workspace || workspace_bytes < need || !saved || saved_bytes < keep)) return CONV_ERR_WORKSPACE;
    const int Fp = padded(F, dtype), piece = dtype == CONV_DTYPE_FP32 ? 32 : 64;
    FfnGateGrad d{};
    d.dh = dh, d.dhs = dh_stride, d.saved = (const float *)saved, d.pitch = saved_pitch(F), d.dgu = workspace;
    d.T = T, d.F = F, d.Fp = Fp, d.act = act;
    FfnGemmArgs a{};
    a.a = workspace, a.as = 2 * (int64_t)Fp, a.N = D;
    if (T) {
        char *rest = (char *)workspace + dgu_bytes(T, F, dtype);
        a.part = (float *)(rest + range_bytes(dtype));
        if (dtype == CONV_DTYPE_FP16) a.factor = d.range = (float *)rest;
    }
    // dx = [dg du] [w_gate; w_up]
    FfnGemmArgs x1 = a;
    x1.b0 = w_gate, x1.b1 = w_up, x1.bs = D, x1.M = T, x1.K = 2 * Fp, x1.ktsplit = Fp / piece, x1.brows = F;
    x1.out = dx, x1.split = T, x1.rows = T;
    // [dw_gate; dw_up] = [dg du]' x
    FfnGemmArgs w1 = a;
    w1.b0 = w1.b1 = x, w1.bs = x_stride, w1.M = 2 * (int64_t)Fp, w1.K = (int)T, w1.ktsplit = INT32_MAX, w1.brows = (int)T;
    w1.out = dw_gate, w1.out2 = dw_up, w1.split = Fp, w1.rows = F;
    const bool want_dx = T && dx, want_dw = dw_gate;
    if (want_dx && !ffn_choose(x1, dtype, true, false, true)) return CONV_ERR_UNSUPPORTED;
    if (want_dw && !ffn_choose(w1, dtype, true, true, true)) return CONV_ERR_UNSUPPORTED;
    if (!want_dx && !want_dw) return CONV_OK;
    hipError_t e = launch_ffn_gate_grad(d, dtype, (hipStream_t)stream);
    if (e == hipSuccess && want_dx) e = launch_ffn_dx(x1, dtype, (hipStream_t)stream);
    if (e == hipSuccess && want_dw) e = launch_ffn_dw(w1, dtype, (hipStream_t)stream);
    return hip_status(e);
}

conv_status_t gated_ffn_bwd(const void *dh, int64_t dh_stride, const void *x, int64_t x_stride, const void *w_gate,
                            const void *w_up, const void *saved, size_t saved_bytes, void *dx, void *dw_gate,
                            void *dw_up, int64_t T, int D, int F, ffn_act_t act, conv_dtype_t dtype,
                            conv_stream_t stream, void *workspace, size_t workspace_bytes) {
    if ((T && !dx) || !dw_gate || !dw_up) return CONV_ERR_INVALID_ARG;
    return gated_ffn_bwd_some(dh, dh_stride, x, x_stride, w_gate, w_up, saved, saved_bytes, dx, dw_gate, dw_up, T, D, F, act,
                              dtype, stream, workspace, workspace_bytes);
}

conv_status_t gated_ffn8_fwd(const void *x, int64_t x_stride, const float *x_scale, const void *w_gate,
                             const float *gate_scale, const void *w_up, const float *up_scale, void *h, int64_t T,
                             int D, int F, ffn_act_t act, conv_dtype_t dtype, conv_stream_t stream) {
    if (dtype != CONV_DTYPE_BF16 && dtype != CONV_DTYPE_FP16) return CONV_ERR_INVALID_ARG;
    const conv_status_t st = ffn_sizes(T, D, F, act, x_stride);
    if (st != CONV_OK) return st;
    if (!T) return CONV_OK;
    if (!x || !w_gate || !w_up || !pointers_ok({x_scale, gate_scale, up_scale}, {}, 4) || !pointers_ok({h}, {}, 2))
        return CONV_ERR_INVALID_ARG;
    FfnGemmArgs a{};
    a.a = x, a.b0 = w_gate, a.b1 = w_up, a.as = x_stride, a.bs = D, a.M = T, a.N = F, a.K = D, a.act = act, a.out = h;
    a.a_scale = x_scale, a.b0_scale = gate_scale, a.b1_scale = up_scale;
    if (!ffn_choose(a, CONV_DTYPE_FP8_E4M3, false, false, false)) return CONV_ERR_UNSUPPORTED;
    return hip_status(launch_ffn_gated(a, FFN_SCALED, CONV_DTYPE_FP8_E4M3, dtype, (hipStream_t)stream));
}

conv_status_t linear_w4_fwd(const void *x, int64_t x_stride, const void *w, const void *scales, const void *zeros,
                            void *y, int64_t R, int D, int F, int group, conv_dtype_t dtype, conv_stream_t stream) {
    const conv_status_t st = w4_check(x, x_stride, y, R, D, F, group, dtype);
    if (st != CONV_OK || !R) return st;
    if (!w4_weights_ok(w, scales, zeros, dtype)) return CONV_ERR_INVALID_ARG;
    W4Args a{};
    a.x = x, a.xs = x_stride, a.w[0] = (const uint8_t *)w, a.scales[0] = scales, a.y = y;
    a.has_zeros = zeros != nullptr, a.zeros[0] = zeros ? zeros : scales;
    a.R = R, a.D = D, a.F = F, a.groups = (D + group - 1) / group;
    return hip_status(launch_w4(a, group, false, dtype, (hipStream_t)stream));
}

conv_status_t gated_ffn_w4_fwd(const void *x, int64_t x_stride, const void *w_gate, const void *gate_scales,
                               const void *gate_zeros, const void *w_up, const void *up_scales, const void *up_zeros,
                               void *h, int64_t R, int D, int F, int group, ffn_act_t act, conv_dtype_t dtype,
                               conv_stream_t stream) {
    const conv_status_t st = w4_check(x, x_stride, h, R, D, F, group, dtype);
    if (st != CONV_OK) return st;
    if (!act_ok(act)) return CONV_ERR_INVALID_ARG;
    if (!R) return CONV_OK;
    if (!w4_weights_ok(w_gate, gate_scales, gate_zeros, dtype) || !w4_weights_ok(w_up, up_scales, up_zeros, dtype) ||
        (gate_zeros != nullptr) != (up_zeros != nullptr))
        return CONV_ERR_INVALID_ARG;
    W4Args a{};
    a.x = x, a.xs = x_stride, a.y = h, a.R = R, a.D = D, a.F = F, a.groups = (D + group - 1) / group, a.act = act;
    a.w[0] = (const uint8_t *)w_gate, a.scales[0] = gate_scales, a.w[1] = (const uint8_t *)w_up, a.scales[1] = up_scales;
    a.has_zeros = gate_zeros != nullptr;
    a.zeros[0] = gate_zeros ? gate_zeros : gate_scales, a.zeros[1] = up_zeros ? up_zeros : up_scales;
    return hip_status(launch_w4(a, group, true, dtype, (hipStream_t)stream));
}

conv_status_t norm_quant_fwd(const void *x, const void *res, const void *w, void *r, void *q, float *scale, int64_t R,
                             int D, float eps, conv_dtype_t dtype, conv_stream_t stream) {
    if (R < 0 || D < 1 || !ffn_dtype_ok(dtype) || !(eps >= 0.f)) return CONV_ERR_INVALID_ARG;
    if (D > FFN_MAX_NORM_WIDTH || R > kMaxRows) return CONV_ERR_UNSUPPORTED;
    if (!R) return CONV_OK;
    if (!pointers_ok({x, w}, {res, r}, bytes_of(dtype)) || !q || !pointers_ok({scale}, {}, 4) || (r && !res))
        return CONV_ERR_INVALID_ARG;
    NormQuantArgs a{};
    a.x = x, a.res = res, a.w = w, a.r = r, a.q = (uint8_t *)q, a.scale = scale, a.R = R, a.D = D, a.eps = eps;
    return hip_status(launch_norm_quant(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
