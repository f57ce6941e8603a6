// The C ABI of include/convlower_mixer.h: argument checks and launches.
// Every check is on the host, before the first launch.
#include <initializer_list>

#include "delta_chunk.h"

namespace convlower {
namespace {

constexpr int64_t kMaxTokens = (1LL << 31) - 1 - 256;
constexpr int kMaxChannels = 1 << 24;

bool mix_dtype_ok(conv_dtype_t d) { return d == CONV_DTYPE_FP32 || d == CONV_DTYPE_BF16 || d == CONV_DTYPE_FP16; }
size_t bytes_of(conv_dtype_t d) { return d == CONV_DTYPE_FP32 ? 4 : 2; }

// Whether every pointer of `must` is there and all are aligned to `es` bytes.
bool pointers_ok(std::initializer_list<const void *> must, std::initializer_list<const void *> may, size_t es) {
    for (const void *p : must)
        if (!p || (uintptr_t)p % es) return false;
    for (const void *p : may)
        if ((uintptr_t)p % es) return false;
    return true;
}

// Sequences of a packed axis: T tokens, N sequences.
conv_status_t seqs_of(const int32_t *cu, int64_t T, int N, Seqs *s) {
    if (T < 0 || N < 1 || (uintptr_t)cu % 4) return CONV_ERR_INVALID_ARG;
    if (!cu && T % N) return CONV_ERR_INVALID_ARG;
    if (T > kMaxTokens) return CONV_ERR_UNSUPPORTED;
    *s = Seqs{cu, T, N, cu ? 0 : T / N};
    return CONV_OK;
}

conv_status_t conv1d_sizes(int D, int W, mix_act_t act, conv_dtype_t dtype) {
    if (D < 1 || W < 1 || !mix_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    if (act != MIX_ACT_NONE && act != MIX_ACT_SILU) return CONV_ERR_INVALID_ARG;
    if (W > MIX_CONV1D_MAX_WIDTH || D > kMaxChannels) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

conv_status_t delta_sizes(int Hk, int Hv, int dk, int dv, conv_dtype_t dtype, conv_dtype_t beta_dtype) {
    if (Hk < 1 || Hv < 1 || dk < 1 || dv < 1 || Hv % Hk || !mix_dtype_ok(dtype)) return CONV_ERR_INVALID_ARG;
    if (beta_dtype != dtype && beta_dtype != CONV_DTYPE_FP32) return CONV_ERR_INVALID_ARG;
    if (dk > MIX_DELTA_MAX_DK || dv > MIX_DELTA_MAX_DV || Hv > 65535) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

conv_status_t norm_sizes(int64_t R, int D, int64_t G, bool gate, float eps, mix_act_t act, conv_dtype_t dtype) {
    if (R < 0 || D < 1 || !mix_dtype_ok(dtype) || !(eps >= 0.f)) return CONV_ERR_INVALID_ARG;
    if (act != MIX_ACT_NONE && act != MIX_ACT_SILU && act != MIX_ACT_SIGMOID) return CONV_ERR_INVALID_ARG;
    // (no rows: a gate of as many, or one that rows would share)
    if (gate && (G < 0 || (R ? !G || G > R || R % G : false))) return CONV_ERR_INVALID_ARG;
    if (D > MIX_NORM_MAX_WIDTH || R > kMaxTokens || (gate && G != R && G > 60000)) return CONV_ERR_UNSUPPORTED;
    return CONV_OK;
}

// Checks and fills in what delta_rule_fwd and _bwd share.
conv_status_t delta_inputs(const void *q, int64_t qs, const void *k, int64_t ks, const void *v, int64_t vs,
                           const float *g, const void *beta, const int32_t *cu, int64_t T, int N, int Hk, int Hv,
                           int dk, int dv, float scale, int qk_norm, conv_dtype_t dtype, conv_dtype_t beta_dtype,
                           DeltaArgs *a) {
    conv_status_t st = delta_sizes(Hk, Hv, dk, dv, dtype, beta_dtype);
    if (st != CONV_OK) return st;
    if ((st = seqs_of(cu, T, N, &a->s)) != CONV_OK) return st;
    if (T && (!q || !k || !v || !g || !beta)) return CONV_ERR_INVALID_ARG;
    if (!pointers_ok({}, {q, k, v}, bytes_of(dtype)) || !pointers_ok({}, {beta}, bytes_of(beta_dtype)) ||
        !pointers_ok({}, {g}, 4))
        return CONV_ERR_INVALID_ARG;
    if (qs < (int64_t)Hk * dk || ks < (int64_t)Hk * dk || vs < (int64_t)Hv * dv) return CONV_ERR_INVALID_ARG;
    // a chunk's 64 tokens are addressed by 32-bit byte offsets
    if (vs > MIX_DELTA_MAX_STRIDE || (int64_t)Hv * dv > MIX_DELTA_MAX_STRIDE) return CONV_ERR_UNSUPPORTED;
    a->q = q, a->qs = qs, a->k = k, a->ks = ks, a->v = v, a->vs = vs, a->g = g, a->beta = beta;
    a->Hk = Hk, a->Hv = Hv, a->dk = dk, a->dv = dv, a->qk_norm = qk_norm != 0, a->scale = scale;
    a->beta_f32 = beta_dtype == CONV_DTYPE_FP32;
    return CONV_OK;
}

// The buffers of the chunked form: PART_FWD and PART_BWD are workspaces (that
// of a forward call which saves is a part of PART_FWD), PART_SAVED goes from
// the forward call to the backward one.
enum Part { PART_FWD, PART_FWD_SAVING, PART_BWD, PART_SAVED };

DeltaBuf delta_buf(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype) {
    DeltaBuf b{};
    b.slots = (int)(T / kC + N);
    b.dkp = dk <= 64 ? 64 : 128;
    b.dvp = (dv + kSlab - 1) / kSlab * kSlab;
    b.planes = dtype == CONV_DTYPE_FP32 ? 2 : 1;
    return b;
}
// Gives b its part of the buffer at p; returns the bytes (p null: only that).
size_t lay_out(DeltaBuf *b, int Hk, int Hv, Part part, void *p) {
    size_t at = 0;
    auto take = [&](size_t values, size_t each) {
        void *r = p ? (char *)p + at : nullptr;
        at += (values * each + 255) / 256 * 256;
        return r;
    };
    const size_t kh = (size_t)b->slots * Hk, vh = (size_t)b->slots * Hv;
    const size_t state = vh * b->dkp * b->dvp, tokens = vh * kC * b->dvp, tiles = vh * (b->dvp / 16);
    const size_t kq = kh * 2 * b->planes * kC * b->dkp;
    if (part == PART_BWD) {
        b->G = (float *)take(state, 4);
        b->E = (float *)take(tokens, 4);
        b->Gmax = (float *)take(tiles, 4);
        return at;
    }
    if (part == PART_FWD || part == PART_FWD_SAVING) b->tp = (char *)take(vh, kTpBytes);
    if (part == PART_FWD || part == PART_SAVED) b->kq = (_Float16 *)take(kq, 2);
    if (part == PART_SAVED) {
        b->tpg = (char *)take(vh, kTpBytes);
        b->rowk = (float *)take(kh * 4 * kC, 4);
        b->gam = (double *)take(vh * kC, 8);
        b->S = (float *)take(state, 4);
        b->Y = (float *)take(tokens, 4);
        b->Smax = (float *)take(tiles, 4);
    }
    return at;
}
conv_status_t delta_bytes(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype, Part part,
                          size_t *bytes_out) {
    if (!bytes_out || T < 0 || N < 1) return CONV_ERR_INVALID_ARG;
    const conv_status_t st = delta_sizes(Hk, Hv, dk, dv, dtype, dtype);
    if (st != CONV_OK) return st;
    // blocks are counted in 32 bits
    if (T > kMaxTokens || T / kC + N > kMaxTokens || (int64_t)N * Hv * (MIX_DELTA_MAX_DV / 16) > kMaxTokens)
        return CONV_ERR_UNSUPPORTED;
    DeltaBuf b = delta_buf(T, N, Hk, Hv, dk, dv, dtype);
    *bytes_out = lay_out(&b, Hk, Hv, part, nullptr);
    return CONV_OK;
}

conv_status_t hip_status(hipError_t e) {
    return e == hipSuccess ? CONV_OK : e == kTooLarge ? CONV_ERR_UNSUPPORTED : CONV_ERR_HIP;
}

}  // namespace
}  // namespace convlower

using namespace convlower;

extern "C" {

conv_status_t conv1d_causal_fwd(const void *x, int64_t x_stride, const void *w, const void *bias, const void *state,
                                const int32_t *cu_seqlens, void *y, void *state_out, int64_t T, int N, int D, int W,
                                mix_act_t act, conv_dtype_t dtype, conv_stream_t stream) {
    conv_status_t st = conv1d_sizes(D, W, act, dtype);
    if (st != CONV_OK) return st;
    Conv1dArgs a{};
    if ((st = seqs_of(cu_seqlens, T, N, &a.s)) != CONV_OK) return st;
    const size_t es = bytes_of(dtype);
    if (x_stride < D || !pointers_ok({w}, {x, bias, state, y, state_out}, es)) return CONV_ERR_INVALID_ARG;
    if (T && (!x || !y)) return CONV_ERR_INVALID_ARG;
    a.x = x, a.xs = x_stride, a.w = w, a.bias = bias, a.state = state, a.y = y, a.state_out = state_out;
    a.D = D, a.W = W, a.act = act;
    return hip_status(launch_conv1d_fwd(a, dtype, (hipStream_t)stream));
}

conv_status_t conv1d_causal_bwd_workspace_size(int64_t T, int N, int D, int W, size_t *bytes_out) {
    if (!bytes_out || T < 0 || N < 1) return CONV_ERR_INVALID_ARG;
    const conv_status_t st = conv1d_sizes(D, W, MIX_ACT_NONE, CONV_DTYPE_FP32);
    if (st != CONV_OK) return st;
    if (T > kMaxTokens) return CONV_ERR_UNSUPPORTED;
    const int64_t tokens = (int64_t)conv1d_bwd_tile(T, D) * kConvRuns;
    *bytes_out = (size_t)((T + tokens - 1) / tokens) * (W + 1) * D * sizeof(float);
    return CONV_OK;
}

conv_status_t conv1d_causal_bwd(const void *dy, int64_t dy_stride, const void *dstate_out, const void *x,
                                int64_t x_stride, const void *w, const void *bias, const void *state,
                                const int32_t *cu_seqlens, void *dx, void *dw, void *dbias, void *dstate, int64_t T,
                                int N, int D, int W, mix_act_t act, conv_dtype_t dtype, conv_stream_t stream,
                                void *workspace, size_t workspace_bytes) {
    conv_status_t st = conv1d_sizes(D, W, act, dtype);
    if (st != CONV_OK) return st;
    Conv1dArgs a{};
    if ((st = seqs_of(cu_seqlens, T, N, &a.s)) != CONV_OK) return st;
    const size_t es = bytes_of(dtype);
    if (x_stride < D || dy_stride < D || !pointers_ok({w, dw}, {x, dy, bias, dbias, state, dstate, dstate_out, dx}, es))
        return CONV_ERR_INVALID_ARG;
    if ((T && (!x || !dy || !dx)) || (!bias && dbias) || (uintptr_t)workspace % 16) return CONV_ERR_INVALID_ARG;
    size_t need = 0;
    if ((st = conv1d_causal_bwd_workspace_size(T, N, D, W, &need)) != CONV_OK) return st;
    if (need && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    a.x = x, a.xs = x_stride, a.dy = dy, a.dys = dy_stride, a.w = w, a.bias = bias, a.state = state;
    a.dstate_out = W > 1 ? dstate_out : nullptr, a.dx = dx, a.dw = dw, a.dbias = dbias, a.dstate = dstate;
    a.part = (float *)workspace, a.D = D, a.W = W, a.act = act;
    return hip_status(launch_conv1d_bwd(a, dtype, (hipStream_t)stream));
}

conv_status_t conv1d_causal_step(const void *x, int64_t x_stride, const void *w, const void *bias, void *pool,
                                 const int32_t *slots, void *y, int R, int P, int D, int W, mix_act_t act,
                                 conv_dtype_t dtype, conv_stream_t stream) {
    const conv_status_t st = conv1d_sizes(D, W, act, dtype);
    if (st != CONV_OK) return st;
    if (R < 0 || P < 0 || (!slots && R > P)) return CONV_ERR_INVALID_ARG;
    if (!R) return CONV_OK;
    if (x_stride < D || !pointers_ok({x, w, y}, {bias, pool}, bytes_of(dtype)) || (uintptr_t)slots % 4)
        return CONV_ERR_INVALID_ARG;
    if (!pool && W > 1 && P) return CONV_ERR_INVALID_ARG;
    return hip_status(launch_conv1d_step(x, x_stride, w, bias, pool, slots, y, R, P, D, W, act, dtype,
                                         (hipStream_t)stream));
}

conv_status_t delta_rule_step(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                              int64_t v_stride, const float *g, const void *beta, float *pool, const int32_t *slots,
                              void *o, int R, int L, int P, int Hk, int Hv, int dk, int dv, float scale, int qk_norm,
                              conv_dtype_t dtype, conv_dtype_t beta_dtype, conv_stream_t stream) {
    const conv_status_t st = delta_sizes(Hk, Hv, dk, dv, dtype, beta_dtype);
    if (st != CONV_OK) return st;
    if (R < 0 || L < 0 || P < 0 || (!slots && R > P)) return CONV_ERR_INVALID_ARG;
    // one wavefront for 32 columns, threads counted in 32 bits
    if ((int64_t)R * L > kMaxTokens || (int64_t)R * Hv > kMaxTokens ||
        (int64_t)R * Hv * ((dv + 31) / 32) > kMaxTokens / 64)
        return CONV_ERR_UNSUPPORTED;
    if (!R || !L) return CONV_OK;
    if (!pointers_ok({q, k, v, o}, {}, bytes_of(dtype)) || !pointers_ok({beta}, {}, bytes_of(beta_dtype)) ||
        !pointers_ok({g, pool}, {slots}, 4))
        return CONV_ERR_INVALID_ARG;
    if (q_stride < (int64_t)Hk * dk || k_stride < (int64_t)Hk * dk || v_stride < (int64_t)Hv * dv)
        return CONV_ERR_INVALID_ARG;
    DeltaArgs a{};
    a.q = q, a.qs = q_stride, a.k = k, a.ks = k_stride, a.v = v, a.vs = v_stride, a.g = g, a.beta = beta, a.o = o;
    a.pool = pool, a.slots = slots, a.R = R, a.L = L, a.P = P;
    a.Hk = Hk, a.Hv = Hv, a.dk = dk, a.dv = dv, a.qk_norm = qk_norm != 0, a.scale = scale;
    a.beta_f32 = beta_dtype == CONV_DTYPE_FP32;
    return hip_status(launch_delta_tokens(a, dtype, (hipStream_t)stream));
}

conv_status_t delta_rule_fwd_workspace_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                            size_t *bytes_out) {
    return delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_FWD, bytes_out);
}

conv_status_t delta_rule_saved_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                    size_t *bytes_out) {
    return delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_SAVED, bytes_out);
}

conv_status_t delta_rule_bwd_workspace_size(int64_t T, int N, int Hk, int Hv, int dk, int dv, conv_dtype_t dtype,
                                            size_t *bytes_out) {
    return delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_BWD, bytes_out);
}

conv_status_t delta_rule_fwd(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const float *g, const void *beta, const float *state,
                             const int32_t *cu_seqlens, void *o, float *state_out, int64_t T, int N, int Hk, int Hv,
                             int dk, int dv, float scale, int qk_norm, conv_dtype_t dtype, conv_dtype_t beta_dtype,
                             conv_stream_t stream, void *workspace, size_t workspace_bytes, void *saved,
                             size_t saved_bytes) {
    DeltaArgs a{};
    conv_status_t st = delta_inputs(q, q_stride, k, k_stride, v, v_stride, g, beta, cu_seqlens, T, N, Hk, Hv, dk, dv,
                                    scale, qk_norm, dtype, beta_dtype, &a);
    if (st != CONV_OK) return st;
    if ((T && !o) || !pointers_ok({}, {o}, bytes_of(dtype)) || !pointers_ok({}, {state, state_out}, 4) ||
        !pointers_ok({}, {workspace, saved}, 16))
        return CONV_ERR_INVALID_ARG;
    size_t need = 0, keep = 0;
    if ((st = delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_FWD, &need)) != CONV_OK) return st;
    if ((st = delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_SAVED, &keep)) != CONV_OK) return st;
    if (!workspace || workspace_bytes < need || (saved && saved_bytes < keep)) return CONV_ERR_WORKSPACE;
    a.o = o, a.state = state, a.state_out = state_out;
    DeltaBuf b = delta_buf(T, N, Hk, Hv, dk, dv, dtype);
    lay_out(&b, Hk, Hv, saved ? PART_FWD_SAVING : PART_FWD, workspace);
    if (saved) lay_out(&b, Hk, Hv, PART_SAVED, saved);
    hipError_t e = launch_delta_prep(a, b, saved != nullptr, dtype, (hipStream_t)stream);
    if (e == hipSuccess) e = launch_delta_scan(a, b, false, dtype, (hipStream_t)stream);
    return hip_status(e);
}

conv_status_t delta_rule_bwd(const void *d_o, int64_t do_stride, const float *dstate_out, const void *q,
                             int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             const float *g, const void *beta, const int32_t *cu_seqlens, const void *saved,
                             size_t saved_bytes, void *dq, void *dk_out, void *dv_out, float *dg, void *dbeta,
                             float *dstate, int64_t T, int N, int Hk, int Hv, int dk, int dv, float scale,
                             int qk_norm, conv_dtype_t dtype, conv_dtype_t beta_dtype, conv_stream_t stream,
                             void *workspace, size_t workspace_bytes) {
    DeltaArgs a{};
    conv_status_t st = delta_inputs(q, q_stride, k, k_stride, v, v_stride, g, beta, cu_seqlens, T, N, Hk, Hv, dk, dv,
                                    scale, qk_norm, dtype, beta_dtype, &a);
    if (st != CONV_OK) return st;
    if (T && (!d_o || !dq || !dk_out || !dv_out || !dg || !dbeta)) return CONV_ERR_INVALID_ARG;
    if (do_stride < (int64_t)Hv * dv || !pointers_ok({}, {d_o, dq, dk_out, dv_out}, bytes_of(dtype)) ||
        !pointers_ok({}, {dbeta}, bytes_of(beta_dtype)) || !pointers_ok({}, {dg, dstate, dstate_out}, 4) ||
        !pointers_ok({}, {workspace, saved}, 16))
        return CONV_ERR_INVALID_ARG;
    if (do_stride > MIX_DELTA_MAX_STRIDE) return CONV_ERR_UNSUPPORTED;
    size_t need = 0, keep = 0;
    if ((st = delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_BWD, &need)) != CONV_OK) return st;
    if ((st = delta_bytes(T, N, Hk, Hv, dk, dv, dtype, PART_SAVED, &keep)) != CONV_OK) return st;
    if (!workspace || workspace_bytes < need || !saved || saved_bytes < keep) return CONV_ERR_WORKSPACE;
    a.d_o = d_o, a.dos = do_stride, a.dstate_out = dstate_out;
    a.dq = dq, a.dk_out = dk_out, a.dv_out = dv_out, a.dg = dg, a.dbeta = dbeta, a.dstate = dstate;
    DeltaBuf b = delta_buf(T, N, Hk, Hv, dk, dv, dtype);
    lay_out(&b, Hk, Hv, PART_BWD, workspace);
    lay_out(&b, Hk, Hv, PART_SAVED, const_cast<void *>(saved));
    hipError_t e = launch_delta_scan(a, b, true, dtype, (hipStream_t)stream);
    if (e == hipSuccess) e = launch_delta_grad(a, b, dtype, (hipStream_t)stream);
    return hip_status(e);
}

conv_status_t branch_norm_fwd(const void *x, const void *y, const void *w_post, const void *gate, const void *w_next,
                              void *r, void *h, float *stats, int64_t R, int D, int64_t G, float alpha, float eps,
                              mix_act_t act, conv_dtype_t dtype, conv_stream_t stream) {
    const conv_status_t st = norm_sizes(R, D, G, gate != nullptr, eps, act, dtype);
    if (st != CONV_OK) return st;
    if (!R) return CONV_OK;
    if (!pointers_ok({y, w_post, r}, {x, gate, w_next, h}, bytes_of(dtype)) || (uintptr_t)stats % 4)
        return CONV_ERR_INVALID_ARG;
    if ((w_next != nullptr) != (h != nullptr)) return CONV_ERR_INVALID_ARG;
    NormArgs a{};
    a.x = x, a.y = y, a.w_post = w_post, a.gate = gate, a.w_next = w_next, a.r = r, a.h = h, a.stats = stats;
    a.R = R, a.D = D, a.G = gate ? G : R, a.rows_per_gate = R / a.G, a.alpha = alpha, a.eps = eps, a.act = act;
    return hip_status(launch_branch_norm_fwd(a, dtype, (hipStream_t)stream));
}

conv_status_t branch_norm_bwd_workspace_size(int64_t R, int D, int64_t G, size_t *bytes_out) {
    if (!bytes_out) return CONV_ERR_INVALID_ARG;
    const conv_status_t st = norm_sizes(R, D, G, true, 0.f, MIX_ACT_NONE, CONV_DTYPE_FP32);
    if (st != CONV_OK) return st;
    int per = 0, blocks = 0;
    if (R) branch_norm_bwd_plan(R, D, G, &per, &blocks);
    *bytes_out = (size_t)blocks * D * 3 * sizeof(float);
    return CONV_OK;
}

conv_status_t branch_norm_bwd(const void *dr, const void *dh, const void *x, const void *y, const void *w_post,
                              const void *gate, const void *w_next, const float *stats, void *dx, void *dy,
                              void *dw_post, void *dgate, void *dw_next, int64_t R, int D, int64_t G, float alpha,
                              float eps, mix_act_t act, conv_dtype_t dtype, conv_stream_t stream, void *workspace,
                              size_t workspace_bytes) {
    conv_status_t st = norm_sizes(R, D, G, gate != nullptr, eps, act, dtype);
    if (st != CONV_OK) return st;
    const size_t es = bytes_of(dtype);
    if (!pointers_ok({w_post, dw_post}, {dr, dh, x, y, gate, w_next, dx, dy, dgate, dw_next}, es))
        return CONV_ERR_INVALID_ARG;
    if (R && (!y || !dy || !stats || (uintptr_t)stats % 4)) return CONV_ERR_INVALID_ARG;
    // each input's gradient goes with the input (that of a gate without rows may be anywhere); dh only where there is an h
    if ((!gate || G) && (gate != nullptr) != (dgate != nullptr)) return CONV_ERR_INVALID_ARG;
    if ((w_next != nullptr) != (dw_next != nullptr)) return CONV_ERR_INVALID_ARG;
    if (R && (x != nullptr) != (dx != nullptr)) return CONV_ERR_INVALID_ARG;
    if (dh && !w_next) return CONV_ERR_INVALID_ARG;
    if ((uintptr_t)workspace % 16) return CONV_ERR_INVALID_ARG;
    NormArgs a{};
    a.G = gate ? G : R, a.rows_per_gate = a.G ? R / a.G : 0;
    if (R) branch_norm_bwd_plan(R, D, a.G, &a.per_group, &a.blocks);
    const size_t need = (size_t)a.blocks * D * 3 * sizeof(float);
    if (need && (!workspace || workspace_bytes < need)) return CONV_ERR_WORKSPACE;
    a.dr = dr, a.dh = dh, a.x = x, a.y = y, a.w_post = w_post, a.gate = gate, a.w_next = w_next;
    a.stats = const_cast<float *>(stats), a.dx = dx, a.dy = dy, a.dw_post = dw_post, a.dgate = dgate, a.dw_next = dw_next;
    a.part = (float *)workspace;
    a.R = R, a.D = D, a.alpha = alpha, a.eps = eps, a.act = act;
    return hip_status(launch_branch_norm_bwd(a, dtype, (hipStream_t)stream));
}

}  // extern "C"
