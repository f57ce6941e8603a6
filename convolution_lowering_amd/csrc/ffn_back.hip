// What the gradients of the gated product need laid out before their products:
// the gradients of g and u,
//
//   du = dh act(g),   dg = dh u act'(g),
//
// along the features (for dx) and along the tokens (for the weights'), and x and
// the weights with their other axis contiguous.  HBM bound; tiles of 64 x 64 pass
// through LDS.
#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int kTile = 64;

// One tile transposed: from in[r][c] (R x C, any addresses) to out[c][r], rows of
// out up to Rp, zeros from R on.
template <typename S>
__device__ __forceinline__ void transpose_tile(const S *in, int64_t is, int64_t R, int C, S *out, int64_t os, int64_t Rp,
                                               int64_t r0, int c0, S (&buf)[kTile][kTile + 2]) {
    const int x = threadIdx.x & 63, y0 = threadIdx.x >> 6;
    for (int y = y0; y < kTile; y += 4) {
        S v = S(0);
        if (r0 + y < R && c0 + x < C) v = in[(r0 + y) * is + c0 + x];
        buf[y][x] = v;
    }
    __syncthreads();
    for (int y = y0; y < kTile; y += 4)
        if (c0 + y < C && r0 + x < Rp) out[(int64_t)(c0 + y) * os + r0 + x] = buf[x][y];
}

template <typename S>
__global__ __launch_bounds__(256) void ffn_transpose_kernel(const S *in, int64_t is, int64_t R, int C, S *out, int64_t os,
                                                            int64_t Rp) {
    __shared__ S buf[kTile][kTile + 2];
    transpose_tile<S>(in, is, R, C, out, os, Rp, (int64_t)blockIdx.x * kTile, blockIdx.y * kTile, buf);
}

template <typename S>
__global__ __launch_bounds__(256) void ffn_gate_grad_kernel(FfnBack A) {
    __shared__ S bg[kTile][kTile + 2], bu[kTile][kTile + 2];
    const int x = threadIdx.x & 63, y0 = threadIdx.x >> 6;
    const int64_t t0 = (int64_t)blockIdx.x * kTile;
    const int f0 = blockIdx.y * kTile;
    const S *dh = (const S *)A.dh;
    for (int y = y0; y < kTile; y += 4) {
        const int64_t t = t0 + y;
        const int f = f0 + x;
        float dg = 0.f, du = 0.f;
        if (t < A.T && f < A.F) {
            const float g = A.saved[t * A.pitch + f], u = A.saved[(A.T + t) * A.pitch + f], d = mix_f32(dh[t * A.dhs + f]);
            float a, slope;
            ffn_act_grad<S>(g, A.act, &a, &slope);
            dg = d * u * slope;
            du = d * a;
        }
        bg[y][x] = mix_out<S>(dg);
        bu[y][x] = mix_out<S>(du);
        if (t < A.T && f < A.Fp) {
            S *row = (S *)A.dgu + t * 2 * A.Fp + f;
            row[0] = bg[y][x];
            row[A.Fp] = bu[y][x];
        }
    }
    __syncthreads();
    for (int y = y0; y < kTile; y += 4)
        if (f0 + y < A.F && t0 + x < A.Tp) {
            S *row = (S *)A.dguT + (int64_t)(f0 + y) * A.Tp + t0 + x;
            row[0] = bg[x][y];
            row[(int64_t)A.F * A.Tp] = bu[x][y];
        }
}

template <typename S>
hipError_t back_prep(const FfnBack &a, hipStream_t st) {
    const int64_t tt = a.Tp / kTile + (a.Tp % kTile != 0);
    const int ft = (a.Fp + kTile - 1) / kTile, dt = (a.D + kTile - 1) / kTile, wt = (a.Fp + kTile - 1) / kTile;
    if (!grid_fits(tt, 256, ft > dt ? ft : dt) || !grid_fits(wt, 256, dt)) return kTooLarge;
    if (tt) {
        hipLaunchKernelGGL((ffn_gate_grad_kernel<S>), dim3((unsigned)tt, ft), dim3(256), 0, st, a);
        if (const hipError_t e = hipGetLastError()) return e;
        hipLaunchKernelGGL((ffn_transpose_kernel<S>), dim3((unsigned)tt, dt), dim3(256), 0, st, (const S *)a.x, a.xs, a.T, a.D,
                           (S *)a.xT, a.Tp, a.Tp);
        if (const hipError_t e = hipGetLastError()) return e;
    }
    for (int h = 0; h < 2; ++h) {
        hipLaunchKernelGGL((ffn_transpose_kernel<S>), dim3(wt, dt), dim3(256), 0, st, (const S *)(h ? a.w_up : a.w_gate),
                           (int64_t)a.D, (int64_t)a.F, a.D, (S *)a.wT + (int64_t)h * a.Fp, 2 * (int64_t)a.Fp, (int64_t)a.Fp);
        if (const hipError_t e = hipGetLastError()) return e;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_ffn_back_prep(const FfnBack &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return back_prep<float>(a, st);
    if (dtype == CONV_DTYPE_FP16) return back_prep<_Float16>(a, st);
    return back_prep<uint16_t>(a, st);
}

}  // namespace convlower
