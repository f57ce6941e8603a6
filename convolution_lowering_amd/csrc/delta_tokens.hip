// The gated delta rule token by token:
//
//   S <- exp(g) S;  u = beta (v - S'k);  S <- S + k u';  o = scale S'q
//
// The state [dk][dv] is read and written once, in fp32, however many tokens a
// request brings: HBM bound.  Columns of S do not meet, so a wavefront takes
// 32 columns of one head: 8 lanes of 4 columns, 8 groups of rows, all of it in
// registers.  Both products with S come out of one pass, since
// S_new'q = (exp(g) S)'q + u (k'q): one reduction a token.
#include "mixer_internal.h"

namespace convlower {
namespace {

constexpr int kStepCols = 32;

// Sum over the 8 row groups (lanes that differ in bits 3 to 5).
__device__ __forceinline__ float rows_sum(float v) {
    v += __shfl_xor(v, 8, 64);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// One head's 32 columns over the tokens [t0, t1), S in and out at st.
template <typename S, int NR, bool VEC>
__device__ __forceinline__ void run_tokens(const DeltaArgs &A, float *st, int h, int c0, int64_t t0, int64_t t1) {
    const int lane = threadIdx.x, rg = lane >> 3, c = c0 + (lane & 7) * 4;
    const int hk = h / (A.Hv / A.Hk);
    float s[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = i * 8 + rg;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
        if (row < A.dk) {
            const float *p = st + (int64_t)row * A.dv + c;
            if (VEC) {
                if (c < A.dv) mix_load<float, 4>(p, s[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < A.dv) s[i][j] = p[j];
            }
        }
    }
    for (int64_t t = t0; t < t1; ++t) {
        const S *qp = (const S *)A.q + t * A.qs + (int64_t)hk * A.dk;
        const S *kp = (const S *)A.k + t * A.ks + (int64_t)hk * A.dk;
        const S *vp = (const S *)A.v + t * A.vs + (int64_t)h * A.dv;
        const int64_t th = t * A.Hv + h;
        float q[NR], k[NR], v[4];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int row = i * 8 + rg;
            q[i] = row < A.dk ? mix_f32(qp[row]) : 0.f;
            k[i] = row < A.dk ? mix_f32(kp[row]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = c + j < A.dv ? mix_f32(vp[c + j]) : 0.f;
        const float decay = expf(A.g[th]);
        const float beta = A.beta_f32 ? ((const float *)A.beta)[th] : mix_f32(((const S *)A.beta)[th]);
        float kq = 0.f, kk = 0.f, qq = 0.f, a[4], b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) a[j] = b[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            kq = fmaf(k[i], q[i], kq);
            kk = fmaf(k[i], k[i], kk);
            qq = fmaf(q[i], q[i], qq);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] *= decay;
                a[j] = fmaf(k[i], s[i][j], a[j]);
                b[j] = fmaf(q[i], s[i][j], b[j]);
            }
        }
        float rk = 1.f, rq = A.scale;
        if (A.qk_norm) {
            rk = 1.f / sqrtf(rows_sum(kk) + kDeltaEps);
            rq *= 1.f / sqrtf(rows_sum(qq) + kDeltaEps);
        }
        kq = rows_sum(kq) * rk * rq;
        float o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float u = beta * (v[j] - rk * rows_sum(a[j]));
            o[j] = fmaf(u, kq, rq * rows_sum(b[j]));
            const float ku = rk * u;
#pragma unroll
            for (int i = 0; i < NR; ++i) s[i][j] = fmaf(k[i], ku, s[i][j]);
        }
        if (rg == 0) {
            S *op = (S *)A.o + th * A.dv + c;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < A.dv) op[j] = mix_out<S>(o[j]);
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = i * 8 + rg;
        if (row >= A.dk) continue;
        float *p = st + (int64_t)row * A.dv + c;
        if (VEC) {
            if (c < A.dv) mix_store<float, 4>(p, s[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < A.dv) p[j] = s[i][j];
        }
    }
}

// blockIdx.x: request * Hv + head; blockIdx.y: 32 columns.
template <typename S, int NR, bool VEC>
__global__ __launch_bounds__(64) void delta_tokens_kernel(DeltaArgs A) {
    const int n = blockIdx.x / A.Hv, h = blockIdx.x % A.Hv, c0 = blockIdx.y * kStepCols;
    const int slot = A.slots ? A.slots[n] : n;
    const int64_t t0 = (int64_t)n * A.L;
    if (slot < 0 || slot >= A.P) {  // a padding request: zeros, and no state
        for (int64_t t = t0; t < t0 + A.L; ++t)
            for (int c = threadIdx.x; c < kStepCols; c += 64)
                if (c0 + c < A.dv) ((S *)A.o)[(t * A.Hv + h) * A.dv + c0 + c] = mix_out<S>(0.f);
        return;
    }
    run_tokens<S, NR, VEC>(A, A.pool + ((int64_t)slot * A.Hv + h) * A.dk * A.dv, h, c0, t0, t0 + A.L);
}

template <typename S>
hipError_t tokens_typed(const DeltaArgs &a, hipStream_t st) {
    if (!a.R) return hipSuccess;
    const dim3 grid((unsigned)((int64_t)a.R * a.Hv), (a.dv + kStepCols - 1) / kStepCols);
    const bool vec = a.dv % 4 == 0 && (uintptr_t)a.pool % 16 == 0;
    if (a.dk <= 64) {
        if (vec) hipLaunchKernelGGL((delta_tokens_kernel<S, 8, true>), grid, dim3(64), 0, st, a);
        else hipLaunchKernelGGL((delta_tokens_kernel<S, 8, false>), grid, dim3(64), 0, st, a);
    } else {
        if (vec) hipLaunchKernelGGL((delta_tokens_kernel<S, 16, true>), grid, dim3(64), 0, st, a);
        else hipLaunchKernelGGL((delta_tokens_kernel<S, 16, false>), grid, dim3(64), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_tokens(const DeltaArgs &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return tokens_typed<float>(a, st);
    if (dtype == CONV_DTYPE_FP16) return tokens_typed<_Float16>(a, st);
    return tokens_typed<uint16_t>(a, st);
}

}  // namespace convlower
