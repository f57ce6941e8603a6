// The gated delta rule token by token:
//
//   S <- exp(g) S;  u = beta (v - S'k);  S <- S + k u';  o = scale S'q
//
// The state [dk][dv] is read and written once, in fp32, however many tokens a
// request brings: HBM bound.  Columns of S do not meet, so a wavefront takes
// 32 columns of one head: 8 lanes of 4 columns, 8 groups of rows, all of it in
// registers.  Both products with S come out of one pass, since
// S_new'q = (exp(g) S)'q + u (k'q): one reduction a token.
//
// A head's wavefronts are neighbours in the grid, so that its rows' pieces are
// fetched together, and four to a SIMD (128 registers) keep more of them under
// way.  The state is not read again before a whole model's worth of other
// data, so its stores pass the caches.  A token's q, k and v are fetched while
// the one before is computed, once a wavefront, and shared through LDS.
//
// 64 requests x 32 heads x 128 x 128 (268 MB): 50 us, 5.3 TB/s; heads apart in
// the grid, three wavefronts and plain stores: 72 us; q and k fetched by every
// lane for itself: 55 us.  67 requests of 4 tokens, 16 heads (140 MB): 38 us,
// was 57.
#include "mixer_internal.h"

namespace convlower {
namespace {

constexpr int kStepCols = 32;
typedef float f4 __attribute__((ext_vector_type(4)));

// Sum over the 8 row groups (lanes that differ in bits 3 to 5).
__device__ __forceinline__ float rows_sum(float v) {
    v += __shfl_xor(v, 8, 64);
    v += __shfl_xor(v, 16, 64);
    return v + __shfl_xor(v, 32, 64);
}

// One head's 32 columns over the tokens [t0, t1), S in and out at st.
template <typename S, int NR, bool VEC>
__device__ __forceinline__ void run_tokens(const DeltaArgs &A, float *st, int h, int c0, int64_t t0, int64_t t1) {
    // q and k of a token, row group rg's rows side by side, and v
    __shared__ __align__(16) float rows[2][2][8 * NR];
    __shared__ __align__(16) float cols[2][kStepCols];
    const int lane = threadIdx.x, rg = lane >> 3, cl = (lane & 7) * 4, c = c0 + cl;
    const int hk = h / (A.Hv / A.Hk);
    S fq[NR / 8], fk[NR / 8], fv;
    auto fetch = [&](int64_t t) {
        const S *qp = (const S *)A.q + t * A.qs + (int64_t)hk * A.dk;
        const S *kp = (const S *)A.k + t * A.ks + (int64_t)hk * A.dk;
        const S *vp = (const S *)A.v + t * A.vs + (int64_t)h * A.dv + c0;
#pragma unroll
        for (int i = 0; i < NR / 8; ++i) {
            const int row = lane + 64 * i;
            fq[i] = row < A.dk ? qp[(uint32_t)row] : S{};
            fk[i] = row < A.dk ? kp[(uint32_t)row] : S{};
        }
        fv = lane < kStepCols && c0 + lane < A.dv ? vp[(uint32_t)lane] : S{};
    };
    if (t0 < t1) fetch(t0);
    float s[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int row = i * 8 + rg;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
        if (row < A.dk) {
            const float *p = st + (uint32_t)(row * A.dv + c);
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
#pragma unroll
        for (int i = 0; i < NR / 8; ++i) {
            const int at = (lane & 7) * NR + (lane >> 3) + 8 * i;
            rows[t & 1][0][at] = mix_f32(fq[i]);
            rows[t & 1][1][at] = mix_f32(fk[i]);
        }
        if (lane < kStepCols) cols[t & 1][lane] = mix_f32(fv);
        __syncthreads();
        if (t + 1 < t1) fetch(t + 1);
        const int64_t th = t * A.Hv + h;
        float q[NR], k[NR], v[4];
#pragma unroll
        for (int i = 0; i < NR; i += 4) {
            const f4 qq = *(const f4 *)&rows[t & 1][0][rg * NR + i], kk = *(const f4 *)&rows[t & 1][1][rg * NR + i];
#pragma unroll
            for (int j = 0; j < 4; ++j) q[i + j] = qq[j], k[i + j] = kk[j];
        }
        const f4 vv = *(const f4 *)&cols[t & 1][cl];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = vv[j];
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
        float *p = st + (uint32_t)(row * A.dv + c);
        if (VEC) {
            if (c < A.dv) __builtin_nontemporal_store(f4{s[i][0], s[i][1], s[i][2], s[i][3]}, (f4 *)p);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j < A.dv) p[j] = s[i][j];
        }
    }
}

// blockIdx.x: (request * Hv + head) * groups of 32 columns + group.
template <typename S, int NR, bool VEC>
__global__ __launch_bounds__(64, 4) void delta_tokens_kernel(DeltaArgs A) {
    const int groups = (A.dv + kStepCols - 1) / kStepCols, c0 = blockIdx.x % groups * kStepCols, u = blockIdx.x / groups;
    const int n = u / A.Hv, h = u % A.Hv;
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
    const dim3 grid((unsigned)((int64_t)a.R * a.Hv * ((a.dv + kStepCols - 1) / kStepCols)));
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
