// Residual sum and norm that leave 8-bit rows:
//
//   r = x + res,  n = r rstd(r) w,  scale = max(max |n|, 2^-100) / 448,  q = e4m3(n / scale)
//
// A few operations for each value read: HBM bound.  A row is held in the
// registers of TPR threads (V values of 16 bytes at a time, NV times) through both
// of its reductions, so each tensor is read once; a short row takes part of a
// wavefront and a block holds several: 16384 x 4096 bf16 with res 82 us (470 MB, 5.7
// TB/s; a copy 5.1, half of whose bytes are writes), 7 x 4000 fp16 3.7 us.  n / scale is n times 448 / max: two
// roundings of 2^-24 each, beside which e4m3's half step is 2^-4.
#include "mixer_internal.h"
#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int nq_block(int tpr) { return tpr > 64 ? tpr : 256; }
constexpr float kE4m3Max = 448.f, kLeast = 7.888609052210118e-31f;  // 2^-100

// Over the TPR threads of a row (at most 64 lanes of one wavefront, or the whole
// block); every thread gets it.  MAX: the largest, a NaN if there is one.
template <int TPR, bool MAX>
__device__ __forceinline__ float nq_reduce(float v, float *red) {
    auto join = [](float a, float b) { return MAX ? __builtin_elementwise_maximum(a, b) : a + b; };
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m > 0; m >>= 1) v = join(v, __shfl_xor(v, m, 64));
    if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) v = join(v, red[i]);
    }
    return v;
}

template <typename S, int V, bool ANY>
__device__ __forceinline__ void nq_load(const S *p, int c, int D, float (&f)[V]) {
    if (ANY ? c + V <= D : c < D) {
        const FfnAnyVec<S, V> t = *(const FfnAnyVec<S, V> *)(p + c);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = mix_f32(t.v[j]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = ANY && c + j < D ? mix_f32(p[c + j]) : 0.f;
    }
}
template <typename S, int V, bool ANY>
__device__ __forceinline__ void nq_store(S *p, int c, int D, const S (&f)[V]) {
    if (ANY ? c + V <= D : c < D) {
        FfnAnyVec<S, V> t;
#pragma unroll
        for (int j = 0; j < V; ++j) t.v[j] = f[j];
        if constexpr (ANY) *(FfnAnyVec<S, V> *)(p + c) = t;
        else __builtin_memcpy(__builtin_assume_aligned(p + c, sizeof(S) * V), &t, sizeof(S) * V);
    } else if (ANY) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < D) p[c + j] = f[j];
    }
}

template <typename S, int V, int TPR, int NV, bool ANY>
__global__ __launch_bounds__(nq_block(TPR)) void norm_quant_kernel(NormQuantArgs A) {
    constexpr int TB = nq_block(TPR), ROWS = TB / TPR;
    __shared__ float red[2][TB / 64];
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool live = row < A.R;  // a block of one row each is always live: the reductions meet all its threads
    const int64_t at = (live ? row : 0) * A.D;
    float r[NV][V], w[NV][V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) nq_load<S, V, ANY>((const S *)A.x + at, (i * TPR + lane) * V, A.D, r[i]);
    if (A.res) {
#pragma unroll
        for (int i = 0; i < NV; ++i) nq_load<S, V, ANY>((const S *)A.res + at, (i * TPR + lane) * V, A.D, w[i]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) r[i][j] += w[i][j];
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) nq_load<S, V, ANY>((const S *)A.w, (i * TPR + lane) * V, A.D, w[i]);
    if (A.r && live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            S t[V];
#pragma unroll
            for (int j = 0; j < V; ++j) t[j] = mix_out<S>(r[i][j]);
            nq_store<S, V, ANY>((S *)A.r + at, (i * TPR + lane) * V, A.D, t);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    ss = nq_reduce<TPR, false>(ss, red[0]);
    const float rs = 1.f / sqrtf(ss / A.D + A.eps);
    float most = ss * 0.f;  // NaN where the sum is not finite
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            r[i][j] *= rs * w[i][j];
            most = __builtin_elementwise_maximum(most, fabsf(r[i][j]));
        }
    most = __builtin_elementwise_maximum(nq_reduce<TPR, true>(most, red[1]), kLeast);
    const float inv = kE4m3Max / most;
    if (!live) return;
    if (lane == 0) A.scale[row] = most / kE4m3Max;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        uint8_t q[V];
        uint32_t words[V / 4];
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            // a product may round to just above 448; NaN stays NaN
            float c[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                c[e] = __builtin_elementwise_minimum(__builtin_elementwise_maximum(r[i][j + e] * inv, -kE4m3Max), kE4m3Max);
            int t = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
            words[j / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], t, true);
        }
        __builtin_memcpy(q, words, V);
        nq_store<uint8_t, V, ANY>(A.q + at, (i * TPR + lane) * V, A.D, q);
    }
}

template <typename S, int V, int TPR, int NV, bool ANY>
hipError_t nq_run(const NormQuantArgs &a, hipStream_t st) {
    constexpr int TB = nq_block(TPR), rows = TB / TPR;
    const int64_t blocks = (a.R + rows - 1) / rows;
    if (!grid_fits(blocks, TB, 1)) return kTooLarge;
    hipLaunchKernelGGL((norm_quant_kernel<S, V, TPR, NV, ANY>), dim3((unsigned)blocks), dim3(TB), 0, st, a);
    return hipGetLastError();
}

// The fewest threads that hold a row in one 16-byte piece each, and more pieces
// only past 1024 threads.
template <typename S, bool ANY>
hipError_t nq_width(const NormQuantArgs &a, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    if (a.D <= 16 * V) return nq_run<S, V, 16, 1, ANY>(a, st);
    if (a.D <= 32 * V) return nq_run<S, V, 32, 1, ANY>(a, st);
    if (a.D <= 64 * V) return nq_run<S, V, 64, 1, ANY>(a, st);
    if (a.D <= 128 * V) return nq_run<S, V, 128, 1, ANY>(a, st);
    if (a.D <= 256 * V) return nq_run<S, V, 256, 1, ANY>(a, st);
    if (a.D <= 512 * V) return nq_run<S, V, 512, 1, ANY>(a, st);
    if (a.D <= 1024 * V) return nq_run<S, V, 1024, 1, ANY>(a, st);
    if (a.D <= 2048 * V) return nq_run<S, V, 1024, 2, ANY>(a, st);
    if constexpr (V == 4)
        if (a.D > 4096 * V) return nq_run<S, V, 1024, 8, ANY>(a, st);  // to 32768 float32
    return nq_run<S, V, 1024, 4, ANY>(a, st);
}

template <typename S>
hipError_t nq_typed(const NormQuantArgs &a, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    bool vec = a.D % V == 0 && (uintptr_t)a.q % V == 0;
    for (const void *p : {a.x, a.res, a.w, (const void *)a.r}) vec = vec && (uintptr_t)p % 16 == 0;
    return vec ? nq_width<S, false>(a, st) : nq_width<S, true>(a, st);
}

}  // namespace

hipError_t launch_norm_quant(const NormQuantArgs &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return nq_typed<float>(a, st);
    if (dtype == CONV_DTYPE_FP16) return nq_typed<_Float16>(a, st);
    return nq_typed<uint16_t>(a, st);
}

}  // namespace convlower
