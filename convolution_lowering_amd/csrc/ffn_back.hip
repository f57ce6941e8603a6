// The gradients of g and u, which the products for dx and for the weights' gradients
// take:
//
//   du = dh act(g),   dg = dh u act'(g).
//
// HBM bound: each thread takes 16 bytes of results of both (8192 x 8192 bf16: 940 MB in
// 216 us, 4.4 TB/s, 8 % of a training step; dg and du belong to both products that
// follow, each of which reads them several times, so they are not made inside one).
// g and u were saved in fp32: dg and du are rounded to the operands' type, which is
// what the matrix instructions take, and that is the only rounding a gradient has
// beside its own (bf16: error against 64 bits 2.3e-3, in float32 operators 1.7e-3;
// with g and u rounded as well it would be 2.9e-3).
//
// fp16 has digits from 2^-24 to 2^16 only, and dh u may lie outside where dx and the
// weights' gradients do not.  So dg and du are kept times a power of two that
// puts their largest value between 2^14 and 2^15, one for all of them (dW adds up
// tokens), which the products' results are divided by: a pass before looks for that
// value and reads what this one reads (8192 x 8192: 124 us of a backward pass of
// 1970).  What is below 2^-38 of it counts as zero.
#include <type_traits>

#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int kThreads = 256;

// The largest over the block; every thread gets it.
__device__ __forceinline__ float block_most(float v) {
    __shared__ float red[kThreads / 64];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor(v, m, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// put(t, f, dg, du) for each 16 bytes of results.
template <typename S, int ACT, typename Fn>
__device__ __forceinline__ void each_piece(const FfnGateGrad &A, Fn &&put) {
    constexpr int V = 16 / (int)sizeof(S);
    const int per = A.Fp / V;
    const int64_t total = A.T * per;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int64_t t = i / per;
        const int f = (int)(i - t * per) * V;
        const float *g = A.saved + t * A.pitch + f, *u = g + A.T * A.pitch;
        const S *dh = (const S *)A.dh + t * A.dhs + f;
        float gv[V] = {}, uv[V] = {}, d[V] = {};
#pragma unroll
        for (int j = 0; j < V; j += 4)
            if (f + j < A.pitch) {  // (rows of the saved values are whole 16-byte pieces)
                const float4 x = *(const float4 *)(g + j), y = *(const float4 *)(u + j);
                gv[j] = x.x, gv[j + 1] = x.y, gv[j + 2] = x.z, gv[j + 3] = x.w;
                uv[j] = y.x, uv[j + 1] = y.y, uv[j + 2] = y.z, uv[j + 3] = y.w;
            }
        if (f + V <= A.F) {
            const FfnAnyVec<S, V> x = *(const FfnAnyVec<S, V> *)dh;
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] = mix_f32(x.v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (f + j < A.F) d[j] = mix_f32(dh[j]);
        }
        float dg[V], du[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float a, slope;
            ffn_act_grad<S>(gv[j], ACT, &a, &slope);
            const bool in = f + j < A.F;
            dg[j] = in ? d[j] * uv[j] * slope : 0.f;
            du[j] = in ? d[j] * a : 0.f;
        }
        put(t, f, dg, du);
    }
}
template <typename S, int ACT>
__global__ __launch_bounds__(kThreads) void ffn_gate_grad_kernel(FfnGateGrad A) {
    constexpr int V = 16 / (int)sizeof(S);
    float by = 1.f;
    if constexpr (__is_same(S, _Float16)) {
        float most = 0.f;
#pragma unroll
        for (int i = 0; i < kFfnRangeBlocks; i += kThreads) most = fmaxf(most, A.range[kFfnRangeAt + i + threadIdx.x]);
        most = block_most(most);
        int e = 0;  // most = x 2^e, x from 1/2 to 1
        if (most > 0.f) frexpf(most, &e);
        const int k = min(15 - e, 126);
        by = ldexpf(1.f, k);
        if (blockIdx.x == 0 && threadIdx.x == 0) A.range[0] = ldexpf(1.f, -k);
    }
    each_piece<S, ACT>(A, [&](int64_t t, int f, float (&dg)[V], float (&du)[V]) {
        if constexpr (__is_same(S, _Float16)) {
#pragma unroll
            for (int j = 0; j < V; ++j) dg[j] *= by, du[j] *= by;
        }
        S *out = (S *)A.dgu + t * 2 * A.Fp + f;
        mix_store<S, V>(out, dg);
        mix_store<S, V>(out + A.Fp, du);
    });
}
// Each block's largest finite value, kFfnRangeBlocks of them.
template <typename S, int ACT>
__global__ __launch_bounds__(kThreads) void ffn_gate_range_kernel(FfnGateGrad A) {
    constexpr int V = 16 / (int)sizeof(S);
    constexpr float top = 3.402823466e38f;
    float most = 0.f;
    each_piece<S, ACT>(A, [&](int64_t, int, float (&dg)[V], float (&du)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float x = fabsf(dg[j]), y = fabsf(du[j]);
            most = fmaxf(most, fmaxf(x <= top ? x : 0.f, y <= top ? y : 0.f));
        }
    });
    most = block_most(most);
    if (threadIdx.x == 0) A.range[kFfnRangeAt + blockIdx.x] = most;
}

template <typename S, int ACT>
hipError_t run_act(const FfnGateGrad &a, hipStream_t st) {
    if constexpr (__is_same(S, _Float16)) {
        hipLaunchKernelGGL((ffn_gate_range_kernel<S, ACT>), dim3(kFfnRangeBlocks), dim3(kThreads), 0, st, a);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    // (fp16: each block reads the range kernel's results first)
    const int64_t blocks = (a.T * (a.Fp / (16 / (int)sizeof(S))) + kThreads - 1) / kThreads, most = __is_same(S, _Float16) ? 1 << 13 : 1 << 20;
    hipLaunchKernelGGL((ffn_gate_grad_kernel<S, ACT>), dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
}
template <typename S>
hipError_t run(const FfnGateGrad &a, hipStream_t st) {
    switch (a.act) {
        case FFN_ACT_SILU: return run_act<S, FFN_ACT_SILU>(a, st);
        case FFN_ACT_SIGMOID: return run_act<S, FFN_ACT_SIGMOID>(a, st);
        case FFN_ACT_GELU: return run_act<S, FFN_ACT_GELU>(a, st);
        default: return run_act<S, FFN_ACT_NONE>(a, st);
    }
}

}  // namespace

hipError_t launch_ffn_gate_grad(const FfnGateGrad &a, int dtype, hipStream_t st) {
    if (!a.T) return hipSuccess;
    if (dtype == CONV_DTYPE_FP32) return run<float>(a, st);
    if (dtype == CONV_DTYPE_FP16) return run<_Float16>(a, st);
    return run<uint16_t>(a, st);
}

}  // namespace convlower
