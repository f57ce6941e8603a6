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
#include <type_traits>

#include "ffn_internal.h"

namespace convlower {
namespace {

template <typename S, int ACT>
__device__ __forceinline__ void gate_grad(const FfnGateGrad &A) {
    constexpr int V = 16 / (int)sizeof(S);
    const int per = A.Fp / V;
    const int64_t total = A.T * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
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
        S *out = (S *)A.dgu + t * 2 * A.Fp + f;
        mix_store<S, V>(out, dg);
        mix_store<S, V>(out + A.Fp, du);
    }
}
template <typename S, int ACT>
__global__ __launch_bounds__(256) void ffn_gate_grad_kernel(FfnGateGrad A) {
    gate_grad<S, ACT>(A);
}

template <typename S>
hipError_t run(const FfnGateGrad &a, hipStream_t st) {
    const int64_t blocks = (a.T * (a.Fp / (16 / (int)sizeof(S))) + 255) / 256;
    const dim3 grid((unsigned)(blocks < 1 << 20 ? blocks : 1 << 20));
    switch (a.act) {
        case FFN_ACT_SILU: hipLaunchKernelGGL((ffn_gate_grad_kernel<S, FFN_ACT_SILU>), grid, dim3(256), 0, st, a); break;
        case FFN_ACT_SIGMOID: hipLaunchKernelGGL((ffn_gate_grad_kernel<S, FFN_ACT_SIGMOID>), grid, dim3(256), 0, st, a); break;
        case FFN_ACT_GELU: hipLaunchKernelGGL((ffn_gate_grad_kernel<S, FFN_ACT_GELU>), grid, dim3(256), 0, st, a); break;
        default: hipLaunchKernelGGL((ffn_gate_grad_kernel<S, FFN_ACT_NONE>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_ffn_gate_grad(const FfnGateGrad &a, int dtype, hipStream_t st) {
    if (!a.T) return hipSuccess;
    if (dtype == CONV_DTYPE_FP32) return run<float>(a, st);
    if (dtype == CONV_DTYPE_FP16) return run<_Float16>(a, st);
    return run<uint16_t>(a, st);
}

}  // namespace convlower
