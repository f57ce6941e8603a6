// Internal declarations of the sequence-mixing operators (convlower_mixer.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "convlower_mixer.h"

namespace convlower {

// ---- element access: uint16_t holds bf16 bits, as in the convolution kernels
__device__ __forceinline__ float mix_f32(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float mix_f32(_Float16 v) { return (float)v; }
__device__ __forceinline__ float mix_f32(float v) { return v; }
template <typename S>
__device__ __forceinline__ S mix_out(float v);  // round to nearest, ties to even
template <>
__device__ __forceinline__ uint16_t mix_out<uint16_t>(float v) {
    return __builtin_bit_cast(uint16_t, (__bf16)v);
}
template <>
__device__ __forceinline__ _Float16 mix_out<_Float16>(float v) {
    return (_Float16)v;
}
template <>
__device__ __forceinline__ float mix_out<float>(float v) {
    return v;
}

// V consecutive elements, loaded and stored as 16-byte (or smaller) words.
template <typename S, int V>
struct alignas(sizeof(S) * V) MixVec {
    S v[V];
};
template <typename S, int V>
__device__ __forceinline__ void mix_load(const S *p, float (&f)[V]) {
    const MixVec<S, V> t = *(const MixVec<S, V> *)p;
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = mix_f32(t.v[i]);
}
template <typename S, int V>
__device__ __forceinline__ void mix_store(S *p, const float (&f)[V]) {
    MixVec<S, V> t;
#pragma unroll
    for (int i = 0; i < V; ++i) t.v[i] = mix_out<S>(f[i]);
    *(MixVec<S, V> *)p = t;
}

// For results of 16 bits the exponential and reciprocal instructions do: what
// they lose, |z| 2^-24 and a unit in the last place, is far below half a step.
// A float32 result would lose five bits to them at z = -80: there the exponent
// -z log2(e) is taken in two floats, the second by its slope, and the quotient
// is improved once (r + r (1 - d r)).  (8192 x 8192 float32 convolved: 120 us,
// with expf and a division 125, the instructions alone 118.)
template <typename S>
__device__ __forceinline__ float mix_sigmoid(float z) {
    if constexpr (sizeof(S) != 4) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
    constexpr double kLog2e = 1.4426950408889634074;
    constexpr float hi = (float)kLog2e, lo = (float)(kLog2e - (double)hi), ln2 = 0.69314718f;
    // (past 87 e^-z is nothing beside 1; below -87 the result is less than the smallest normal number)
    const float c = -__builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -87.f), 87.f);
    const float t = c * hi, rest = fmaf(c, lo, fmaf(c, hi, -t));
    float e = __builtin_amdgcn_exp2f(t);
    e = fmaf(e * ln2, rest, e);
    const float d = 1.f + e, r = __builtin_amdgcn_rcpf(d);
    return z < -87.f ? 0.f : fmaf(r, fmaf(-d, r, 1.f), r);
}

// ---- packed sequences.  cu null: every sequence holds T / N tokens.  Values
// outside [0, T] are clamped, so that a bad array reads and writes nothing
// outside the caller's buffers.
struct Seqs {
    const int32_t *cu;
    int64_t T;
    int N;
    int64_t each;  // T / N where cu is null
};
__device__ __forceinline__ int64_t seq_start(const Seqs &s, int n) {
    if (!s.cu) return s.each * n;
    const int64_t v = s.cu[n];
    return v < 0 ? 0 : v > s.T ? s.T : v;
}
__device__ __forceinline__ void seq_range(const Seqs &s, int n, int64_t *a, int64_t *e) {
    *a = seq_start(s, n);
    const int64_t z = seq_start(s, n + 1);
    *e = z < *a ? *a : z;
}
// The last sequence that starts at or before token t (the one that holds it).
__device__ __forceinline__ int seq_of(const Seqs &s, int64_t t) {
    if (!s.cu) return (int)(s.each ? t / s.each : 0);
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (seq_start(s, mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// ---- launchers; dtype: conv_dtype_t (fp32, bf16, fp16).  Before its first
// launch a launcher looks whether its grids fit (threads of an axis are counted
// in 32 bits, blocks of the second one go to 65536), and else returns
// kTooLarge, which callers see as CONV_ERR_UNSUPPORTED.
constexpr hipError_t kTooLarge = hipErrorInvalidConfiguration;
inline bool grid_fits(int64_t blocks_x, int threads, int64_t blocks_y) {
    return blocks_x * threads < (1LL << 32) && blocks_y <= 65536;
}
struct Conv1dArgs {
    const void *x, *w, *bias, *state, *dy, *dstate_out;
    void *y, *state_out, *dx, *dw, *dbias, *dstate;
    float *part;  // bwd: [blocks][W + 1][D] partial sums
    int64_t xs, dys;
    Seqs s;
    int D, W, act, tiles, tile;
};
constexpr int kConvRuns = 4;  // runs of tokens whose sums a backward block adds up
int conv1d_bwd_tile(int64_t T, int D);  // tokens of one run
hipError_t launch_conv1d_fwd(Conv1dArgs a, int dtype, hipStream_t st);
hipError_t launch_conv1d_bwd(Conv1dArgs a, int dtype, hipStream_t st);
hipError_t launch_conv1d_step(const void *x, int64_t xs, const void *w, const void *bias, void *pool,
                              const int32_t *slots, void *y, int R, int P, int D, int W, int act, int dtype,
                              hipStream_t st);

struct NormArgs {
    const void *x, *y, *w_post, *gate, *w_next, *dr, *dh;
    void *r, *h, *dx, *dy, *dw_post, *dgate, *dw_next;
    float *stats;  // [2][R]
    float *part;   // bwd: [3][blocks][D] partial sums
    int64_t R, G, rows_per_gate;
    int D, act;
    int per_group, blocks;  // bwd: blocks of one gate row, blocks in all
    float alpha, eps;
};
void branch_norm_bwd_plan(int64_t R, int D, int64_t G, int *per_group, int *blocks);
hipError_t launch_branch_norm_fwd(const NormArgs &a, int dtype, hipStream_t st);
hipError_t launch_branch_norm_bwd(const NormArgs &a, int dtype, hipStream_t st);

struct DeltaArgs {
    const void *q, *k, *v, *beta, *d_o;
    const float *g, *state, *dstate_out;
    void *o, *dq, *dk_out, *dv_out, *dbeta;
    float *state_out, *dg, *dstate;
    int64_t qs, ks, vs, dos;  // token strides
    Seqs s;
    int Hk, Hv, dk, dv, qk_norm, beta_f32;
    float scale;
    // token-by-token form
    float *pool;
    const int32_t *slots;
    int R, L, P;
};
// qk_norm's term under the root
constexpr float kDeltaEps = 1e-6f;
hipError_t launch_delta_tokens(const DeltaArgs &a, int dtype, hipStream_t st);

}  // namespace convlower
