// Internal declarations of the feed-forward operators (convlower_ffn.h).
#pragma once

#include "convlower_ffn.h"
#include "igemm_impl.h"
#include "mixer_internal.h"

namespace convlower {

// ---- the gate's activation: value, and value and slope.  S: the type whose
// digits the result needs (mix_sigmoid).  In the tanh form's polynomial z stops
// at +-30, far past where the sigmoid is 0 or 1 in 32 bits, so that no z
// overflows it.
template <typename S>
__device__ __forceinline__ float gelu_gate(float z, float *inner) {
    constexpr float k2c = 1.5957691216057308f;  // 2 sqrt(2 / pi)
    const float c = __builtin_elementwise_minimum(__builtin_elementwise_maximum(z, -30.f), 30.f);
    *inner = c * k2c * fmaf(0.134145f, c * c, 1.f);  // z times the argument's slope
    return mix_sigmoid<S>(c * k2c * fmaf(0.044715f, c * c, 1.f));
}
template <typename S>
__device__ __forceinline__ float ffn_act(float z, int act) {
    float inner;
    switch (act) {
        case FFN_ACT_SILU: return z * mix_sigmoid<S>(z);
        case FFN_ACT_SIGMOID: return mix_sigmoid<S>(z);
        case FFN_ACT_GELU: return z * gelu_gate<S>(z, &inner);
        default: return z;
    }
}
// A slope takes 1 - s(z) as s(-z): beside an s(z) near 1 the difference would
// cancel (sigmoid's float32 slope would be zero from z = 17 on).  The kernel waits for memory
// (8192 x 8192 bf16: 152 us either way).
template <typename S>
__device__ __forceinline__ void ffn_act_grad(float z, int act, float *a, float *da) {
    if (act == FFN_ACT_NONE) {
        *a = z;
        *da = 1.f;
    } else if (act == FFN_ACT_GELU) {
        float inner;
        const float q = gelu_gate<S>(-z, &inner), p = gelu_gate<S>(z, &inner);
        *a = z * p;
        *da = fmaf(p * q, inner, p);
    } else {
        const float p = mix_sigmoid<S>(z), q = mix_sigmoid<S>(-z);
        *a = act == FFN_ACT_SILU ? z * p : p;
        *da = act == FFN_ACT_SILU ? p * fmaf(z, q, 1.f) : p * q;
    }
}

// V consecutive elements at any multiple of an element's size.
template <typename S, int V>
struct __attribute__((packed, aligned(sizeof(S)))) FfnAnyVec {
    S v[V];
};

// lds_dma16 (igemm_dma.h) of rows that begin `at` bytes further on.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void ffn_dma16(__amdgpu_buffer_rsrc_t rsrc, uint32_t voff, uint32_t at, uint32_t lds_base) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %3 offen lds"
                 :
                 : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(lds_base)), "s"(__builtin_amdgcn_readfirstlane(at))
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// 16 bytes at an address in LDS.
__device__ __forceinline__ uint4 ffn_lds_at(uint32_t at) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = *(const __attribute__((address_space(3))) u32x4 *)at;
    return __builtin_bit_cast(uint4, v);
}

// ---- products: out[m][n] = sum_k a[m][k] b[n][k] (ffn_gemm.h)
enum FfnEpilogue {
    FFN_GATED,   // h = act(a b0') * (a b1')
    FFN_SAVING,  // ... and both products, fp32
    FFN_SCALED,  // ... each times its row's and its column's factor (8-bit operands)
    FFN_PLAIN,   // out = a b0'
};
struct FfnGemmArgs {
    const void *a, *b0, *b1;
    int64_t as, bs;  // strides of rows of k or of rows of m, elements
    int64_t M;
    int N, K;  // columns (of each of b0, b1), products summed
    // b as rows of m: `brows` of them in b0, and from K tile `ktsplit` on in b1
    int ktsplit, brows;
    int act;
    // plain: row m < rows of out, row m - split < rows of out2; other rows go nowhere
    void *out, *out2;  // [..][N]
    int64_t split, rows;
    float *saved;  // [2][M][pitch]
    int64_t pitch;
    const float *a_scale, *b0_scale, *b1_scale;
    // how the product is made (ffn_choose); plain: the K tiles shared out to `splits` grids, whose sums go to part
    bool vec;
    int tile, splits;
    float *part;  // [splits][M][ffn_part_pitch(N)]
    const float *factor;  // plain, fp16: the results times this; NULL: as they are
};
__host__ __device__ inline int64_t ffn_part_pitch(int N) { return ((int64_t)N + 3) / 4 * 4; }

// The tile and the number of parts of a product.  vec: rows at multiples of 16
// bytes (else there is a loop for 64 x 32 only); a_of_m: a as rows of m (not 32 x 32).
enum FfnTileKind { FFN_TILE_256x128, FFN_TILE_256x64, FFN_TILE_128x64, FFN_TILE_64x32, FFN_TILE_32x32 };  // of m, of each half of b
struct FfnPlan {
    int tile, splits;
};
FfnPlan ffn_plan(int64_t M, int N, int K, int value_bytes, bool plain, bool vec, bool a_of_m);
// The plan of a product, into a; a_of_m, b_of_m: operands as rows of m.  False:
// one launch does not hold its blocks.
bool ffn_choose(FfnGemmArgs &a, int dtype, bool plain, bool a_of_m, bool b_of_m);
// The launches take a plan that was chosen.
hipError_t launch_ffn_gated(const FfnGemmArgs &a, FfnEpilogue e, int dtype, int out_dtype, hipStream_t st);
hipError_t launch_ffn_dx(const FfnGemmArgs &a, int dtype, hipStream_t st);  // a: rows of k, b: rows of m
hipError_t launch_ffn_dw(const FfnGemmArgs &a, int dtype, hipStream_t st);  // both: rows of m

// The gradients of g and u, [T][2][Fp], zeros from F to Fp.
struct FfnGateGrad {
    const void *dh;
    int64_t dhs;
    const float *saved;
    int64_t pitch;
    void *dgu;
    int64_t T;
    int F, Fp, act;
    float *range;  // fp16: 2^-k, which the products' results meet, and from kFfnRangeAt on the blocks' largest values
};
constexpr int kFfnRangeBlocks = 1024, kFfnRangeAt = 4;  // floats
hipError_t launch_ffn_gate_grad(const FfnGateGrad &a, int dtype, hipStream_t st);

struct W4Args {
    const void *x;
    const uint8_t *w[2];
    const void *scales[2], *zeros[2];
    void *y;
    int64_t xs, R;
    int D, F, groups, act;
    int has_zeros;  // (without, zeros point to the scales)
};
hipError_t launch_w4(const W4Args &a, int group, bool gated, int dtype, hipStream_t st);

struct NormQuantArgs {
    const void *x, *res, *w;
    void *r;
    uint8_t *q;
    float *scale;
    int64_t R;
    int D;
    float eps;
};
hipError_t launch_norm_quant(const NormQuantArgs &a, int dtype, hipStream_t st);

}  // namespace convlower
