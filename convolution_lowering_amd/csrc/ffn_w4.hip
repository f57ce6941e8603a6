// Products with 4-bit weights for a few tokens:
//
//   y[r,f] = sum over groups G of s[f,G] (sum_{d in G} x[r,d] code[f,d] - z[f,G] sum_{d in G} x[r,d])
//
// Each weight is read once, for up to 64 tokens: HBM bound for few of them.  The codes
// become operands of the matrix instructions exactly, so that nothing is
// rounded before the sums of a group (fp32), and a group's scale meets its sum.
//   * 16-bit x: a code's four bits are set into the low digits of 128 (bf16) or
//     1024 (fp16), one instruction for two codes; the 128 joins the zero point, whose
//     term needs sum x of the group: one more product, with ones, that leaves it
//     in the lanes that use it.  The two codes are four places apart, so x's
//     eight values of a fragment are put in the same order.
//   * fp32 x: three bf16 parts of 8 bits each, cut, not rounded, so that they add
//     up to x exactly; codes as integers (128 would cost seven of the sum's digits).
// A block has 16 FT features of each matrix; its wavefronts share out the 128-value
// pieces of the rows, and their sums meet in LDS in a fixed order.
#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int kWaves = 8;
constexpr int kPiece = 128;  // values of a row that a wavefront takes at once: 16 bytes of codes a lane

template <typename S>
struct W4Type {  // 16-bit x: one part, codes behind a leading digit
    static constexpr int PARTS = 1;
    static constexpr uint32_t LEAD = sizeof(S) == 2 && __is_same(S, _Float16) ? 0x64006400u : 0x43004300u;
    static constexpr float OFFSET = __is_same(S, _Float16) ? 1024.f : 128.f;
    typedef S mma_t;
};
template <>
struct W4Type<float> {
    static constexpr int PARTS = 3;
    static constexpr uint32_t LEAD = 0;
    static constexpr float OFFSET = 0.f;
    typedef uint16_t mma_t;
};

// Eight codes as a fragment: (0,4), (1,5), (2,6), (3,7), or in their order for fp32 x.
template <typename S>
__device__ __forceinline__ uint4 w4_codes(uint32_t d) {
    if constexpr (sizeof(S) == 2) {
        constexpr uint32_t lead = W4Type<S>::LEAD, mask = 0x000f000fu;
        return make_uint4((d & mask) | lead, ((d >> 4) & mask) | lead, ((d >> 8) & mask) | lead, ((d >> 12) & mask) | lead);
    } else {
        uint32_t f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __float_as_uint((float)((d >> (4 * i)) & 15));
        // (whole numbers up to 15: the upper half holds them)
        return make_uint4(__builtin_amdgcn_perm(f[1], f[0], 0x07060302), __builtin_amdgcn_perm(f[3], f[2], 0x07060302),
                          __builtin_amdgcn_perm(f[5], f[4], 0x07060302), __builtin_amdgcn_perm(f[7], f[6], 0x07060302));
    }
}
// Eight values of x as fragments, in the codes' order.
template <typename S>
__device__ __forceinline__ void w4_x(const FfnAnyVec<S, 8> &v, uint4 (&out)[W4Type<S>::PARTS]) {
    if constexpr (sizeof(S) == 2) {
        uint4 t;
        __builtin_memcpy(&t, &v, 16);
        out[0] = make_uint4(__builtin_amdgcn_perm(t.z, t.x, 0x05040100), __builtin_amdgcn_perm(t.z, t.x, 0x07060302),
                            __builtin_amdgcn_perm(t.w, t.y, 0x05040100), __builtin_amdgcn_perm(t.w, t.y, 0x07060302));
    } else {
        uint32_t p[3][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float x = v.v[i];
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                p[k][i] = __float_as_uint(x) & 0xffff0000u;
                x -= __uint_as_float(p[k][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < 3; ++k)
            out[k] = make_uint4(__builtin_amdgcn_perm(p[k][1], p[k][0], 0x07060302), __builtin_amdgcn_perm(p[k][3], p[k][2], 0x07060302),
                                __builtin_amdgcn_perm(p[k][5], p[k][4], 0x07060302), __builtin_amdgcn_perm(p[k][7], p[k][6], 0x07060302));
    }
}
// d[j] of lane row q (16 lanes) becomes d[q] of lane row j.
__device__ __forceinline__ void w4_transpose(uint32_t (&d)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = c[0], d[1] = c[1], d[2] = e[0], d[3] = e[1];
}

// NT: 16-token tiles; FT: 16-feature tiles of each of NM matrices.
template <typename S, int NT, int FT, int GROUP, bool GATED>
__device__ __forceinline__ void w4_body(const W4Args &A) {
    using T = W4Type<S>;
    constexpr int NM = GATED ? 2 : 1, TILES = NM * FT, SUB = kPiece / GROUP, STEPS = 4 / SUB;
    constexpr int AHEAD = NT == 1 ? 4 : NT == 2 ? 2 : 1;  // pieces under way
    typedef MfmaShape<typename T::mma_t, 16> MF;
    __shared__ f32x4_t sums[kWaves][TILES][64];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
    const int f0 = blockIdx.x * 16 * FT;
    const int64_t r0 = (int64_t)blockIdx.y * 16 * NT;
    const int pieces = (A.D + kPiece - 1) / kPiece;
    const int first = (int)((int64_t)pieces * wave / kWaves), last = (int)((int64_t)pieces * (wave + 1) / kWaves);
    const int64_t pitch = A.D / 2;

    struct Piece {
        uint32_t w[TILES][4];
        S s[TILES][SUB], z[TILES][SUB];
        FfnAnyVec<S, 8> x[NT][4];
    } buf[AHEAD];
    auto load = [&](Piece &p, int at) {
        const int d0 = at * kPiece;
        if (at >= last) return;
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
            const int m = t / FT;
            const int f = min(f0 + (t % FT) * 16 + (lane & 15), A.F - 1);
            const uint8_t *row = A.w[m] + f * pitch + (d0 + q * 32) / 2;
            if (d0 + q * 32 + 32 <= A.D) {
                const FfnAnyVec<uint32_t, 4> v = *(const FfnAnyVec<uint32_t, 4> *)row;
#pragma unroll
                for (int j = 0; j < 4; ++j) p.w[t][j] = v.v[j];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) p.w[t][j] = d0 + q * 32 + j * 8 < A.D ? *(const uint32_t *)(row + j * 4) : 0u;
            }
#pragma unroll
            for (int g = 0; g < SUB; ++g) {
                const int64_t i = (int64_t)f * A.groups + min(at * SUB + g, A.groups - 1);
                p.s[t][g] = ((const S *)A.scales[m])[i];
                if (A.zeros[m]) p.z[t][g] = ((const S *)A.zeros[m])[i];
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int64_t r = r0 + 16 * n + (lane & 15);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int d = d0 + (SUB == 1 ? q * 32 + j * 8 : j * 32 + q * 8);
                FfnAnyVec<S, 8> v = {};
                if (r < A.R && d < A.D) v = *(const FfnAnyVec<S, 8> *)((const S *)A.x + r * A.xs + d);
                p.x[n][j] = v;
            }
        }
    };

    f32x4_t acc[NT][TILES] = {};
    uint4 ones;
    {
        constexpr uint32_t one = __is_same(S, _Float16) ? 0x3c003c00u : 0x3f803f80u;
        ones = make_uint4(one, one, one, one);
    }
    auto work = [&](Piece &p) {
        if constexpr (SUB > 1) {  // a product's 32 values lie in one group
#pragma unroll
            for (int t = 0; t < TILES; ++t) w4_transpose(p.w[t]);
        }
#pragma unroll
        for (int g = 0; g < SUB; ++g) {
            f32x4_t part[NT][TILES] = {}, all[NT] = {};
#pragma unroll
            for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) {
                uint4 c[TILES];
#pragma unroll
                for (int t = 0; t < TILES; ++t) c[t] = w4_codes<S>(p.w[t][j]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint4 x[T::PARTS];
                    w4_x<S>(p.x[n][j], x);
#pragma unroll
                    for (int k = 0; k < T::PARTS; ++k) {
                        MF::mma(x[k], ones, all[n]);
#pragma unroll
                        for (int t = 0; t < TILES; ++t) MF::mma(x[k], c[t], part[n][t]);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < TILES; ++t) {
                const float s = mix_f32(p.s[t][g]), z = T::OFFSET + (A.zeros[t / FT] ? mix_f32(p.z[t][g]) : 8.f);
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][t][i] = fmaf(s, fmaf(-z, all[n][i], part[n][t][i]), acc[n][t][i]);
            }
        }
    };

#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(buf[i], first + i);
    for (int at = first; at < last; at += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (at + i < last) {
                work(buf[i]);
                load(buf[i], at + i + AHEAD);
            }
    }

    // Result: lane l holds feature l % 16 and tokens 4 (l / 16) .. + 3 of a tile.
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n) __syncthreads();
#pragma unroll
        for (int t = 0; t < TILES; ++t) sums[wave][t][lane] = acc[n][t];
        __syncthreads();
        for (int i = threadIdx.x; i < FT * 256; i += kWaves * 64) {
            const int f = (i & 15) + 16 * (i >> 8), tok = (i >> 4) & 15, at = (tok >> 2) * 16 + (i & 15);
            const int64_t r = r0 + 16 * n + tok;
            if (r >= A.R || f0 + f >= A.F) continue;
            float y[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                y[m] = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) y[m] += sums[w][m * FT + (i >> 8)][at][tok & 3];
            }
            ((S *)A.y)[r * A.F + f0 + f] = mix_out<S>(GATED ? ffn_act<S>(y[0], A.act) * y[NM - 1] : y[0]);
        }
    }
}
template <typename S, int NT, int FT, int GROUP, bool GATED>
__global__ __launch_bounds__(kWaves * 64) void w4_kernel(W4Args A) {
    w4_body<S, NT, FT, GROUP, GATED>(A);
}

template <typename S, int NT, int FT, int GROUP, bool GATED>
hipError_t w4_run(const W4Args &a, hipStream_t st) {
    const int64_t x = (a.F + 16 * FT - 1) / (16 * FT), y = (a.R + 16 * NT - 1) / (16 * NT);
    if (!grid_fits(x, kWaves * 64, y)) return kTooLarge;
    hipLaunchKernelGGL((w4_kernel<S, NT, FT, GROUP, GATED>), dim3((unsigned)x, (unsigned)y), dim3(kWaves * 64), 0, st, a);
    return hipGetLastError();
}
template <typename S, int GROUP, bool GATED>
hipError_t w4_tokens(const W4Args &a, hipStream_t st) {
    if (a.R <= 16) return w4_run<S, 1, 1, GROUP, GATED>(a, st);
    if (a.R <= 32) return w4_run<S, 2, 1, GROUP, GATED>(a, st);
    return w4_run<S, 4, 1, GROUP, GATED>(a, st);
}
template <typename S>
hipError_t w4_typed(const W4Args &a, int group, bool gated, hipStream_t st) {
    if (group == 32) return gated ? w4_tokens<S, 32, true>(a, st) : w4_tokens<S, 32, false>(a, st);
    if (group == 64) return gated ? w4_tokens<S, 64, true>(a, st) : w4_tokens<S, 64, false>(a, st);
    return gated ? w4_tokens<S, 128, true>(a, st) : w4_tokens<S, 128, false>(a, st);
}

}  // namespace

hipError_t launch_w4(const W4Args &a, int group, bool gated, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return w4_typed<float>(a, group, gated, st);
    if (dtype == CONV_DTYPE_FP16) return w4_typed<_Float16>(a, group, gated, st);
    return w4_typed<uint16_t>(a, group, gated, st);
}

}  // namespace convlower
