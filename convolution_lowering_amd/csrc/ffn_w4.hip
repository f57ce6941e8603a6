// Products with 4-bit weights for a few tokens:
//
//   y[r,f] = sum over groups G of s[f,G] (sum_{d in G} x[r,d] code[f,d] - z[f,G] sum_{d in G} x[r,d])
//
// Each weight is read once for up to 64 tokens (32 gated ones of groups of 32; 16 of
// float32, and of 16-bit rows at odd multiples of 2 bytes), bound by its way here for few
// of them.  The codes
// become operands of the matrix instructions exactly, so that nothing is
// rounded before the sums of a group (fp32), and a group's scale meets its sum.
//   * 16-bit x: a code's four bits are set into the low digits of 128 (bf16; of 2^-9, in
//     units of 2^-16) or 1024 (fp16), one instruction for two codes; the 128 joins the zero point, whose
//     term needs sum x of the group: one more product, with ones, that leaves it
//     in the lanes that use it.  The two codes are four places apart, so x's
//     eight values of a fragment are put in the same order.
//   * fp32 x: three bf16 parts of 8 bits each, cut, not rounded, so that they add
//     up to x exactly; codes as integers (128 would cost seven of the sum's digits).
// A block has 16 features of each matrix; its wavefronts share out the 128-value
// pieces of the rows and run apart from one another, their sums meet in LDS in a
// fixed order.  Codes and x go from memory to registers, the next pieces' on their
// way and no branch between them (each would end in a wait for all of them).  They
// are loaded along the rows, neighbouring lanes side by side, and come into the
// matrix instructions' order (neighbouring lanes in different rows) by LDS: loaded
// in that order each lane's 16 bytes are an access of its own to the first cache, which
// bounds the kernel from some 8 tokens on (4096 to 10240 gated, bf16, groups of 128: 16 and
// 32 tokens 22 and 33 us, by LDS 16.6 and 22.6).  Up to 4 tokens there is little of x, and
// both are loaded in that order (DIRECT; 1 token 15 us, by LDS 17).  Scales pass
// through LDS as well.
//
// Inside a captured graph, bf16: 10240 to 4096, groups of 128: 1 token 8.5 us, of 21.6
// MB, 32 tokens 16.4, 64 tokens 26.7; 4096 to 10240 gated: 1 token 14.3 us (45 MB),
// 32 tokens 21.6, 64 tokens 40.4; groups of 32: 23.1, 43.6, 65.9, bound by the
// arithmetic on scales, which is four times as much.  (That is of one layer again and
// again, out of the Infinity Cache.  Of 48 in turn, from HBM: 1 token 10.3 us, 2.1 TB/s,
// and 15.8, 2.8 TB/s, 32 tokens 18.4 and 24.8; the launch and the first pieces' way
// are some 5 us of each.)
#include "ffn_internal.h"

namespace convlower {
namespace {

constexpr int kPiece = 128;  // values of a row that a wavefront takes at once: 16 bytes of codes a lane

// Codes and the ones beside them count in units of 1 / UNIT: 2^-16 where the exponent
// has the room, so that no sum of x times 128 or times 15 passes the largest float32
// number where y does not.  The results meet it at the end.
template <typename S>
struct W4Type {  // 16-bit x: one part, codes behind a leading digit
    static constexpr int PARTS = 1;
    static constexpr uint32_t LEAD = __is_same(S, _Float16) ? 0x64006400u : 0x3b003b00u;
    static constexpr float OFFSET = __is_same(S, _Float16) ? 1024.f : 128.f;
    static constexpr uint32_t ONES = __is_same(S, _Float16) ? 0x3c003c00u : 0x37803780u;
    static constexpr float UNIT = __is_same(S, _Float16) ? 1.f : 65536.f;
    typedef S mma_t;
};
template <>
struct W4Type<float> {
    static constexpr int PARTS = 3;
    static constexpr uint32_t LEAD = 0;
    static constexpr float OFFSET = 0.f;
    static constexpr uint32_t ONES = 0x37803780u;
    static constexpr float UNIT = 65536.f;
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
        for (int i = 0; i < 8; ++i) f[i] = __float_as_uint((float)((d >> (4 * i)) & 15) * (1.f / W4Type<S>::UNIT));
        // (four digits: the upper half holds them)
        return make_uint4(__builtin_amdgcn_perm(f[1], f[0], 0x07060302), __builtin_amdgcn_perm(f[3], f[2], 0x07060302),
                          __builtin_amdgcn_perm(f[5], f[4], 0x07060302), __builtin_amdgcn_perm(f[7], f[6], 0x07060302));
    }
}
// Eight 16-bit values of x in the codes' order.
__device__ __forceinline__ uint4 w4_order(const uint4 &t) {
    return make_uint4(__builtin_amdgcn_perm(t.z, t.x, 0x05040100), __builtin_amdgcn_perm(t.z, t.x, 0x07060302),
                      __builtin_amdgcn_perm(t.w, t.y, 0x05040100), __builtin_amdgcn_perm(t.w, t.y, 0x07060302));
}
// Eight float32 values as three bf16 fragments.
__device__ __forceinline__ void w4_parts(const uint4 &lo, const uint4 &hi, uint4 (&out)[3]) {
    const uint32_t v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t p[3][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float x = __uint_as_float(v[i]);
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
// d[j] of lane row q (16 lanes) becomes d[q] of lane row j.
__device__ __forceinline__ void w4_transpose(uint32_t (&d)[4]) {
    const auto a = __builtin_amdgcn_permlane32_swap(d[0], d[2], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(d[1], d[3], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto e = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    d[0] = c[0], d[1] = c[1], d[2] = e[0], d[3] = e[1];
}

// Between a wavefront's lanes that write LDS and those of it that read it, either way:
// its accesses are made in their order, the compiler has to keep it as well.
__device__ __forceinline__ void w4_between_lanes() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

constexpr int kScaleBytes = 8192;  // scales and zero points in LDS at a time (32 gated tokens, groups of 128: 24 us, with 16 KB 30)

template <typename S>
struct W4Scale {
    S scale, zero;
};

// NT: 16-token tiles, all of them a wavefront's; WAVES of them share out the pieces.
// VEC: rows of x at multiples of 4 bytes.
template <typename S, int NT, int WAVES, int GROUP, bool GATED, bool VEC, bool DIRECT>
__device__ __forceinline__ void w4_body(const W4Args &A) {
    using T = W4Type<S>;
    constexpr int NM = GATED ? 2 : 1, SUB = kPiece / GROUP, STEPS = 4 / SUB;
    constexpr int ES = (int)sizeof(S), UNIT = 16 / ES, XL = ES / 2;  // values of a 16-byte load, loads of eight
    constexpr int AHEAD = NT * XL * NM * (SUB == 4 ? 2 : 1) <= 2 ? 2 : 1;                      // pieces under way beside the one worked with
    constexpr int THREADS = WAVES * 64, ROWS = 16 * NM;
    constexpr int SPAN = kScaleBytes / (ROWS * SUB * (int)sizeof(W4Scale<S>)) / (WAVES * AHEAD) * AHEAD;  // turns whose scales have room
    constexpr int PER = SPAN * WAVES * SUB;                          // scales of a row and span
    static_assert(SPAN >= AHEAD && PER % 16 == 0, "scales have room");
    typedef MfmaShape<typename T::mma_t, 16> MF;
    __shared__ W4Scale<S> scales[ROWS * PER];
    // a wavefront's piece of x and of codes; in the end its sums
    constexpr int ROOM = ((DIRECT ? 0 : NT * 16 * kPiece * ES) + NM * 1024) / 16;
    __shared__ uint4 turned[WAVES][ROOM];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), q = lane >> 4;
    const int f0 = blockIdx.x * 16;
    const int64_t r0 = (int64_t)blockIdx.y * 16 * NT;
    const int rows = (int)min((int64_t)16 * NT, A.R - r0);
    const int full = A.D / kPiece, turns = (full + WAVES - 1) / WAVES;  // whole pieces of a row
    const int64_t pitch = A.D / 2;

    // ---- loads: what is not there (rows, pieces) reads as zeros
    __amdgpu_buffer_rsrc_t rw[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) rw[m] = make_rsrc(A.w[m] + f0 * pitch, (uint32_t)(min(16, A.F - f0) * pitch));
    const S *const x0 = (const S *)A.x + r0 * A.xs;
    const __amdgpu_buffer_rsrc_t rx = make_rsrc(x0, (uint32_t)(((int64_t)(rows - 1) * A.xs + A.D) * ES));
    // Load i of a tile's x: rows RPL i + lane / UNITS, unit lane % UNITS of a piece; of
    // codes: row lane / 4, 16 bytes lane % 4.  In LDS unit u of row r lies in place u ^ r,
    // 16 bytes c of row r of codes in c ^ r / 4, so that both ways take all banks.
    constexpr int UNITS = kPiece / UNIT, RPL = 64 / UNITS, LOADS = 16 / RPL;
    const uint32_t code_at = DIRECT ? (uint32_t)((lane & 15) * pitch) + q * 16 : (uint32_t)((lane >> 2) * pitch) + (lane & 3) * 16;
    const int code_first = (DIRECT ? q : lane & 3) * 32;  // its first value of a piece
    auto unit_of = [&](int i) {
        if constexpr (!DIRECT) return lane % UNITS;
        const int j = i / XL;
        return (SUB == 1 ? q * 4 + j : j * 4 + q) * XL + i % XL;
    };
    auto row_of = [&](int i) { return DIRECT ? lane & 15 : RPL * i + lane / UNITS; };
    struct Piece {
        uint4 w[NM], x[NT][LOADS];
    };
    auto load_x = [&](Piece &p, int piece) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int row = 16 * n + row_of(i), unit = unit_of(i);
                const bool in = piece * kPiece + unit * UNIT < A.D;
                if constexpr (VEC) {
                    p.x[n][i] = __builtin_bit_cast(
                        uint4, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)(in ? (uint32_t)(row * A.xs * ES) + unit * 16 : kOutOfRange), piece * kPiece * ES, 0));
                } else {  // (the first values in their place, and zeros)
                    const bool here = in && row < rows;
                    const FfnAnyVec<S, UNIT> v = *(const FfnAnyVec<S, UNIT> *)(x0 + (here ? row * A.xs + piece * kPiece + unit * UNIT : 0));
                    __builtin_memcpy(&p.x[n][i], &v, 16);
                    if (!here) p.x[n][i] = make_uint4(0, 0, 0, 0);
                }
            }
    };
    auto load = [&](Piece &p, int turn) {
        const int piece = turn * WAVES + wave;
#pragma unroll
        for (int m = 0; m < NM; ++m)
            p.w[m] = __builtin_bit_cast(
                uint4, __builtin_amdgcn_raw_buffer_load_b128(rw[m], (int)(piece < full ? code_at : kOutOfRange), piece * (kPiece / 2), 0));
        load_x(p, piece);
    };
    // This wavefront's piece in LDS, and its way there.
    uint4 *const mine = turned[wave];
    const int code_to = (lane >> 2) * 4 + ((lane & 3) ^ (lane >> 4)), code_from = (lane & 15) * 4 + (q ^ ((lane & 15) >> 2));
    auto turn_x = [&](const Piece &p) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int row = row_of(i);
                mine[(n * 16 + row) * UNITS + (unit_of(i) ^ row)] = p.x[n][i];
            }
    };
    // (16 rows of one group lie on different banks: gated groups of 32, one token 27.5 us, unmixed 34.7)
    auto scale_at = [](int row, int g) { return row * PER + (g ^ (row & 15)); };
    auto scales_of = [&](int turn) {  // of the span that begins with this turn
        const int g0 = turn * WAVES * SUB, per = min(PER, (A.groups + SUB - 1) / SUB * SUB - g0);
#pragma unroll 4
        for (int u = threadIdx.x; u < ROWS * per; u += THREADS) {
            const int row = u / per, g = g0 + u % per;
            const bool up = GATED && row >= 16;
            W4Scale<S> v = {S(0), S(0)};
            if (g < A.groups) {
                const int64_t at = (int64_t)min(f0 + (row & 15), A.F - 1) * A.groups + g;
                v.scale = ((const S *)(up ? A.scales[1] : A.scales[0]))[at];
                v.zero = A.has_zeros ? ((const S *)(up ? A.zeros[1] : A.zeros[0]))[at] : mix_out<S>(8.f);
            }
            scales[scale_at(row, g - g0)] = v;
        }
    };

    f32x4_t acc[NT][NM] = {};
    const uint4 ones = make_uint4(T::ONES, T::ONES, T::ONES, T::ONES);
    // Piece `in` of the span; if not `there`, to no effect (a code of 0 is not a weight of 0).
    auto work = [&](const Piece &p, int in, bool there) {
        if constexpr (!DIRECT) {
            w4_between_lanes();  // the last piece has been read
            turn_x(p);
#pragma unroll
            for (int m = 0; m < NM; ++m) mine[NT * 16 * UNITS + m * 64 + code_to] = p.w[m];
            w4_between_lanes();
        }
        uint32_t w[NM][4];
#pragma unroll
        for (int m = 0; m < NM; ++m) {
            const uint4 v = DIRECT ? p.w[m] : mine[NT * 16 * UNITS + m * 64 + code_from];
            w[m][0] = v.x, w[m][1] = v.y, w[m][2] = v.z, w[m][3] = v.w;
            if constexpr (SUB > 1) w4_transpose(w[m]);  // a product's 32 values lie in one group
        }
#pragma unroll
        for (int g = 0; g < SUB; ++g) {
            f32x4_t part[NT][NM] = {}, all[NT] = {};
#pragma unroll
            for (int j = g * STEPS; j < (g + 1) * STEPS; ++j) {
                uint4 codes[NM];
#pragma unroll
                for (int m = 0; m < NM; ++m) codes[m] = w4_codes<S>(w[m][j]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int first = (SUB == 1 ? q * 4 + j : j * 4 + q) * XL, row = lane & 15;
                    const uint4 *at = mine + (n * 16 + row) * UNITS;
                    uint4 x[T::PARTS];
                    if constexpr (DIRECT && ES == 2) x[0] = w4_order(p.x[n][j]);
                    else if constexpr (DIRECT) w4_parts(p.x[n][j * XL], p.x[n][j * XL + XL - 1], x);
                    else if constexpr (ES == 2) x[0] = w4_order(at[first ^ row]);
                    else w4_parts(at[first ^ row], at[(first + 1) ^ row], x);
#pragma unroll
                    for (int k = 0; k < T::PARTS; ++k) {
                        MF::mma(x[k], ones, all[n]);
#pragma unroll
                        for (int m = 0; m < NM; ++m) MF::mma(x[k], codes[m], part[n][m]);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                const W4Scale<S> sz = scales[scale_at(m * 16 + (lane & 15), in * SUB + g)];
                const float s = there ? mix_f32(sz.scale) : 0.f, z = there ? T::OFFSET + mix_f32(sz.zero) : 0.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[n][m][i] = fmaf(s, fmaf(-z, all[n][i], part[n][m][i]), acc[n][m][i]);
            }
            __builtin_amdgcn_sched_barrier(0);  // (one group's operands at a time: there are no registers for more)
        }
    };

    Piece piece[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) load(piece[i], i);
    scales_of(0);
    __syncthreads();
    int in_span = 0;
#pragma nounroll
    for (int turn = 0; turn < turns; turn += AHEAD) {
        if (in_span == SPAN) {
            __syncthreads();  // nobody reads the last span's scales any more
            scales_of(turn);
            __syncthreads();
            in_span = 0;
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            work(piece[i], (in_span + i) * WAVES + wave, (turn + i) * WAVES + wave < full);
            load(piece[i], turn + i + AHEAD);
        }
        in_span += AHEAD;
    }
    if (A.D % kPiece) {  // what is left of a row, word by word
        const int first = full / (SPAN * WAVES) * SPAN;
        __syncthreads();
        scales_of(first);
        __syncthreads();
        if (full % WAVES == wave) {
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                uint32_t v[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    v[j] = __builtin_amdgcn_raw_buffer_load_b32(
                        rw[m], (int)(full * kPiece + code_first + j * 8 < A.D ? code_at + j * 4 : kOutOfRange), full * (kPiece / 2), 0);
                piece[0].w[m] = make_uint4(v[0], v[1], v[2], v[3]);
            }
            load_x(piece[0], full);
            work(piece[0], full - first * WAVES, true);
        }
    }

    // Result: lane l holds feature l % 16 and tokens 4 (l / 16) .. + 3 of a tile.
    static_assert(NM * 64 <= ROOM, "the sums' room");
    w4_between_lanes();
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        if (n) __syncthreads();
#pragma unroll
        for (int m = 0; m < NM; ++m) mine[m * 64 + lane] = __builtin_bit_cast(uint4, acc[n][m]);
        __syncthreads();
        const int tok = threadIdx.x >> 4, f = threadIdx.x & 15, at = (tok >> 2) * 16 + f;
        const int64_t r = r0 + 16 * n + tok;
        if (tok < 16 && r < A.R && f0 + f < A.F) {
            float y[NM];
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                y[m] = 0.f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) y[m] += ((const float *)&turned[w][m * 64 + at])[tok & 3];
                y[m] *= T::UNIT;
            }
            ((S *)A.y)[r * A.F + f0 + f] = mix_out<S>(GATED ? ffn_act<S>(y[0], A.act) * y[NM - 1] : y[0]);
        }
    }
}
template <typename S, int NT, int WAVES, int GROUP, bool GATED, bool VEC, bool DIRECT>
__global__ __launch_bounds__(WAVES * 64, NT == 1 ? (GROUP == 128 ? 4 : 3) : NT == 2 && GROUP == 128 ? 3 : 2) void w4_kernel(W4Args A) {
    w4_body<S, NT, WAVES, GROUP, GATED, VEC, DIRECT>(A);
}

template <typename S, int NT, int WAVES, int GROUP, bool GATED, bool VEC, bool DIRECT>
hipError_t w4_run(const W4Args &a, hipStream_t st) {
    const int64_t x = (a.F + 15) / 16, y = (a.R + 16 * NT - 1) / (16 * NT);
    if (!grid_fits(x, WAVES * 64, y)) return kTooLarge;
    hipLaunchKernelGGL((w4_kernel<S, NT, WAVES, GROUP, GATED, VEC, DIRECT>), dim3((unsigned)x, (unsigned)y), dim3(WAVES * 64), 0, st, a);
    return hipGetLastError();
}
// Blocks of eight wavefronts where all of them are on the CUs at once: one a CU (256
// blocks, 4096 wide gated bf16, one token 6.6 us, with four wavefronts 7.6; 32 tokens 10.1
// and 12.3), two where a second one fits beside it, which several token tiles and
// float32's LDS leave no room for (512 blocks, one token 10.7 and 11.2, groups of 32 16.0
// and 20.7; but 32 tokens 19.6 and 17.8, float32, 8 tokens 25.3 and 23.5).  Else four, of which a CU
// holds more (640 blocks, one token 15.6 and 14.3, 32 tokens 26.2 and 21.3; 128 tokens of 4096
// features 29.1 and 26.2).  (Eight, not sixteen: one token of 4096 x 4096 5.4 us against 7.1.)
// Four token tiles at once but for the groups whose sums do not fit the registers (gated,
// 32, 64 tokens: two by two 74 us; with the scales' rows still on one bank 84, and 114
// four at once).
template <typename S, int NT, int GROUP, bool GATED, bool DIRECT>
hipError_t w4_waves(const W4Args &a, hipStream_t st) {
    const int64_t blocks = ((a.F + 15) / 16) * ((a.R + 16 * NT - 1) / (16 * NT));
    constexpr int at_once = NT == 1 && (DIRECT || sizeof(S) == 2) ? 512 : 256;
    return blocks > at_once ? w4_run<S, NT, 4, GROUP, GATED, true, DIRECT>(a, st) : w4_run<S, NT, 8, GROUP, GATED, true, DIRECT>(a, st);
}
template <typename S, int GROUP, bool GATED>
hipError_t w4_tokens(const W4Args &a, hipStream_t st) {
    if constexpr (sizeof(S) == 4) {
        return a.R <= 4 ? w4_waves<S, 1, GROUP, GATED, true>(a, st) : w4_waves<S, 1, GROUP, GATED, false>(a, st);
    } else {
        if ((uintptr_t)a.x % 4 || a.xs % 2) return w4_run<S, 1, 8, GROUP, GATED, false, false>(a, st);
        if (a.R <= 4) return w4_waves<S, 1, GROUP, GATED, true>(a, st);
        if (a.R <= 16) return w4_waves<S, 1, GROUP, GATED, false>(a, st);
        if (a.R <= 32 || (GROUP == 32 && GATED)) return w4_waves<S, 2, GROUP, GATED, false>(a, st);
        if constexpr (GROUP != 32 || !GATED) return w4_waves<S, 4, GROUP, GATED, false>(a, st);
    }
    return hipErrorInvalidValue;
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
