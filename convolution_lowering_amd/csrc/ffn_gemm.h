// Products on the matrix cores: out[m][n] = sum_k a[m][k] b[n][k].  An operand
// lies with its k together ("rows of k": activations and weights on the way
// forward) or with its m or n together ("rows of m": what the gradients' products
// sum over runs down the columns of the same tensors).
//
// A K tile is 128 bytes of each row of k (64 16-bit values, 32 float32, 128 e4m3),
// or as many rows of m.  In LDS it lies in regions of W rows or columns:
//   * rows of k: W rows of 8 chunks of 16 bytes; chunk c of row r in slot 8 r + (c
//     ^ (r / 2) % 8).  A fragment read takes 16 rows of one chunk: this puts them on
//     the 16 groups of banks of a 256-byte line.  Which values a lane's chunk holds
//     does not matter to a sum as long as both operands agree, so all types read
//     the same two chunks of a row, c = lane / 16 and that plus 4, and differ only in
//     the instruction that takes them.
//   * rows of m: one LDS row for each k.  16-bit fragments come by the transposing
//     read: 16 lanes read 16 columns of four rows and each gets its column of
//     them, the same values a chunk of k would hold.  float32 ones are read one by
//     one (their matrix instructions are 16 times slower).  Chunks are exchanged
//     within a row so that the rows of one read lie on different banks.
//
// b is the matrix instruction's left operand, so that a lane's four results are
// four neighbours of one output row.
//
// Bound by the matrix cores from some hundred tokens on, below by the weights' way
// from HBM.  Kernel times, MI355X (an 8192 cubed bf16 product of the library 1413
// TFLOP/s, e4m3 2676): gated forward, 5003 tokens, 4096 to 10240: bf16 591 to 660 us (1270 to
// 1420 TFLOP/s); 8192 tokens e4m3 509 to 590 (2330 to 2700); training, 8192 tokens, 4096 to
// 8192: forward with g and u saved 940 us (1170; 671 MB of
// results, of which 764 MB leave: h goes in pieces of 32 bytes, and between two of one 64-byte
// piece lie stores of g and u), dx 730 (1500), dw 790
// (1390); 200 tokens 59 us, 4 tokens 39 (168 MB of weights,
// all from HBM, 4.3 TB/s; of one layer again and again, mostly from the Infinity Cache, 25).  The matrix
// cores are busy 64 to 87 % of the time, no LDS access meets another's bank.
#pragma once

#include <type_traits>

#include "ffn_internal.h"

namespace convlower {
namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// acc += b's rows x a's rows over the two chunks of each.
template <typename S>
__device__ __forceinline__ void ffn_mma(const uint4 (&b)[2], const uint4 (&a)[2], f32x4_t &acc) {
    if constexpr (sizeof(S) == 1) {
        i32x8_t x, y;
        __builtin_memcpy(&x, &b, 32);
        __builtin_memcpy(&y, &a, 32);
        // (e4m3 both; without block scales, which zeros ask for)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);
    } else if constexpr (sizeof(S) == 4) {
        // The tile's 32 products are added up by themselves: in one chain of K
        // additions a float32 result loses sqrt(K / 32) times as much.
        f32x4_t part = {};
        MfmaShape<S, 16>::mma(b[0], a[0], part);
        MfmaShape<S, 16>::mma(b[1], a[1], part);
        acc += part;
    } else {
        MfmaShape<S, 16>::mma(b[0], a[0], acc);
        MfmaShape<S, 16>::mma(b[1], a[1], acc);
    }
}

// A region of W rows of k, or of W columns of rows of m (MM).
template <typename S, bool MM, int W>
struct FfnRegion {
    static constexpr int ES = (int)sizeof(S);
    static constexpr int KROWS = 128 / ES;               // rows of m in a K tile
    static constexpr int PITCH = MM ? W * ES : 128;      // bytes of an LDS row
    static constexpr int CHUNKS = PITCH / 16;
    static constexpr int LOADS = W / 8;                  // 1 KB loads that fill it
    static constexpr int ROWS_PER_LOAD = 64 / CHUNKS;
    __device__ static __forceinline__ int swizzle(int row) {
        if constexpr (!MM) return (row >> 1) & 7;
        else if constexpr (ES == 4) return 4 * ((row >> 2) & 3);
        else if constexpr (W == 128) return 2 * ((row & 3) | (((row >> 3) & 1) << 2));
        else return 2 * (((row >> 1) & 1) | (((row >> 3) & 1) << 1));
    }
    // Which LDS row, and which of its chunks, lane `lane` of load q brings.
    __device__ static __forceinline__ int load_row(int q, int lane) { return q * ROWS_PER_LOAD + lane / CHUNKS; }
    __device__ static __forceinline__ int load_chunk(int q, int lane) {
        return (lane % CHUNKS) ^ swizzle(load_row(q, lane));
    }
};

// A wavefront's fragments of NT tiles of 16, from row or column `first` of a region.
template <typename S, bool MM, int W, int NT>
struct FfnFragments {
    using R = FfnRegion<S, MM, W>;
    uint32_t at[MM ? NT : 2];
    __device__ __forceinline__ void init(uint32_t region, int first, int lane) {
        const int g = lane >> 4, t = lane & 15;
        if constexpr (!MM) {
#pragma unroll
            for (int j = 0; j < 2; ++j) at[j] = region + (first + t) * 128 + (((j * 4 + g) ^ (t >> 1)) * 16);
        } else if constexpr (R::ES == 2) {
            const int row = 8 * g + (t >> 2);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                at[i] = region + row * R::PITCH + ((((first >> 3) + 2 * i) ^ R::swizzle(row)) + ((t & 3) >> 1)) * 16 + (t & 1) * 8;
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i)
                at[i] = region + 4 * g * R::PITCH + ((((first >> 2) + 4 * i) ^ (4 * g)) + (t >> 2)) * 16 + (t & 3) * 4;
        }
    }
    // The same `by` times 4 KB on.  A read's constant offset reaches 64 KB, and what
    // lies further would cost the compiler one register a fragment; behind the
    // asm these addresses are registers of their own (with known alignment).
    __device__ __forceinline__ FfnFragments moved(uint32_t by) const {
        FfnFragments f = *this;
        asm("" : "+v"(by));
#pragma unroll
        for (int i = 0; i < (MM ? NT : 2); ++i) f.at[i] += by << 12;
        return f;
    }
    // Chunk j of tile i; add: the stage, or another region like this one.
    __device__ __forceinline__ uint4 get(int i, int j, uint32_t add) const {
        if constexpr (!MM) {
            return ffn_lds_at(at[j] + add + i * 2048);
        } else if constexpr (R::ES == 2) {
            typedef short s16x4 __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4 *ptr;
            const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(at[i] + add + 32 * j * R::PITCH));
            const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(at[i] + add + (32 * j + 4) * R::PITCH));
            return __builtin_bit_cast(uint4, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            uint32_t v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                v[e] = *(const __attribute__((address_space(3))) uint32_t *)(at[i] + add + (16 * j + e) * R::PITCH);
            return make_uint4(v[0], v[1], v[2], v[3]);
        }
    }
};

// Tiles in an order that keeps what the blocks of one XCD work on at a time
// nearly square: XCD x (blocks x, x + 8, ...) has a contiguous run of the list,
// in which groups of up to `group` row tiles go through all column tiles.
__device__ __forceinline__ void ffn_tile(int mt, int nt, int group, int *m, int *n) {
    const uint32_t b = blockIdx.x, total = (uint32_t)mt * nt;
    const uint32_t xcd = b & 7, q = total >> 3, r = total & 7;
    const uint32_t l = xcd * q + min(xcd, r) + (b >> 3);
    const uint32_t span = (uint32_t)group * nt, g = l / span, in = l - g * span;
    const uint32_t rows = min((uint32_t)group, (uint32_t)mt - g * group);
    *n = (int)(in / rows);
    *m = (int)(g * group + (in - (uint32_t)*n * rows));
}

// Four neighbouring results of row m from column n.
template <typename O>
__device__ __forceinline__ void ffn_put4(O *row, int n, int N, const float (&v)[4]) {
    if (n + 4 <= N && (uintptr_t)(row + n) % (4 * sizeof(O)) == 0) {
        store4(row + n, v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (n + i < N) row[n + i] = mix_out<O>(v[i]);
    }
}
template <typename O, FfnEpilogue EPI, int ACT>
__device__ __forceinline__ void ffn_gated_out(const FfnGemmArgs &A, int64_t m, int n, const f32x4_t &ga,
                                              const f32x4_t &ua) {
    float g[4], u[4], h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = ga[i], u[i] = ua[i];
    if constexpr (EPI == FFN_SCALED) {
        const float s = A.a_scale[m];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = min(n + i, A.N - 1);
            g[i] *= s * A.b0_scale[c];
            u[i] *= s * A.b1_scale[c];
        }
    }
    if constexpr (EPI == FFN_SAVING) {  // (rows of the saved values are whole 16-byte pieces)
        float *p = A.saved + m * A.pitch + n;
        store4(p, g[0], g[1], g[2], g[3]);
        store4(p + A.M * A.pitch, u[0], u[1], u[2], u[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = ffn_act<O>(g[i], ACT) * u[i];
    ffn_put4((O *)A.out + m * A.N, n, A.N, h);
}
// f with the activation as a constant: one branch for all results.
template <typename F>
__device__ __forceinline__ void ffn_with_act(int act, F &&f) {
    switch (act) {
        case FFN_ACT_SILU: f(std::integral_constant<int, FFN_ACT_SILU>()); break;
        case FFN_ACT_SIGMOID: f(std::integral_constant<int, FFN_ACT_SIGMOID>()); break;
        case FFN_ACT_GELU: f(std::integral_constant<int, FFN_ACT_GELU>()); break;
        default: f(std::integral_constant<int, FFN_ACT_NONE>());
    }
}
template <typename O>
__device__ __forceinline__ float ffn_factor(const FfnGemmArgs &A) {
    if constexpr (__is_same(O, _Float16)) return A.factor ? *A.factor : 1.f;
    return 1.f;
}
template <typename O>
__device__ __forceinline__ void ffn_plain_out(const FfnGemmArgs &A, int64_t m, int n, const f32x4_t &acc, float by) {
    if (A.splits > 1) {  // this part's sums; their rows are whole 16-byte pieces
        *(float4 *)(A.part + ((int64_t)blockIdx.y * A.M + m) * ffn_part_pitch(A.N) + n) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        return;
    }
    const float v[4] = {acc[0] * by, acc[1] * by, acc[2] * by, acc[3] * by};
    const bool second = m >= A.split;
    const int64_t row = second ? m - A.split : m;
    if (row < A.rows) ffn_put4((O *)(second ? A.out2 : A.out) + row * A.N, n, A.N, v);
}

// The K tiles of an operand of rows of m, one after another: `rows` of them from
// p0 and, from tile `split` on, as many from p1, `width` bytes of each.
template <typename S>
struct FfnRowsOfM {
    static constexpr int KROWS = 128 / (int)sizeof(S);
    const char *p, *p1;
    uint32_t step, behind;  // behind: what of a row is past its `width` bytes
    int rows, left, until;  // left: rows from here on; until: tiles before p1's
    __device__ __forceinline__ void init(const void *p0, const void *p1_, int64_t stride, int rows_, int64_t width, int split, int first) {
        step = (uint32_t)(stride * (int64_t)sizeof(S));
        behind = step - (uint32_t)(width * (int64_t)sizeof(S));
        const bool other = first >= split;
        first -= other ? split : 0;
        p = (const char *)(other ? p1_ : p0) + (uint64_t)step * KROWS * (uint32_t)first;
        p1 = (const char *)p1_, rows = rows_, left = rows_ - first * KROWS;
        until = other ? INT32_MAX : split - first;
    }
    __device__ __forceinline__ void next() {
        const bool other = --until == 0;
        p = other ? p1 : p + (uint64_t)step * KROWS;
        left = other ? rows : left - KROWS;
    }
    // The tile as a buffer: no bytes where no rows are left.
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t tile() const {
        const int n = left < KROWS ? left : KROWS;
        return make_rsrc(p, n > 0 ? (uint32_t)n * step - behind : 0u);
    }
};

// ---- the loop for any size: four wavefronts, 2 x 2, over BM of a's m and BH of
// each of b0 and b1 (or 2 BH of b0 alone).  Chunks at multiples of 16 bytes are
// copied into LDS by the load instructions that write there (three stages, two
// tiles under way); others (ANY) pass through registers, one tile ahead, the last
// values of a row one by one.
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY, bool AM, bool BMM>
__device__ __forceinline__ void ffn_small_body(const FfnGemmArgs &A) {
    constexpr bool PLAIN = EPI == FFN_PLAIN;
    constexpr int ES = (int)sizeof(S), V = 16 / ES, ST = ANY ? 2 : 3;
    constexpr int TM = BM / 32, TN = BH / 32;  // 16-wide tiles of a wavefront: of a, and of each half of b
    using RA = FfnRegion<S, AM, BM>;
    using RB = FfnRegion<S, BMM, 2 * BH>;
    constexpr int IA = RA::LOADS / 4, IB = RB::LOADS / 4, IPW = IA + IB;  // loads of a wavefront per tile
    static_assert(BM % 32 == 0 && BH % 32 == 0 && (PLAIN || !BMM), "loads and wavefronts split evenly");
    constexpr uint32_t STAGE = (BM + 2 * BH) * 128;
    __shared__ alignas(16) char lds[ST * STAGE];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    constexpr int BN = PLAIN ? 2 * BH : BH;
    ffn_tile((int)((A.M + BM - 1) / BM), (A.N + BN - 1) / BN, 8, &mt, &nt);
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;
    const uint32_t kbytes = (uint32_t)A.K * ES, abytes = (uint32_t)(A.as * ES), bbytes = (uint32_t)(A.bs * ES);
    const int tiles = (A.K + RA::KROWS - 1) / RA::KROWS;
    const int k0 = PLAIN ? (int)((int64_t)tiles * blockIdx.y / A.splits) : 0;  // this part's tiles
    const int nk = (PLAIN ? (int)((int64_t)tiles * (blockIdx.y + 1) / A.splits) : tiles) - k0;
    const int am = (int)min((int64_t)BM, A.M - m0);  // a's m that are there
    const char *abase = (const char *)A.a + m0 * (AM ? ES : A.as * ES);
    FfnRowsOfM<S> ma, mb;
    if constexpr (AM) ma.init(abase, nullptr, A.as, A.K, A.M - m0, INT32_MAX, k0);
    if constexpr (BMM) mb.init((const char *)A.b0 + (int64_t)n0 * ES, (const char *)A.b1 + (int64_t)n0 * ES, A.bs, A.brows, A.N - n0, A.ktsplit, k0);

    // Load i of this wavefront is load 4 i + wave of its region.
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
    f32x4_t acc[TM][2][TN] = {};
    const int wm = wave >> 1, wn = wave & 1;
    FfnFragments<S, AM, BM, TM> fa;
    FfnFragments<S, BMM, 2 * BH, TN> fb[2];
    fa.init(lds0, wm * TM * 16, lane);
#pragma unroll
    for (int h = 0; h < 2; ++h) fb[h].init(lds0 + BM * 128, h * BH + wn * TN * 16, lane);
    auto compute = [&](uint32_t stage) {
        uint4 b[2][TN][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) b[h][t][j] = fb[h].get(t, j, stage);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            uint4 a[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) a[j] = fa.get(t, j, stage);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < TN; ++f) ffn_mma<S>(b[h][f], a, acc[t][h][f]);
        }
    };
    auto next = [](uint32_t stage) { return stage + STAGE == ST * STAGE ? 0u : stage + STAGE; };

    if constexpr (!ANY) {
        const int gate = min(BH, A.N - n0), up = min(BH, A.N - n0 - (PLAIN ? BH : 0));
        const int64_t up0 = (int64_t)(n0 + (PLAIN ? BH : 0)) * A.bs * ES;
        const __amdgpu_buffer_rsrc_t ka = make_rsrc(abase, (uint32_t)(am - 1) * abytes + kbytes),
                                     kg = make_rsrc((const char *)A.b0 + (int64_t)n0 * A.bs * ES, (uint32_t)(gate - 1) * bbytes + kbytes),
                                     ku = make_rsrc((const char *)(PLAIN ? A.b0 : A.b1) + (up > 0 ? up0 : 0),
                                                    up > 0 ? (uint32_t)(up - 1) * bbytes + kbytes : 0u);
        uint32_t off[IPW];
#pragma unroll
        for (int i = 0; i < IPW; ++i) {
            const bool of_a = i < IA;
            const int q = 4 * (of_a ? i : i - IA) + wave;
            const int row = of_a ? RA::load_row(q, lane) : RB::load_row(q, lane);
            const int chunk = of_a ? RA::load_chunk(q, lane) : RB::load_chunk(q, lane);
            if (of_a ? AM : BMM) {
                const bool in = chunk * V < (of_a ? am : A.N - n0);
                off[i] = in ? (uint32_t)row * (of_a ? abytes : bbytes) + chunk * 16 : kOutOfRange;
            } else {
                off[i] = (uint32_t)(of_a ? row : row % BH) * (of_a ? abytes : bbytes) + chunk * 16;
            }
        }
        // (in rows of k all loads of a lane bring the same chunk, as 8 q + lane / 8 keep (row / 2) % 8)
        const uint32_t chunk = (uint32_t)FfnRegion<S, false, 128>::load_chunk(wave, lane) * 16;
        auto issue = [&](int kt, uint32_t stage) {  // tiles past the end and what lies behind a row read as zeros
            const uint32_t at = (uint32_t)(k0 + kt) * 128;
            const bool in = at + chunk < kbytes;
            const uint32_t dst = lds0 + stage + wave * 1024;
            __amdgpu_buffer_rsrc_t ta, tb;
            if constexpr (AM) ta = ma.tile(), ma.next();
            if constexpr (BMM) tb = mb.tile(), mb.next();
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                if (i < IA) {
                    if constexpr (AM) lds_dma16(ta, off[i], dst + i * 4096);
                    else ffn_dma16(ka, in ? off[i] : kOutOfRange, at, dst + i * 4096);
                } else {
                    if constexpr (BMM) lds_dma16(tb, off[i], dst + i * 4096);
                    else ffn_dma16(i - IA < BH / 32 ? kg : ku, in ? off[i] : kOutOfRange, at, dst + i * 4096);
                }
            }
        };
        issue(0, 0);
        issue(1, STAGE);
        uint32_t stage = 0, filled = 2 * STAGE;
#pragma nounroll
        for (int kt = 0; kt < nk; ++kt) {
            CONVLOWER_WAIT_VMCNT_LDS(IPW);
            block_barrier();  // tile kt has landed for all, and nobody reads tile kt - 1's stage any more
            __builtin_amdgcn_sched_barrier(0);
            issue(kt + 2, filled);
            __builtin_amdgcn_sched_barrier(0);
            compute(stage);
            __builtin_amdgcn_sched_barrier(0);
            stage = next(stage);
            filled = next(filled);
        }
        CONVLOWER_WAIT_VMCNT(0);  // no load may still write LDS when the block ends
    } else {
        uint4 reg[IPW];
        // V values of a row from value k on, of which there are `have`.
        auto values = [&](const char *row, int k, int have) {
            const S *src = (const S *)row + k;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (k + V <= have) {
                const FfnAnyVec<S, V> t = *(const FfnAnyVec<S, V> *)src;
                __builtin_memcpy(&v, &t, 16);
            } else if (k < have) {
                S t[V] = {};
#pragma unroll
                for (int j = 0; j < V; ++j)
                    if (k + j < have) t[j] = src[j];
                __builtin_memcpy(&v, t, 16);
            }
            return v;
        };
        auto fetch = [&](int kt) {
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                const bool of_a = i < IA;
                const int q = 4 * (of_a ? i : i - IA) + wave;
                const int row = of_a ? RA::load_row(q, lane) : RB::load_row(q, lane);
                const int first = (of_a ? RA::load_chunk(q, lane) : RB::load_chunk(q, lane)) * V;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (of_a ? AM : BMM) {
                    const FfnRowsOfM<S> &m = of_a ? ma : mb;
                    if (row < m.left) v = values(m.p + (int64_t)row * m.step, first, of_a ? am : A.N - n0);
                } else {
                    const bool up = !of_a && !PLAIN && row >= BH;
                    const int64_t r = of_a ? m0 + row : n0 + (up ? row - BH : row);
                    const char *p = (const char *)(of_a ? A.a : up ? A.b1 : A.b0) + r * (of_a ? A.as : A.bs) * ES;
                    if (r < (of_a ? A.M : (int64_t)A.N)) v = values(p, (k0 + kt) * RA::KROWS + first, A.K);
                }
                reg[i] = v;
            }
            if constexpr (AM) ma.next();
            if constexpr (BMM) mb.next();
        };
        auto keep = [&](uint32_t stage) {
#pragma unroll
            for (int i = 0; i < IPW; ++i) *(uint4 *)(lds + stage + (4 * i + wave) * 1024 + lane * 16) = reg[i];
        };
        if (nk > 0) {
            fetch(0);
            keep(0);
        }
        uint32_t stage = 0;
#pragma nounroll
        for (int kt = 0; kt < nk; ++kt) {
            __syncthreads();
            if (kt + 1 < nk) fetch(kt + 1);
            compute(stage);
            stage = next(stage);
            if (kt + 1 < nk) keep(stage);
        }
    }

    const float by = PLAIN ? ffn_factor<O>(A) : 1.f;
    auto results = [&](auto act) {
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            const int64_t m = m0 + (wm * TM + t) * 16 + (lane & 15);
            if (m >= A.M) continue;
#pragma unroll
            for (int f = 0; f < TN; ++f) {
                const int n = n0 + (wn * TN + f) * 16 + 4 * (lane >> 4);
                if constexpr (PLAIN) {
                    if (n < A.N) ffn_plain_out<O>(A, m, n, acc[t][0][f], by);
                    if (n + BH < A.N) ffn_plain_out<O>(A, m, n + BH, acc[t][1][f], by);
                } else if (n < A.N) {
                    ffn_gated_out<O, EPI, decltype(act)::value>(A, m, n, acc[t][0][f], acc[t][1][f]);
                }
            }
        }
    };
    if constexpr (PLAIN) results(0);
    else ffn_with_act(A.act, results);
}
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY, bool AM, bool BMM>
__global__ __launch_bounds__(256) void ffn_small_kernel(FfnGemmArgs A) {
    ffn_small_body<S, O, EPI, BM, BH, ANY, AM, BMM>(A);
}

// ---- large tiles: one block of eight wavefronts on a CU, two on each SIMD, WM x 8 /
// WM over 32 WM TA of a's m by 16 (8 / WM) TB of each half of b.  Wavefronts 0-3 and
// 4-7 alternate: while one group multiplies, the other reads LDS and issues loads,
// with a barrier at each change, so that a SIMD's matrix core always has a
// wavefront whose operands are in registers.
//
// A wavefront goes through a K tile in four phases, (A0, F), (A0, L), (A1, L),
// (A1, F): A0, A1 are the halves of its part of a; F and L, the first and the
// last, its parts of b's halves, B0 and B1 in even tiles, B1 and B0 in odd ones. The
// next tile's F is then this tile's L, whose registers are free one phase early,
// and each phase reads one region: L and A1 for the next phase of the tile, F and
// A0 for the next tile's.  There are two stages, and a region takes the tile after
// next as soon as both groups have read it.  Every wavefront's loads of a phase
// fill one region, in the order in which they are read, seven phases ahead: the
// wait at the end of a phase's reads leaves those of six under way.
template <int WM_, int TA_, int TB_>
struct FfnLarge {
    static constexpr int WM = WM_, WN = 8 / WM_, TA = TA_, TB = TB_;
    static constexpr int RA = WM * TA * 16, RB = WN * TB * 16;  // rows of a region
    static constexpr int BM = 2 * RA, BH = RB;
};
template <typename S, typename O, FfnEpilogue EPI, bool AM, bool BMM, typename C>
__device__ __forceinline__ void ffn_large_body(const FfnGemmArgs &A) {
    constexpr int BM = C::BM, BH = C::BH, TA = C::TA, TB = C::TB, ES = (int)sizeof(S), V = 16 / ES;
    constexpr bool PLAIN = EPI == FFN_PLAIN;
    static_assert(PLAIN || !BMM, "two matrices of rows of k, or one of either kind");
    constexpr uint32_t SIZE_A = C::RA * 128, SIZE_B = C::RB * 128, STAGE = 2 * (SIZE_A + SIZE_B);
    using RA = FfnRegion<S, AM, C::RA>;
    using RB = FfnRegion<S, BMM, C::RB>;
    constexpr int LA = RA::LOADS / 8, LB = RB::LOADS / 8;  // a wavefront's loads of a region
    static_assert(LA * 8 == RA::LOADS && LB * 8 == RB::LOADS && STAGE % 4096 == 0, "regions split evenly");
    __shared__ alignas(16) char lds[2 * STAGE];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    constexpr int BN = PLAIN ? 2 * BH : BH;
    ffn_tile((int)((A.M + BM - 1) / BM), (A.N + BN - 1) / BN, 8, &mt, &nt);
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;
    const uint32_t kbytes = (uint32_t)A.K * ES, abytes = (uint32_t)(A.as * ES), bbytes = (uint32_t)(A.bs * ES);
    const int tiles = (A.K + RA::KROWS - 1) / RA::KROWS;
    const int k0 = PLAIN ? (int)((int64_t)tiles * blockIdx.y / A.splits) : 0;  // this part's tiles
    const int nk = (PLAIN ? (int)((int64_t)tiles * (blockIdx.y + 1) / A.splits) : tiles) - k0;

    auto rows_at = [&](const void *p, int64_t first, int64_t rows, int64_t most, uint32_t step) {
        const int64_t n = rows - first < most ? rows - first : most;
        return make_rsrc((const char *)p + (n > 0 ? first : 0) * (int64_t)step, n > 0 ? (uint32_t)(n - 1) * step + kbytes : 0u);
    };
    // Regions 0, 1: the first and second half of each wavefront's part of a; 2, 3: the halves of b.
    __amdgpu_buffer_rsrc_t rs[4];
    constexpr int HA = TA * 16;  // a half
    if constexpr (!AM) rs[0] = rows_at(A.a, m0, A.M, BM - HA, abytes), rs[1] = rows_at(A.a, m0 + HA, A.M, BM - HA, abytes);
    if constexpr (!BMM) {
        rs[2] = rows_at(A.b0, n0, A.N, BH, bbytes);
        rs[3] = rows_at(PLAIN ? A.b0 : A.b1, n0 + (PLAIN ? BH : 0), A.N, BH, bbytes);
    }

    // Load j of this wavefront is load LA wave + j, or LB wave + j, of a region.
    uint32_t off_a[2][LA], off_b[2][LB];  // rows of k: the same for both regions of an operand
    uint32_t chunk_a[LA], chunk_b[LB];
#pragma unroll
    for (int j = 0; j < LA; ++j) {
        const int q = LA * wave + j, row = RA::load_row(q, lane), c = RA::load_chunk(q, lane) * V;
        chunk_a[j] = c * ES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = AM ? c : row, at = m / HA * 2 * HA + m % HA + (AM ? h * HA : 0);
            if constexpr (AM) off_a[h][j] = m0 + at < A.M ? (uint32_t)row * abytes + at * ES : kOutOfRange;
            else off_a[h][j] = (uint32_t)at * abytes + c * ES;
        }
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
        const int q = LB * wave + j, row = RB::load_row(q, lane), c = RB::load_chunk(q, lane) * V;
        chunk_b[j] = c * ES;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (BMM) off_b[h][j] = n0 + c + h * BH < A.N ? (uint32_t)row * bbytes + (c + h * BH) * ES : kOutOfRange;
            else off_b[h][j] = (uint32_t)row * bbytes + c * ES;
        }
    }
    FfnRowsOfM<S> ma, mb;
    if constexpr (AM) ma.init((const char *)A.a + m0 * ES, nullptr, A.as, A.K, min(A.M - m0, (int64_t)BM), INT32_MAX, k0);
    if constexpr (BMM)
        mb.init((const char *)A.b0 + (int64_t)n0 * ES, (const char *)A.b1 + (int64_t)n0 * ES, A.bs, A.brows, min(A.N - n0, BN), A.ktsplit, k0);
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
    auto issue = [&](auto region_c, auto stage_c, int kt) {  // tiles past the end read as zeros
        constexpr int region = decltype(region_c)::value, h = region & 1;
        constexpr bool of_a = region < 2;
        const uint32_t at = (uint32_t)(k0 + kt) * 128,
                       dst = lds0 + decltype(stage_c)::value * STAGE + (of_a ? h * SIZE_A : 2 * SIZE_A + h * SIZE_B) + wave * ((of_a ? LA : LB) * 1024);
#pragma unroll
        for (int j = 0; j < (of_a ? LA : LB); ++j) {
            const uint32_t off = of_a ? off_a[h][j] : off_b[h][j];
            if constexpr (of_a ? AM : BMM) lds_dma16(rs[region], off, dst + j * 1024);
            else ffn_dma16(rs[region], at + (of_a ? chunk_a[j] : chunk_b[j]) < kbytes ? off : kOutOfRange, at, dst + j * 1024);
        }
    };
    // The next tile of an operand of rows of m.
    auto turn_a = [&] {
        if constexpr (AM) rs[0] = rs[1] = ma.tile(), ma.next();
    };
    auto turn_b = [&] {
        if constexpr (BMM) rs[2] = rs[3] = mb.tile(), mb.next();
    };

    const int wm = wave / C::WN, wn = wave % C::WN;
    f32x4_t acc[2][2][TA][TB] = {};  // [half of a][half of b][tile of a][tile of b]
    uint4 fa[TA][2], fb[2][TB][2];
    FfnFragments<S, AM, C::RA, TA> pa[2];
    FfnFragments<S, BMM, C::RB, TB> pb[2];
    pa[0].init(lds0, wm * HA, lane);
    pb[0].init(lds0 + 2 * SIZE_A, wn * TB * 16, lane);
    pa[1] = pa[0].moved(STAGE / 4096);
    pb[1] = pb[0].moved(STAGE / 4096);
    auto read_a = [&](int h, int stage) {
#pragma unroll
        for (int t = 0; t < TA; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) fa[t][j] = pa[stage].get(t, j, h * SIZE_A);
    };
    auto read_b = [&](int h, int stage) {
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[h][t][j] = pb[stage].get(t, j, h * SIZE_B);
    };
    auto multiply = [&](int ha, int hb) {
        // This wavefront's reads have come, and all but its loads of the last six phases.
        CONVLOWER_WAIT_VMCNT_LDS(3 * (LA + LB));
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < TA; ++t) {
#pragma unroll
            for (int f = 0; f < TB; ++f) ffn_mma<S>(fb[hb][f], fa[t], acc[ha][hb][t][f]);
            if constexpr (ES == 4) __builtin_amdgcn_sched_barrier(0);  // (else the tiles' own sums are kept side by side, and spill)
        }
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    constexpr std::integral_constant<int, 0> even;
    constexpr std::integral_constant<int, 1> odd;
    constexpr std::integral_constant<int, 0> A0;
    constexpr std::integral_constant<int, 1> A1;
    constexpr std::integral_constant<int, 2> B0;
    constexpr std::integral_constant<int, 3> B1;
    auto tile = [&](int kt, auto parity) {
        constexpr int F = decltype(parity)::value, L = 1 - F;
        read_a(0, F);
        turn_b();
        issue(std::integral_constant<int, 2 + F>(), parity, kt + 2);
        multiply(0, F);
        read_b(L, F);
        turn_a();
        issue(A0, parity, kt + 2);
        multiply(0, L);
        read_a(1, F);
        issue(std::integral_constant<int, 2 + L>(), parity, kt + 2);
        multiply(1, L);
        read_b(L, L);
        issue(A1, parity, kt + 2);
        multiply(1, F);
    };

    turn_a();
    turn_b();
    issue(B0, even, 0);
    issue(A0, even, 0);
    issue(B1, even, 0);
    issue(A1, even, 0);
    turn_a();
    turn_b();
    issue(B1, odd, 1);
    issue(A0, odd, 1);
    issue(B0, odd, 1);
    issue(A1, odd, 1);
    CONVLOWER_WAIT_VMCNT(4 * LA + 3 * LB);
    block_barrier();
    read_b(0, 0);
    CONVLOWER_WAIT_VMCNT_LDS(3 * (LA + LB));
    block_barrier();
    if (wave >= 4) block_barrier();
    int kt = 0;
#pragma nounroll
    for (; kt + 1 < nk; kt += 2) {
        tile(kt, even);
        tile(kt + 1, odd);
    }
    if (kt < nk) tile(kt, even);
    if (wave < 4) block_barrier();
    CONVLOWER_WAIT_VMCNT(0);  // no load may still write LDS when the block ends

    const float by = PLAIN ? ffn_factor<O>(A) : 1.f;
    auto results = [&](auto act) {
#pragma unroll
        for (int ha = 0; ha < 2; ++ha)
#pragma unroll
            for (int t = 0; t < TA; ++t) {
                const int64_t m = m0 + (wm * 2 + ha) * HA + 16 * t + (lane & 15);
                if (m >= A.M) continue;
#pragma unroll
                for (int f = 0; f < TB; ++f) {
                    const int n = n0 + (wn * TB + f) * 16 + 4 * (lane >> 4);
                    if constexpr (PLAIN) {
                        if (n < A.N) ffn_plain_out<O>(A, m, n, acc[ha][0][t][f], by);
                        if (n + BH < A.N) ffn_plain_out<O>(A, m, n + BH, acc[ha][1][t][f], by);
                    } else if (n < A.N) {
                        ffn_gated_out<O, EPI, decltype(act)::value>(A, m, n, acc[ha][0][t][f], acc[ha][1][t][f]);
                    }
                }
            }
    };
    if constexpr (PLAIN) results(0);
    else ffn_with_act(A.act, results);
}
template <typename S, typename O, FfnEpilogue EPI, bool AM, bool BMM, typename C>
__global__ __launch_bounds__(512) void ffn_large_kernel(FfnGemmArgs A) {
    ffn_large_body<S, O, EPI, AM, BMM, C>(A);
}
typedef FfnLarge<2, 4, 2> FfnTile256x128;  // 128 x (32 + 32) of a wavefront
typedef FfnLarge<4, 2, 2> FfnTile256x64;   // 64 x (32 + 32)
typedef FfnLarge<2, 2, 1> FfnTile128x64;   // 64 x (16 + 16), two blocks on a CU

// out from the parts' sums, added in their order.
template <typename O>
__global__ __launch_bounds__(256) void ffn_sum_kernel(FfnGemmArgs A) {
    const int64_t pitch = ffn_part_pitch(A.N), per = pitch / 4, total = A.M * per;
    const float by = ffn_factor<O>(A);
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t m = i / per;
        const int n = (int)(i - m * per) * 4;
        const bool second = m >= A.split;
        const int64_t row = second ? m - A.split : m;
        if (row >= A.rows) continue;
        float v[4] = {};
        for (int s = 0; s < A.splits; ++s) {
            const float4 x = *(const float4 *)(A.part + (s * A.M + m) * pitch + n);
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] *= by;
        ffn_put4((O *)(second ? A.out2 : A.out) + row * A.N, n, A.N, v);
    }
}

// ---- launches
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY, bool AM, bool BMM>
hipError_t ffn_run_small(const FfnGemmArgs &a, hipStream_t st) {
    constexpr int BN = EPI == FFN_PLAIN ? 2 * BH : BH;
    const int64_t blocks = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    hipLaunchKernelGGL((ffn_small_kernel<S, O, EPI, BM, BH, ANY, AM, BMM>), dim3((unsigned)blocks, a.splits), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <typename S, typename O, FfnEpilogue EPI, bool AM, bool BMM, typename C>
hipError_t ffn_run_large(const FfnGemmArgs &a, hipStream_t st) {
    constexpr int BN = EPI == FFN_PLAIN ? 2 * C::BH : C::BH;
    const int64_t blocks = ((a.M + C::BM - 1) / C::BM) * ((a.N + BN - 1) / BN);
    hipLaunchKernelGGL((ffn_large_kernel<S, O, EPI, AM, BMM, C>), dim3((unsigned)blocks, a.splits), dim3(512), 0, st, a);
    return hipGetLastError();
}

// AM, BMM: a, b as rows of m (of columns that are there: M and N values wide).
template <typename S, typename O, FfnEpilogue EPI, bool AM, bool BMM>
hipError_t ffn_run(const FfnGemmArgs &a, hipStream_t st) {
    hipError_t e = hipErrorInvalidValue;
    if (!a.vec) e = ffn_run_small<S, O, EPI, 64, 32, true, AM, BMM>(a, st);
    else if (a.tile == FFN_TILE_256x128) e = ffn_run_large<S, O, EPI, AM, BMM, FfnTile256x128>(a, st);
    else if (a.tile == FFN_TILE_256x64) e = ffn_run_large<S, O, EPI, AM, BMM, FfnTile256x64>(a, st);
    else if (a.tile == FFN_TILE_128x64) e = ffn_run_large<S, O, EPI, AM, BMM, FfnTile128x64>(a, st);
    else if (AM || a.tile == FFN_TILE_64x32) e = ffn_run_small<S, O, EPI, 64, 32, false, AM, BMM>(a, st);
    else if constexpr (!AM) e = ffn_run_small<S, O, EPI, 32, 32, false, AM, BMM>(a, st);
    if constexpr (EPI == FFN_PLAIN) {
        if (e != hipSuccess || a.splits == 1) return e;
        const int64_t blocks = (a.M * (ffn_part_pitch(a.N) / 4) + 255) / 256;
        hipLaunchKernelGGL((ffn_sum_kernel<O>), dim3((unsigned)(blocks < 1 << 16 ? blocks : 1 << 16)), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    return e;
}

}  // namespace
}  // namespace convlower
