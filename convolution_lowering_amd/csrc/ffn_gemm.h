// Products of rows on the matrix cores: every a[m] with every b[n], both
// contiguous along what is summed.  A K tile is 128 bytes of each row (64
// 16-bit values, 32 float32, 128 e4m3), in LDS as 8 chunks of 16 bytes.
//
// Chunk c of row r lies in slot 8 r + (c ^ (r / 2) % 8): a fragment read takes
// 16 rows of one chunk, and this puts them on the 16 groups of banks of a 256-byte
// line.  Which values a lane's chunk holds does not matter to a sum as long as
// both operands agree, so all types read the same two chunks of a row, c = lane
// / 16 and that plus 4, and differ only in the instruction that takes them.
//
// The rows of b are the matrix instruction's left operand, so that a lane's four
// results are four neighbours of one output row.
#pragma once

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
        // (e4m3 both; the scale operands are unused exponents of 1)
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
    } else {
        MfmaShape<S, 16>::mma(b[0], a[0], acc);
        MfmaShape<S, 16>::mma(b[1], a[1], acc);
    }
}

__device__ __forceinline__ int ffn_slot(int r, int c) { return r * 8 + (c ^ ((r >> 1) & 7)); }

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
template <typename O, FfnEpilogue EPI>
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
    for (int i = 0; i < 4; ++i) h[i] = ffn_act<O>(g[i], A.act) * u[i];
    ffn_put4((O *)A.out + m * A.N, n, A.N, h);
}
template <typename O>
__device__ __forceinline__ void ffn_plain_out(const FfnGemmArgs &A, int64_t m, int n, const f32x4_t &acc) {
    const float v[4] = {acc[0], acc[1], acc[2], acc[3]};
    O *row = m < A.split ? (O *)A.out + m * A.N : (O *)A.out2 + (m - A.split) * A.N;
    ffn_put4(row, n, A.N, v);
}

// ---- the loop for any size: four wavefronts, 2 x 2, over BM rows of a and BH
// of each of b0 and b1 (or 2 BH of b0 alone).  Rows at multiples of 16 bytes are
// copied into LDS by the load instructions that write there (three stages, two
// tiles under way); others (ANY) pass through registers, one tile ahead, their
// last values one by one.
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY>
__device__ __forceinline__ void ffn_small_body(const FfnGemmArgs &A) {
    constexpr int V = 16 / (int)sizeof(S), ROWS = BM + 2 * BH, ST = ANY ? 2 : 3;
    constexpr int IPW = ROWS / 32;              // 1 KB loads of a wavefront per tile
    constexpr int TM = BM / 32, TN = BH / 32;   // 16-row tiles of a wavefront: of a, and of each half of b
    constexpr bool PLAIN = EPI == FFN_PLAIN;
    static_assert(ROWS % 32 == 0 && BM % 32 == 0 && BH % 32 == 0, "loads and wavefronts split evenly");
    __shared__ uint4 lds[ST][ROWS * 8];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    constexpr int BN = PLAIN ? 2 * BH : BH;
    ffn_tile((int)((A.M + BM - 1) / BM), (A.N + BN - 1) / BN, 8, &mt, &nt);
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;
    const uint32_t kbytes = (uint32_t)A.K * (uint32_t)sizeof(S), abytes = (uint32_t)(A.as * sizeof(S)),
                   bbytes = (uint32_t)(A.bs * sizeof(S));
    const int nk = (int)((kbytes + 127) / 128);

    // Bases of the three groups of rows and how many rows are there.
    const char *base[3] = {(const char *)A.a + m0 * A.as * (int64_t)sizeof(S),
                           (const char *)A.b0 + (int64_t)n0 * A.bs * (int64_t)sizeof(S),
                           (const char *)(PLAIN ? A.b0 : A.b1) + (int64_t)(n0 + (PLAIN ? BH : 0)) * A.bs * (int64_t)sizeof(S)};
    const int have[3] = {(int)min((int64_t)BM, A.M - m0), min(BH, A.N - n0), min(BH, A.N - n0 - (PLAIN ? BH : 0))};

    // Load i of this wavefront covers rows 8 (4 i + wave) + lane / 8 of one group; each lane always has the same chunk.
    const int chunk = (lane & 7) ^ (((wave & 1) << 2) + (lane >> 4));
    auto part_of = [&](int row) { return row < BM ? 0 : row < BM + BH ? 1 : 2; };
    auto row_in = [&](int row) { return row < BM ? row : row < BM + BH ? row - BM : row - BM - BH; };

    f32x4_t acc[TM][2][TN] = {};
    const int wm = wave >> 1, wn = wave & 1;
    auto compute = [&](const uint4 *st) {
        uint4 b[2][TN][2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int t = 0; t < TN; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    b[h][t][j] = st[ffn_slot(BM + h * BH + (wn * TN + t) * 16 + (lane & 15), j * 4 + (lane >> 4))];
#pragma unroll
        for (int t = 0; t < TM; ++t) {
            uint4 a[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) a[j] = st[ffn_slot((wm * TM + t) * 16 + (lane & 15), j * 4 + (lane >> 4))];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int f = 0; f < TN; ++f) ffn_mma<S>(b[h][f], a, acc[t][h][f]);
        }
    };

    if constexpr (!ANY) {
        __amdgpu_buffer_rsrc_t rs[3];
#pragma unroll
        for (int p = 0; p < 3; ++p)
            rs[p] = make_rsrc(base[p], have[p] > 0 ? (uint32_t)(have[p] - 1) * (p ? bbytes : abytes) + kbytes : 0u);
        uint32_t off[IPW];
#pragma unroll
        for (int i = 0; i < IPW; ++i) {
            const int row = 8 * (4 * i + wave) + (lane >> 3), p = part_of(32 * i);
            off[i] = (uint32_t)row_in(row) * (p ? bbytes : abytes) + chunk * 16;
        }
        auto issue = [&](int kt) {  // tiles past the end and what lies behind a row read as zeros
            const uint32_t at = (uint32_t)kt * 128;
            const bool in = at + chunk * 16 < kbytes;
            const uint32_t dst = (uint32_t)(uintptr_t)(lds_ptr_t)&lds[kt % ST][0] + wave * 1024;
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                const int p = part_of(32 * i);
                lds_dma16(rs[p], in ? off[i] + at : kOutOfRange, dst + i * 4096);
            }
        };
        if (nk > 0) {
            issue(0);
            issue(1);
        }
        for (int kt = 0; kt < nk; ++kt) {
            CONVLOWER_WAIT_VMCNT_LDS(IPW);
            block_barrier();  // tile kt has landed for all, and nobody reads tile kt - 1's stage any more
            __builtin_amdgcn_sched_barrier(0);
            issue(kt + 2);
            __builtin_amdgcn_sched_barrier(0);
            compute(lds[kt % ST]);
            __builtin_amdgcn_sched_barrier(0);
        }
        CONVLOWER_WAIT_VMCNT(0);  // no load may still write LDS when the block ends
    } else {
        uint4 reg[IPW];
        auto fetch = [&](int kt) {
            const int k = kt * (128 / (int)sizeof(S)) + chunk * V;
#pragma unroll
            for (int i = 0; i < IPW; ++i) {
                const int row = 8 * (4 * i + wave) + (lane >> 3), p = part_of(32 * i), in = row_in(row);
                uint4 v = make_uint4(0, 0, 0, 0);
                if (in < have[p] && k < A.K) {
                    const S *src = (const S *)base[p] + (int64_t)in * (p ? A.bs : A.as) + k;
                    if (k + V <= A.K) {
                        const FfnAnyVec<S, V> t = *(const FfnAnyVec<S, V> *)src;
                        __builtin_memcpy(&v, &t, 16);
                    } else {
                        S t[V] = {};
#pragma unroll
                        for (int j = 0; j < V; ++j)
                            if (k + j < A.K) t[j] = src[j];
                        __builtin_memcpy(&v, t, 16);
                    }
                }
                reg[i] = v;
            }
        };
        auto keep = [&](int kt) {
#pragma unroll
            for (int i = 0; i < IPW; ++i) lds[kt % ST][(4 * i + wave) * 64 + lane] = reg[i];
        };
        if (nk > 0) {
            fetch(0);
            keep(0);
        }
        for (int kt = 0; kt < nk; ++kt) {
            __syncthreads();
            if (kt + 1 < nk) fetch(kt + 1);
            compute(lds[kt % ST]);
            if (kt + 1 < nk) keep(kt + 1);
        }
    }

#pragma unroll
    for (int t = 0; t < TM; ++t) {
        const int64_t m = m0 + (wm * TM + t) * 16 + (lane & 15);
        if (m >= A.M) continue;
#pragma unroll
        for (int f = 0; f < TN; ++f) {
            const int n = n0 + (wn * TN + f) * 16 + 4 * (lane >> 4);
            if constexpr (PLAIN) {
                if (n < A.N) ffn_plain_out<O>(A, m, n, acc[t][0][f]);
                if (n + BH < A.N) ffn_plain_out<O>(A, m, n + BH, acc[t][1][f]);
            } else if (n < A.N) {
                ffn_gated_out<O, EPI>(A, m, n, acc[t][0][f], acc[t][1][f]);
            }
        }
    }
}
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY>
__global__ __launch_bounds__(256) void ffn_small_kernel(FfnGemmArgs A) {
    ffn_small_body<S, O, EPI, BM, BH, ANY>(A);
}

// ---- the large tile: 256 rows of a by 128 of each half of b, one block of
// eight wavefronts on a CU, two on each SIMD, each with 128 x (32 + 32) of the
// tile.  Wavefronts 0-3 and 4-7 alternate: while one group multiplies, the other
// reads LDS and issues loads, with a barrier at each change, so that a SIMD's
// matrix core always has a wavefront whose operands are in registers.
//
// A wavefront goes through a K tile in four phases, (A0, B0), (A0, B1), (A1, B1),
// (A1, B0): A0, A1 are the halves of its rows of a, B0 and B1 its rows of the
// halves of b.  Each of the four is 16 KB of a stage, its own region; there are
// two stages, and a region takes the tile after next as soon as both groups
// have read it.  Two 1 KB loads of each phase and wavefront fill one region, in
// the order in which they are read, five phases ahead: the wait at the end of a
// phase's reads leaves ten loads under way.
template <typename S, typename O, FfnEpilogue EPI>
__device__ __forceinline__ void ffn_large_body(const FfnGemmArgs &A) {
    constexpr int BM = 256, BH = 128;
    constexpr bool PLAIN = EPI == FFN_PLAIN;
    constexpr uint32_t REGION = 16384, STAGE = 4 * REGION;
    __shared__ alignas(16) char lds[2 * STAGE];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int mt, nt;
    constexpr int BN = PLAIN ? 2 * BH : BH;
    ffn_tile((int)((A.M + BM - 1) / BM), (A.N + BN - 1) / BN, 8, &mt, &nt);
    const int64_t m0 = (int64_t)mt * BM;
    const int n0 = nt * BN;
    const uint32_t kbytes = (uint32_t)A.K * (uint32_t)sizeof(S), abytes = (uint32_t)(A.as * sizeof(S)),
                   bbytes = (uint32_t)(A.bs * sizeof(S));
    const int nk = (int)((kbytes + 127) / 128);

    auto rows_at = [&](const void *p, int64_t first, int64_t rows, int64_t most, uint32_t step) {
        const int64_t n = rows - first < most ? rows - first : most;
        return make_rsrc((const char *)p + (n > 0 ? first : 0) * (int64_t)step, n > 0 ? (uint32_t)(n - 1) * step + kbytes : 0u);
    };
    // Regions 0, 1: the first and second 64 of each 128 rows of a; 2, 3: the halves of b.
    const __amdgpu_buffer_rsrc_t rs[4] = {rows_at(A.a, m0, A.M, 192, abytes), rows_at(A.a, m0 + 64, A.M, 192, abytes),
                                          rows_at(A.b0, n0, A.N, BH, bbytes),
                                          rows_at(PLAIN ? A.b0 : A.b1, n0 + (PLAIN ? BH : 0), A.N, BH, bbytes)};

    // Load j of this wavefront: rows 16 wave + 8 j + lane / 8 of a region.
    uint32_t off[2][2];  // [of a, of b][j]
    int chunk[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        chunk[j] = (lane & 7) ^ (4 * j + (lane >> 4));
        const int row = 16 * wave + 8 * j + (lane >> 3);
        off[0][j] = (uint32_t)((row >> 6) * 128 + (row & 63)) * abytes + chunk[j] * 16;
        off[1][j] = (uint32_t)row * bbytes + chunk[j] * 16;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
    auto issue = [&](int region, int kt) {
        const uint32_t at = (uint32_t)kt * 128, dst = lds0 + (kt & 1) * STAGE + region * REGION + wave * 2048;
#pragma unroll
        for (int j = 0; j < 2; ++j)
            lds_dma16(rs[region], at + chunk[j] * 16 < kbytes ? off[region >> 1][j] + at : kOutOfRange, dst + j * 1024);
    };

    const int wm = wave >> 2, wn = wave & 3;
    f32x4_t acc[2][2][4][2] = {};  // [half of a][half of b][tile of a][tile of b]
    uint4 fa[4][2], fb[2][2][2];
    // Fragments of a region's rows r0 + 16 t + lane % 16.
    auto frag = [&](int stage, int region, int r0, int t, int j) {
        return *(const uint4 *)(lds + stage * STAGE + region * REGION + (r0 + 16 * t + (lane & 15)) * 128 +
                                ((j * 4 + (lane >> 4)) ^ ((lane & 15) >> 1)) * 16);
    };
    auto read_a = [&](int stage, int h) {
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) fa[t][j] = frag(stage, h, wm * 64, t, j);
    };
    auto read_b = [&](int stage, int h) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) fb[h][t][j] = frag(stage, 2 + h, wn * 32, t, j);
    };
    auto multiply = [&](int ha, int hb) {
        // This wavefront's reads have come, and all but its last ten loads.
        CONVLOWER_WAIT_VMCNT_LDS(10);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int f = 0; f < 2; ++f) ffn_mma<S>(fb[hb][f], fa[t], acc[ha][hb][t][f]);
        __builtin_amdgcn_s_setprio(0);
        __builtin_amdgcn_sched_barrier(0);
        block_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    auto tile = [&](int kt, int stage) {
        read_a(stage, 0);
        read_b(stage, 0);
        issue(1, kt + 1);
        multiply(0, 0);
        read_b(stage, 1);
        issue(0, kt + 2);
        multiply(0, 1);
        read_a(stage, 1);
        issue(2, kt + 2);
        multiply(1, 1);
        issue(3, kt + 2);
        multiply(1, 0);
    };

    issue(0, 0);
    issue(2, 0);
    issue(3, 0);
    issue(1, 0);
    issue(0, 1);
    issue(2, 1);
    issue(3, 1);
    CONVLOWER_WAIT_VMCNT(10);
    block_barrier();
    if (wave >= 4) block_barrier();
    // (an odd number of tiles ends with one of zeros)
    for (int kt = 0; kt < nk; kt += 2) {
        tile(kt, 0);
        tile(kt + 1, 1);
    }
    if (wave < 4) block_barrier();
    CONVLOWER_WAIT_VMCNT(0);  // no load may still write LDS when the block ends

#pragma unroll
    for (int ha = 0; ha < 2; ++ha)
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const int64_t m = m0 + wm * 128 + ha * 64 + 16 * t + (lane & 15);
            if (m >= A.M) continue;
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                const int n = n0 + wn * 32 + 16 * f + 4 * (lane >> 4);
                if constexpr (PLAIN) {
                    if (n < A.N) ffn_plain_out<O>(A, m, n, acc[ha][0][t][f]);
                    if (n + BH < A.N) ffn_plain_out<O>(A, m, n + BH, acc[ha][1][t][f]);
                } else if (n < A.N) {
                    ffn_gated_out<O, EPI>(A, m, n, acc[ha][0][t][f], acc[ha][1][t][f]);
                }
            }
        }
}
template <typename S, typename O, FfnEpilogue EPI>
__global__ __launch_bounds__(512) void ffn_large_kernel(FfnGemmArgs A) {
    ffn_large_body<S, O, EPI>(A);
}

// ---- launches
template <typename S, typename O, FfnEpilogue EPI, int BM, int BH, bool ANY>
hipError_t ffn_run_small(const FfnGemmArgs &a, hipStream_t st) {
    constexpr int BN = EPI == FFN_PLAIN ? 2 * BH : BH;
    const int64_t blocks = ((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    if (!grid_fits(blocks, 256, 1)) return kTooLarge;
    hipLaunchKernelGGL((ffn_small_kernel<S, O, EPI, BM, BH, ANY>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <typename S, typename O, FfnEpilogue EPI>
hipError_t ffn_run_large(const FfnGemmArgs &a, hipStream_t st) {
    constexpr int BN = EPI == FFN_PLAIN ? 256 : 128;
    const int64_t blocks = ((a.M + 255) / 256) * ((a.N + BN - 1) / BN);
    if (!grid_fits(blocks, 512, 1)) return kTooLarge;
    hipLaunchKernelGGL((ffn_large_kernel<S, O, EPI>), dim3((unsigned)blocks), dim3(512), 0, st, a);
    return hipGetLastError();
}

template <typename S, typename O, FfnEpilogue EPI>
hipError_t ffn_run(const FfnGemmArgs &a, hipStream_t st) {
    bool vec = a.K % (16 / (int)sizeof(S)) == 0 && a.as * sizeof(S) % 16 == 0 && a.bs * sizeof(S) % 16 == 0;
    for (const void *p : {a.a, a.b0, a.b1}) vec = vec && (uintptr_t)p % 16 == 0;
    constexpr int BN = EPI == FFN_PLAIN ? 2 : 1;
    if (vec) {
        const int64_t large = ((a.M + 255) / 256) * ((a.N + 128 * BN - 1) / (128 * BN));
        if (large >= 192) return ffn_run_large<S, O, EPI>(a, st);
        const int64_t mid = ((a.M + 127) / 128) * ((a.N + 64 * BN - 1) / (64 * BN));
        if (mid >= 256) return ffn_run_small<S, O, EPI, 128, 64, false>(a, st);
        return ffn_run_small<S, O, EPI, 64, 32, false>(a, st);
    }
    // (the backward pass lays its operands out aligned)
    if constexpr (EPI == FFN_PLAIN) return hipErrorInvalidValue;
    else return ffn_run_small<S, O, EPI, 64, 32, true>(a, st);
}

}  // namespace
}  // namespace convlower
