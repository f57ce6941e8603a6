// The part of the chunked gated delta rule that runs along the sequence, and
// its mirror image for the gradients.
//
// Columns of the state never meet, so a wavefront takes 16 NT columns of one
// value head and holds them, [dk][16 NT] in float32, in registers from the
// first chunk to the last.  A chunk is five products whose right operands come
// out of registers.  The left operands (K, Q, the inverse and P, 58 KB for a
// 16-bit dk = 128) are the same for all columns: the block's wavefronts copy
// the next chunk's into the other half of LDS while they work on this one's,
// with one barrier a chunk.  K', Q', and on the way back the transposes of the
// triangular operands, are read from the same bytes by the transposing LDS
// read.
#include "delta_chunk.h"

namespace convlower {
namespace {

template <int BYTES>
struct Bits {
    typedef uint16_t type;
};
template <>
struct Bits<4> {
    typedef uint32_t type;
};

template <int N, int NT>
__device__ __forceinline__ void zero(f32x4 (&v)[NT][N]) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < N; ++i) v[t][i] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// What a wavefront works on, and where things lie.
template <typename S, int DKP, int NT, int NW>
struct Scan {
    static constexpr bool SPLIT = sizeof(S) == 4;
    static constexpr int KS = DKP / 32, MT = DKP / 16, PL = SPLIT ? 2 : 1;
    static constexpr int kMat = kC * DKP * 2;                  // bytes of one half of K or Q
    static constexpr int kIn = 2 * PL * kMat;                  // K and Q
    static constexpr int kStage = kIn + kTpBytes;
    static constexpr int STAGES = 2 * kStage <= 160 * 1024 ? 2 : 1;
    static constexpr int kTi = kIn, kP = kIn + kTpRows / 2, kRows = kIn + kTpRows;

    int n, h, hk, tile, g, m, tl;
    int64_t a, e, base, chunks;
    bool live[NT];

    // Blocks of one query/key head go to one XCD (every eighth block), whose
    // L2 then serves K and Q to all of them.
    __device__ __forceinline__ bool place(const DeltaArgs &A, int groups) {
        const int rep = A.Hv / A.Hk, inner = groups * rep;
        const int64_t b = blockIdx.x;
        const int64_t unit = b / (8 * inner) * 8 + b % 8;
        const int in = (int)(b / 8 % inner);
        if (unit >= (int64_t)A.s.N * A.Hk) return false;
        n = (int)(unit / A.Hk);
        hk = (int)(unit % A.Hk);
        h = hk * rep + in / groups;
        tile = ((in % groups) * NW + (threadIdx.x >> 6)) * NT;
        const int lane = threadIdx.x & 63;
        g = lane >> 4, m = lane & 15, tl = trans_lane();
        for (int t = 0; t < NT; ++t) live[t] = (tile + t) * 16 + m < A.dv;
        seq_range(A.s, n, &a, &e);
        base = slot_base(A.s, n);
        chunks = (e - a + kC - 1) / kC;
        return true;
    }
    __device__ __forceinline__ int len_of(int64_t c) const {
        const int64_t left = e - a - c * kC;
        return left < kC ? (int)left : kC;
    }
    __device__ __forceinline__ void issue(const DeltaArgs &A, const DeltaBuf &B, int64_t c, const char *tp, char *lds) const {
        const int64_t slot = base + c;
        copy_in<NW, kIn / 1024>((const char *)B.kq + (slot * A.Hk + hk) * kIn, lds);
        copy_in<NW, kTpBytes / 1024>(tp + (slot * A.Hv + h) * kTpBytes, lds + kIn);
    }
    // Columns of a [64][..] tensor of the caller's in result order, by buffer
    // accesses: rows past the chunk's end and columns past the last read as
    // zeros and are not written, being past the buffer's end.
    __device__ __forceinline__ void load(const S *p, int64_t stride, int len, uint32_t (&v)[NT][16]) const {
        const __amdgpu_buffer_rsrc_t r = rows_of(p);
        const int st = (int)stride * (int)sizeof(S);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int at = live[t] ? 4 * g * st + ((tile + t) * 16 + m) * (int)sizeof(S) : (int)kOutOfRange;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 16 * (i / 4) + i % 4;  // and 4 g
                const int o = len == kC || row + 4 * g < len ? at : (int)kOutOfRange;
                if constexpr (sizeof(S) == 2) v[t][i] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, row * st, 0);
                else v[t][i] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, o, row * st, 0);
            }
        }
    }
    __device__ __forceinline__ void store(S *p, int64_t stride, int len, const f32x4 (&v)[NT][4]) const {
        const __amdgpu_buffer_rsrc_t r = rows_of(p);
        const int st = (int)stride * (int)sizeof(S);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int at = live[t] ? 4 * g * st + ((tile + t) * 16 + m) * (int)sizeof(S) : (int)kOutOfRange;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = 16 * (i / 4) + i % 4;
                const int o = len == kC || row + 4 * g < len ? at : (int)kOutOfRange;
                const S x = mix_out<S>(v[t][i / 4][i % 4]);
                if constexpr (sizeof(S) == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(short, x), r, o, row * st, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(int, x), r, o, row * st, 0);
            }
        }
    }
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rows_of(const void *p) {
        const uint64_t a = (uint64_t)p;
        const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)a);
        const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32));
        return make_rsrc((const void *)(lo | hi << 32), 0x7fffffff);
    }
    template <int N>
    __device__ __forceinline__ void store_result(float *p, int tiles, const f32x4 (&v)[NT][N]) const {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (tile + t < tiles) *(f32x4 *)(p + (((tile + t) * N + i) * 64 + (threadIdx.x & 63)) * 4) = v[t][i];
    }
    // [dk][dv] float32 of the caller's.
    __device__ __forceinline__ void load_state(const DeltaArgs &A, const float *p, f32x4 (&v)[NT][MT]) const {
        const int64_t at = ((int64_t)n * A.Hv + h) * A.dk * A.dv;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 4 * g + r;
                    v[t][i][r] = p && live[t] && row < A.dk ? p[at + (int64_t)row * A.dv + (tile + t) * 16 + m] : 0.f;
                }
    }
    __device__ __forceinline__ void store_state(const DeltaArgs &A, float *p, const f32x4 (&v)[NT][MT]) const {
        if (!p) return;
        const int64_t at = ((int64_t)n * A.Hv + h) * A.dk * A.dv;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 4 * g + r;
                    if (live[t] && row < A.dk) p[at + (int64_t)row * A.dv + (tile + t) * 16 + m] = v[t][i][r];
                }
    }

    // Products with what lies in LDS.  Consecutive products go to different
    // results, so that none waits for the one before it.
    __device__ __forceinline__ void by_rows(const char *x, int s, const Split (&b)[NT][KS], f32x4 (&c)[NT][4]) const {
        f16x8 f[4];
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) f[mt] = frag_at(x + (mt * KS + s) * 1024);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) c[t][mt] = mma(f[mt], b[t][s].lo, c[t][mt]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) c[t][mt] = mma(f[mt], b[t][s].hi, c[t][mt]);
        if constexpr (SPLIT) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) f[mt] = frag_at(x + kMat + (mt * KS + s) * 1024);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) c[t][mt] = mma(f[mt], b[t][s].hi, c[t][mt]);
        }
    }
    // c[t] = (rows 16 mt.. of the transpose) b[t]
    __device__ __forceinline__ void by_cols(const char *x, int mt, const Split (&b)[NT][2], f32x4 (&c)[NT]) const {
#pragma unroll
        for (int t = 0; t < NT; ++t) c[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const char *p = x + (2 * s * KS + mt / 2) * 1024;
            const f16x8 f = trans_at(p, p + KS * 1024, mt, tl);
#pragma unroll
            for (int t = 0; t < NT; ++t) c[t] = mma2(f, b[t][s], c[t]);
            if constexpr (SPLIT) {
                const f16x8 l = trans_at(p + kMat, p + kMat + KS * 1024, mt, tl);
#pragma unroll
                for (int t = 0; t < NT; ++t) c[t] = mma(l, b[t][s].hi, c[t]);
            }
        }
    }
    template <bool TRANS>
    __device__ __forceinline__ void by_tri(const char *x, const Split (&b)[NT][2], f32x4 (&c)[NT][4]) const {
        zero(c);
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (TRANS ? s < mt / 2 : s > mt / 2) continue;
                f16x8 hi, lo;
                if constexpr (TRANS) {
                    const char *p = x + tri_lower(2 * s, mt / 2) * 1024, *q = x + tri_lower(2 * s + 1, mt / 2) * 1024;
                    hi = trans_at(p, q, mt, tl), lo = trans_at(p + kTri * 1024, q + kTri * 1024, mt, tl);
                } else {
                    const char *p = x + tri_lower(mt, s) * 1024;
                    hi = frag_at(p), lo = frag_at(p + kTri * 1024);
                }
#pragma unroll
                for (int t = 0; t < NT; ++t) c[t][mt] = mma3(hi, lo, b[t][s], c[t][mt]);
            }
    }
};

// Starts a chunk: its operands are in LDS, its own rows in registers, and
// nobody reads the other half of LDS any more.  Waiting for this wavefront's
// copies before the barrier makes everybody's visible after it.  The rows are
// taken over before new loads are issued, which the compiler counts without
// the copies to LDS.
template <typename S, int NT>
__device__ __forceinline__ void chunk_ready(uint32_t (&rows)[NT][16], f32x4 (&v)[NT][4]) {
    CONVLOWER_WAIT_VMCNT_LDS(0);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            asm volatile("" : "+v"(rows[t][i]));
            v[t][i / 4][i % 4] = mix_f32(__builtin_bit_cast(S, (typename Bits<sizeof(S)>::type)rows[t][i]));
        }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(v[t][i]));
    block_barrier();
}

template <typename S, int DKP, int NT, int NW, bool SAVE>
__global__ __launch_bounds__(64 * NW) void delta_scan_kernel(DeltaArgs A, DeltaBuf B, int groups) {
    typedef Scan<S, DKP, NT, NW> W;
    constexpr int MT = W::MT, KS = W::KS;
    __shared__ __align__(16) char lds[W::STAGES * W::kStage];
    W w;
    if (!w.place(A, groups)) return;
    f32x4 st[NT][MT];
    w.load_state(A, A.state, st);
    uint32_t next[NT][16] = {};
    auto values = [&](int64_t c) {
        w.load((const S *)A.v + (w.a + c * kC) * A.vs + (int64_t)w.h * A.dv, A.vs, w.len_of(c), next);
    };
    // stored after the next chunk has begun: a chunk begins by waiting for all memory accesses before it
    f32x4 o[NT][4];
    auto results = [&](int64_t c) {
        w.store((S *)A.o + ((w.a + c * kC) * A.Hv + w.h) * A.dv, (int64_t)A.Hv * A.dv, w.len_of(c), o);
    };
    if (w.chunks > 0) {
        if (W::STAGES == 2) w.issue(A, B, 0, B.tp, lds);
        values(0);
    }
    for (int64_t c = 0; c < w.chunks; ++c) {
        const char *x = lds + (W::STAGES == 2 && (c & 1) ? W::kStage : 0);
        if (W::STAGES == 1) {
            block_barrier();
            w.issue(A, B, c, B.tp, lds);
        }
        f32x4 z[NT][4];
        chunk_ready<S>(next, z);
        const int64_t vh = (w.base + c) * A.Hv + w.h;
        if (c > 0) results(c - 1);
        if (c + 1 < w.chunks) {
            if (W::STAGES == 2) w.issue(A, B, c + 1, B.tp, lds + (c & 1 ? 0 : W::kStage));
            values(c + 1);
        }
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + 4 * kC;
        const float last = sc[0], it = sc[1], ip = sc[2];
        Split sb[NT][KS], xb[NT][2];
        float is[NT], inv[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) is[t] = split_cols<MT>(st[t], sb[t]);
        if constexpr (SAVE) {
            w.store_result(B.S + vh * DKP * B.dvp, B.dvp / 16, st);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < MT; ++i) mx = max4(st[t][i], mx);
                mx = tile_max(mx);
                if ((threadIdx.x & 63) == 0 && w.tile + t < B.dvp / 16) B.Smax[vh * (B.dvp / 16) + w.tile + t] = mx;
            }
        }
        f32x4 y[NT][4];
        zero(y);
        zero(o);
#pragma unroll
        for (int s = 0; s < KS; ++s) w.by_rows(x, s, sb, y);
#pragma unroll
        for (int s = 0; s < KS; ++s) w.by_rows(x + W::kIn / 2, s, sb, o);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[t][i] -= y[t][i] * (*(const f32x4 *)(f + 16 * i) * is[t]);
            inv[t] = split_cols<4>(z[t], xb[t]) * it;
        }
        w.template by_tri<false>(x + W::kTi, xb, y);
        if constexpr (SAVE) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) z[t][i] = y[t][i] * inv[t];
            w.store_result(B.Y + vh * kC * B.dvp, B.dvp / 16, z);
        }
        Split ub[NT][2];
        float iu[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[t][i] *= *(const f32x4 *)(f + 3 * kC + 16 * i) * inv[t];  // U
                z[t][i] = y[t][i] * *(const f32x4 *)(f + 2 * kC + 16 * i);
            }
            iu[t] = split_cols<4>(z[t], ub[t]);
            inv[t] = split_cols<4>(y[t], xb[t]) * ip;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f32x4 d[NT];
            w.by_cols(x, mt, ub, d);
#pragma unroll
            for (int t = 0; t < NT; ++t) st[t][mt] = st[t][mt] * last + d[t] * iu[t];
        }
        w.template by_tri<false>(x + W::kP, xb, y);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[t][i] = o[t][i] * (*(const f32x4 *)(f + kC + 16 * i) * is[t]) + y[t][i] * inv[t];
    }
    if (w.chunks > 0) results(w.chunks - 1);
    w.store_state(A, A.state_out, st);
}

// From the last chunk to the first, with G, the gradient of the state.
template <typename S, int DKP, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void delta_scan_grad_kernel(DeltaArgs A, DeltaBuf B, int groups) {
    typedef Scan<S, DKP, NT, NW> W;
    constexpr int MT = W::MT, KS = W::KS;
    __shared__ __align__(16) char lds[W::STAGES * W::kStage];
    W w;
    if (!w.place(A, groups)) return;
    f32x4 G[NT][MT];
    w.load_state(A, A.dstate_out, G);
    uint32_t next[NT][16] = {};
    auto values = [&](int64_t c) {
        w.load((const S *)A.d_o + (w.a + c * kC) * A.dos + (int64_t)w.h * A.dv, A.dos, w.len_of(c), next);
    };
    f32x4 e[NT][4], dz[NT][4];  // stored after the next chunk has begun
    auto results = [&](int64_t c) {
        w.store_result(B.E + ((w.base + c) * A.Hv + w.h) * kC * B.dvp, B.dvp / 16, e);
        w.store((S *)A.dv_out + ((w.a + c * kC) * A.Hv + w.h) * A.dv, (int64_t)A.Hv * A.dv, w.len_of(c), dz);
    };
    if (w.chunks > 0) {
        if (W::STAGES == 2) w.issue(A, B, w.chunks - 1, B.tpg, lds);
        values(w.chunks - 1);
    }
    int half = 0;
    for (int64_t c = w.chunks - 1; c >= 0; --c) {
        const char *x = lds + half * W::kStage;
        if (W::STAGES == 1) {
            block_barrier();
            w.issue(A, B, c, B.tpg, lds);
        } else {
            half ^= 1;
        }
        f32x4 d[NT][4];
        chunk_ready<S>(next, d);
        const int64_t vh = (w.base + c) * A.Hv + w.h;
        if (c + 1 < w.chunks) results(c + 1);
        if (c > 0) {
            if (W::STAGES == 2) w.issue(A, B, c - 1, B.tpg, lds + half * W::kStage);
            values(c - 1);
        }
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + 4 * kC;
        const float last = sc[0], it = sc[1], ip = sc[2];
        Split gb[NT][KS], xb[NT][2];
        float ig[NT], inv[NT];
        w.store_result(B.G + vh * DKP * B.dvp, B.dvp / 16, G);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            ig[t] = split_cols<MT>(G[t], gb[t]);
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) mx = max4(G[t][i], mx);
            mx = tile_max(mx);
            if ((threadIdx.x & 63) == 0 && w.tile + t < B.dvp / 16) B.Gmax[vh * (B.dvp / 16) + w.tile + t] = mx;
            inv[t] = split_cols<4>(d[t], xb[t]) * ip;
        }
        f32x4 y[NT][4];
        w.template by_tri<true>(x + W::kP, xb, y);
        zero(e);
#pragma unroll
        for (int s = 0; s < KS; ++s) w.by_rows(x, s, gb, e);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) e[t][i] = e[t][i] * (*(const f32x4 *)(f + 2 * kC + 16 * i) * ig[t]) + y[t][i] * inv[t];
            inv[t] = split_cols<4>(e[t], xb[t]) * it;
        }
        w.template by_tri<true>(x + W::kTi, xb, e);
        Split db[NT][2];
        float id[NT], iy[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                e[t][i] *= inv[t];
                dz[t][i] = e[t][i] * *(const f32x4 *)(f + 3 * kC + 16 * i);
                d[t][i] *= *(const f32x4 *)(f + kC + 16 * i);
                y[t][i] = dz[t][i] * *(const f32x4 *)(f + 16 * i);
            }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            id[t] = split_cols<4>(d[t], db[t]);
            iy[t] = split_cols<4>(y[t], xb[t]);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f32x4 p[NT], q[NT];
            w.by_cols(x + W::kIn / 2, mt, db, p);
            w.by_cols(x, mt, xb, q);
#pragma unroll
            for (int t = 0; t < NT; ++t) G[t][mt] = G[t][mt] * last + p[t] * id[t] - q[t] * iy[t];
        }
    }
    if (w.chunks > 0) results(0);
    w.store_state(A, A.dstate, G);
}

template <typename S, int DKP, int NT, int NW>
hipError_t scan_run(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    // saved matrices are written in whole slabs of columns
    const int cols = grad || b.S ? b.dvp : a.dv;
    const int groups = (cols + 16 * NT * NW - 1) / (16 * NT * NW);
    const int64_t units = ((int64_t)a.s.N * a.Hk + 7) / 8 * 8;
    const dim3 grid((unsigned)(units * groups * (a.Hv / a.Hk)));
    auto run = [&](auto kern) {
        hipLaunchKernelGGL(kern, grid, dim3(64 * NW), 0, st, a, b, groups);
        return hipGetLastError();
    };
    if (grad) return run(delta_scan_grad_kernel<S, DKP, NT, NW>);
    if (b.S) return run(delta_scan_kernel<S, DKP, NT, NW, true>);
    return run(delta_scan_kernel<S, DKP, NT, NW, false>);
}

template <typename S, int DKP>
hipError_t scan_typed(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    return scan_run<S, DKP, 1, 2>(a, b, grad, st);
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? scan_typed<float, 64>(a, b, grad, st) : scan_typed<float, 128>(a, b, grad, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? scan_typed<_Float16, 64>(a, b, grad, st) : scan_typed<_Float16, 128>(a, b, grad, st);
    return b.dkp == 64 ? scan_typed<uint16_t, 64>(a, b, grad, st) : scan_typed<uint16_t, 128>(a, b, grad, st);
}

}  // namespace convlower
