// The part of the chunked gated delta rule that runs along the sequence, and
// its mirror image for the gradients.
//
// Columns of the state never meet, so a wavefront takes 16 columns of one
// value head and holds them, [dk][16] in float32, in registers from the first
// chunk to the last.  A chunk is five products whose right operands come out
// of registers, each from the result before it, so what counts is how long
// that chain is.  The left operands (K, Q, the inverse and P, 58 KB for a
// 16-bit dk = 128) and the rows of V are the same for all columns or lie
// across them: one more wavefront of the block copies the next chunk's into the other half of LDS and
// takes the last chunk's results from there to memory (issuing those accesses
// took a fifth of a chunk's time from the wavefronts that compute).  One
// barrier a chunk.  K', Q', and on the way back the transposes of the
// triangular operands, are read from the same bytes by the transposing LDS
// read.
#include "delta_chunk.h"

namespace convlower {
namespace {

template <int N>
__device__ __forceinline__ void zero(f32x4 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
}

// A block has fewer threads; but with room for 512 in a kernel's bounds the
// compiler keeps to 256 registers and leaves products' results among the
// ordinary ones (otherwise 160 moves a chunk from the others).
constexpr int kScanBounds = 512;

// What a block works on, and where things lie.
template <typename S, int DKP, int NW>
struct Scan {
    static constexpr bool SPLIT = sizeof(S) == 4;
    static constexpr int KS = DKP / 32, MT = DKP / 16, PL = SPLIT ? 2 : 1, COLS = 16 * NW, ES = sizeof(S);
    static constexpr int kMat = kC * DKP * 2;                  // bytes of one half of K or Q
    static constexpr int kIn = 2 * PL * kMat;                  // K and Q
    static constexpr int kStage = kIn + kTpBytes;
    static constexpr int kRow = COLS * ES, kTile = kC * kRow;  // a row and all rows of V, dO, O or dV
    static constexpr int STAGES = 2 * kStage + 4 * kTile <= 160 * 1024 ? 2 : 1;
    static constexpr int kTi = kIn, kP = kIn + kTpRows / 2, kRows = kIn + kTpRows;
    static constexpr int kVals = STAGES * kStage, kOuts = kVals + 2 * kTile, kLds = kOuts + 2 * kTile;

    int n, h, hk, c0, w, g, m, tl;  // c0: the block's first column; w: the wavefront
    int64_t a, e, base, chunks;

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
        c0 = (in % groups) * COLS;
        w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int lane = threadIdx.x & 63;
        g = lane >> 4, m = lane & 15, tl = trans_lane();
        seq_range(A.s, n, &a, &e);
        base = slot_base(A.s, n);
        chunks = (e - a + kC - 1) / kC;
        return true;
    }
    __device__ __forceinline__ int len_of(int64_t c) const {
        const int64_t left = e - a - c * kC;
        return left < kC ? (int)left : kC;
    }

    // ---- the copying wavefront
    __device__ __forceinline__ static __amdgpu_buffer_rsrc_t rows_of(const void *p) { return uniform_rsrc(p, 0x7fffffff); }
    // Rows of the block's columns, [64][..] of the caller's, to LDS: 16 bytes a
    // lane, or one value at a time where the rows do not lie that way.  What is
    // past the chunk's end or the last column reads as zero.
    __device__ __forceinline__ void rows_in(const S *p, int64_t stride, int len, int dv, bool vec, char *lds) const {
        const __amdgpu_buffer_rsrc_t r = rows_of(p + c0);
        const int lane = threadIdx.x & 63, st = (int)stride * ES;
        if (vec) {
            constexpr int L = kRow / 16;  // lanes of a row
            const uint32_t d = (uint32_t)(uintptr_t)(lds_ptr_t)lds;
            const int col = lane % L * 16;
#pragma unroll
            for (int u = 0; u < kTile / 1024; ++u) {
                const int row = u * (64 / L) + lane / L;
                lds_dma16(r, row < len && c0 + col / ES < dv ? (uint32_t)(row * st + col) : kOutOfRange, d + u * 1024);
            }
        } else {
            for (int u = lane; u < kC * COLS; u += 64) {
                const int row = u / COLS, col = u % COLS;
                const int o = row < len && c0 + col < dv ? row * st + col * ES : (int)kOutOfRange;
                if constexpr (ES == 2) ((uint16_t *)lds)[u] = __builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0);
                else ((uint32_t *)lds)[u] = __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
            }
        }
    }
    __device__ __forceinline__ void rows_out(S *p, int64_t stride, int len, int dv, bool vec, const char *lds) const {
        const __amdgpu_buffer_rsrc_t r = rows_of(p + c0);
        const int lane = threadIdx.x & 63, st = (int)stride * ES;
        typedef int i32x4 __attribute__((ext_vector_type(4)));
        if (vec) {
            constexpr int L = kRow / 16;
            const int col = lane % L * 16;
            i32x4 v[kTile / 1024];
#pragma unroll
            for (int u = 0; u < kTile / 1024; ++u) v[u] = *(const i32x4 *)(lds + u * 1024 + lane * 16);
#pragma unroll
            for (int u = 0; u < kTile / 1024; ++u) {
                const int row = u * (64 / L) + lane / L;
                const int o = row < len && c0 + col / ES < dv ? row * st + col : (int)kOutOfRange;
                __builtin_amdgcn_raw_buffer_store_b128(v[u], r, o, 0, 0);
            }
        } else {
            for (int u = lane; u < kC * COLS; u += 64) {
                const int row = u / COLS, col = u % COLS;
                const int o = row < len && c0 + col < dv ? row * st + col * ES : (int)kOutOfRange;
                if constexpr (ES == 2) __builtin_amdgcn_raw_buffer_store_b16(((const short *)lds)[u], r, o, 0, 0);
                else __builtin_amdgcn_raw_buffer_store_b32(((const int *)lds)[u], r, o, 0, 0);
            }
        }
    }
    // The copying wavefront's whole life.  LAG: after how many barriers a
    // chunk's results are in LDS.
    template <bool BACK, int LAG>
    __device__ __forceinline__ void copy(const DeltaArgs &A, const DeltaBuf &B, bool vec, char *lds) const {
        const char *tp = BACK ? B.tpg : B.tp;
        const S *in = BACK ? (const S *)A.d_o : (const S *)A.v;
        S *out = BACK ? (S *)A.dv_out : (S *)A.o;
        const int64_t is = BACK ? A.dos : A.vs, os = (int64_t)A.Hv * A.dv;
        auto chunk = [&](int64_t i) { return BACK ? chunks - 1 - i : i; };
        auto issue = [&](int64_t i) {
            const int64_t c = chunk(i), slot = base + c;
            char *d = lds + (STAGES == 2 ? i & 1 : 0) * kStage;
            rows_in(in + (a + c * kC) * is + (int64_t)h * A.dv, is, len_of(c), A.dv, vec, lds + kVals + (i & 1) * kTile);
            copy_in<1, kIn / 1024>((const char *)B.kq + (slot * A.Hk + hk) * kIn, d);
            copy_in<1, kTpBytes / 1024>(tp + (slot * A.Hv + h) * kTpBytes, d + kIn);
        };
        auto results = [&](int64_t i) {
            const int64_t c = chunk(i);
            rows_out(out + (a + c * kC) * os + (int64_t)h * A.dv, os, len_of(c), A.dv, vec, lds + kOuts + (i & 1) * kTile);
        };
        if (STAGES == 2 && chunks > 0) issue(0);
        for (int64_t i = 0; i < chunks; ++i) {
            if (STAGES == 1) {
                block_barrier();  // nobody reads the chunk before any more
                issue(i);
                if (i >= LAG) results(i - LAG);
            }
            CONVLOWER_WAIT_VMCNT_LDS(0);
            block_barrier();  // the chunk is in LDS, the results of the one before too
            if (STAGES == 2) {
                if (i >= LAG) results(i - LAG);
                if (i + 1 < chunks) issue(i + 1);
            }
        }
        block_barrier();
        for (int64_t i = chunks > LAG ? chunks - LAG : 0; i < chunks; ++i) results(i);
    }
    // The other wavefronts' side of it.
    __device__ __forceinline__ static void next_chunk() {
        CONVLOWER_WAIT_LDS();
        if (STAGES == 1) block_barrier();
        block_barrier();
    }

    // ---- the computing wavefronts
    __device__ __forceinline__ void values(const char *lds, f32x4 (&v)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (ES == 2) {
                const char *p = lds + (16 * i + 4 * g + (m >> 2)) * kRow + (16 * w + 4 * (m & 3)) * 2;
                const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)p));
#pragma unroll
                for (int r = 0; r < 4; ++r) v[i][r] = mix_f32(__builtin_bit_cast(S, (short)x[r]));
            } else {
#pragma unroll
                for (int r = 0; r < 4; ++r) v[i][r] = *(const float *)(lds + (16 * i + 4 * g + r) * kRow + (16 * w + m) * 4);
            }
        }
    }
    __device__ __forceinline__ void results(char *lds, const f32x4 (&v)[4]) const {
        S *p = (S *)(lds + 4 * g * kRow) + 16 * w + m;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) p[(16 * i + r) * COLS] = mix_out<S>(v[i][r]);
    }
    // Result order, for the gradient kernel; tile: of 16 columns.
    template <int N>
    __device__ __forceinline__ void keep(float *p, int tile, const f32x4 (&v)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) *(f32x4 *)(p + ((tile * N + i) * 64 + (threadIdx.x & 63)) * 4) = v[i];
    }
    // [dk][dv] float32 of the caller's.
    __device__ __forceinline__ void load_state(const DeltaArgs &A, const float *p, f32x4 (&v)[MT]) const {
        const int col = c0 + 16 * w + m;
        const int64_t at = ((int64_t)n * A.Hv + h) * A.dk * A.dv + col;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * g + r;
                v[i][r] = p && col < A.dv && row < A.dk ? p[at + (int64_t)row * A.dv] : 0.f;
            }
    }
    __device__ __forceinline__ void store_state(const DeltaArgs &A, float *p, const f32x4 (&v)[MT]) const {
        const int col = c0 + 16 * w + m;
        const int64_t at = ((int64_t)n * A.Hv + h) * A.dk * A.dv + col;
        if (!p || col >= A.dv) return;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * i + 4 * g + r;
                if (row < A.dk) p[at + (int64_t)row * A.dv] = v[i][r];
            }
    }

    // Products with what lies in LDS.  Consecutive products go to different
    // results, so that none waits for the one before it.
    struct Rows {
        f16x8 f[KS][4];
    };
    __device__ __forceinline__ static void rows_load(const char *x, int s0, int s1, Rows &f) {
#pragma unroll
        for (int s = s0; s < s1; ++s)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) f.f[s][mt] = frag_at(x + (mt * KS + s) * 1024);
    }
    __device__ __forceinline__ static void rows_mul(const char *x, const Rows &f, const Split (&b)[KS], f32x4 (&c)[4]) {
        zero(c);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) c[mt] = mma(f.f[s][mt], b[s].lo, c[mt]);
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) c[mt] = mma(f.f[s][mt], b[s].hi, c[mt]);
            if constexpr (SPLIT) {
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) c[mt] = mma(frag_at(x + kMat + (mt * KS + s) * 1024), b[s].hi, c[mt]);
            }
        }
    }
    // Rows 16 mt.. of the transpose (four tiles of them) times b, added to c.
    struct Cols {
        f16x8 f[2][4];
    };
    __device__ __forceinline__ void cols_load(const char *x, int mt, Cols &f) const {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char *p = x + (2 * s * KS + (mt + i) / 2) * 1024;
                f.f[s][i] = trans_at(p, p + KS * 1024, mt + i, tl);
            }
    }
    __device__ __forceinline__ void cols_mul(const char *x, int mt, const Cols &f, const Split (&b)[2], f32x4 (&c)[MT]) const {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[mt + i] = mma(f.f[s][i], b[s].lo, c[mt + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) c[mt + i] = mma(f.f[s][i], b[s].hi, c[mt + i]);
            if constexpr (SPLIT) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const char *p = x + kMat + (2 * s * KS + (mt + i) / 2) * 1024;
                    c[mt + i] = mma(trans_at(p, p + KS * 1024, mt + i, tl), b[s].hi, c[mt + i]);
                }
            }
        }
    }
    // A triangular operand's fragments, or its transpose's, and its product;
    // ONE: the right operand has no second half.
    struct Tri {
        f16x8 hi[4][2], lo[4][2];
    };
    static constexpr int kLo = kTri * 1024;  // from a triangular operand's first half to its second
    template <bool TRANS>
    __device__ __forceinline__ void tri_load(const char *x, f16x8 (&f)[4][2]) const {
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                if (TRANS ? s < mt / 2 : s > mt / 2) continue;
                if constexpr (TRANS)
                    f[mt][s] = trans_at(x + tri_lower(2 * s, mt / 2) * 1024, x + tri_lower(2 * s + 1, mt / 2) * 1024, mt, tl);
                else f[mt][s] = frag_at(x + tri_lower(mt, s) * 1024);
            }
    }
    template <bool TRANS, bool ONE>
    __device__ __forceinline__ static void tri_mul(const Tri &f, const Split (&b)[2], f32x4 (&c)[4]) {
        zero(c);
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int mt = 0; mt < 4; ++mt) {
                    if ((TRANS ? s < mt / 2 : s > mt / 2) || (ONE && k == 1)) continue;
                    c[mt] = mma(k == 2 ? f.lo[mt][s] : f.hi[mt][s], k == 1 ? b[s].lo : b[s].hi, c[mt]);
                }
    }
};

// A phase of a chunk ends here: its accesses to LDS, which serve the next
// one, are not moved into that.
__device__ __forceinline__ void phase() { __builtin_amdgcn_sched_barrier(0); }

template <typename S, int DKP, int NW, bool SAVE>
__global__ __launch_bounds__(kScanBounds) void delta_scan_kernel(DeltaArgs A, DeltaBuf B, int groups, bool vec) {
    typedef Scan<S, DKP, NW> W;
    constexpr int MT = W::MT, KS = W::KS;
    __shared__ __align__(16) char lds[W::kLds];
    W w;
    if (!w.place(A, groups)) return;
    if (w.w == NW) return w.template copy<false, 2>(A, B, vec, lds);
    const int tile = w.c0 / 16 + w.w;
    const bool kept = SAVE && tile < B.dvp / 16;
    // The state, each column times a power of two that keeps it in f16's
    // range; is: the inverse.  What a chunk adds is bounded before it is
    // known, and comes in the same measure.
    f32x4 st[MT];
    w.load_state(A, A.state, st);
    float is, smax = col_max(max_of(st));
    {
        const float s = pow2_to(smax, kTop, &is);
#pragma unroll
        for (int i = 0; i < MT; ++i) st[i] *= s;
        smax *= s;
    }
    // The last product of a chunk, (P b) Y, waits for the next chunk, whose
    // own first product has to wait for the state to be split.
    typename W::Tri pf = {};
    Split yb[2] = {};
    f32x4 o[4];
    float iy = 0.f;
    zero(o);
    auto finish = [&](int64_t c) {
        f32x4 y[4];
        W::template tri_mul<false, false>(pf, yb, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += y[i] * iy;
        w.results(lds + W::kOuts + (c & 1) * W::kTile, o);
    };
    for (int64_t c = 0; c < w.chunks; ++c) {
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? c & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        auto row = [&](int which, int i) { return *(const f32x4 *)(f + which * kC + 16 * i); };
        // the state in two halves; the chunk before is finished meanwhile
        f32x4 z[4], y[4], f1[4], f2[4];
        typename W::Rows kf, qf;
        W::rows_load(x, 0, KS / 2, kf);
        if constexpr (SAVE) {
            if (kept) {
                const int64_t vh = (w.base + c) * A.Hv + w.h;
                f32x4 s[MT];
#pragma unroll
                for (int i = 0; i < MT; ++i) s[i] = st[i] * is;
                w.keep(B.S + vh * DKP * B.dvp, tile, s);
                const float mx = tile_max(smax * is);
                if ((threadIdx.x & 63) == 0) B.Smax[vh * (B.dvp / 16) + tile] = mx;
            }
        }
        Split sb[KS], zb[2], wb[2];
#pragma unroll
        for (int s = 0; s < KS; ++s) sb[s] = split8(st[2 * s], st[2 * s + 1]);
        finish(c - 1);  // (before the first chunk: zeros, which nobody takes)
        phase();
        // K S
        W::rows_load(x, KS / 2, KS, kf);
        w.values(lds + W::kVals + (c & 1) * W::kTile, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) f1[i] = row(ROW_F1, i);
        W::rows_load(x + W::kIn / 2, 0, KS / 2, qf);
        W::rows_mul(x, kf, sb, y);
        phase();
        // Q S; Z
        typename W::Tri tf;
        W::rows_load(x + W::kIn / 2, KS / 2, KS, qf);
        w.template tri_load<false>(x + W::kTi, tf.hi);
        const float last = sc[SC_LAST], it = sc[SC_IT], ip = sc[SC_IP], bt = sc[SC_T], bw = sc[SC_TF3];
        W::rows_mul(x + W::kIn / 2, qf, sb, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] -= y[i] * (f1[i] * is);
        float iz;
        const float zmax = col_max(max_of(z));
        split_by(z, pow2_to(zmax, kTop, &iz), zb);
        iz *= it;
        phase();
        // Y
        typename W::Cols kc[MT / 4];
        w.template tri_load<false>(x + W::kTi + W::kLo, tf.lo);
        f32x4 f3b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f3b[i] = row(ROW_F3B, i), f2[i] = row(ROW_F2, i);
        w.cols_load(x, 0, kc[0]);
        W::template tri_mul<false, false>(tf, zb, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= f2[i] * is;
        // the next power of two, and the state in it
        const float ss = pow2_to(smax * is * last + kRowSum * (zmax * bw), kBound, &iy);
        const float step = last * (ss * is);
        is = iy;
#pragma unroll
        for (int i = 0; i < MT; ++i) st[i] *= step;
        phase();
        // W, and K' W into the state
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = y[i] * f3b[i];
        split_by(z, iz * ss, wb);
        if (MT > 4) w.cols_load(x, 4, kc[MT / 4 - 1]);
        phase();
        w.template tri_load<false>(x + W::kP, pf.hi);
        w.template tri_load<false>(x + W::kP + W::kLo, pf.lo);
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) w.cols_mul(x, 4 * i, kc[i], wb, st);
        if constexpr (SAVE) {
            if (kept) {
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = y[i] * iz;
                w.keep(B.Y + ((w.base + c) * A.Hv + w.h) * kC * B.dvp, tile, z);
            }
        }
        split_by(y, iz * pow2_to(zmax * bt, kBound, &iy), yb);
        iy *= ip;
        phase();
        smax = col_max(max_of(st));
    }
    finish(w.chunks - 1);
    CONVLOWER_WAIT_LDS();
    block_barrier();
#pragma unroll
    for (int i = 0; i < MT; ++i) st[i] *= is;
    w.store_state(A, A.state_out, st);
}

// From the last chunk to the first, with G, the gradient of the state.
template <typename S, int DKP, int NW>
__global__ __launch_bounds__(kScanBounds) void delta_scan_grad_kernel(DeltaArgs A, DeltaBuf B, int groups, bool vec) {
    typedef Scan<S, DKP, NW> W;
    constexpr int MT = W::MT, KS = W::KS;
    __shared__ __align__(16) char lds[W::kLds];
    W w;
    if (!w.place(A, groups)) return;
    if (w.w == NW) return w.template copy<true, 1>(A, B, vec, lds);
    const int tile = w.c0 / 16 + w.w;
    const bool kept = tile < B.dvp / 16;
    f32x4 G[MT];
    w.load_state(A, A.dstate_out, G);
    float is, gmax = col_max(max_of(G));
    {
        const float s = pow2_to(gmax, kTop, &is);
#pragma unroll
        for (int i = 0; i < MT; ++i) G[i] *= s;
        gmax *= s;
    }
    for (int64_t j = 0; j < w.chunks; ++j) {
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? j & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        auto row = [&](int which, int i) { return *(const f32x4 *)(f + which * kC + 16 * i); };
        const int64_t vh = (w.base + w.chunks - 1 - j) * A.Hv + w.h;
        f32x4 d[4], y[4], e[4], f3[4], f1b[4], f2[4], b[4];
        typename W::Rows kf;
        typename W::Tri pf, tf;
        W::rows_load(x, 0, KS / 2, kf);
        w.values(lds + W::kVals + (j & 1) * W::kTile, d);
        w.template tri_load<true>(x + W::kP, pf.hi);
        w.template tri_load<true>(x + W::kP + W::kLo, pf.lo);
        if (kept) {
            f32x4 s[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) s[i] = G[i] * is;
            w.keep(B.G + vh * DKP * B.dvp, tile, s);
            const float mx = tile_max(gmax * is);
            if ((threadIdx.x & 63) == 0) B.Gmax[vh * (B.dvp / 16) + tile] = mx;
        }
        float id, ie;
        Split gb[KS], db[2], eb[2], yb[2];
#pragma unroll
        for (int s = 0; s < KS; ++s) gb[s] = split8(G[2 * s], G[2 * s + 1]);
        phase();
        // K G, P' dO (16-bit dO is exact in one half)
        W::rows_load(x, KS / 2, KS, kf);
        w.template tri_load<true>(x + W::kTi, tf.hi);
        w.template tri_load<true>(x + W::kTi + W::kLo, tf.lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) f3[i] = row(ROW_F3, i), f2[i] = row(ROW_F2, i);
        const float last = sc[SC_LAST], it = sc[SC_IT], ip = sc[SC_IP], bf1 = sc[SC_TF1], bf2 = sc[SC_F2];
        W::rows_mul(x, kf, gb, e);
        const float dmax = col_max(max_of(d));
        split_by(d, pow2_to(dmax, kTop, &id), db);
        W::template tri_mul<true, !W::SPLIT>(pf, db, y);
        id *= ip;
        phase();
        // X, E
        typename W::Cols kc, qc;
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = e[i] * (f3[i] * is) + y[i] * id;
        const float emax = col_max(max_of(e));
        split_by(e, pow2_to(emax, kTop, &ie), eb);
        ie *= it;
        w.cols_load(x, 0, kc);
        phase();
#pragma unroll
        for (int i = 0; i < 4; ++i) f1b[i] = row(ROW_F1B, i), b[i] = row(ROW_B, i);
        W::template tri_mul<true, false>(tf, eb, e);
        float ig;
        const float ss = pow2_to(gmax * is * last + kRowSum * (emax * bf1 + dmax * bf2), kBound, &ig);
        const float step = last * (ss * is);
        is = ig;
#pragma unroll
        for (int i = 0; i < MT; ++i) G[i] *= step;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] *= f2[i];
        split_by(d, ss, db);
        w.cols_load(x + W::kIn / 2, 0, qc);
        phase();
        // dS = .. + Q' (f2 dO) - K' (f1 b E)
        w.cols_mul(x + W::kIn / 2, 0, qc, db, G);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            e[i] *= ie;
            y[i] = e[i] * f1b[i];
        }
        split_by(y, -ss, yb);
        phase();
        w.cols_mul(x, 0, kc, yb, G);
        if (MT > 4) {
            w.cols_load(x, 4, kc);
            w.cols_load(x + W::kIn / 2, 4, qc);
        }
        if (kept) w.keep(B.E + vh * kC * B.dvp, tile, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] *= b[i];  // dZ
        w.results(lds + W::kOuts + (j & 1) * W::kTile, e);
        phase();
        if (MT > 4) {
            w.cols_mul(x + W::kIn / 2, 4, qc, db, G);
            w.cols_mul(x, 4, kc, yb, G);
        }
        gmax = col_max(max_of(G));
    }
    CONVLOWER_WAIT_LDS();
    block_barrier();
#pragma unroll
    for (int i = 0; i < MT; ++i) G[i] *= is;
    w.store_state(A, A.dstate, G);
}

template <typename S, int DKP, int NW>
hipError_t scan_run(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    // saved matrices are written in whole slabs of columns
    const int cols = grad || b.S ? b.dvp : a.dv;
    const int groups = (cols + 16 * NW - 1) / (16 * NW);
    const int64_t units = ((int64_t)a.s.N * a.Hk + 7) / 8 * 8;
    const dim3 grid((unsigned)(units * groups * (a.Hv / a.Hk)));
    const int64_t is = (grad ? a.dos : a.vs) * sizeof(S);
    const uintptr_t in = (uintptr_t)(grad ? a.d_o : a.v), out = (uintptr_t)(grad ? a.dv_out : a.o);
    const bool vec = a.dv * sizeof(S) % 16 == 0 && is % 16 == 0 && in % 16 == 0 && out % 16 == 0;
    auto run = [&](auto kern) {
        hipLaunchKernelGGL(kern, grid, dim3(64 * NW + 64), 0, st, a, b, groups, vec);
        return hipGetLastError();
    };
    if (grad) return run(delta_scan_grad_kernel<S, DKP, NW>);
    if (b.S) return run(delta_scan_kernel<S, DKP, NW, true>);
    return run(delta_scan_kernel<S, DKP, NW, false>);
}

template <typename S, int DKP>
hipError_t scan_typed(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    return scan_run<S, DKP, 2>(a, b, grad, st);
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? scan_typed<float, 64>(a, b, grad, st) : scan_typed<float, 128>(a, b, grad, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? scan_typed<_Float16, 64>(a, b, grad, st) : scan_typed<_Float16, 128>(a, b, grad, st);
    return b.dkp == 64 ? scan_typed<uint16_t, 64>(a, b, grad, st) : scan_typed<uint16_t, 128>(a, b, grad, st);
}

}  // namespace convlower
