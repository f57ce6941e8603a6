// The part of the chunked gated delta rule that runs along the sequence, and
// its mirror image for the gradients.
//
// Columns of the state never meet, so a wavefront takes 16 columns of one
// value head and holds them, [dk][16] in float32, in registers from the first
// chunk to the last.  A chunk is five products whose right operands come out
// of registers, each from the result before it, so what counts is how long
// that chain is, and what is not in it is taken elsewhere:
//
//   - A second wavefront does what the chain does not wait for: the outputs
//     Q S and P U and the copies kept for the gradients; on the way back P' dO
//     and Q' (f2 dO), which need no state, before the chain asks for them, and
//     dV.  The two hand over operands and results through LDS, lane by lane.
//   - The left operands (K, Q, the inverse and P, 58 KB for a 16-bit dk = 128)
//     and the rows of V are the same for all columns or lie across them: a
//     third kind of wavefront, one for the block, copies the next chunk's into
//     the other half of LDS and takes the last chunk's results to memory.  It
//     also brings the chunk after that into L2, each block of a query/key head
//     an equal part of the lines: otherwise all of them wait for memory at once.
//
// One barrier a chunk, and one or two inside it for the pair.  K', Q', and on
// the way back the transposes of the triangular operands, are read from the
// same bytes by the transposing LDS read.
//
// 16384 tokens in 6 sequences, the longest of 129 chunks, 32 heads of 128 x 128:
// 300 us, 4450 cycles a chunk of which the chain's products are 1312 (82 of
// 16x16x32); one wavefront doing all of it 338 us, without the lines brought to
// L2 322 us.  32 chunks x 64 heads, with what is kept for the gradients (200 MB)
// 91 us, was 111; back 103 us, was 113.  Two more pairs of columns in a block do
// not fit LDS, and a wavefront's columns cannot be fewer than a product's 16.
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
    // what a pair of wavefronts hand each other: a state's operands, a result of four tiles, scalars
    static constexpr int kPairTiles = 2 * KS * 1024, kPairRows = kPairTiles + 4096, kPair = kPairRows + 1024;
    static constexpr int STAGES = 2 * kStage + 4 * kTile + NW * kPair + 1024 <= 160 * 1024 ? 2 : 1;
    static constexpr int kTi = kIn, kP = kIn + kTpRows / 2, kRows = kIn + kTpRows;
    static constexpr int kVals = STAGES * kStage, kOuts = kVals + 2 * kTile, kPairs = kOuts + 2 * kTile;
    static constexpr int kTouch = kPairs + NW * kPair, kLds = kTouch + 1024;  // (and 1 KB that nobody reads)
    static constexpr int kTouches = 5;

    int n, h, hk, c0, w, role, g, m, tl;  // c0: the block's first column; w: which 16 of its columns
    int inner, share, groups;             // blocks of a query/key head, this one's number, those of a value head
    int64_t a, e, base, chunks;

    // Blocks of one query/key head go to one XCD (every eighth block), whose
    // L2 then serves K and Q to all of them.
    __device__ __forceinline__ bool place(const DeltaArgs &A, int groups_) {
        groups = groups_;
        const int rep = A.Hv / A.Hk;
        inner = groups * rep;
        const int64_t b = blockIdx.x;
        const int64_t unit = b / (8 * inner) * 8 + b % 8;
        const int in = (int)(b / 8 % inner);
        share = in;
        if (unit >= (int64_t)A.s.N * A.Hk) return false;
        n = (int)(unit / A.Hk);
        hk = (int)(unit % A.Hk);
        h = hk * rep + in / groups;
        c0 = (in % groups) * COLS;
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        w = wave % NW, role = wave / NW;
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
    // The copying wavefront's whole life.  A chunk's results are in LDS at the
    // next chunk's barrier.
    template <bool BACK>
    __device__ __forceinline__ void copy(const DeltaArgs &A, const DeltaBuf &B, bool vec, char *lds) const {
        const char *tp = BACK ? B.tpg : B.tp;
        const S *in = BACK ? (const S *)A.d_o : (const S *)A.v;
        S *out = BACK ? (S *)A.dv_out : (S *)A.o;
        const int64_t is = BACK ? A.dos : A.vs, os = (int64_t)A.Hv * A.dv;
        auto chunk = [&](int64_t i) { return BACK ? chunks - 1 - i : i; };
        auto issue = [&](int64_t i, int part) {
            const int64_t c = chunk(i), slot = base + c;
            char *d = lds + (STAGES == 2 ? i & 1 : 0) * kStage;
            if (part != 1) {
                rows_in(in + (a + c * kC) * is + (int64_t)h * A.dv, is, len_of(c), A.dv, vec, lds + kVals + (i & 1) * kTile);
                copy_in<1, kIn / 1024>((const char *)B.kq + (slot * A.Hk + hk) * kIn, d);
            }
            if (part != 0) copy_in<1, kTpBytes / 1024>(tp + (slot * A.Hv + h) * kTpBytes, d + kIn);
        };
        // One access a line brings a later chunk's bytes as far as L2 (what it
        // copies is not looked at): this block's share of q's, k's and the
        // triangular operands', and its columns' of V.  Always kTouches of them.
        auto touch = [&](int64_t i) {
            const int64_t c = chunk(i < chunks ? i : chunks - 1), slot = base + c;
            const int lane = threadIdx.x & 63;
            const uint32_t d = (uint32_t)(uintptr_t)(lds_ptr_t)(lds + kTouch);
            const __amdgpu_buffer_rsrc_t rk = uniform_rsrc((const char *)B.kq + (slot * A.Hk + hk) * kIn, kIn);
            const __amdgpu_buffer_rsrc_t rt = uniform_rsrc(tp + (slot * A.Hv + h) * kTpBytes, kTpBytes);
            const __amdgpu_buffer_rsrc_t rv = rows_of(in + (a + c * kC) * is + (int64_t)h * A.dv + c0);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                lds_dma16(rk, (uint32_t)((lane + 64 * u) * inner + share) * 128, d);
                lds_dma16(rt, (uint32_t)((lane + 64 * u) * groups + c0 / COLS) * 128, d);
            }
            lds_dma16(rv, vec && c0 < A.dv && lane < len_of(c) ? (uint32_t)(lane * (int)is * ES) : kOutOfRange, d);
        };
        auto results = [&](int64_t i) {
            const int64_t c = chunk(i);
            rows_out(out + (a + c * kC) * os + (int64_t)h * A.dv, os, len_of(c), A.dv, vec, lds + kOuts + (i & 1) * kTile);
        };
        if (STAGES == 2 && chunks > 0) issue(0, 2), touch(1);
        for (int64_t i = 0; i < chunks; ++i) {
            if (STAGES == 1) {
                block_barrier();  // nobody reads the chunk before any more
                issue(i, 2);
                if (i > 0) results(i - 1);
            }
            CONVLOWER_WAIT_VMCNT_LDS(STAGES == 2 ? kTouches : 0);
            block_barrier();  // the chunk is in LDS, the results of the one before too
            const bool more = STAGES == 2 && i + 1 < chunks;
            // The way back's first barrier comes soon, and issuing the copies
            // takes a third of a chunk's time.
            if (!BACK && more) issue(i + 1, 2);
            block_barrier();
            if (BACK && more) issue(i + 1, 0);
            if (BACK) block_barrier();
            if (BACK && more) issue(i + 1, 1);
            if (STAGES == 2 && i > 0) results(i - 1);
            touch(i + STAGES);
        }
        block_barrier();
        if (chunks > 0) results(chunks - 1);
        CONVLOWER_WAIT_VMCNT(0);  // nothing is on its way into LDS when the block ends
    }
    // The other wavefronts' side of it.
    __device__ __forceinline__ static void next_chunk() {
        asm volatile("" ::: "memory");
        CONVLOWER_WAIT_LDS();
        if (STAGES == 1) block_barrier();
        block_barrier();
    }

    // Inside a chunk: what this wavefront wrote is there for its partner.
    __device__ __forceinline__ static void hand_over() {
        asm volatile("" ::: "memory");
        CONVLOWER_WAIT_LDS();
        block_barrier();
    }

    // ---- the computing wavefronts
    template <int N>
    __device__ __forceinline__ static void put(char *p, const f32x4 (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) *(f32x4 *)(p + i * 1024 + (threadIdx.x & 63) * 16) = v[i];
    }
    template <int N>
    __device__ __forceinline__ static void get(const char *p, f32x4 (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = *(const f32x4 *)(p + i * 1024 + (threadIdx.x & 63) * 16);
    }
    __device__ __forceinline__ static void put(char *p, const Split (&v)[KS]) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            *(f16x8 *)(p + 2 * s * 1024 + (threadIdx.x & 63) * 16) = v[s].hi;
            *(f16x8 *)(p + (2 * s + 1) * 1024 + (threadIdx.x & 63) * 16) = v[s].lo;
        }
    }
    __device__ __forceinline__ static void get(const char *p, Split (&v)[KS]) {
#pragma unroll
        for (int s = 0; s < KS; ++s) v[s].hi = frag_at(p + 2 * s * 1024), v[s].lo = frag_at(p + (2 * s + 1) * 1024);
    }
    // A float a lane; which: 0 the state's measure, 1 of the chunk.
    __device__ __forceinline__ static float &scalar(char *pair, int which) {
        return ((float *)(pair + kPairRows) + which * 64)[threadIdx.x & 63];
    }
    // The state that a pair's operands stand for, 16 rows by 16.  22 bits: all
    // that the gradients' products take of it, and its float32 values would be
    // another 8 KB a pair to hand over.
    __device__ __forceinline__ static void unsplit(const Split (&b)[KS], float is, f32x4 (&v)[MT]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                v[i][r] = ((float)b[i / 2].hi[4 * (i & 1) + r] + (float)b[i / 2].lo[4 * (i & 1) + r]) * is;
    }
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
    // One half of that product: rows 32 s.. of b.
    __device__ __forceinline__ void cols_step(const char *x, int mt, int s, const Cols &f, const Split &b, f32x4 (&c)[MT]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt + i] = mma(f.f[s][i], b.lo, c[mt + i]);
#pragma unroll
        for (int i = 0; i < 4; ++i) c[mt + i] = mma(f.f[s][i], b.hi, c[mt + i]);
        if constexpr (SPLIT) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const char *p = x + kMat + (2 * s * KS + (mt + i) / 2) * 1024;
                c[mt + i] = mma(trans_at(p, p + KS * 1024, mt + i, tl), b.hi, c[mt + i]);
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

// The wavefront that keeps the state: from it the rows that the chunk's tokens
// miss, and the next state.
template <typename W, typename S>
__device__ __forceinline__ void scan_state(const W &w, const DeltaArgs &A, char *lds) {
    constexpr int MT = W::MT, KS = W::KS;
    char *pair = lds + W::kPairs + w.w * W::kPair;
    // The state, each column times a power of two that keeps it in f16's
    // range; is: the inverse.  What a chunk adds comes in the same measure,
    // which therefore follows from the largest of the state and of W, not from
    // bounds on them: those are loose by up to 2^27 where a chunk's large
    // values have decayed by its end, more than f16's range makes up for.
    f32x4 st[MT];
    Split sb[KS];
    w.load_state(A, A.state, st);
    float is;
    {
        const float s = pow2_to(col_max(max_of(st)), kTop, &is);
#pragma unroll
        for (int i = 0; i < MT; ++i) st[i] *= s;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) sb[s] = split8(st[2 * s], st[2 * s + 1]);
    for (int64_t c = 0; c < w.chunks; ++c) {
#pragma unroll
        for (int s = 2; s < KS; ++s) sb[s] = split8(st[2 * s], st[2 * s + 1]);
        W::put(pair, sb);
        W::scalar(pair, 0) = is;
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? c & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        auto row = [&](int which, int i) { return *(const f32x4 *)(f + which * kC + 16 * i); };
        f32x4 z[4], y[4], f1[4], f3b[4];
        Split zb[2], wb[2];
        // K S
        typename W::Rows kf;
        typename W::Tri tf;
        W::rows_load(x, 0, KS, kf);
        w.values(lds + W::kVals + (c & 1) * W::kTile, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) f1[i] = row(ROW_F1, i);
        const float last = sc[SC_LAST], it = sc[SC_IT];
        w.template tri_load<false>(x + W::kTi, tf.hi);
        W::rows_mul(x, kf, sb, y);
        const float smax = col_max(max_of(st));
        phase();
        // Z
        typename W::Cols kc[MT / 4];
        w.template tri_load<false>(x + W::kTi + W::kLo, tf.lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) f3b[i] = row(ROW_F3B, i);
        w.cols_load(x, 0, kc[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] -= y[i] * (f1[i] * is);
        float iz;
        split_by(z, pow2_to(col_max(max_of(z)), kTop, &iz), zb);
        iz *= it;
        phase();
        // Y
        W::template tri_mul<false, false>(tf, zb, y);
        W::scalar(pair, 1) = iz;
        phase();
        // W, the next power of two, and K' W into the state in it
        W::put(pair + W::kPairTiles, y);
        if (MT > 4) w.cols_load(x, 4, kc[MT / 4 - 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = y[i] * f3b[i];
        float in;
        const float ss = pow2_to(smax * is * last + kRowSum * (col_max(max_of(z)) * iz), kTop, &in);
        const float step = state_step(last, is, ss), sw = held(iz * ss);
        is = in;
        wb[0] = split8(z[0], z[1], sw);
        W::hand_over();
        phase();
#pragma unroll
        for (int i = 0; i < MT; ++i) st[i] *= step;
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) w.cols_step(x, 4 * i, 0, kc[i], wb[0], st);
        wb[1] = split8(z[2], z[3], sw);
        phase();
        w.cols_step(x, 0, 1, kc[0], wb[1], st);
        phase();
        // (the state's first rows are split while its last ones are still to come)
        if (MT > 4) w.cols_step(x, MT - 4, 1, kc[MT / 4 - 1], wb[1], st);
#pragma unroll
        for (int s = 0; s < 2; ++s) sb[s] = split8(st[2 * s], st[2 * s + 1]);
        phase();
    }
    W::hand_over();
#pragma unroll
    for (int i = 0; i < MT; ++i) st[i] *= is;
    w.store_state(A, A.state_out, st);
}

// Its partner: the outputs, and what is kept for the gradients.
template <typename W, typename S, bool SAVE>
__device__ __forceinline__ void scan_outputs(const W &w, const DeltaArgs &A, const DeltaBuf &B, char *lds) {
    constexpr int MT = W::MT, KS = W::KS, DKP = 16 * MT;
    char *pair = lds + W::kPairs + w.w * W::kPair;
    const int tile = w.c0 / 16 + w.w;
    const bool kept = SAVE && tile < B.dvp / 16;
    for (int64_t c = 0; c < w.chunks; ++c) {
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? c & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        const int64_t vh = (w.base + c) * A.Hv + w.h;
        f32x4 o[4], y[4], f2[4];
        Split sb[KS], yb[2];
        typename W::Rows qf;
        typename W::Tri pf;
        // Q S
        W::get(pair, sb);
        const float is = W::scalar(pair, 0);
        W::rows_load(x + W::kIn / 2, 0, KS, qf);
#pragma unroll
        for (int i = 0; i < 4; ++i) f2[i] = *(const f32x4 *)(f + ROW_F2 * kC + 16 * i);
        const float ip = sc[SC_IP];
        W::rows_mul(x + W::kIn / 2, qf, sb, o);
        phase();
        w.template tri_load<false>(x + W::kP, pf.hi);
        w.template tri_load<false>(x + W::kP + W::kLo, pf.lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= f2[i] * is;
        if constexpr (SAVE) {
            if (kept) {
                f32x4 s[MT];
                W::unsplit(sb, is, s);
                w.keep(B.S + vh * DKP * B.dvp, tile, s);
                const float mx = tile_max(max_of(s));
                if ((threadIdx.x & 63) == 0) B.Smax[vh * (B.dvp / 16) + tile] = mx;
            }
        }
        W::hand_over();
        phase();
        // P Y
        W::get(pair + W::kPairTiles, y);
        const float iz = W::scalar(pair, 1);
        float iy;
        split_by(y, pow2_to(col_max(max_of(y)), kTop, &iy), yb);
        iy *= iz * ip;
        if constexpr (SAVE) {
            if (kept) {
                f32x4 z[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = y[i] * iz;
                w.keep(B.Y + vh * kC * B.dvp, tile, z);
            }
        }
        W::template tri_mul<false, false>(pf, yb, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] += y[i] * iy;
        w.results(lds + W::kOuts + (c & 1) * W::kTile, o);
    }
    W::hand_over();
}

template <typename S, int DKP, int NW, bool SAVE>
__global__ __launch_bounds__(kScanBounds) void delta_scan_kernel(DeltaArgs A, DeltaBuf B, int groups, bool vec) {
    typedef Scan<S, DKP, NW> W;
    __shared__ __align__(16) char lds[W::kLds];
    W w;
    if (!w.place(A, groups)) return;
    if (w.role == 0) scan_outputs<W, S, SAVE>(w, A, B, lds);
    else if (w.role == 1) scan_state<W, S>(w, A, lds);
    else w.template copy<false>(A, B, vec, lds);
}

// From the last chunk to the first, with G, the gradient of the state.
template <typename W, typename S>
__device__ __forceinline__ void scan_grad_state(const W &w, const DeltaArgs &A, char *lds) {
    constexpr int MT = W::MT, KS = W::KS;
    char *pair = lds + W::kPairs + w.w * W::kPair;
    f32x4 G[MT];
    w.load_state(A, A.dstate_out, G);
    float is;
    {
        const float s = pow2_to(col_max(max_of(G)), kTop, &is);
#pragma unroll
        for (int i = 0; i < MT; ++i) G[i] *= s;
    }
    for (int64_t j = 0; j < w.chunks; ++j) {
        Split gb[KS], eb[2], yb[2];
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? j & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        auto row = [&](int which, int i) { return *(const f32x4 *)(f + which * kC + 16 * i); };
        f32x4 e[4], y[4], f3[4], f1b[4], q[MT];
        // K G
        typename W::Rows kf;
        typename W::Tri tf;
        W::rows_load(x, 0, KS, kf);
        w.template tri_load<true>(x + W::kTi, tf.hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) f3[i] = row(ROW_F3, i);
        const float last = sc[SC_LAST], it = sc[SC_IT];
#pragma unroll
        for (int s = 0; s < KS; ++s) gb[s] = split8(G[2 * s], G[2 * s + 1]);
        W::put(pair, gb);
        W::scalar(pair, 0) = is;
        W::hand_over();
        phase();
        W::get(pair + W::kPairTiles, y);
        const float dmax = W::scalar(pair, 1);
        w.template tri_load<true>(x + W::kTi + W::kLo, tf.lo);
        W::rows_mul(x, kf, gb, e);
        const float gmax = col_max(max_of(G));
        phase();
        // X = .. + P' dO, E
        typename W::Cols kc[MT / 4];
        w.cols_load(x, 0, kc[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) f1b[i] = row(ROW_F1B, i);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = e[i] * (f3[i] * is) + y[i];
        float ie;
        split_by(e, pow2_to(col_max(max_of(e)), kTop, &ie), eb);
        ie *= it;
        phase();
        W::template tri_mul<true, false>(tf, eb, e);
        phase();
        // dS = .. + Q' (f2 dO) - K' (f1 b E)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] *= ie;
        W::put(pair + W::kPairTiles, e);
        if (MT > 4) w.cols_load(x, 4, kc[MT / 4 - 1]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = e[i] * f1b[i];
        float ig;  // the next power of two, as for the state
        const float ss = pow2_to(gmax * is * last + kRowSum * (col_max(max_of(y)) + dmax), kTop, &ig);
        const float step = state_step(last, is, ss);
        is = ig;
        split_by(y, -ss, yb);
        W::hand_over();
        W::get(pair, q);
#pragma unroll
        for (int i = 0; i < MT; ++i) G[i] *= step;
#pragma unroll
        for (int i = 0; i < MT; ++i) G[i] += q[i] * ss;
        phase();
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) w.cols_mul(x, 4 * i, kc[i], yb, G);
        phase();
    }
    W::hand_over();
#pragma unroll
    for (int i = 0; i < MT; ++i) G[i] *= is;
    w.store_state(A, A.dstate, G);
}

// Its partner: what needs dO alone, P' dO and Q' (f2 dO); dV, and what is kept.
template <typename W, typename S>
__device__ __forceinline__ void scan_grad_outputs(const W &w, const DeltaArgs &A, const DeltaBuf &B, char *lds) {
    constexpr int MT = W::MT, KS = W::KS, DKP = 16 * MT;
    char *pair = lds + W::kPairs + w.w * W::kPair;
    const int tile = w.c0 / 16 + w.w;
    const bool kept = tile < B.dvp / 16;
    for (int64_t j = 0; j < w.chunks; ++j) {
        W::next_chunk();
        const char *x = lds + (W::STAGES == 2 ? j & 1 : 0) * W::kStage;
        const float *f = (const float *)(x + W::kRows) + 4 * w.g;
        const float *sc = (const float *)(x + W::kRows) + ROW_SCALARS * kC;
        auto row = [&](int which, int i) { return *(const f32x4 *)(f + which * kC + 16 * i); };
        const int64_t vh = (w.base + w.chunks - 1 - j) * A.Hv + w.h;
        f32x4 d[4], y[4], f2[4], q[MT];
        Split gb[KS], db[2];
        typename W::Tri pf;
        // P' dO (16-bit dO is exact in one half)
        w.values(lds + W::kVals + (j & 1) * W::kTile, d);
        w.template tri_load<true>(x + W::kP, pf.hi);
        w.template tri_load<true>(x + W::kP + W::kLo, pf.lo);
#pragma unroll
        for (int i = 0; i < 4; ++i) f2[i] = row(ROW_F2, i);
        const float ip = sc[SC_IP];
        float id;
        split_by(d, pow2_to(col_max(max_of(d)), kTop, &id), db);
        W::template tri_mul<true, !W::SPLIT>(pf, db, y);
        id *= ip;
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] *= f2[i];
        const float dmax = col_max(max_of(d));
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= id;
        W::put(pair + W::kPairTiles, y);
        W::scalar(pair, 1) = dmax;
        phase();
        // Q' (f2 dO)
        typename W::Cols qc[MT / 4];
        w.cols_load(x + W::kIn / 2, 0, qc[0]);
        W::hand_over();
        W::get(pair, gb);
        const float is = W::scalar(pair, 0);
        if (kept) {
            f32x4 s[MT];
            W::unsplit(gb, is, s);
            w.keep(B.G + vh * DKP * B.dvp, tile, s);
            const float mx = tile_max(max_of(s));
            if ((threadIdx.x & 63) == 0) B.Gmax[vh * (B.dvp / 16) + tile] = mx;
        }
        if (MT > 4) w.cols_load(x + W::kIn / 2, 4, qc[MT / 4 - 1]);
        split_by(d, pow2_to(dmax, kTop, &id), db);
        phase();
        zero(q);
#pragma unroll
        for (int i = 0; i < MT / 4; ++i) w.cols_mul(x + W::kIn / 2, 4 * i, qc[i], db, q);
#pragma unroll
        for (int i = 0; i < MT; ++i) q[i] *= id;
        W::put(pair, q);
        W::hand_over();
        phase();
        // E, dV = b E
        f32x4 e[4];
        W::get(pair + W::kPairTiles, e);
        if (kept) w.keep(B.E + vh * kC * B.dvp, tile, e);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] *= row(ROW_B, i);
        w.results(lds + W::kOuts + (j & 1) * W::kTile, e);
    }
    W::hand_over();
}

template <typename S, int DKP, int NW>
__global__ __launch_bounds__(kScanBounds) void delta_scan_grad_kernel(DeltaArgs A, DeltaBuf B, int groups, bool vec) {
    typedef Scan<S, DKP, NW> W;
    __shared__ __align__(16) char lds[W::kLds];
    W w;
    if (!w.place(A, groups)) return;
    if (w.role == 0) scan_grad_outputs<W, S>(w, A, B, lds);
    else if (w.role == 1) scan_grad_state<W, S>(w, A, lds);
    else w.template copy<true>(A, B, vec, lds);
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
        hipLaunchKernelGGL(kern, grid, dim3(64 * (2 * NW + 1)), 0, st, a, b, groups, vec);
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
