// Shared by the kernels of the chunked gated delta rule.
//
// A chunk is C = 64 tokens of one sequence.  With gam the running sum of g
// inside the chunk, G_ij = exp(gam_i - gam_j) and S the state before it:
//
//   L_ij = (k_i . k_j) G_ij, i > j        P_ij = (q_i . k_j) G_ij, i >= j
//   Z = V - diag(e^gam) K S               what the state alone predicts wrongly
//   Y = (1 + L diag(b))^-1 Z              v - S'k at each token's turn
//   U = diag(b) Y
//   O = diag(e^gam) Q S + P U
//   S' = e^gam_C S + K' diag(e^(gam_C - gam)) U
//
// and backwards, with X the gradient of U as an output, G that of S':
//
//   X = P' dO + diag(e^(gam_C - gam)) K G
//   E = (1 + L' diag(b))^-1 X             the gradient of U in full
//   dZ = diag(b) E = dV,   db_i = Y_i . E_i
//   dS = e^gam_C G + Q' diag(e^gam) dO - K' diag(e^gam) dZ
//
// (q holds the scale; q and k their norms where asked for.)
//
// Products run on the f16 matrix cores, with float32 results.  An operand
// that is a bf16 or f16 input is exact there: each token's row is moved by a
// power of two to the middle of f16's range.  Any other operand is split in
// two, x = hi + lo, each 11 bits, after moving its column (or the whole
// tile) by a power of two: 22 bits, two fewer than float32 has (measured: 3e-7
// of a float32 state's norm, 6e-7 of the outputs'); hi alone (or bf16) would
// leave three digits in the state.  What is carried from chunk to chunk stays
// float32.  A product of two split operands leaves out lo * lo.  float32
// inputs are split as well.
//
// The 16x16x32 product takes column (row) k of its left (right) operand from
// lane group k / 8.  Results lie otherwise: row 4 g + r in group g.  So that
// a result can be the next right operand without leaving its lanes, every
// left operand's columns are stored in the order in which results lie:
// place (g, j) of the 32-column step s holds column
//   kappa(s, g, j) = 32 s + (j < 4 ? 4 g + j : 16 + 4 g + j - 4).
#pragma once

#include "igemm_impl.h"
#include "mixer_internal.h"

namespace convlower {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kC = 64;        // tokens of a chunk
constexpr int kFrag = 512;    // f16 values of one operand fragment: 64 lanes x 8
constexpr int kTri = 6;       // fragments of a triangular 64 x 64 operand: 16 rows x 32 columns each
constexpr int kSlab = 64;     // value columns the gradient kernel takes at once

// Fragment of a lower triangular left operand: rows 16 mt.., columns 32 s..
__device__ __forceinline__ constexpr int tri_lower(int mt, int s) { return mt < 2 ? mt : 2 * mt - 2 + s; }

// Everything the kernels hand one another.  A "slot" is a chunk's place:
// sequence n's chunk c is slot start(n) / 64 + n + c, which needs no sums over
// the sequences' lengths (T / 64 + N slots hold any T tokens of N sequences).
// Matrices in "result order" lie as the lanes hold them: [tile of 16 columns]
// [tile of 16 rows][lane][4 rows].
struct DeltaBuf {
    int slots, dkp, dvp;  // dk in 64 or 128 columns, dv in whole slabs
    int planes;           // 2: q and k in two halves (float32 inputs)
    _Float16 *kq;  // [slots][Hk][K, Q][planes][64 * dkp] as left operands
    char *tp;      // [slots][Hv] of kTpBytes: the inverse, P, and the rows' factors
    char *tpg;     // the same for the way back (saved): the other inverse, P, factors
    float *rowk;   // saved: [slots][Hk][4][64]: factor of k's row, 1 / k's norm, the same of q
    double *gam;   // saved: [slots][Hv][64]
    float *S, *Y;  // saved: [slots][Hv], [dkp][dvp] and [64][dvp] in result order
    float *Smax;   // saved: [slots][Hv][dvp / 16]: largest |S| of the tile
    float *G, *E, *Gmax;  // gradients: the same of G and E
};
// One chunk of one value head: 6 + 6 fragments of each triangular operand (hi,
// lo), then rows of 64 factors and, in the last row, scalars.
enum TpRow {
    ROW_F1 = 0,   // rho_k e^gam
    ROW_F2 = 1,   // rho_q e^gam
    ROW_F3 = 2,   // rho_k e^(gam_C - gam)
    ROW_B = 3,    // b
    ROW_F3B = 4,  // f3 b
    ROW_F1B = 5,  // f1 b
    ROW_SCALARS = 7,
};
enum TpScalar {
    SC_LAST = 0,  // e^gam_C
    SC_IT = 1,    // 1 / (the inverse's factor)
    SC_IP = 2,    // 1 / (P's factor)
};
// P stands with its columns times b on the way forward (P U = (P b) Y).
constexpr int kTpRows = 4 * kTri * kFrag * 2;  // bytes before the factors
constexpr int kTpBytes = kTpRows + 2048;

hipError_t launch_delta_prep(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st);
hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st);
hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaBuf &b, int dtype, hipStream_t st);

struct DeltaChunk {
    int n, c;       // sequence, chunk in it
    int64_t t0;     // first token
    int len;        // tokens, 0: the slot is not used
};
__device__ __forceinline__ int64_t slot_base(const Seqs &s, int n) {
    return s.cu ? seq_start(s, n) / kC + n : (int64_t)n * ((s.each + kC - 1) / kC);
}
// All 64 lanes take part: they look at 64 sequences at once.
__device__ __forceinline__ DeltaChunk chunk_of(const Seqs &s, int slot) {
    int lo = 0;
    if (!s.cu) {
        const int64_t per = (s.each + kC - 1) / kC;
        lo = per ? (int)(slot / per) : 0;
        if (lo > s.N - 1) lo = s.N - 1;
    } else {
        // the last sequence whose first slot is not past this one
        for (int span = s.N; span > 1;) {
            const int step = (span + 63) / 64;
            const int n = lo + (int)(threadIdx.x & 63) * step;
            const uint64_t before = __ballot(n < lo + span && slot_base(s, n) <= slot);
            const int k = before ? 63 - __builtin_clzll(before) : 0;
            const int left = lo + span - (lo + k * step);
            lo += k * step;
            span = left < step ? left : step;
        }
        lo = __builtin_amdgcn_readfirstlane(lo);
    }
    DeltaChunk r;
    r.n = lo;
    int64_t a, e;
    seq_range(s, lo, &a, &e);
    const int64_t base = s.cu ? a / kC + lo : slot_base(s, lo);
    const int64_t c = slot - base;
    r.c = (int)c;
    r.t0 = a + c * kC;
    const int64_t left = c < 0 ? 0 : e - r.t0;
    r.len = left < 0 ? 0 : left > kC ? kC : (int)left;
    return r;
}

// The power of two that brings m to [2^t, 2^(t+1)), and its inverse.
__device__ __forceinline__ float pow2_to(float m, int t, float *inv) {
    int e = 254 + t - (int)((__float_as_uint(m) >> 23) & 255);
    e = e < 3 ? 3 : e > 251 ? 251 : e;
    *inv = __uint_as_float((uint32_t)(254 - e) << 23);
    return __uint_as_float((uint32_t)e << 23);
}
// A state's next power of two is ss, its present one 1 / is, and `last` what a
// chunk leaves of it: the factor that takes it there.  Either power of two may
// lie near the end of the range (a bound of zero gives the largest), their
// product past it.  Taken in this order and held below infinity, what is zero
// (a cleared state, `last` = 0, or one of zeros) stays zero; a state that is
// neither, and so small that the limit is met, is below float32 anyway.
__device__ __forceinline__ float held(float v) { return __builtin_elementwise_minimum(v, 0x1p126f); }
__device__ __forceinline__ float state_step(float last, float is, float ss) { return held(last * is * ss); }
// Split operands: the largest value (of a state: what it can become in a
// chunk) in [2^14, 2^15).  Halves reach down to 2^-25, so values down to 2^-17 of the
// largest keep all 22 bits.
constexpr int kTop = 14;
// Rows of q and k: largest value in [1, 2).  What f16 then loses of a bf16 or
// f16 row is below 2^-25 of its largest value.
constexpr int kRowTop = 0;
constexpr float kRowSum = 2.f * kC;  // so |K' u| <= kRowSum max |u|

struct Split {
    f16x8 hi, lo;
};
// Two pieces of four rows that are in f16's range already.
__device__ __forceinline__ Split split8(f32x4 a, f32x4 b) {
    typedef float f32x8 __attribute__((ext_vector_type(8)));
    const f32x8 v = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    float one = 1.f;
    asm("" : "+v"(one));  // or the multiply-add is taken apart again
    Split r;
    r.hi = __builtin_convertvector(v, f16x8);
#pragma unroll
    for (int j = 0; j < 8; ++j) r.lo[j] = (_Float16)fmaf(v[j], one, -(float)r.hi[j]);
    return r;
}
__device__ __forceinline__ Split split8(f32x4 a, f32x4 b, float scale) {
    Split r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        // written as fused multiply-adds, which the mixed-precision instructions do in one step each
        r.hi[j] = (_Float16)fmaf(a[j], scale, 0.f);
        r.hi[j + 4] = (_Float16)fmaf(b[j], scale, 0.f);
        r.lo[j] = (_Float16)fmaf(a[j], scale, -(float)r.hi[j]);
        r.lo[j + 4] = (_Float16)fmaf(b[j], scale, -(float)r.hi[j + 4]);
    }
    return r;
}
__device__ __forceinline__ f32x4 mma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma2(f16x8 a, const Split &b, f32x4 c) { return mma(a, b.hi, mma(a, b.lo, c)); }
__device__ __forceinline__ f32x4 mma3(f16x8 ah, f16x8 al, const Split &b, f32x4 c) {
    return mma(ah, b.hi, mma(ah, b.lo, mma(al, b.hi, c)));
}
// (NaN if there is one: two values an instruction, without quieting them first)
__device__ __forceinline__ float max2(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ __forceinline__ float max4(f32x4 v, float m) {
    return max2(max2(fabsf(v[2]), fabsf(v[3])), max2(max2(fabsf(v[0]), fabsf(v[1])), m));
}
// Largest over the four lane groups: of one column of a result.
__device__ __forceinline__ float col_max(float m) {
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const uint32_t a = __float_as_uint(m);
    const u32x2 x = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane16_swap(a, a, false, false));
    const uint32_t b = __float_as_uint(max2(__uint_as_float(x[0]), __uint_as_float(x[1])));
    const u32x2 y = __builtin_bit_cast(u32x2, __builtin_amdgcn_permlane32_swap(b, b, false, false));
    return max2(__uint_as_float(y[0]), __uint_as_float(y[1]));
}
// Largest over a wavefront.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float m) {
    const int x = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), CTRL, 0xf, 0xf, true);
    return max2(m, __builtin_bit_cast(float, x));
}
__device__ __forceinline__ float tile_max(float m) {
    m = dpp_max<0x121>(m);  // row_ror 1, 2, 4, 8: the 16 lanes of a group
    m = dpp_max<0x122>(m);
    m = dpp_max<0x124>(m);
    return col_max(dpp_max<0x128>(m));
}
// Sum over the 16 lanes of a group, to all of them.
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
    return v + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float group_sum(float v) {
    return dpp_add<0x121>(dpp_add<0x122>(dpp_add<0x124>(dpp_add<0x128>(v))));
}
// Right operands of 32 rows each from a result of N tiles of 16 rows.
template <int N>
__device__ __forceinline__ void split_by(const f32x4 (&v)[N], float sc, Split (&out)[N / 2]) {
#pragma unroll
    for (int s = 0; s < N / 2; ++s) out[s] = split8(v[2 * s], v[2 * s + 1], sc);
}
template <int N>
__device__ __forceinline__ float max_of(const f32x4 (&v)[N]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) m = max4(v[i], m);
    return m;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 *lds_s16x4;
typedef __attribute__((address_space(3))) char *lds_bytes;

// A left operand's fragment in LDS.
__device__ __forceinline__ f16x8 frag_at(const char *p) { return *(const f16x8 *)(p + (threadIdx.x & 63) * 16); }
// Where this lane reads in a fragment for its transpose: lane t of a group of
// 16 reads columns 4 (t % 4) .. + 3 of row 4 g + t / 4 and gets column t of
// the group's four rows.
__device__ __forceinline__ int trans_lane() {
    const int lane = threadIdx.x & 63, g = lane >> 4, t = lane & 15;
    return (4 * g + (t >> 2) + 16 * (t & 3)) * 16;
}
// Fragment (mt, s) of the transpose: a and b hold rows 32 s.. and 32 s + 16..,
// both their fragment of columns 32 (mt / 2)...
__device__ __forceinline__ f16x8 trans_at(const char *a, const char *b, int mt, int tl) {
    const int o = tl + (mt & 1) * 8;
    const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)a + o));
    const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)b + o));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
}

// The bytes at p as a buffer.  p is the same for the whole wavefront, whatever
// it was computed from.  A buffer access may read scalars that a vector
// instruction wrote only five cycles later; the compiler does not see into the
// copies below, so the wait is here.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void *p, uint32_t bytes) {
    const uint64_t a = (uint64_t)p;
    uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)a);
    uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32));
    asm volatile("s_nop 4" : "+s"(lo), "+s"(hi));
    return make_rsrc((const void *)(lo | (uint64_t)hi << 32), bytes);
}

// 16-byte copies into LDS, 1 KB an instruction, shared by the block's NW
// wavefronts (NW = 1: done by the one that calls).
template <int NW, int UNITS>
__device__ __forceinline__ void copy_in(const void *src, char *dst) {
    const __amdgpu_buffer_rsrc_t r = uniform_rsrc(src, UNITS * 1024);
    const int w = NW == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t d = (uint32_t)(uintptr_t)(lds_ptr_t)dst + w * 1024, v = (threadIdx.x & 63) * 16 + w * 1024;
#pragma unroll
    for (int u = 0; u < UNITS; u += NW)
        if (u + NW <= UNITS || u + w < UNITS) lds_dma16(r, v + u * 1024, d + u * 1024);
}

}  // namespace convlower
