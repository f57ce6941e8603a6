// The part of the chunked gated delta rule that runs along the sequence, and
// its mirror image for the gradients.
//
// Columns of the state never meet, so a wavefront takes 16 columns of one
// value head and holds them, [dk][16] in float32, in registers from the first
// chunk to the last.  A chunk is five products whose right operands come out
// of registers and whose left operands are read in place; nothing passes
// through LDS and no wavefront waits for another.
#include "delta_chunk.h"

namespace convlower {
namespace {

// Rows 16 i + 4 g + r, one column: a result-shaped piece of a [64][..] tensor
// of the caller's; tokens past the chunk's end are zero.
template <typename S>
__device__ __forceinline__ void load_tile(const S *p, int64_t stride, int len, bool col, f32x4 (&v)[4]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * g + r;
            v[i][r] = col && t < len ? mix_f32(p[t * stride]) : 0.f;
        }
}
template <typename S>
__device__ __forceinline__ void store_tile(S *p, int64_t stride, int len, bool col, const f32x4 (&v)[4]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * i + 4 * g + r;
            if (col && t < len) p[t * stride] = mix_out<S>(v[i][r]);
        }
}
// float32 matrices of N tiles of 16 rows.
template <int N>
__device__ __forceinline__ void store_mat(float *p, int64_t stride, const f32x4 (&v)[N]) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) p[(16 * i + 4 * g + r) * stride] = v[i][r];
}

// Triangular left operand (hi, then lo) times a right operand of 64 rows.
template <bool UPPER>
__device__ __forceinline__ void tri_mul(const _Float16 *a, const Split (&b)[2], f32x4 (&c)[4]) {
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (UPPER ? s < mt / 2 : s > mt / 2) continue;
            const _Float16 *f = a + (UPPER ? tri_upper(mt, s) : tri_lower(mt, s)) * kFrag;
            c[mt] = mma3(*(const f16x8 *)f, *(const f16x8 *)(f + kTri * kFrag), b[s], c[mt]);
        }
}
template <int N>
__device__ __forceinline__ void zero(f32x4 (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = f32x4{0.f, 0.f, 0.f, 0.f};
}

template <typename S, int DKP, bool SAVE>
__global__ __launch_bounds__(64) void delta_scan_kernel(DeltaArgs A, DeltaBuf B, int tiles) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int KS = DKP / 32, MT = DKP / 16, PL = SPLIT ? 2 : 1, HALF = kC * DKP;
    const int lane = threadIdx.x, g = lane >> 4;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % A.Hv, n = blockIdx.x / tiles / A.Hv;
    const int hk = h / (A.Hv / A.Hk), col = tile * 16 + (lane & 15);
    const bool live = col < A.dv;
    int64_t a, e;
    seq_range(A.s, n, &a, &e);
    const int64_t base = slot_base(A.s, n), chunks = (e - a + kC - 1) / kC;
    const int64_t st = ((int64_t)n * A.Hv + h) * A.dk * A.dv + col;
    f32x4 S0[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * g + r;
            S0[i][r] = A.state && live && row < A.dk ? A.state[st + (int64_t)row * A.dv] : 0.f;
        }
    for (int64_t c = 0; c < chunks; ++c) {
        const int64_t slot = base + c, kh = slot * A.Hk + hk, vh = slot * A.Hv + h, t0 = a + c * kC;
        const int len = e - t0 < kC ? (int)(e - t0) : kC;
        const _Float16 *pk = B.k + kh * PL * HALF + lane * 8, *pq = B.q + kh * PL * HALF + lane * 8;
        const _Float16 *pkt = B.kt + kh * PL * HALF + lane * 8;
        const _Float16 *pt = B.t + vh * 2 * kTri * kFrag + lane * 8, *pp = B.p + vh * 2 * kTri * kFrag + lane * 8;
        const float *f = B.rowf + vh * 4 * kC + 4 * g;
        const float last = B.scal[vh * 4], it = B.scal[vh * 4 + 1], ip = B.scal[vh * 4 + 2];
        f32x4 z[4];
        load_tile((const S *)A.v + t0 * A.vs + (int64_t)h * A.dv + col, A.vs, len, live, z);
        Split sb[KS], xb[2];
        const float is = split_cols<MT>(S0, sb);
        f32x4 x[4], o[4];
        zero(x);
        zero(o);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) {
                x[mt] = mma_in<SPLIT>(pk + (mt * KS + s) * kFrag, HALF, sb[s], x[mt]);
                o[mt] = mma_in<SPLIT>(pq + (mt * KS + s) * kFrag, HALF, sb[s], o[mt]);
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            z[i] -= x[i] * (*(const f32x4 *)(f + 16 * i) * is);
            o[i] *= *(const f32x4 *)(f + kC + 16 * i) * is;
        }
        float inv = split_cols<4>(z, xb) * it;
        zero(x);
        tri_mul<false>(pt, xb, x);
        if (SAVE) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = x[i] * inv;
            store_mat(B.Y + vh * kC * B.dvp + col, B.dvp, z);
            store_mat(B.S + vh * DKP * B.dvp + col, B.dvp, S0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] *= *(const f32x4 *)(f + 3 * kC + 16 * i) * inv;  // U
        inv = split_cols<4>(x, xb) * ip;
        zero(z);
        tri_mul<false>(pp, xb, z);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            o[i] += z[i] * inv;
            x[i] *= *(const f32x4 *)(f + 2 * kC + 16 * i);
        }
        store_tile((S *)A.o + (t0 * A.Hv + h) * A.dv + col, (int64_t)A.Hv * A.dv, len, live, o);
        inv = split_cols<4>(x, xb);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f32x4 d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s) d = mma_in<SPLIT>(pkt + (mt * 2 + s) * kFrag, HALF, xb[s], d);
            S0[mt] = S0[mt] * last + d * inv;
        }
    }
    if (!A.state_out) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * g + r;
            if (live && row < A.dk) A.state_out[st + (int64_t)row * A.dv] = S0[i][r];
        }
}

// From the last chunk to the first, with G, the gradient of the state.
template <typename S, int DKP>
__global__ __launch_bounds__(64) void delta_scan_grad_kernel(DeltaArgs A, DeltaBuf B, int tiles) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int KS = DKP / 32, MT = DKP / 16, PL = SPLIT ? 2 : 1, HALF = kC * DKP;
    const int lane = threadIdx.x, g = lane >> 4;
    const int tile = blockIdx.x % tiles, h = blockIdx.x / tiles % A.Hv, n = blockIdx.x / tiles / A.Hv;
    const int hk = h / (A.Hv / A.Hk), col = tile * 16 + (lane & 15);
    const bool live = col < A.dv;
    int64_t a, e;
    seq_range(A.s, n, &a, &e);
    const int64_t base = slot_base(A.s, n), chunks = (e - a + kC - 1) / kC;
    const int64_t st = ((int64_t)n * A.Hv + h) * A.dk * A.dv + col;
    f32x4 G[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * g + r;
            G[i][r] = A.dstate_out && live && row < A.dk ? A.dstate_out[st + (int64_t)row * A.dv] : 0.f;
        }
    for (int64_t c = chunks - 1; c >= 0; --c) {
        const int64_t slot = base + c, kh = slot * A.Hk + hk, vh = slot * A.Hv + h, t0 = a + c * kC;
        const int len = e - t0 < kC ? (int)(e - t0) : kC;
        const _Float16 *pk = B.k + kh * PL * HALF + lane * 8;
        const _Float16 *pkt = B.kt + kh * PL * HALF + lane * 8, *pqt = B.qt + kh * PL * HALF + lane * 8;
        const _Float16 *pt = B.t + vh * 2 * kTri * kFrag + lane * 8, *pp = B.p + vh * 2 * kTri * kFrag + lane * 8;
        const float *f = B.rowf + vh * 4 * kC + 4 * g;
        const float last = B.scal[vh * 4], it = B.scal[vh * 4 + 1], ip = B.scal[vh * 4 + 2];
        store_mat(B.G + vh * DKP * B.dvp + col, B.dvp, G);
        f32x4 d[4], x[4], y[4];
        load_tile((const S *)A.d_o + t0 * A.dos + (int64_t)h * A.dv + col, A.dos, len, live, d);
        Split gb[KS], xb[2];
        const float ig = split_cols<MT>(G, gb);
        zero(x);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int mt = 0; mt < 4; ++mt) x[mt] = mma_in<SPLIT>(pk + (mt * KS + s) * kFrag, HALF, gb[s], x[mt]);
        float inv = split_cols<4>(d, xb) * ip;
        zero(y);
        tri_mul<true>(pp, xb, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = x[i] * (*(const f32x4 *)(f + 2 * kC + 16 * i) * ig) + y[i] * inv;
        inv = split_cols<4>(x, xb) * it;
        zero(y);
        tri_mul<true>(pt, xb, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= inv;
        store_mat(B.E + vh * kC * B.dvp + col, B.dvp, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] *= *(const f32x4 *)(f + 3 * kC + 16 * i);  // dZ
        store_tile((S *)A.dv_out + (t0 * A.Hv + h) * A.dv + col, (int64_t)A.Hv * A.dv, len, live, y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] *= *(const f32x4 *)(f + kC + 16 * i);
            y[i] *= *(const f32x4 *)(f + 16 * i);
        }
        Split yb[2];
        const float id = split_cols<4>(d, xb), iy = split_cols<4>(y, yb);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            f32x4 p = {0.f, 0.f, 0.f, 0.f}, q = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                p = mma_in<SPLIT>(pqt + (mt * 2 + s) * kFrag, HALF, xb[s], p);
                q = mma_in<SPLIT>(pkt + (mt * 2 + s) * kFrag, HALF, yb[s], q);
            }
            G[mt] = G[mt] * last + p * id - q * iy;
        }
    }
    if (!A.dstate) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = 16 * i + 4 * g + r;
            if (live && row < A.dk) A.dstate[st + (int64_t)row * A.dv] = G[i][r];
        }
}

template <typename S, int DKP>
hipError_t scan_typed(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    // saved matrices are written in whole slabs of columns
    const int tiles = grad || b.S ? b.dvp / 16 : (a.dv + 15) / 16;
    const dim3 grid((unsigned)((int64_t)a.s.N * a.Hv * tiles));
    if (grad) hipLaunchKernelGGL((delta_scan_grad_kernel<S, DKP>), grid, dim3(64), 0, st, a, b, tiles);
    else if (b.S) hipLaunchKernelGGL((delta_scan_kernel<S, DKP, true>), grid, dim3(64), 0, st, a, b, tiles);
    else hipLaunchKernelGGL((delta_scan_kernel<S, DKP, false>), grid, dim3(64), 0, st, a, b, tiles);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_scan(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? scan_typed<float, 64>(a, b, grad, st) : scan_typed<float, 128>(a, b, grad, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? scan_typed<_Float16, 64>(a, b, grad, st) : scan_typed<_Float16, 128>(a, b, grad, st);
    return b.dkp == 64 ? scan_typed<uint16_t, 64>(a, b, grad, st) : scan_typed<uint16_t, 128>(a, b, grad, st);
}

}  // namespace convlower
