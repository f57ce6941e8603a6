// Last step of the delta rule's gradients: everything of a chunk once the
// state S before it and G, the gradient of the state after it, are known.
// With D_ij = (dO_i . U_j) G_ij (i >= j) and F_ij = -(dZ_i . U_j) G_ij (i > j),
// the gradients of P and L through their decays,
//
//   dq_i  = e^gam_i S dO_i + sum_j D_ij k_j
//   dkr_i = -e^gam_i S dZ_i + sum_j F_ij k_j                       k as a row
//   dkc_j = e^(gam_C - gam_j) G' U_j + sum_i D_ij q_i + F_ij k_i   k as a column
//   dgam_i = q_i . dq_i + k_i . dkr_i - k_i . dkc_i,  and <S', G> at the end
//   dg_t = sum over i >= t of dgam_i,   db_j = Y_j . E_j
//
// since e^gam_i stands beside q_i and k_i as a row, e^-gam_i beside k_i as a
// column.  A block takes one chunk of one query/key head and adds up the value
// heads that share it; its four wavefronts take 16 tokens each.
#include "delta_chunk.h"

namespace convlower {
namespace {

constexpr int kLs = kSlab + 8;  // f16 values from row to row of a slab in LDS
constexpr int kLd = 68;         // floats from row to row of D and F

// Rows of a left operand, 16 values a lane: moved row by row.  Returns the
// inverse factors of rows 4 g .. 4 g + 3, where their results lie.
__device__ __forceinline__ f32x4 split_rows(const float (&v)[2][8], Split (&out)[2]) {
    float m = 0.f, inv;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[s][j]));
    const float sc = pow2_to(col_max(m), kTop, &inv);
#pragma unroll
    for (int s = 0; s < 2; ++s)
        out[s] = split8(f32x4{v[s][0], v[s][1], v[s][2], v[s][3]}, f32x4{v[s][4], v[s][5], v[s][6], v[s][7]}, sc);
    f32x4 r;
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __shfl(inv, 4 * g + i, 64);
    return r;
}

// A row of 64 values of a slab to LDS in two halves, N threads a row.
template <int N>
__device__ __forceinline__ void put_row(const float (&v)[kSlab / N], _Float16 *hi, _Float16 *lo, float *inv_out, int q) {
    float m = 0.f, inv;
#pragma unroll
    for (int i = 0; i < kSlab / N; ++i) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int d = 1; d < N; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    const float sc = pow2_to(m, kTop, &inv);
#pragma unroll
    for (int i = 0; i < kSlab / N; i += 8) {
        const Split s = split8(f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]}, f32x4{v[i + 4], v[i + 5], v[i + 6], v[i + 7]}, sc);
        *(f16x8 *)(hi + i) = s.hi;
        *(f16x8 *)(lo + i) = s.lo;
    }
    if (q == 0) *inv_out = inv;
}
__device__ __forceinline__ Split lds_frag(const _Float16 *hi, const _Float16 *lo, int row, int s) {
    const int g = (threadIdx.x & 63) >> 4;
    Split r;
    r.hi = *(const f16x8 *)(hi + row * kLs + 32 * s + 8 * g);
    r.lo = *(const f16x8 *)(lo + row * kLs + 32 * s + 8 * g);
    return r;
}
__device__ __forceinline__ f32x4 mma_split(const Split &a, const Split &b, f32x4 c) { return mma3(a.hi, a.lo, b, c); }

template <typename S, int DKP>
__global__ __launch_bounds__(256) void delta_grad_kernel(DeltaArgs A, DeltaBuf B) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int MT = DKP / 16, PL = SPLIT ? 2 : 1, HALF = kC * DKP, TR = 256 / DKP;
    constexpr int kIn = 2 * DKP * kLs * 2, kMat = 2 * kC * kLd * 4;
    __shared__ __align__(16) char first[kIn > kMat ? kIn : kMat];  // a slab of S or G, then D and F
    _Float16 *sh = (_Float16 *)first, *sl = sh + DKP * kLs;
    float *dm = (float *)first, *fm = dm + kC * kLd;
    __shared__ __align__(16) _Float16 uh[kC * kLs], ul[kC * kLs];
    __shared__ float is[DKP], iu[kC], sb[kC], rise[kC], fall[kC], rk[kC], nk[kC], rq[kC], nq[kC], red[4];
    __shared__ double sg[kC];
    __shared__ float dgam[kC];
    const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int g = lane >> 4, m = lane & 15;
    const Chunk ch = chunk_of(A.s, slot);
    if (ch.len == 0) return;
    const int64_t head = (int64_t)slot * A.Hk + hk;
    if (tid < kC) {
        const float *o = B.rowk + head * 4 * kC + tid;
        rk[tid] = o[0], nk[tid] = o[kC], rq[tid] = o[2 * kC], nq[tid] = o[3 * kC];
    }
    const _Float16 *pkt = B.kt + head * PL * HALF + lane * 8, *pqt = B.qt + head * PL * HALF + lane * 8;
    const int row = 16 * w + m;  // this lane's row of left operands
    const bool in = row < ch.len;
    // q and k (with their norms, q without the scale) where results lie
    auto raw = [&](const void *p, int64_t stride, const float *norm, int nt, int r) {
        const int t = 16 * w + 4 * g + r, c = 16 * nt + m;
        return t < ch.len && c < A.dk ? mix_f32(((const S *)p)[(ch.t0 + t) * stride + (int64_t)hk * A.dk + c]) * norm[t]
                                      : 0.f;
    };
    f32x4 dqt[MT], dkt[MT], dotq = {0.f, 0.f, 0.f, 0.f}, dotk = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < MT; ++i) dqt[i] = dkt[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int rep = A.Hv / A.Hk;
    for (int v = 0; v < rep; ++v) {
        const int h = hk * rep + v;
        const int64_t vh = (int64_t)slot * A.Hv + h;
        const float *gS = B.S + vh * DKP * B.dvp, *gG = B.G + vh * DKP * B.dvp;
        const float *gY = B.Y + vh * kC * B.dvp, *gE = B.E + vh * kC * B.dvp;
        __syncthreads();
        if (tid < kC) {
            const double x = ((const double *)B.gam)[vh * kC + tid], all = ((const double *)B.gam)[vh * kC + kC - 1];
            sg[tid] = x;
            rise[tid] = expf((float)x);
            fall[tid] = expf((float)(all - x));
            sb[tid] = B.rowf[vh * 4 * kC + 3 * kC + tid];
        }
        const float last = B.scal[vh * 4];
        f32x4 dq[MT], dk[MT], gu[MT], dp[4], dl[4];
#pragma unroll
        for (int i = 0; i < MT; ++i) dq[i] = dk[i] = gu[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) dp[i] = dl[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        float sgsum = 0.f, db = 0.f;
        for (int c0 = 0; c0 < B.dvp; c0 += kSlab) {
            __syncthreads();  // sb above; the slab before
            {
                constexpr int W = kSlab / TR;
                const int r = tid / TR, q = tid % TR;
                float x[W];
#pragma unroll
                for (int i = 0; i < W; i += 4) mix_load<float, 4>(gS + (int64_t)r * B.dvp + c0 + q * W + i, *(float(*)[4]) & x[i]);
                put_row<TR>(x, sh + r * kLs + q * W, sl + r * kLs + q * W, is + r, q);
            }
            {
                const int r = tid >> 2, q = tid & 3;
                float x[16];
#pragma unroll
                for (int i = 0; i < 16; i += 4) mix_load<float, 4>(gY + (int64_t)r * B.dvp + c0 + q * 16 + i, *(float(*)[4]) & x[i]);
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] *= sb[r];
                put_row<4>(x, uh + r * kLs + q * 16, ul + r * kLs + q * 16, iu + r, q);
            }
            float xo[2][8], xe[2][8];
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int c = c0 + 32 * s + 8 * g;
                const S *po = (const S *)A.d_o + (ch.t0 + row) * A.dos + (int64_t)h * A.dv + c;
#pragma unroll
                for (int j = 0; j < 8; ++j) xo[s][j] = in && c + j < A.dv ? mix_f32(po[j]) : 0.f;
                float y[8];
                mix_load<float, 4>(gE + (int64_t)row * B.dvp + c, *(float(*)[4]) & xe[s][0]);
                mix_load<float, 4>(gE + (int64_t)row * B.dvp + c + 4, *(float(*)[4]) & xe[s][4]);
                mix_load<float, 4>(gY + (int64_t)row * B.dvp + c, *(float(*)[4]) & y[0]);
                mix_load<float, 4>(gY + (int64_t)row * B.dvp + c + 4, *(float(*)[4]) & y[4]);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    db = fmaf(y[j], xe[s][j], db);
                    xe[s][j] *= -sb[row];  // -dZ
                }
            }
            Split fo[2], fe[2];
            const f32x4 io = split_rows(xo, fo), ie = split_rows(xe, fe);
            __syncthreads();
#pragma unroll
            for (int nt = 0; nt < MT; ++nt) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = lds_frag(sh, sl, 16 * nt + m, s);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                const float f = is[16 * nt + m];
                dq[nt] += a * (io * f);
                dk[nt] += b * (ie * f);
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                if (nt > w) continue;
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = lds_frag(uh, ul, 16 * nt + m, s);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                const float f = iu[16 * nt + m];
                dp[nt] += a * (io * f);
                dl[nt] += b * (ie * f);
            }
            __syncthreads();
            {
                constexpr int W = kSlab / TR;
                const int r = tid / TR, q = tid % TR;
                float x[W], y[4];
#pragma unroll
                for (int i = 0; i < W; i += 4) {
                    mix_load<float, 4>(gG + (int64_t)r * B.dvp + c0 + q * W + i, *(float(*)[4]) & x[i]);
                    mix_load<float, 4>(gS + (int64_t)r * B.dvp + c0 + q * W + i, y);
#pragma unroll
                    for (int j = 0; j < 4; ++j) sgsum = fmaf(x[i + j], y[j], sgsum);
                }
                put_row<TR>(x, sh + r * kLs + q * W, sl + r * kLs + q * W, is + r, q);
            }
            __syncthreads();
            f32x4 iur;
#pragma unroll
            for (int r = 0; r < 4; ++r) iur[r] = iu[16 * w + 4 * g + r];
            const Split u0 = lds_frag(uh, ul, row, 0), u1 = lds_frag(uh, ul, row, 1);
#pragma unroll
            for (int nt = 0; nt < MT; ++nt) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
                a = mma_split(u0, lds_frag(sh, sl, 16 * nt + m, 0), a);
                a = mma_split(u1, lds_frag(sh, sl, 16 * nt + m, 1), a);
                gu[nt] += a * (iur * is[16 * nt + m]);
            }
        }
        // db: this lane's quarter of row `row`
        db += __shfl_xor(db, 16, 64);
        db += __shfl_xor(db, 32, 64);
        if (g == 0 && in) {
            const int64_t th = (ch.t0 + row) * A.Hv + h;
            if (A.beta_f32) ((float *)A.dbeta)[th] = db;
            else ((S *)A.dbeta)[th] = mix_out<S>(db);
        }
        __syncthreads();
        // D and F, the decays in place
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * g + r, j = 16 * nt + m;
                const float d = j <= i ? expf((float)(sg[i] - sg[j])) : 0.f;
                dm[i * kLd + j] = j <= i ? dp[nt][r] * d : 0.f;
                fm[i * kLd + j] = j < i ? dl[nt][r] * d : 0.f;
            }
        f32x4 up, down;
#pragma unroll
        for (int r = 0; r < 4; ++r) up[r] = rise[16 * w + 4 * g + r], down[r] = fall[16 * w + 4 * g + r];
        f32x4 dot = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            dq[nt] *= up;
            dk[nt] *= up;
            gu[nt] *= down;
#pragma unroll
            for (int r = 0; r < 4; ++r) dot[r] = fmaf(gu[nt][r], raw(A.k, A.ks, nk, nt, r), dot[r]);
        }
        // <S', G> = e^gam_C <S, G> + sum_j k_j . (its column part from the state)
        float end = last * sgsum + dot[0] + dot[1] + dot[2] + dot[3];
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) end += __shfl_xor(end, d, 64);
        if (lane == 0) red[w] = end;
        __syncthreads();
        // products inside the chunk: D and F by K, their transposes by Q and K
        Split fa[2], fb[2];
        float xa[2][8], xb[2][8];
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 32 * s + (j < 4 ? 4 * g + j : 16 + 4 * g + j - 4);
                xa[s][j] = dm[row * kLd + c] * rk[c];
                xb[s][j] = fm[row * kLd + c] * rk[c];
            }
        f32x4 ia = split_rows(xa, fa), ib = split_rows(xb, fb);
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const _Float16 *p = pkt + (nt * 2 + s) * kFrag;
                const f16x8 x = *(const f16x8 *)p;
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, x, mma(fb[s].lo, x, b));
                if (SPLIT) {
                    const f16x8 y = *(const f16x8 *)(p + HALF);
                    a = mma(fa[s].hi, y, a);
                    b = mma(fb[s].hi, y, b);
                }
            }
            dq[nt] += a * ia;
            dk[nt] += b * ib;
        }
        f32x4 dg = {0.f, 0.f, 0.f, 0.f}, dr = dg;
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            dqt[nt] += dq[nt];
            dkt[nt] += dk[nt];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dg[r] = fmaf(dq[nt][r] * A.scale, raw(A.q, A.qs, nq, nt, r), dg[r]);
                dr[r] = fmaf(dk[nt][r], raw(A.k, A.ks, nk, nt, r), dr[r]);
            }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int c = 32 * s + (j < 4 ? 4 * g + j : 16 + 4 * g + j - 4);
                xa[s][j] = dm[c * kLd + row] * rq[c];
                xb[s][j] = fm[c * kLd + row] * rk[c];
            }
        ia = split_rows(xa, fa);
        ib = split_rows(xb, fb);
        f32x4 dc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const _Float16 *p = pqt + (nt * 2 + s) * kFrag, *q = pkt + (nt * 2 + s) * kFrag;
                const f16x8 x = *(const f16x8 *)p, y = *(const f16x8 *)q;
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, y, mma(fb[s].lo, y, b));
                if (SPLIT) {
                    a = mma(fa[s].hi, *(const f16x8 *)(p + HALF), a);
                    b = mma(fb[s].hi, *(const f16x8 *)(q + HALF), b);
                }
            }
            gu[nt] += a * ia + b * ib;
            dkt[nt] += gu[nt];
#pragma unroll
            for (int r = 0; r < 4; ++r) dc[r] = fmaf(gu[nt][r], raw(A.k, A.ks, nk, nt, r), dc[r]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dg[r] += __shfl_xor(dg[r], d, 64);
                dr[r] += __shfl_xor(dr[r], d, 64);
                dc[r] += __shfl_xor(dc[r], d, 64);
            }
        dotq += dg;
        dotk += dr + dc;
        if (m == 0)
#pragma unroll
            for (int r = 0; r < 4; ++r) dgam[16 * w + 4 * g + r] = dg[r] + dr[r] - dc[r];
        __syncthreads();
        if (w == 0) {  // sums from each token to the chunk's end
            double x = dgam[lane];
            if (lane == 63) x += (double)red[0] + red[1] + red[2] + red[3];
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_down(x, d, 64);
                if (lane + d < 64) x += o;
            }
            if (lane < ch.len) A.dg[(ch.t0 + lane) * A.Hv + h] = (float)x;
        }
    }
    // back through the scale and the norms
#pragma unroll
    for (int nt = 0; nt < MT; ++nt)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * w + 4 * g + r, c = 16 * nt + m;
            if (t >= ch.len || c >= A.dk) continue;
            float x = dqt[nt][r] * A.scale, y = dkt[nt][r];
            if (A.qk_norm) {
                x = nq[t] * (x - raw(A.q, A.qs, nq, nt, r) * dotq[r]);
                y = nk[t] * (y - raw(A.k, A.ks, nk, nt, r) * dotk[r]);
            }
            const int64_t o = ((ch.t0 + t) * A.Hk + hk) * A.dk + c;
            ((S *)A.dq)[o] = mix_out<S>(x);
            ((S *)A.dk_out)[o] = mix_out<S>(y);
        }
}

template <typename S>
hipError_t grad_typed(const DeltaArgs &a, const DeltaBuf &b, hipStream_t st) {
    const dim3 grid(b.slots, a.Hk);
    if (b.dkp == 64) hipLaunchKernelGGL((delta_grad_kernel<S, 64>), grid, dim3(256), 0, st, a, b);
    else hipLaunchKernelGGL((delta_grad_kernel<S, 128>), grid, dim3(256), 0, st, a, b);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaBuf &b, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return grad_typed<float>(a, b, st);
    if (dtype == CONV_DTYPE_FP16) return grad_typed<_Float16>(a, b, st);
    return grad_typed<uint16_t>(a, b, st);
}

}  // namespace convlower
