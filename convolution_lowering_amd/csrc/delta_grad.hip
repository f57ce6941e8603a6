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
//
// S, G, Y and E come in result order, one column and four rows a lane.  They
// are put into LDS as [column][row], split in two, and read as operands by the
// transposing read, 64 columns at a time.
#include "delta_chunk.h"

namespace convlower {
namespace {

constexpr int kLd = 68;          // floats from row to row of D and F
constexpr int kTokLd = kC + 8;   // f16 values from column to column of U and dZ

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
__device__ __forceinline__ f32x4 mma_split(const Split &a, const Split &b, f32x4 c) { return mma3(a.hi, a.lo, b, c); }

// Four rows of one column into LDS, hi and lo.
__device__ __forceinline__ void put4(f32x4 v, float sc, _Float16 *hi, _Float16 *lo) {
    f16x4 h, l;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        h[r] = (_Float16)fmaf(v[r], sc, 0.f);
        l[r] = (_Float16)fmaf(v[r], sc, -(float)h[r]);
    }
    *(f16x4 *)hi = h;
    *(f16x4 *)lo = l;
}
// An operand of rows 16 rt.. and the 32 columns 32 s.. of the slab, from
// [column][row]: place (g, j) holds column 32 s + 8 g + j.  `o` is trans_off.
template <int LD>
__device__ __forceinline__ int trans_off() {
    const int lane = threadIdx.x & 63, g = lane >> 4, t = lane & 15;
    return ((8 * g + (t >> 2)) * LD + 4 * (t & 3)) * 2;
}
template <int LD>
__device__ __forceinline__ f16x8 slab_at(const _Float16 *x, int rt, int s, int o) {
    const char *p = (const char *)x + o + (32 * s * LD + 16 * rt) * 2;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)p));
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)(p + 4 * LD * 2)));
    return __builtin_bit_cast(f16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}
template <int LD>
__device__ __forceinline__ Split slab_split(const _Float16 *hi, const _Float16 *lo, int rt, int s, int o) {
    Split r;
    r.hi = slab_at<LD>(hi, rt, s, o);
    r.lo = slab_at<LD>(lo, rt, s, o);
    return r;
}

template <typename S, int DKP, bool GROUP>
__global__ __launch_bounds__(256, 1) void delta_grad_kernel(DeltaArgs A, DeltaBuf B, bool vec) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int KS = DKP / 32, MT = DKP / 16, PL = SPLIT ? 2 : 1, MAT = kC * DKP * 2, IN = 2 * PL * MAT;
    constexpr int SLD = DKP + 8;
    constexpr int kState = 2 * kSlab * SLD * 2, kDF = 2 * kC * kLd * 4, kTok = 4 * kSlab * kTokLd * 2;
    // a slab of S or G, then D and F
    __shared__ __align__(16) char first[kState > kDF ? kState : kDF];
    // U and dZ of a slab, then K and Q
    __shared__ __align__(16) char second[kTok > IN ? kTok : IN];
    _Float16 *sh = (_Float16 *)first, *sl = sh + kSlab * SLD;
    float *dm = (float *)first, *fm = dm + kC * kLd;
    _Float16 *uh = (_Float16 *)second, *ul = uh + kSlab * kTokLd, *eh = ul + kSlab * kTokLd, *el = eh + kSlab * kTokLd;
    const char *kq = second;
    __shared__ __align__(16) float sb[kC], rise[kC], fall[kC], rk[kC], nk[kC], rq[kC], nq[kC], dgam[kC];
    __shared__ __align__(16) float dbs[4][kC], red[4], mx[2][4];
    __shared__ double sg[kC];
    const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int g = lane >> 4, m = lane & 15, tl = trans_lane(), so = trans_off<SLD>(), to = trans_off<kTokLd>();
    const DeltaChunk ch = chunk_of(A.s, slot);
    if (ch.len == 0) return;
    const int64_t head = (int64_t)slot * A.Hk + hk;
    if (tid < kC) {
        const float *o = B.rowk + head * 4 * kC + tid;
        rk[tid] = o[0], nk[tid] = o[kC], rq[tid] = o[2 * kC], nq[tid] = o[3 * kC];
    }
    const int row = 16 * w + m;  // this lane's row of left operands
    const bool in = row < ch.len;
    // k or q with its norm (q with the scale too), four rows of column 16 nt + m as results lie
    auto unit = [&](const char *x, const float *rho, int nt) {
        const char *p = x + (w * KS + nt / 2) * 1024 + (4 * g + 16 * (m >> 2)) * 16 + ((nt & 1) * 4 + (m & 3)) * 2;
        f32x4 v;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            v[r] = (float)*(const _Float16 *)(p + r * 16);
            if (SPLIT) v[r] += (float)*(const _Float16 *)(p + MAT + r * 16);
        }
        return v * *(const f32x4 *)(rho + 16 * w + 4 * g);
    };
    f32x4 dqt[GROUP ? MT : 1], dkt[GROUP ? MT : 1], dotq = {0.f, 0.f, 0.f, 0.f}, dotk = dotq;
    f32x4 dq[MT], dk[MT], gu[MT];
    if constexpr (GROUP)
#pragma unroll
        for (int i = 0; i < MT; ++i) dqt[i] = dkt[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int rep = GROUP ? A.Hv / A.Hk : 1;
    for (int v = 0; v < rep; ++v) {
        const int h = hk * rep + v;
        const int64_t vh = (int64_t)slot * A.Hv + h;
        const float *gS = B.S + vh * DKP * B.dvp + lane * 4, *gG = B.G + vh * DKP * B.dvp + lane * 4;
        const float *gY = B.Y + vh * kC * B.dvp + lane * 4, *gE = B.E + vh * kC * B.dvp + lane * 4;
        const float *fac = (const float *)(B.tpg + vh * kTpBytes + kTpRows);
        __syncthreads();
        if (tid < kC) {
            const double x = B.gam[vh * kC + tid], all = B.gam[vh * kC + kC - 1];
            sg[tid] = x;
            rise[tid] = expf((float)x);
            fall[tid] = expf((float)(all - x));
            sb[tid] = fac[ROW_B * kC + tid];
        }
        const float last = fac[ROW_SCALARS * kC + SC_LAST];
        f32x4 dp[4], dl[4], dbp[4];
#pragma unroll
        for (int i = 0; i < MT; ++i) dq[i] = dk[i] = gu[i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) dp[i] = dl[i] = dbp[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        float sgsum = 0.f;
        __syncthreads();
        for (int c0 = 0; c0 < B.dvp; c0 += kSlab) {
            const int tile = c0 / 16 + w;  // this wavefront's columns of the slab: 16 w..
            f32x4 s4[MT], y4[4], e4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) y4[i] = *(const f32x4 *)(gY + (tile * 4 + i) * 256);
#pragma unroll
            for (int i = 0; i < 4; ++i) e4[i] = *(const f32x4 *)(gE + (tile * 4 + i) * 256);
#pragma unroll
            for (int i = 0; i < MT; ++i) s4[i] = *(const f32x4 *)(gS + (tile * MT + i) * 256);
            float xo[2][8];
            const S *po = (const S *)A.d_o + (ch.t0 + (in ? row : 0)) * A.dos + (int64_t)h * A.dv + c0 + 8 * g;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                if (vec) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) xo[s][j] = 0.f;
                    if (c0 + 32 * s + 8 * g < A.dv) mix_load<S, 8>(po + 32 * s, xo[s]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) xo[s][j] = c0 + 32 * s + 8 * g + j < A.dv ? mix_f32(po[32 * s + j]) : 0.f;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) xo[s][j] = in ? xo[s][j] : 0.f;
            }
            float smax = 0.f, gmax = 0.f, is, ig, iu, ie;
#pragma unroll
            for (int i = 0; i < kSlab / 16; ++i) {
                smax = fmaxf(smax, B.Smax[vh * (B.dvp / 16) + c0 / 16 + i]);
                gmax = fmaxf(gmax, B.Gmax[vh * (B.dvp / 16) + c0 / 16 + i]);
            }
            const float ss = pow2_to(smax, kTop, &is), sgs = pow2_to(gmax, kTop, &ig);
            float um = 0.f, em = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const f32x4 b = *(const f32x4 *)(sb + 16 * i + 4 * g);
                dbp[i] += y4[i] * e4[i];
                y4[i] *= b;    // U
                e4[i] *= -b;   // -dZ
                um = max4(y4[i], um);
                em = max4(e4[i], em);
            }
            um = tile_max(um), em = tile_max(em);
            if (lane == 0) mx[0][w] = um, mx[1][w] = em;
            __syncthreads();  // mx; and the slab before is done with
            const float us = pow2_to(fmaxf(fmaxf(mx[0][0], mx[0][1]), fmaxf(mx[0][2], mx[0][3])), kTop, &iu);
            const float es = pow2_to(fmaxf(fmaxf(mx[1][0], mx[1][1]), fmaxf(mx[1][2], mx[1][3])), kTop, &ie);
            const int col = 16 * w + m;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = col * kTokLd + 16 * i + 4 * g;
                put4(y4[i], us, uh + o, ul + o);
                put4(e4[i], es, eh + o, el + o);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) put4(s4[i], ss, sh + col * SLD + 16 * i + 4 * g, sl + col * SLD + 16 * i + 4 * g);
            // G of the same place, on its way while S is worked with
            f32x4 g4[MT];
#pragma unroll
            for (int i = 0; i < MT; ++i) g4[i] = *(const f32x4 *)(gG + (tile * MT + i) * 256);
            Split fo[2];
            const f32x4 io = split_rows(xo, fo);
            __syncthreads();
            Split fe[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) fe[s] = slab_split<kTokLd>(eh, el, w, s, to);
#pragma unroll
            for (int nt = 0; nt < MT; ++nt) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = slab_split<SLD>(sh, sl, nt, s, so);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                dq[nt] += a * (io * is);
                dk[nt] += b * (ie * is);
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                if (nt > w) continue;
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = slab_split<kTokLd>(uh, ul, nt, s, to);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                dp[nt] += a * (io * iu);
                dl[nt] += b * (ie * iu);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sgsum = fmaf(s4[i][r], g4[i][r], sgsum);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < MT; ++i) put4(g4[i], sgs, sh + col * SLD + 16 * i + 4 * g, sl + col * SLD + 16 * i + 4 * g);
            __syncthreads();
            Split fu[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) fu[s] = slab_split<kTokLd>(uh, ul, w, s, to);
#pragma unroll
            for (int nt = 0; nt < MT; ++nt) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 2; ++s) a = mma_split(fu[s], slab_split<SLD>(sh, sl, nt, s, so), a);
                gu[nt] += a * (iu * ig);
            }
        }
        // db over the columns: 16 lanes, then the wavefronts
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1)
#pragma unroll
                for (int r = 0; r < 4; ++r) dbp[i][r] += __shfl_xor(dbp[i][r], d, 64);
        if (m == 0)
#pragma unroll
            for (int i = 0; i < 4; ++i) *(f32x4 *)&dbs[w][16 * i + 4 * g] = dbp[i];
        __syncthreads();
        copy_in<4, IN / 1024>((const char *)B.kq + head * IN, second);
        if (tid < ch.len) {
            const float db = (dbs[0][tid] + dbs[1][tid]) + (dbs[2][tid] + dbs[3][tid]);
            const int64_t th = (ch.t0 + tid) * A.Hv + h;
            if (A.beta_f32) ((float *)A.dbeta)[th] = db;
            else ((S *)A.dbeta)[th] = mix_out<S>(db);
        }
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
        CONVLOWER_WAIT_VMCNT_LDS(0);  // the copies
        __syncthreads();
        const f32x4 up = *(const f32x4 *)(rise + 16 * w + 4 * g), down = *(const f32x4 *)(fall + 16 * w + 4 * g);
        f32x4 dot = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            dq[nt] *= up;
            dk[nt] *= up;
            gu[nt] *= down;
            dot += gu[nt] * unit(kq, rk, nt);
        }
        // <S', G> = e^gam_C <S, G> + sum_j k_j . (its column part from the state)
        float end = last * sgsum + dot[0] + dot[1] + dot[2] + dot[3];
#pragma unroll
        for (int d = 32; d > 0; d >>= 1) end += __shfl_xor(end, d, 64);
        if (lane == 0) red[w] = end;
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
        f32x4 dg = {0.f, 0.f, 0.f, 0.f}, dr = dg, dc = dg;
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const char *p = kq + (2 * s * KS + nt / 2) * 1024;
                const f16x8 x = trans_at(p, p + KS * 1024, nt, tl);
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, x, mma(fb[s].lo, x, b));
                if constexpr (SPLIT) {
                    const f16x8 y = trans_at(p + MAT, p + MAT + KS * 1024, nt, tl);
                    a = mma(fa[s].hi, y, a);
                    b = mma(fb[s].hi, y, b);
                }
            }
            dq[nt] += a * ia;
            dk[nt] += b * ib;
            dg += dq[nt] * unit(kq + IN / 2, rq, nt);
            dr += dk[nt] * unit(kq, rk, nt);
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
#pragma unroll
        for (int nt = 0; nt < MT; ++nt) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const char *p = kq + (2 * s * KS + nt / 2) * 1024, *q = p + IN / 2;
                const f16x8 x = trans_at(q, q + KS * 1024, nt, tl), y = trans_at(p, p + KS * 1024, nt, tl);
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, y, mma(fb[s].lo, y, b));
                if constexpr (SPLIT) {
                    a = mma(fa[s].hi, trans_at(q + MAT, q + MAT + KS * 1024, nt, tl), a);
                    b = mma(fb[s].hi, trans_at(p + MAT, p + MAT + KS * 1024, nt, tl), b);
                }
            }
            gu[nt] += a * ia + b * ib;
            dc += gu[nt] * unit(kq, rk, nt);
            dk[nt] += gu[nt];
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
        if constexpr (GROUP)
#pragma unroll
            for (int nt = 0; nt < MT; ++nt) dqt[nt] += dq[nt], dkt[nt] += dk[nt];
        if (m == 0) *(f32x4 *)(dgam + 16 * w + 4 * g) = dg + dr - dc;
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
    // back through the scale and the norms: x / |x| of a unit row is the row's value over the scale
    const f32x4 vq = *(const f32x4 *)(nq + 16 * w + 4 * g), vk = *(const f32x4 *)(nk + 16 * w + 4 * g);
#pragma unroll
    for (int nt = 0; nt < MT; ++nt) {
        f32x4 x = (GROUP ? dqt[GROUP ? nt : 0] : dq[nt]), y = (GROUP ? dkt[GROUP ? nt : 0] : dk[nt]);
        x *= A.scale;
        const int c = 16 * nt + m;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int t = 16 * w + 4 * g + r;
            if (t >= ch.len || c >= A.dk) continue;
            float a = x[r], b = y[r];
            if (A.qk_norm) {
                const int64_t qo = (ch.t0 + t) * A.qs + (int64_t)hk * A.dk + c, ko = (ch.t0 + t) * A.ks + (int64_t)hk * A.dk + c;
                a = vq[r] * (a - mix_f32(((const S *)A.q)[qo]) * vq[r] * dotq[r]);
                b = vk[r] * (b - mix_f32(((const S *)A.k)[ko]) * vk[r] * dotk[r]);
            }
            const int64_t o = ((ch.t0 + t) * A.Hk + hk) * A.dk + c;
            ((S *)A.dq)[o] = mix_out<S>(a);
            ((S *)A.dk_out)[o] = mix_out<S>(b);
        }
    }
}

template <typename S, int DKP>
hipError_t grad_run(const DeltaArgs &a, const DeltaBuf &b, hipStream_t st) {
    const dim3 grid(b.slots, a.Hk);
    const bool vec = a.dv % 8 == 0 && a.dos % 8 == 0 && (uintptr_t)a.d_o % (8 * sizeof(S)) == 0;
    if (a.Hv > a.Hk) hipLaunchKernelGGL((delta_grad_kernel<S, DKP, true>), grid, dim3(256), 0, st, a, b, vec);
    else hipLaunchKernelGGL((delta_grad_kernel<S, DKP, false>), grid, dim3(256), 0, st, a, b, vec);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaBuf &b, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? grad_run<float, 64>(a, b, st) : grad_run<float, 128>(a, b, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? grad_run<_Float16, 64>(a, b, st) : grad_run<_Float16, 128>(a, b, st);
    return b.dkp == 64 ? grad_run<uint16_t, 64>(a, b, st) : grad_run<uint16_t, 128>(a, b, st);
}

}  // namespace convlower
