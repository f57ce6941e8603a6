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
// heads that share it; each of its eight wavefronts takes 16 tokens and half
// of the key columns.
//
// S, G, Y and E come in result order, one column and four rows a lane.  They
// are put into LDS as [column][row], split in two, and read as operands by the
// transposing read, 64 columns at a time; the next 64 columns' loads are issued
// before the products of these.
//
// 8192 tokens, 8 and 16 heads of 128 x 128 (400 MB of S, G, Y and E: 82 us at a
// copy's rate): 206 us.  Bound by the way through LDS (write, barrier, read, for
// operands that serve one product each) with one block of eight wavefronts a
// CU; four wavefronts of all key columns each spill, 339 us.
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

// The sums of several value heads are kept in one place.  A head's own dot
// products, which its decays' gradients are made of, are taken of what it adds
// before that goes there: a difference of the sums would leave a small head
// after a large one without digits, and a head of NaN none to any.
template <typename S, int DKP>
__global__ __launch_bounds__(512) void delta_grad_kernel(DeltaArgs A, DeltaBuf B, bool vec, bool vec_out) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int KS = DKP / 32, MT = DKP / 16, MH = MT / 2, PL = SPLIT ? 2 : 1, MAT = kC * DKP * 2, IN = 2 * PL * MAT;
    constexpr int SLD = DKP + 8;
    constexpr int kState = 2 * kSlab * SLD * 2, kDF = 2 * kC * kLd * 4, kTok = 4 * kSlab * kTokLd * 2;
    // a slab of S or G, then D and F
    __shared__ __align__(16) char first[kState > kDF ? kState : kDF];
    // U and dZ of a slab
    __shared__ __align__(16) char second[kTok];
    __shared__ __align__(16) char kq[IN];  // K and Q, for the block's whole life
    _Float16 *sh = (_Float16 *)first, *sl = sh + kSlab * SLD;
    float *dm = (float *)first, *fm = dm + kC * kLd;
    _Float16 *uh = (_Float16 *)second, *ul = uh + kSlab * kTokLd, *eh = ul + kSlab * kTokLd, *el = eh + kSlab * kTokLd;
    __shared__ __align__(16) float sb[kC], rise[kC], fall[kC], rk[kC], nk[kC], uq[kC], rq[kC], nq[kC], dgam[2][kC];
    __shared__ __align__(16) float dbs[4][kC], red[8], mx[2][8];
    __shared__ __align__(16) float sums[2][2][kC];  // over the heads: q . dq and k . dk, a half of the columns each
    __shared__ double sg[kC];
    const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6 & 3), hf = __builtin_amdgcn_readfirstlane(tid >> 8);  // rows 16 w.., columns 16 MH hf..
    // Lane numbers, renewed in each part of the loops: or the compiler keeps some
    // hundred LDS addresses made of them in registers throughout, and spills.
    int g = lane >> 4, m = lane & 15, tl = trans_lane(), so = trans_off<SLD>(), to = trans_off<kTokLd>();
    auto renew = [&] { asm volatile("" : "+v"(g), "+v"(m), "+v"(tl), "+v"(so), "+v"(to)); };
    const DeltaChunk ch = chunk_of(A.s, slot);
    if (ch.len == 0) return;
    const int64_t head = (int64_t)slot * A.Hk + hk;
    if (tid < kC) {
        const float *o = B.rowk + head * 4 * kC + tid;
        rk[tid] = o[0], nk[tid] = o[kC], uq[tid] = o[2 * kC], nq[tid] = o[3 * kC];
        rq[tid] = uq[tid] * A.scale;
    }
    // this wavefront's columns: where they begin in K' (fragments), in K (this lane's element) and in a slab of S
    const int fo0 = hf * (MH / 2) * 1024;
    const _Float16 *shh = sh + 16 * MH * hf, *slh = sl + 16 * MH * hf;
    // K's or Q's values where results lie: rows 16 w + 4 g .., column 16 i + m of this wavefront's
    auto rows4 = [&](const char *x, int i) {
        const char *p = x + (w * KS + hf * (MH / 2) + i / 2) * 1024 + tl + (i & 1) * 8;
        auto read = [](const char *at) {
            const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)((lds_bytes)(lds_ptr_t)at));
            return __builtin_convertvector(__builtin_bit_cast(f16x4, v), f32x4);
        };
        f32x4 v = read(p);
        if (SPLIT) v += read(p + MAT);
        return v;
    };
    // a row's dot product, its factor and the sum over its columns
    auto whole = [&](f32x4 v, const float *rho) {
        v *= *(const f32x4 *)(rho + 16 * w + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = group_sum(v[r]);
        return v;
    };
    f32x4 dq[MH], dk[MH];
#pragma unroll
    for (int i = 0; i < MH; ++i) dq[i] = dk[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int rep = A.Hv / A.Hk, slabs = B.dvp / kSlab;
    // What a slab begins with, fetched while the one before it is worked with.
    // Buffer loads: the base in scalar registers, one offset for all of them.
    // (A spill read back in here would wait for these loads; there is none, with
    // the products inside the chunk kept to themselves below: mixed, float32
    // inputs spilled 40 registers and took 213 us for 168.)
    const int l16 = lane * 16;
    auto load4 = [&](__amdgpu_buffer_rsrc_t r, int at) {
        return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, l16, at, 0));
    };
    const int do_at = 16 * w + m < ch.len ? (16 * w + m) * (int)A.dos * (int)sizeof(S) + 8 * g * (int)sizeof(S) : (int)kOutOfRange;
    f32x4 s4[MH], y4[2], e4[2], smax4, gmax4;
    double gam_t = 0., gam_end = 0.;  // of a head's first slab: this thread's token and the last
    float b_t = 0.f, last = 0.f;
    typedef MixVec<S, 8> Do8;
    Do8 do8[2];
    auto fetch = [&](int v, int slab) {
        const int64_t vh = (int64_t)slot * A.Hv + hk * rep + v;
        const int tile = slab * (kSlab / 16) + w;  // this wavefront's columns of the slab: 16 w.., and half their rows
        const __amdgpu_buffer_rsrc_t ry = make_rsrc(B.Y + vh * kC * B.dvp, 0x7fffffff);
        const __amdgpu_buffer_rsrc_t re = make_rsrc(B.E + vh * kC * B.dvp, 0x7fffffff);
        const __amdgpu_buffer_rsrc_t rs = make_rsrc(B.S + vh * DKP * B.dvp, 0x7fffffff);
        if (slab == 0) {
            const float *fac = (const float *)(B.tpg + vh * kTpBytes + kTpRows);
            gam_t = B.gam[vh * kC + lane], gam_end = B.gam[vh * kC + kC - 1];
            b_t = fac[ROW_B * kC + lane], last = fac[ROW_SCALARS * kC + SC_LAST];
        }
        smax4 = *(const f32x4 *)(B.Smax + vh * (B.dvp / 16) + slab * 4);
        gmax4 = *(const f32x4 *)(B.Gmax + vh * (B.dvp / 16) + slab * 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) y4[i] = load4(ry, (tile * 4 + 2 * hf + i) * 1024);
#pragma unroll
        for (int i = 0; i < 2; ++i) e4[i] = load4(re, (tile * 4 + 2 * hf + i) * 1024);
#pragma unroll
        for (int i = 0; i < MH; ++i) s4[i] = load4(rs, (tile * MT + MH * hf + i) * 1024);
        const __amdgpu_buffer_rsrc_t rd = make_rsrc((const S *)A.d_o + ch.t0 * A.dos + (int64_t)(hk * rep + v) * A.dv, 0x7fffffff);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int c = slab * kSlab + 32 * s;  // and 8 g
            if (vec) {
                const int at = c + 8 * g < A.dv ? do_at : (int)kOutOfRange;
                if constexpr (sizeof(S) == 2) {
                    do8[s] = __builtin_bit_cast(Do8, __builtin_amdgcn_raw_buffer_load_b128(rd, at, c * 2, 0));
                } else {
                    ((uint4 *)&do8[s])[0] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rd, at, c * 4, 0));
                    ((uint4 *)&do8[s])[1] = __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(rd, at, c * 4 + 16, 0));
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int at = c + 8 * g + j < A.dv ? do_at : (int)kOutOfRange;
                    if constexpr (sizeof(S) == 2)
                        do8[s].v[j] = __builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b16(rd, at, (c + j) * 2, 0));
                    else do8[s].v[j] = __builtin_bit_cast(S, __builtin_amdgcn_raw_buffer_load_b32(rd, at, (c + j) * 4, 0));
                }
            }
        }
    };
    copy_in<8, IN / 1024>((const char *)B.kq + head * IN, kq);
    fetch(0, 0);
    if (tid < 4 * kC) (&sums[0][0][0])[tid] = 0.f;
    for (int v = 0; v < rep; ++v) {
        const int h = hk * rep + v;
        const int64_t vh = (int64_t)slot * A.Hv + h;
        const __amdgpu_buffer_rsrc_t rg = make_rsrc(B.G + vh * DKP * B.dvp, 0x7fffffff);
        __syncthreads();
        if (tid < kC) {
            sg[tid] = gam_t;
            rise[tid] = expf((float)gam_t);
            fall[tid] = expf((float)(gam_end - gam_t));
            sb[tid] = b_t;
        }
        if (hf == 0) dbs[w][lane] = 0.f;
        const float last_v = last;
        f32x4 dp[2], dl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) dp[i] = dl[i] = f32x4{0.f, 0.f, 0.f, 0.f};
        // of this head: q . dq, k . dkr and k . dkc, this lane's columns and without the rows' factors
        f32x4 pq = {0.f, 0.f, 0.f, 0.f}, pr = pq, pc = pq;
        float sgsum = 0.f;
        __syncthreads();
        const f32x4 up = *(const f32x4 *)(rise + 16 * w + 4 * g), down = *(const f32x4 *)(fall + 16 * w + 4 * g);
        for (int slab = 0; slab < slabs; ++slab) {
            renew();
            const int c0 = slab * kSlab;
            f32x4 g4[MH];
#pragma unroll
            for (int i = 0; i < MH; ++i) g4[i] = load4(rg, ((c0 / 16 + w) * MT + MH * hf + i) * 1024);
            float xo[2][8];
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int j = 0; j < 8; ++j) xo[s][j] = mix_f32(do8[s].v[j]);
            float is, ig, iu, ie;
            const float ss = pow2_to(max4(smax4, 0.f), kTop, &is), sgs = pow2_to(max4(gmax4, 0.f), kTop, &ig);
            float um = 0.f, em = 0.f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = 16 * (2 * hf + i) + 4 * g;
                const f32x4 b = *(const f32x4 *)(sb + t);
                f32x4 p = y4[i] * e4[i];  // b's gradient
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = group_sum(p[r]);
                if (m == 0) *(f32x4 *)&dbs[w][t] += p;
                y4[i] *= b;    // U
                e4[i] *= -b;   // -dZ
                um = max4(y4[i], um);
                em = max4(e4[i], em);
            }
            um = tile_max(um), em = tile_max(em);
            if (lane == 0) mx[0][tid >> 6] = um, mx[1][tid >> 6] = em;
            __syncthreads();  // mx; and the slab before is done with
            const float us = pow2_to(max4(*(const f32x4 *)mx[0], max4(*(const f32x4 *)(mx[0] + 4), 0.f)), kTop, &iu);
            const float es = pow2_to(max4(*(const f32x4 *)mx[1], max4(*(const f32x4 *)(mx[1] + 4), 0.f)), kTop, &ie);
            const int col = 16 * w + m;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int o = col * kTokLd + 16 * (2 * hf + i) + 4 * g;
                put4(y4[i], us, uh + o, ul + o);
                put4(e4[i], es, eh + o, el + o);
            }
#pragma unroll
            for (int i = 0; i < MH; ++i) {
                const int o = col * SLD + 16 * (MH * hf + i) + 4 * g;
                put4(s4[i], ss, sh + o, sl + o);
            }
            Split fo[2];
            f32x4 io = split_rows(xo, fo);
            if (v == 0 && slab == 0) CONVLOWER_WAIT_VMCNT(0);  // K and Q are in LDS (all but G's slab was waited for above)
            if (slab + 1 < slabs) fetch(v, slab + 1);
            else if (v + 1 < rep) fetch(v + 1, 0);
            __syncthreads();
            Split fe[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) fe[s] = slab_split<kTokLd>(eh, el, w, s, to);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int nt = 2 * hf + i;
                if (nt > w) continue;
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = slab_split<kTokLd>(uh, ul, nt, s, to);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                dp[i] += a * (io * iu);
                dl[i] += b * (ie * iu);
            }
            io *= up * is;
            const f32x4 je = up * (ie * is);
#pragma unroll
            for (int i = 0; i < MH; ++i) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    const Split x = slab_split<SLD>(shh, slh, i, s, so);
                    a = SPLIT ? mma_split(fo[s], x, a) : mma2(fo[s].hi, x, a);
                    b = mma_split(fe[s], x, b);
                }
                a *= io, b *= je;
                dq[i] += a, dk[i] += b;
                pq += rows4(kq + IN / 2, i) * a;
                pr += rows4(kq, i) * b;
            }
            __syncthreads();
            float part = 0.f;
#pragma unroll
            for (int i = 0; i < MH; ++i) {  // in the place of this lane's S
                const int o = col * SLD + 16 * (MH * hf + i) + 4 * g;
                _Float16 *h = sh + o, *l = sl + o;
                const f16x4 a = *(const f16x4 *)h, b = *(const f16x4 *)l;
#pragma unroll
                for (int r = 0; r < 4; ++r) part = fmaf(g4[i][r], (float)a[r] + (float)b[r], part);
                put4(g4[i], sgs, h, l);
            }
            sgsum = fmaf(part, is, sgsum);
            __syncthreads();
            Split fu[2];
#pragma unroll
            for (int s = 0; s < 2; ++s) fu[s] = slab_split<kTokLd>(uh, ul, w, s, to);
            const f32x4 ju = down * (iu * ig);
#pragma unroll
            for (int i = 0; i < MH; ++i) {
                f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < 2; ++s) a = mma_split(fu[s], slab_split<SLD>(shh, slh, i, s, so), a);
                a *= ju;
                dk[i] += a;
                pc += rows4(kq, i) * a;
            }
        }
        __syncthreads();
        renew();
        const int row = 16 * w + m;  // this lane's row of left operands
        if (tid < ch.len) {
            const float db = (dbs[0][tid] + dbs[1][tid]) + (dbs[2][tid] + dbs[3][tid]);
            const int64_t th = (ch.t0 + tid) * A.Hv + h;
            if (A.beta_f32) ((float *)A.dbeta)[th] = db;
            else ((S *)A.dbeta)[th] = mix_out<S>(db);
        }
        // D and F, the decays in place
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * g + r, j = 16 * (2 * hf + t) + m;
                const float d = j <= i ? expf((float)(sg[i] - sg[j])) : 0.f;
                dm[i * kLd + j] = j <= i ? dp[t][r] * d : 0.f;
                fm[i * kLd + j] = j < i ? dl[t][r] * d : 0.f;
            }
        __syncthreads();
        // <S', G> = e^gam_C <S, G> + sum_j k_j . (its column part from the state)
        {
            const f32x4 x = pc * *(const f32x4 *)(rk + 16 * w + 4 * g);
            float end = last_v * sgsum + ((x[0] + x[1]) + (x[2] + x[3]));
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) end += __shfl_xor(end, d, 64);
            if (lane == 0) red[tid >> 6] = end;
        }
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
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MH; ++i) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const char *p = kq + fo0 + (2 * s * KS + i / 2) * 1024;
                const f16x8 x = trans_at(p, p + KS * 1024, i, tl);
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, x, mma(fb[s].lo, x, b));
                if constexpr (SPLIT) {
                    const f16x8 y = trans_at(p + MAT, p + MAT + KS * 1024, i, tl);
                    a = mma(fa[s].hi, y, a);
                    b = mma(fb[s].hi, y, b);
                }
            }
            a *= ia, b *= ib;
            dq[i] += a, dk[i] += b;
            pq += rows4(kq + IN / 2, i) * a;
            pr += rows4(kq, i) * b;
        }
        __builtin_amdgcn_sched_barrier(0);
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
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < MH; ++i) {
            f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const char *p = kq + fo0 + (2 * s * KS + i / 2) * 1024, *q = p + IN / 2;
                const f16x8 x = trans_at(q, q + KS * 1024, i, tl), y = trans_at(p, p + KS * 1024, i, tl);
                a = mma(fa[s].hi, x, mma(fa[s].lo, x, a));
                b = mma(fb[s].hi, y, mma(fb[s].lo, y, b));
                if constexpr (SPLIT) {
                    a = mma(fa[s].hi, trans_at(q + MAT, q + MAT + KS * 1024, i, tl), a);
                    b = mma(fb[s].hi, trans_at(p + MAT, p + MAT + KS * 1024, i, tl), b);
                }
            }
            a = a * ia + b * ib;
            dk[i] += a;
            pc += rows4(kq, i) * a;
        }
        renew();
        pq = whole(pq, rq), pr = whole(pr, rk), pc = whole(pc, rk);
        if (m == 0) {
            const int at = 16 * w + 4 * g;
            *(f32x4 *)(dgam[hf] + at) = pq + pr - pc;
            *(f32x4 *)(sums[0][hf] + at) += pq;
            *(f32x4 *)(sums[1][hf] + at) += pr + pc;
        }
        __syncthreads();
        if (tid < 64) {  // sums from each token to the chunk's end
            double x = (double)dgam[0][lane] + dgam[1][lane];
            if (lane == 63)
                for (int i = 0; i < 8; ++i) x += red[i];
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_down(x, d, 64);
                if (lane + d < 64) x += o;
            }
            if (lane < ch.len) A.dg[(ch.t0 + lane) * A.Hv + h] = (float)x;
        }
    }
    // Back through the norms: a unit row is K's or Q's with its factor.  The
    // rows leave by way of LDS, 16 bytes a lane.
    constexpr int OLD = DKP + 16 / sizeof(S);
    S *rows = (S *)first;
    auto leave = [&](const char *x, const float *rho, const float *norm, const f32x4 (&v)[MH], f32x4 dots, float scale, S *out) {
        const f32x4 rh = *(const f32x4 *)(rho + 16 * w + 4 * g), nv = *(const f32x4 *)(norm + 16 * w + 4 * g);
#pragma unroll
        for (int i = 0; i < MH; ++i) {
            const char *p = x + (w * KS + hf * (MH / 2)) * 1024 + (4 * g + 16 * (m >> 2)) * 16 + (m & 3) * 2 + (i / 2) * 1024 + (i & 1) * 8;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float o = v[i][r] * scale;
                if (A.qk_norm) {
                    float u = (float)*(const _Float16 *)(p + r * 16);
                    if (SPLIT) u += (float)*(const _Float16 *)(p + MAT + r * 16);
                    o = nv[r] * (o - u * rh[r] * dots[r]);
                }
                rows[(16 * w + 4 * g + r) * OLD + 16 * (MH * hf + i) + m] = mix_out<S>(o);
            }
        }
        __syncthreads();
        S *to = out + (ch.t0 * A.Hk + hk) * A.dk;
        constexpr int V = 16 / sizeof(S);
        if (vec_out) {
            for (int i = tid; i < kC * DKP / V; i += 512) {
                const int t = i / (DKP / V), c = i % (DKP / V) * V;
                if (t < ch.len && c < A.dk)
                    *(MixVec<S, V> *)(to + (int64_t)t * A.Hk * A.dk + c) = *(const MixVec<S, V> *)(rows + t * OLD + c);
            }
        } else {
            for (int i = tid; i < kC * DKP; i += 512) {
                const int t = i / DKP, c = i % DKP;
                if (t < ch.len && c < A.dk) to[(int64_t)t * A.Hk * A.dk + c] = rows[t * OLD + c];
            }
        }
        __syncthreads();
    };
    const int at = 16 * w + 4 * g;
    const f32x4 sq = *(const f32x4 *)(sums[0][0] + at) + *(const f32x4 *)(sums[0][1] + at);
    const f32x4 sk = *(const f32x4 *)(sums[1][0] + at) + *(const f32x4 *)(sums[1][1] + at);
    leave(kq + IN / 2, uq, nq, dq, sq, A.scale, (S *)A.dq);
    leave(kq, rk, nk, dk, sk, 1.f, (S *)A.dk_out);
}

template <typename S, int DKP>
hipError_t grad_run(const DeltaArgs &a, const DeltaBuf &b, hipStream_t st) {
    const dim3 grid(b.slots, a.Hk);
    const bool vec = a.dv % 8 == 0 && a.dos % 8 == 0 && (uintptr_t)a.d_o % (8 * sizeof(S)) == 0;
    const bool vec_out = a.dk * sizeof(S) % 16 == 0 && (uintptr_t)a.dq % 16 == 0 && (uintptr_t)a.dk_out % 16 == 0;
    hipLaunchKernelGGL((delta_grad_kernel<S, DKP>), grid, dim3(512), 0, st, a, b, vec, vec_out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_grad(const DeltaArgs &a, const DeltaBuf &b, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? grad_run<float, 64>(a, b, st) : grad_run<float, 128>(a, b, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? grad_run<_Float16, 64>(a, b, st) : grad_run<_Float16, 128>(a, b, st);
    return b.dkp == 64 ? grad_run<uint16_t, 64>(a, b, st) : grad_run<uint16_t, 128>(a, b, st);
}

}  // namespace convlower
