// First step of the chunked gated delta rule: everything of a chunk that does
// not need the state.  A block takes one chunk of one query/key head: it puts
// q and k in the order of the matrix cores' left operands, multiplies K K' and
// Q K' once, and for each value head of the group forms the decays, P and the
// inverse of the chunk's unit lower triangular matrix: (1 + L diag(b))^-1 for
// the way forward and, where gradients are wanted, (1 + diag(b) L)^-1 too.
//
// The inverse is built from 16 x 16 diagonal blocks (substitution, a lane a
// column) and joined twice, [A 0; B C]^-1 = [A' 0; -C' B A', C'], on the
// float32 matrix cores.
// Sums of g are held in float64, and as two floats where differences of them
// are taken: gam_i - gam_j loses too many digits in 32 bits where a chunk holds
// strong decays beside weak ones.
//
// 16384 tokens, 16 and 32 heads of 128 (134 MB of q and k, 352 MB of operands
// written, 99 us at a copy's rate): 143 us; 8192 tokens, 8 and 16 heads with
// what the gradients need 57 us.  Bound by the barriers between a head's steps
// (six, three blocks to a CU); the inverse by substitution alone, a lane a
// column of the whole matrix, 246 us.
#include "delta_chunk.h"

namespace convlower {
namespace {

constexpr int kLd = 68;  // floats from row to row of the 64 x 64 matrices in LDS

// A quarter of row `row` a thread, as it lies.
template <typename S, int DKP>
__device__ __forceinline__ void fetch_rows(const S *src, int64_t stride, const DeltaChunk &ch, int dk, bool vec,
                                           S (&f)[DKP / 4]) {
    constexpr int Q = DKP / 4, V = 16 / sizeof(S);
    const int row = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * Q;
#pragma unroll
    for (int i = 0; i < Q; ++i) f[i] = S(0);
    if (row >= ch.len) return;
    const S *p = src + (ch.t0 + row) * stride + c0;
    if (vec) {
#pragma unroll
        for (int i = 0; i < Q; i += V)
            if (c0 + i < dk) *(MixVec<S, V> *)&f[i] = *(const MixVec<S, V> *)(p + i);
    } else {
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (c0 + i < dk) f[i] = p[i];
    }
}
// Its largest value and sum of squares; the row goes to LDS as f16.
template <typename S, int DKP, bool SPLIT>
__device__ __forceinline__ void put_rows(const S (&f)[DKP / 4], int norm, _Float16 *dst, float *rho, float *rnorm) {
    constexpr int Q = DKP / 4, LD = DKP + 8;
    const int row = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * Q;
    float m = 0.f, ss = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        m = max2(m, fabsf(mix_f32(f[i])));
        ss = fmaf(mix_f32(f[i]), mix_f32(f[i]), ss);
    }
    m = max2(m, __shfl_xor(m, 1, 64));
    m = max2(m, __shfl_xor(m, 2, 64));
    ss += __shfl_xor(ss, 1, 64);
    ss += __shfl_xor(ss, 2, 64);
    float inv;
    const float sc = pow2_to(m, kRowTop, &inv);
#pragma unroll
    for (int i = 0; i < Q; i += 8) {
        f16x8 h, l;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = mix_f32(f[i + j]) * sc;
            h[j] = (_Float16)x;
            l[j] = (_Float16)(x - (float)h[j]);
        }
        *(f16x8 *)(dst + row * LD + c0 + i) = h;
        if (SPLIT) *(f16x8 *)(dst + kC * LD + row * LD + c0 + i) = l;
    }
    if ((threadIdx.x & 3) == 0) {
        const float r = norm ? 1.f / sqrtf(ss + kDeltaEps) : 1.f;
        rnorm[row] = r;
        rho[row] = inv * r;
    }
}

// The left operand of rows 16 mt.., columns 32 s.. from LDS rows.
template <int LD>
__device__ __forceinline__ f16x8 row_frag(const _Float16 *x, int mt, int s) {
    const int lane = threadIdx.x & 63;
    const _Float16 *p = x + (16 * mt + (lane & 15)) * LD + 32 * s + 4 * (lane >> 4);
    const f16x4 a = *(const f16x4 *)p, b = *(const f16x4 *)(p + 16);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}
__device__ __forceinline__ f32x4 mma32(float a, float b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// Both inverses of a chunk, from the strictly lower L ([64][kLd] in LDS) and
// b: X[0] = (1 + L diag(b))^-1 and, WAYS = 2, X[1] = (1 + diag(b) L)^-1.
// 256 threads, two barriers inside, none after.  m[way]: the largest value
// this thread wrote.
//
// A float32 product's left operand has row m, step s column 4 s + g in lane
// (g, m).  The second product of a join takes the columns in the order
// 4 g + r instead: then the first one's result is its right operand as it is.
template <int WAYS>
__device__ __forceinline__ void invert(const float *L, const float *b, float *X, float (&mx)[2]) {
    const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, g = lane >> 4, m = lane & 15;
    constexpr int kX = kC * kLd;
    mx[0] = mx[1] = 0.f;
    if (g < WAYS) {  // column m of diagonal block w
        const float *l = L + 16 * w * (kLd + 1);
        float v[16], big = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < i; j += 4) {
                const f32x4 r = *(const f32x4 *)(l + i * kLd + j);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (j + k < i) s = fmaf(r[k], v[j + k], s);
            }
            const float bi = b[16 * w + i];
            const float x = (i == m ? 1.f : 0.f) - (g ? bi * s : s);
            v[i] = g ? x : bi * x;
            X[g * kX + (16 * w + i) * kLd + 16 * w + m] = x;
            big = max2(big, fabsf(x));
        }
        mx[0] = g ? 0.f : big, mx[1] = g ? big : 0.f;
    }
    __syncthreads();
    if ((w >> 1) < WAYS) {  // rows 16.., columns 0.. of each half: a pair and a way a wavefront
        const int o = 32 * (w & 1), way = w >> 1;
        float *x = X + way * kX;
        f32x4 t = {0.f, 0.f, 0.f, 0.f}, c = t;
#pragma unroll
        for (int s = 0; s < 4; ++s)
            t = mma32(L[(o + 16 + m) * kLd + o + 4 * s + g] * b[way ? o + 16 + m : o + 4 * s + g], x[(o + 4 * s + g) * kLd + o + m], t);
#pragma unroll
        for (int r = 0; r < 4; ++r) c = mma32(x[(o + 16 + m) * kLd + o + 16 + 4 * g + r], t[r], c);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[(o + 16 + 4 * g + r) * kLd + o + m] = -c[r];
        mx[way] = max4(c, mx[way]);
    }
    __syncthreads();
    {  // rows 32.., columns 0..31: a tile of columns a wavefront; two ways, or two tiles of rows
        const int tj = w & 1, way = WAYS == 2 ? w >> 1 : 0;
        float *x = X + way * kX;
        f32x4 t[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            t[k] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int l = 0; l < 2; ++l) {
                if (l < tj) continue;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const int row = 32 + 16 * k + m, col = 16 * l + 4 * s + g;
                    t[k] = mma32(L[row * kLd + col] * b[way ? row : col], x[col * kLd + 16 * tj + m], t[k]);
                }
            }
        }
#pragma unroll
        for (int ti = 0; ti < 2; ++ti) {
            if (WAYS == 1 && ti != w >> 1) continue;
            f32x4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k <= ti; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r) c = mma32(x[(32 + 16 * ti + m) * kLd + 32 + 16 * k + 4 * g + r], t[k][r], c);
#pragma unroll
            for (int r = 0; r < 4; ++r) x[(32 + 16 * ti + 4 * g + r) * kLd + 16 * tj + m] = -c[r];
            mx[way] = max4(c, mx[way]);
        }
    }
}

// The triangular matrix in LDS, its columns times `by` where that is given,
// as six left operands in two halves.  Six wavefront-sized pieces over four
// wavefronts.
__device__ __forceinline__ void store_tri(const float *x, const float *by, float scale, char *out) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    for (int f = threadIdx.x >> 6; f < kTri; f += 4) {
        const int mt = f < 2 ? f : f / 2 + 1, s = f < 2 ? 0 : f % 2;
        const float *p = x + (16 * mt + r) * kLd + 32 * s + 4 * g;
        f32x4 a = *(const f32x4 *)p, c = *(const f32x4 *)(p + 16);
        if (by) a *= *(const f32x4 *)(by + 32 * s + 4 * g), c *= *(const f32x4 *)(by + 32 * s + 4 * g + 16);
        const Split v = split8(a, c, scale);
        const int at = (f * kFrag + lane * 8) * 2;
        *(f16x8 *)(out + at) = v.hi;
        *(f16x8 *)(out + at + kTri * kFrag * 2) = v.lo;
    }
}

// Bounds: the blocks that a CU's LDS and registers hold; a fourth, with the
// registers that leaves it, gains nothing (151 us where three took 149).
constexpr int blocks_of(int bytes, int dkp, bool grad) { return grad || (bytes == 4 && dkp == 128) ? 2 : 3; }
template <typename S, int DKP, bool GRAD>
__global__ __launch_bounds__(256, blocks_of(sizeof(S), DKP, GRAD)) void delta_prep_kernel(DeltaArgs A, DeltaBuf B, bool vec) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int LD = DKP + 8, KS = DKP / 32, PL = SPLIT ? 2 : 1, WAYS = GRAD ? 2 : 1;
    // q and k first, then a value head's L and inverses (P before those)
    constexpr int kIn = PL * 2 * kC * LD * 2, kMat = (1 + WAYS) * kC * kLd * 4;
    __shared__ __align__(16) char both[kIn > kMat ? kIn : kMat];
    _Float16 *sk = (_Float16 *)both, *sq = sk + PL * kC * LD;
    float *lm = (float *)both, *xi = lm + kC * kLd;
    __shared__ __align__(16) float rk[kC], nk[kC], uq[kC], nq[kC], sb[4][kC], red[4][4];
    __shared__ __align__(16) float gh[4][kC], gl[4][kC];  // gam / log 2 in two floats
    const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, lane = tid & 63, g = lane >> 4, m = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const DeltaChunk ch = chunk_of(A.s, slot);
    if (ch.len == 0) return;
    const int rep = A.Hv / A.Hk;
    // g and b of one value head a wavefront, four heads at a time
    float gt, bt;
    auto fetch_gates = [&](int v) {
        gt = bt = 0.f;
        if (v < rep && lane < ch.len) {
            const int64_t th = (ch.t0 + lane) * A.Hv + hk * rep + v;
            gt = A.g[th];
            bt = A.beta_f32 ? ((const float *)A.beta)[th] : mix_f32(((const S *)A.beta)[th]);
        }
    };
    {
        S fk[DKP / 4], fq[DKP / 4];
        fetch_rows<S, DKP>((const S *)A.k + (int64_t)hk * A.dk, A.ks, ch, A.dk, vec, fk);
        fetch_rows<S, DKP>((const S *)A.q + (int64_t)hk * A.dk, A.qs, ch, A.dk, vec, fq);
        fetch_gates(w);
        put_rows<S, DKP, SPLIT>(fk, A.qk_norm, sk, rk, nk);
        put_rows<S, DKP, SPLIT>(fq, A.qk_norm, sq, uq, nq);
    }
    __syncthreads();
    const int64_t head = (int64_t)slot * A.Hk + hk;
    const int64_t at = head * 2 * PL * kC * DKP;
    if (GRAD && tid < kC) {
        float *o = B.rowk + head * 4 * kC + tid;
        o[0] = rk[tid], o[kC] = nk[tid], o[2 * kC] = uq[tid], o[3 * kC] = nq[tid];
    }
#pragma unroll
    for (int pl = 0; pl < PL; ++pl) {
        const _Float16 *k = sk + pl * kC * LD, *q = sq + pl * kC * LD;
        const int64_t o = at + (int64_t)pl * kC * DKP + lane * 8;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            *(f16x8 *)(B.kq + o + (w * KS + s) * kFrag) = row_frag<LD>(k, w, s);
            *(f16x8 *)(B.kq + o + PL * kC * DKP + (w * KS + s) * kFrag) = row_frag<LD>(q, w, s);
        }
    }
    // K K' and Q K', rows 16 w.. of the lower triangle: they stay in registers
    f32x4 kk[4], qk[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) kk[nt] = qk[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < KS; ++s) {
        const f16x8 kh = row_frag<LD>(sk, w, s), qh = row_frag<LD>(sq, w, s);
        f16x8 kl, ql;
        if (SPLIT) kl = row_frag<LD>(sk + kC * LD, w, s), ql = row_frag<LD>(sq + kC * LD, w, s);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt > w) continue;
            const f16x8 rh = row_frag<LD>(sk, nt, s);
            if (SPLIT) {
                const f16x8 rl = row_frag<LD>(sk + kC * LD, nt, s);
                kk[nt] = mma(kl, rh, mma(kh, rl, kk[nt]));
                qk[nt] = mma(ql, rh, mma(qh, rl, qk[nt]));
            }
            kk[nt] = mma(kh, rh, kk[nt]);
            qk[nt] = mma(qh, rh, qk[nt]);
        }
    }
    const int row = 16 * w + 4 * g;  // of this lane's four
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        const float rj = rk[16 * nt + m];
        kk[nt] *= *(const f32x4 *)(rk + row) * rj;
        qk[nt] *= *(const f32x4 *)(uq + row) * (A.scale * rj);
    }
    for (int v0 = 0; v0 < rep; v0 += 4) {
        __syncthreads();  // q and k, or the heads before, are done with
        if (v0 + w < rep) {
            const int64_t vh = (int64_t)slot * A.Hv + hk * rep + v0 + w;
            char *tp = B.tp + vh * kTpBytes;
            const float ga = gt < -1e4f ? -1e4f : gt;  // -inf too: e^-1e4 is zero, and differences stay numbers
            double s = ga;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_up(s, d, 64);
                if (lane >= d) s += o;
            }
            const double all = __shfl(s, 63, 64);
            const double s2 = s * 1.4426950408889634;
            gh[w][lane] = (float)s2;
            gl[w][lane] = (float)(s2 - (double)(float)s2);
            sb[w][lane] = bt;
            const float rise = expf((float)s), last = expf((float)all);
            const float f1 = rk[lane] * rise, f2 = uq[lane] * A.scale * rise, f3 = rk[lane] * expf((float)(all - s));
            auto put = [&](char *p) {
                float *f = (float *)(p + kTpRows) + lane;
                f[ROW_F1 * kC] = f1, f[ROW_F2 * kC] = f2, f[ROW_F3 * kC] = f3, f[ROW_B * kC] = bt;
                f[ROW_F3B * kC] = f3 * bt, f[ROW_F1B * kC] = f1 * bt;
                if (lane == 0) f[ROW_SCALARS * kC + SC_LAST] = last;
            };
            put(tp);
            if (GRAD) {
                put(B.tpg + vh * kTpBytes);
                B.gam[vh * kC + lane] = s;
            }
        }
        fetch_gates(v0 + 4 + w);
        // tiles right of the diagonal that the operands of 32 columns reach into: (0, 1) and (2, 3)
        for (int i = tid; i < WAYS * 512; i += 256) {
            const int x = i >> 9, t = i >> 8 & 1, e = i & 255;
            xi[x * kC * kLd + (32 * t + (e >> 4)) * kLd + 32 * t + 16 + (e & 15)] = 0.f;
        }
        const int heads = rep - v0 < 4 ? rep - v0 : 4;
        for (int v = 0; v < heads; ++v) {
            const int64_t vh = (int64_t)slot * A.Hv + hk * rep + v0 + v;
            char *tp = B.tp + vh * kTpBytes, *tpg = GRAD ? B.tpg + vh * kTpBytes : nullptr;
            __syncthreads();
            // L into lm, P into xi
            float mp = 0.f, mpb = 0.f;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                if (nt > w) continue;
                const int j = 16 * nt + m;
                const float hj = gh[v][j], lj = gl[v][j], bj = sb[v][j];
                const f32x4 hi = *(const f32x4 *)(gh[v] + row), li = *(const f32x4 *)(gl[v] + row);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int i = row + r;
                    const float d = __builtin_amdgcn_exp2f((hi[r] - hj) + (li[r] - lj));
                    const bool in = nt < w || j <= i;
                    const float p = in ? qk[nt][r] * d : 0.f;
                    lm[i * kLd + j] = in && j != i ? kk[nt][r] * d : 0.f;
                    xi[i * kLd + j] = p;
                    mp = max2(mp, fabsf(p));
                    mpb = max2(mpb, fabsf(p * bj));
                }
            }
            mp = tile_max(mp), mpb = tile_max(mpb);
            if (lane == 0) red[0][w] = mp, red[1][w] = mpb;
            __syncthreads();
            float inv;
            float sc = pow2_to(max4(*(const f32x4 *)red[1], 0.f), kTop, &inv);
            store_tri(xi, sb[v], sc, tp + kTpRows / 2);
            if (tid == 0) ((float *)(tp + kTpRows))[ROW_SCALARS * kC + SC_IP] = inv;
            if (GRAD) {
                sc = pow2_to(max4(*(const f32x4 *)red[0], 0.f), kTop, &inv);
                store_tri(xi, nullptr, sc, tpg + kTpRows / 2);
                if (tid == 0) ((float *)(tpg + kTpRows))[ROW_SCALARS * kC + SC_IP] = inv;
            }
            __syncthreads();
            float mx[2];
            invert<WAYS>(lm, sb[v], xi, mx);
#pragma unroll
            for (int way = 0; way < WAYS; ++way) {
                const float x = tile_max(mx[way]);
                if (lane == 0) red[2 + way][w] = x;
            }
            __syncthreads();
#pragma unroll
            for (int way = 0; way < WAYS; ++way) {
                const float big = max4(*(const f32x4 *)red[2 + way], 0.f);
                sc = pow2_to(big, kTop, &inv);
                store_tri(xi + way * kC * kLd, nullptr, sc, way ? tpg : tp);
                if (tid == 0) ((float *)((way ? tpg : tp) + kTpRows))[ROW_SCALARS * kC + SC_IT] = inv;
            }
        }
    }
}

template <typename S, int DKP>
hipError_t prep_typed(const DeltaArgs &a, const DeltaBuf &b, bool grad, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    const bool vec = a.dk % V == 0 && a.qs % V == 0 && a.ks % V == 0 && (uintptr_t)a.q % 16 == 0 && (uintptr_t)a.k % 16 == 0;
    const dim3 grid(b.slots, a.Hk);
    if (grad) hipLaunchKernelGGL((delta_prep_kernel<S, DKP, true>), grid, dim3(256), 0, st, a, b, vec);
    else hipLaunchKernelGGL((delta_prep_kernel<S, DKP, false>), grid, dim3(256), 0, st, a, b, vec);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_prep(const DeltaArgs &a, const DeltaBuf &b, bool grad, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return b.dkp == 64 ? prep_typed<float, 64>(a, b, grad, st) : prep_typed<float, 128>(a, b, grad, st);
    if (dtype == CONV_DTYPE_FP16) return b.dkp == 64 ? prep_typed<_Float16, 64>(a, b, grad, st) : prep_typed<_Float16, 128>(a, b, grad, st);
    return b.dkp == 64 ? prep_typed<uint16_t, 64>(a, b, grad, st) : prep_typed<uint16_t, 128>(a, b, grad, st);
}

}  // namespace convlower
