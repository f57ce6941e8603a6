// First step of the chunked gated delta rule: everything of a chunk that does
// not need the state.  A block takes one chunk of one query/key head: it puts
// q and k in the order of the matrix cores' left operands, multiplies K K' and
// Q K' once, and for each value head of the group forms the decays, P and the
// inverse of the chunk's unit lower triangular matrix: (1 + L diag(b))^-1 for
// the way forward and, where gradients are wanted, (1 + diag(b) L)^-1 too.
//
// The inverse is built from 16 x 16 diagonal blocks (substitution, one
// wavefront each) and joined twice: [A 0; B C]^-1 = [A' 0; -C' B A', C'].
// Sums of g are held in float64: gam_i - gam_j loses too many digits in 32
// bits where a chunk holds strong decays beside weak ones.
#include "delta_chunk.h"

namespace convlower {
namespace {

constexpr int kLd = 68;  // floats from row to row of the 64 x 64 matrices in LDS

// Loads 16-byte pieces of row `row` (a quarter of it a thread), finds its
// largest value and its sum of squares, and leaves it in LDS as f16.
template <typename S, int DKP, bool SPLIT>
__device__ __forceinline__ void load_rows(const S *src, int64_t stride, const DeltaChunk &ch, int dk, bool vec, int norm,
                                          _Float16 *dst, float *rho, float *rnorm) {
    constexpr int Q = DKP / 4, V = 16 / sizeof(S), LD = DKP + 8;
    const int row = threadIdx.x >> 2, c0 = (threadIdx.x & 3) * Q;
    float f[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) f[i] = 0.f;
    if (row < ch.len) {
        const S *p = src + (ch.t0 + row) * stride + c0;
        if (vec) {
#pragma unroll
            for (int i = 0; i < Q; i += V)
                if (c0 + i < dk) mix_load<S, V>(p + i, *(float(*)[V]) & f[i]);
        } else {
#pragma unroll
            for (int i = 0; i < Q; ++i)
                if (c0 + i < dk) f[i] = mix_f32(p[i]);
        }
    }
    float m = 0.f, ss = 0.f;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        m = fmaxf(m, fabsf(f[i]));
        ss = fmaf(f[i], f[i], ss);
    }
    m = fmaxf(m, __shfl_xor(m, 1, 64));
    m = fmaxf(m, __shfl_xor(m, 2, 64));
    ss += __shfl_xor(ss, 1, 64);
    ss += __shfl_xor(ss, 2, 64);
    float inv;
    const float sc = pow2_to(m, kRowTop, &inv);
#pragma unroll
    for (int i = 0; i < Q; i += 8) {
        f16x8 h, l;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float x = f[i + j] * sc;
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
__device__ __forceinline__ float wave_max(float m) { return tile_max(m); }
// Largest of all 256 threads' values, to every thread.
__device__ __forceinline__ float block_max(float m, float *red) {
    m = wave_max(m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

// X = M^-1 for the unit lower triangular M = 1 + (strict part in m), both
// [64][kLd] in LDS.  256 threads; X's upper part is left zero.
__device__ __forceinline__ void invert(const float *m, float *x, float *tmp) {
    const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
    for (int i = tid; i < kC * kLd; i += 256) x[i] = 0.f;
    __syncthreads();
    if (lane < 16) {  // column `lane` of diagonal block w
        const float *b = m + 16 * w * (kLd + 1);
        float col[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s = i == lane ? 1.f : 0.f;
#pragma unroll
            for (int j = 0; j < i; ++j) s = fmaf(-b[i * kLd + j], col[j], s);
            col[i] = s;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) x[(16 * w + i) * kLd + 16 * w + lane] = col[i];
    }
    __syncthreads();
    {  // two 32 x 32 blocks: tmp = B A', then -C' tmp; 128 threads each
        const int h = tid >> 7, r = (tid >> 3) & 15, c = (tid & 7) * 2, o = 32 * h;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float b = m[(o + 16 + r) * kLd + o + j];
            s0 = fmaf(b, x[(o + j) * kLd + o + c], s0);
            s1 = fmaf(b, x[(o + j) * kLd + o + c + 1], s1);
        }
        tmp[(16 * h + r) * kLd + c] = s0;
        tmp[(16 * h + r) * kLd + c + 1] = s1;
        __syncthreads();
        s0 = s1 = 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const float b = x[(o + 16 + r) * kLd + o + 16 + j];
            s0 = fmaf(-b, tmp[(16 * h + j) * kLd + c], s0);
            s1 = fmaf(-b, tmp[(16 * h + j) * kLd + c + 1], s1);
        }
        x[(o + 16 + r) * kLd + o + c] = s0;
        x[(o + 16 + r) * kLd + o + c + 1] = s1;
    }
    __syncthreads();
    {  // the lower left 32 x 32 block
        const int r = tid >> 3, c = (tid & 7) * 4;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int j = 0; j < 32; ++j) s += m[(32 + r) * kLd + j] * *(const f32x4 *)(x + j * kLd + c);
        *(f32x4 *)(tmp + r * kLd + c) = s;
        __syncthreads();
        s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int j = 0; j < 32; ++j) s -= x[(32 + r) * kLd + 32 + j] * *(const f32x4 *)(tmp + j * kLd + c);
        *(f32x4 *)(x + (32 + r) * kLd + c) = s;
    }
    __syncthreads();
}

// The triangular matrix in LDS as six left operands in two halves.  Six
// wavefront-sized pieces over four wavefronts.
__device__ __forceinline__ void store_tri(const float *x, float scale, char *out) {
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    for (int f = threadIdx.x >> 6; f < kTri; f += 4) {
        const int mt = f < 2 ? f : f / 2 + 1, s = f < 2 ? 0 : f % 2;
        const float *p = x + (16 * mt + r) * kLd + 32 * s + 4 * g;
        const Split v = split8(*(const f32x4 *)p, *(const f32x4 *)(p + 16), scale);
        const int at = (f * kFrag + lane * 8) * 2;
        *(f16x8 *)(out + at) = v.hi;
        *(f16x8 *)(out + at + kTri * kFrag * 2) = v.lo;
    }
}

template <typename S, int DKP, bool GRAD>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs A, DeltaBuf B, bool vec) {
    constexpr bool SPLIT = sizeof(S) == 4;
    constexpr int LD = DKP + 8, KS = DKP / 32, PL = SPLIT ? 2 : 1;
    // q and k first, the value heads' matrices afterwards, in one place: 78 KB in all, two blocks a CU
    constexpr int kIn = PL * 2 * kC * LD * 2, kMat = (2 * kC + 32) * kLd * 4;
    __shared__ __align__(16) char both[kIn > kMat ? kIn : kMat];
    _Float16 *sk = (_Float16 *)both, *sq = sk + PL * kC * LD;
    float *lm = (float *)both, *xi = lm + kC * kLd, *tmp = xi + kC * kLd;
    __shared__ __align__(16) float kk[kC * kLd], qk[kC * kLd];
    __shared__ float rk[kC], nk[kC], uq[kC], rq[kC], nq[kC], sb[kC], red[4];
    __shared__ double sg[kC];
    const int slot = blockIdx.x, hk = blockIdx.y, tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const DeltaChunk ch = chunk_of(A.s, slot);
    if (ch.len == 0) return;
    load_rows<S, DKP, SPLIT>((const S *)A.k + (int64_t)hk * A.dk, A.ks, ch, A.dk, vec, A.qk_norm, sk, rk, nk);
    load_rows<S, DKP, SPLIT>((const S *)A.q + (int64_t)hk * A.dk, A.qs, ch, A.dk, vec, A.qk_norm, sq, uq, nq);
    __syncthreads();
    if (tid < kC) rq[tid] = uq[tid] * A.scale;
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
    {  // K K' and Q K': rows 16 w.., lower triangle
        f32x4 a[4], b[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) a[nt] = b[nt] = f32x4{0.f, 0.f, 0.f, 0.f};
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
                    a[nt] = mma(kl, rh, mma(kh, rl, a[nt]));
                    b[nt] = mma(ql, rh, mma(qh, rl, b[nt]));
                }
                a[nt] = mma(kh, rh, a[nt]);
                b[nt] = mma(qh, rh, b[nt]);
            }
        }
        const int g = lane >> 4;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int i = 16 * w + 4 * g + r, j = 16 * nt + (lane & 15);
                const float rj = rk[j];
                kk[i * kLd + j] = a[nt][r] * rk[i] * rj;
                qk[i * kLd + j] = b[nt][r] * rq[i] * rj;
            }
    }
    const int rep = A.Hv / A.Hk;
    float mf[4] = {};
    for (int v = 0; v < rep; ++v) {
        const int h = hk * rep + v;
        const int64_t vh = (int64_t)slot * A.Hv + h;
        char *tp = B.tp + vh * kTpBytes, *tpg = GRAD ? B.tpg + vh * kTpBytes : nullptr;
        if (w == 0) {
            float g = 0.f, b = 0.f;
            if (lane < ch.len) {
                const int64_t th = (ch.t0 + lane) * A.Hv + h;
                g = A.g[th];
                g = g < -1e4f ? -1e4f : g;  // -inf too: e^-1e4 is zero, and differences stay numbers
                b = A.beta_f32 ? ((const float *)A.beta)[th] : mix_f32(((const S *)A.beta)[th]);
            }
            double s = g;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_up(s, d, 64);
                if (lane >= d) s += o;
            }
            const double all = __shfl(s, 63, 64);
            sg[lane] = s;
            sb[lane] = b;
            const float rise = expf((float)s);
            const float f1 = rk[lane] * rise, f2 = rq[lane] * rise, f3 = rk[lane] * expf((float)(all - s));
            const float last = expf((float)all);
            mf[0] = wave_max(fabsf(f3 * b)), mf[1] = wave_max(fabsf(f1 * b)), mf[2] = wave_max(fabsf(f2));
            auto put = [&](char *tp) {
                float *f = (float *)(tp + kTpRows) + lane;
                f[ROW_F1 * kC] = f1, f[ROW_F2 * kC] = f2, f[ROW_F3 * kC] = f3, f[ROW_B * kC] = b;
                f[ROW_F3B * kC] = f3 * b, f[ROW_F1B * kC] = f1 * b;
                if (lane == 0) f[ROW_SCALARS * kC + SC_LAST] = last, f[ROW_SCALARS * kC + SC_F2] = mf[2];
            };
            put(tp);
            if (GRAD) {
                put(tpg);
                B.gam[vh * kC + lane] = s;
            }
        }
        __syncthreads();
        // the matrix to invert into lm, P into xi
        float mp = 0.f;
        for (int e = tid; e < kC * kC; e += 256) {
            const int i = e >> 6, j = e & 63;
            float l = 0.f, p = 0.f;
            if (j <= i) {
                const float d = expf((float)(sg[i] - sg[j]));
                p = qk[i * kLd + j] * d * (GRAD ? 1.f : sb[j]);
                if (j < i) l = kk[i * kLd + j] * d * sb[j];
            }
            lm[i * kLd + j] = l;
            xi[i * kLd + j] = p;
            mp = fmaxf(mp, fabsf(p));
        }
        float inv, sc;
        if (GRAD) {
            sc = pow2_to(block_max(mp, red), kTop, &inv);
            store_tri(xi, sc, tpg + kTpRows / 2);
            if (tid == 0) ((float *)(tpg + kTpRows))[ROW_SCALARS * kC + SC_IP] = inv;
            __syncthreads();
            mp = 0.f;
            for (int e = tid; e < kC * kC; e += 256) {
                const float p = xi[(e >> 6) * kLd + (e & 63)] *= sb[e & 63];
                mp = fmaxf(mp, fabsf(p));
            }
        }
        sc = pow2_to(block_max(mp, red), kTop, &inv);
        store_tri(xi, sc, tp + kTpRows / 2);
        if (tid == 0) ((float *)(tp + kTpRows))[ROW_SCALARS * kC + SC_IP] = inv;
        for (int way = 0; way < (GRAD ? 2 : 1); ++way) {
            __syncthreads();
            if (way) {  // b beside the row instead of the column
                for (int e = tid; e < kC * kC; e += 256) {
                    const int i = e >> 6, j = e & 63;
                    lm[i * kLd + j] = j < i ? kk[i * kLd + j] * expf((float)(sg[i] - sg[j])) * sb[i] : 0.f;
                }
                __syncthreads();
            }
            invert(lm, xi, tmp);
            mp = 0.f;
            for (int e = tid; e < kC * kC; e += 256) mp = fmaxf(mp, fabsf(xi[(e >> 6) * kLd + (e & 63)]));
            mp = block_max(mp, red);
            sc = pow2_to(mp, kTop, &inv);
            store_tri(xi, sc, way ? tpg : tp);
            if (tid == 0) {
                float *o = (float *)((way ? tpg : tp) + kTpRows) + ROW_SCALARS * kC;
                o[SC_IT] = inv;
                o[SC_T] = kC * mp, o[SC_TF3] = kC * mp * mf[0], o[SC_TF1] = kC * mp * mf[1];
            }
        }
        __syncthreads();
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
