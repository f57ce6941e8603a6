// The end of a block on rows of D values, and its gradients:
//
//   u = y rstd(y) w_post,  r = x + alpha act(gate) u,  h = r rstd(r) w_next
//
// A few operations for each value read: HBM bound.  A row is held in the
// registers of TPR threads (V values of 16 bytes at a time, NV times), so each
// tensor is read once and the two norms cost no second pass; a short row takes
// part of a wavefront and a block holds several.  The backward pass gives a
// block a run of rows: weights and a shared gate stay in registers as they
// lie, the next row is on its way while one is worked with, and each thread
// keeps the sums of its own columns for the weights' gradients until the run
// ends.
// Measured (bf16): forward 16384 x 4096 with x, h and a shared gate 107 us,
// 5.0 TB/s; gradients of 8192 x 4096 110 + 7 us (82 us at a copy's rate);
// 131072 x 128 gated rows 21 us forward, 37 + 7 us back.  Rows of odd widths
// are read 16 bytes at a time as well: 72052 x 222 forward 35 us (128 MB), one
// value at a time 66; 30001 x 1061 both ways 494 us, was 714.
#include <algorithm>

#include "mixer_internal.h"

namespace convlower {
namespace {

// Threads of a block: a row of more than one wavefront has it to itself.
constexpr int block_of(int tpr) { return tpr > 64 ? tpr : 256; }

// Sum over the TPR threads of a row (a power of two: at most 64 lanes of one
// wavefront, or the whole block); every thread gets it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
#pragma unroll
    for (int m = (TPR < 64 ? TPR : 64) / 2; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
    if constexpr (TPR > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int i = 0; i < TPR / 64; ++i) v += red[i];
    }
    return v;
}

template <typename S>
__device__ __forceinline__ float act_of(float z, int act) {
    return act == MIX_ACT_NONE ? z : act == MIX_ACT_SILU ? z * mix_sigmoid<S>(z) : mix_sigmoid<S>(z);
}
// Value and slope.
template <typename S>
__device__ __forceinline__ void act_grad(float z, int act, float *a, float *da) {
    if (act == MIX_ACT_NONE) {
        *a = z;
        *da = 1.f;
        return;
    }
    const float s = mix_sigmoid<S>(z);
    *a = act == MIX_ACT_SILU ? z * s : s;
    *da = act == MIX_ACT_SILU ? s * (1.f + z * (1.f - s)) : s * (1.f - s);
}

// V values from column c of a row of D, at p.  ANY: rows that lie at any
// multiple of a value's size (such an access still is one instruction), whose
// last piece may hold fewer; what is past the row reads as zero.
template <typename S, int V>
struct __attribute__((packed, aligned(sizeof(S)))) AnyVec {
    S v[V];
};
template <typename S, int V, bool ANY>
__device__ __forceinline__ MixVec<S, V> piece(const S *p, int c, int D) {
    MixVec<S, V> t = {};
    if constexpr (!ANY) {
        if (c < D) t = *(const MixVec<S, V> *)(p + c);
    } else if (c + V <= D) {
        const AnyVec<S, V> u = *(const AnyVec<S, V> *)(p + c);
#pragma unroll
        for (int j = 0; j < V; ++j) t.v[j] = u.v[j];
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < D) t.v[j] = p[c + j];
    }
    return t;
}
template <typename S, int V, bool ANY>
__device__ __forceinline__ void put_piece(S *p, int c, int D, const float (&f)[V]) {
    if constexpr (!ANY) {
        if (c < D) mix_store<S, V>(p + c, f);
    } else if (c + V <= D) {
        AnyVec<S, V> t;
#pragma unroll
        for (int j = 0; j < V; ++j) t.v[j] = mix_out<S>(f[j]);
        *(AnyVec<S, V> *)(p + c) = t;
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (c + j < D) p[c + j] = mix_out<S>(f[j]);
    }
}

// The columns of a thread: V values from (i * TPR + lane) * V, i < NV.
template <typename S, int V, int TPR, int NV, bool ANY>
__device__ __forceinline__ void load_row(const S *p, int lane, int D, float (&f)[NV][V]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const MixVec<S, V> t = piece<S, V, ANY>(p, (i * TPR + lane) * V, D);
#pragma unroll
        for (int j = 0; j < V; ++j) f[i][j] = mix_f32(t.v[j]);
    }
}
template <typename S, int V, int TPR, int NV, bool ANY>
__device__ __forceinline__ void store_row(S *p, int lane, int D, const float (&f)[NV][V]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) put_piece<S, V, ANY>(p, (i * TPR + lane) * V, D, f[i]);
}

template <typename S, int V, int TPR, int NV, bool ANY>
__global__ __launch_bounds__(block_of(TPR)) void branch_norm_fwd_kernel(NormArgs A) {
    constexpr int TB = block_of(TPR), ROWS = TB / TPR;
    __shared__ float red[TB / 64];
    const int lane = threadIdx.x % TPR;
    const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / TPR;
    const bool live = row < A.R;  // a block of one row each is always live: the sums below meet all its threads
    const int64_t at = (live ? row : 0) * A.D;
    float r[NV][V], f[NV][V], w[NV][V];
    load_row<S, V, TPR, NV, ANY>((const S *)A.y + at, lane, A.D, r);
    if (A.gate) load_row<S, V, TPR, NV, ANY>((const S *)A.gate + (live ? row / A.rows_per_gate : 0) * A.D, lane, A.D, f);
    load_row<S, V, TPR, NV, ANY>((const S *)A.w_post, lane, A.D, w);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) ss = fmaf(r[i][j], r[i][j], ss);
    const float rs = 1.f / sqrtf(row_sum<TPR>(ss, red) / A.D + A.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            r[i][j] *= rs * w[i][j];
            if (A.gate) r[i][j] *= act_of<S>(f[i][j], A.act);
        }
    if (A.x) {
        load_row<S, V, TPR, NV, ANY>((const S *)A.x + at, lane, A.D, f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) r[i][j] = fmaf(A.alpha, r[i][j], f[i][j]);
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) r[i][j] *= A.alpha;
    }
    if (live) store_row<S, V, TPR, NV, ANY>((S *)A.r + at, lane, A.D, r);
    if (A.stats && live && lane == 0) A.stats[row] = rs;
    if (!A.w_next) return;
    load_row<S, V, TPR, NV, ANY>((const S *)A.w_next, lane, A.D, w);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j)
            if ((i * TPR + lane) * V + (ANY ? j : 0) < A.D) ss = fmaf(r[i][j], r[i][j], ss);
    const float rn = 1.f / sqrtf(row_sum<TPR>(ss, red) / A.D + A.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) r[i][j] *= rn * w[i][j];
    if (live) store_row<S, V, TPR, NV, ANY>((S *)A.h + at, lane, A.D, r);
    if (A.stats && live && lane == 0) A.stats[A.R + row] = rn;
}

// The block's sum of each column over the rows it held side by side, to p[D].
template <int V, int TPR, int NV, bool ANY>
__device__ __forceinline__ void block_sums(float (&s)[NV][V], float *p, int lane, int D) {
    if constexpr (TPR > 64) {
#pragma unroll
        for (int i = 0; i < NV; ++i) put_piece<float, V, ANY>(p, (i * TPR + lane) * V, D, s[i]);
    } else {
        __shared__ float all[4][NV * TPR * V];  // one line a wavefront
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
#pragma unroll
                for (int m = TPR; m < 64; m <<= 1) s[i][j] += __shfl_xor(s[i][j], m, 64);
                if ((threadIdx.x & 63) < TPR) all[threadIdx.x >> 6][(i * TPR + lane) * V + j] = s[i][j];
            }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += 256) p[c] = (all[0][c] + all[1][c]) + (all[2][c] + all[3][c]);
        __syncthreads();
    }
}

// dr += rstd(r) (e - rn mean(e rn)), e = dh w_next;  dx = dr
// du = alpha act(gate) dr;  dgate = alpha act'(gate) dr u
// dy = rstd(y) (e - yn mean(e yn)), e = du w_post
// r is built again from x and y: the rounded r would cost digits, and x is
// the same number of bytes.
template <typename S, int V, int TPR, int NV, bool ANY>
__global__ __launch_bounds__(block_of(TPR)) void branch_norm_bwd_kernel(NormArgs A) {
    constexpr int TB = block_of(TPR), ROWS = TB / TPR;
    __shared__ float red[TB / 64];
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const int64_t group = blockIdx.x / A.per_group;
    const int part = blockIdx.x % A.per_group;
    // gate rows of their own: the run of rows of one group is all rows
    const int64_t span = A.G == A.R ? A.R : A.rows_per_gate, base = group * span;
    const int64_t each = ((span + A.per_group - 1) / A.per_group + ROWS - 1) / ROWS * ROWS;
    const int64_t first = part * each, last = first + each < span ? first + each : span;
    const bool per_row = A.gate && A.G == A.R, next = A.w_next && A.dh;
    typedef MixVec<S, V> Raw;
    auto fetch = [&](const void *p, int64_t at, Raw (&f)[NV]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            f[i] = Raw{};
            if (p) f[i] = piece<S, V, ANY>((const S *)p + at, (i * TPR + lane) * V, A.D);
        }
    };
    float sp[NV][V], sg[NV][V], sn[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sp[i][j] = sg[i][j] = sn[i][j] = 0.f;
    Raw w[NV], wn[NV], gate[NV], ry[NV], rx[NV], rd[NV], rh[NV];
    float rs = 0.f, rn = 0.f;
    fetch(A.w_post, 0, w);
    fetch(A.w_next, 0, wn);
    if (A.gate && !per_row) fetch(A.gate, group * A.D, gate);
    // of a row past the run's end, the last one again
    auto fetch_row = [&](int64_t o) {
        const int64_t row = base + (o + sub < last ? o + sub : last - 1), at = row * A.D;
        fetch(A.y, at, ry);
        if (per_row) fetch(A.gate, at, gate);
        fetch(A.dr, at, rd);
        rs = A.stats[row];
        if (next) {
            fetch(A.x, at, rx);
            fetch(A.dh, at, rh);
            rn = A.stats[A.R + row];
        }
    };
    if (first < last) fetch_row(first);
    for (int64_t o = first; o < last; o += ROWS) {
        const bool live = o + sub < last;
        const int64_t at = (base + (live ? o + sub : o)) * A.D;
        float y[NV][V], g[NV][V], d[NV][V], x[NV][V], e[NV][V];
        const float ys = rs, xs = rn;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                y[i][j] = mix_f32(ry[i].v[j]) * ys;
                if (A.gate) g[i][j] = mix_f32(gate[i].v[j]);
                d[i][j] = mix_f32(rd[i].v[j]);
                if (next) x[i][j] = mix_f32(rx[i].v[j]), e[i][j] = mix_f32(rh[i].v[j]);
            }
        if (o + ROWS < last) fetch_row(o + ROWS);
        if (next) {
            float dot = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float u = y[i][j] * mix_f32(w[i].v[j]);
                    if (A.gate) u *= act_of<S>(g[i][j], A.act);
                    x[i][j] = fmaf(A.alpha, u, x[i][j]) * xs;  // (x reads as zero where there is none)
                    if (live) sn[i][j] = fmaf(e[i][j], x[i][j], sn[i][j]);
                    e[i][j] *= mix_f32(wn[i].v[j]);
                    dot = fmaf(e[i][j], x[i][j], dot);
                }
            dot = row_sum<TPR>(dot, red) / A.D;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < V; ++j) d[i][j] = fmaf(xs, e[i][j] - x[i][j] * dot, d[i][j]);
        }
        if (A.dx && live) store_row<S, V, TPR, NV, ANY>((S *)A.dx + at, lane, A.D, d);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float wp = mix_f32(w[i].v[j]);
                float f = A.alpha * d[i][j];
                if (A.gate) {
                    float a, da;
                    act_grad<S>(g[i][j], A.act, &a, &da);
                    g[i][j] = f * y[i][j] * wp * da;
                    if (live) sg[i][j] += g[i][j];
                    f *= a;
                }
                if (live) sp[i][j] = fmaf(f, y[i][j], sp[i][j]);
                f *= wp;
                dot = fmaf(f, y[i][j], dot);
                d[i][j] = f;
            }
        if (per_row && live) store_row<S, V, TPR, NV, ANY>((S *)A.dgate + at, lane, A.D, g);
        dot = row_sum<TPR>(dot, red) / A.D;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) d[i][j] = ys * (d[i][j] - y[i][j] * dot);
        if (live) store_row<S, V, TPR, NV, ANY>((S *)A.dy + at, lane, A.D, d);
    }
    block_sums<V, TPR, NV, ANY>(sp, A.part + (int64_t)blockIdx.x * A.D, lane, A.D);
    const int64_t plane = (int64_t)gridDim.x * A.D;
    if (A.w_next) block_sums<V, TPR, NV, ANY>(sn, A.part + plane + (int64_t)blockIdx.x * A.D, lane, A.D);
    if (A.gate && !per_row) block_sums<V, TPR, NV, ANY>(sg, A.part + 2 * plane + (int64_t)blockIdx.x * A.D, lane, A.D);
}

// Sums of the blocks' partial sums for one output row of D columns: 64
// columns a block, sixteen runs of rows side by side, in a fixed order.
// blockIdx.y: 0 w_post, 1 w_next, 2.. gate row y - 2.
template <typename S>
__global__ __launch_bounds__(1024) void branch_norm_sum_kernel(NormArgs A) {
    __shared__ float sum[16][64];
    const int64_t plane = (int64_t)A.blocks * A.D;
    const int what = blockIdx.y < 2 ? blockIdx.y : 2;
    S *out = what == 0 ? (S *)A.dw_post : what == 1 ? (S *)A.dw_next : (S *)A.dgate;
    if (!out || (what == 2 && A.G == A.R)) return;
    const int64_t group = what == 2 ? blockIdx.y - 2 : 0;
    const int n = what == 2 ? A.per_group : A.blocks;
    const float *p = A.part + what * plane + group * A.per_group * A.D;
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int c = blockIdx.x * 64 + lane;
    float s = 0.f;
    if (c < A.D)
#pragma unroll 4
        for (int t = q; t < n; t += 16) s += p[(int64_t)t * A.D + c];
    sum[q][lane] = s;
    __syncthreads();
    if (q || c >= A.D) return;
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += sum[r][lane];
    out[group * A.D + c] = mix_out<S>(s);
}

template <typename S, int V, int TPR, int NV, bool ANY, bool BWD>
hipError_t norm_run(const NormArgs &a, hipStream_t st) {
    constexpr int TB = block_of(TPR), rows = TB / TPR;
    if constexpr (!BWD) {
        const int64_t blocks = (a.R + rows - 1) / rows;
        if (!grid_fits(blocks, TB, 1)) return kTooLarge;
        hipLaunchKernelGGL((branch_norm_fwd_kernel<S, V, TPR, NV, ANY>), dim3((unsigned)blocks), dim3(TB), 0, st, a);
        return hipGetLastError();
    } else {
        if (a.R) {
            hipLaunchKernelGGL((branch_norm_bwd_kernel<S, V, TPR, NV, ANY>), dim3(a.blocks), dim3(TB), 0, st, a);
            if (const hipError_t e = hipGetLastError()) return e;
        }
        const unsigned gates = a.gate && a.G != a.R ? (unsigned)a.G : 0;
        hipLaunchKernelGGL((branch_norm_sum_kernel<S>), dim3((a.D + 63) / 64, 2 + gates), dim3(1024), 0, st, a);
        return hipGetLastError();
    }
}

// The fewest threads that hold a row in one 16-byte piece each, and more
// pieces only past 1024 threads: registers are what the backward pass runs out
// of (4096 bf16: 512 threads of one piece against 256 of two, 110 against 171
// us).
template <typename S, bool ANY, bool BWD>
hipError_t norm_width(const NormArgs &a, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    if (a.D <= 16 * V) return norm_run<S, V, 16, 1, ANY, BWD>(a, st);
    if (a.D <= 32 * V) return norm_run<S, V, 32, 1, ANY, BWD>(a, st);
    if (a.D <= 64 * V) return norm_run<S, V, 64, 1, ANY, BWD>(a, st);
    if (a.D <= 128 * V) return norm_run<S, V, 128, 1, ANY, BWD>(a, st);
    if (a.D <= 256 * V) return norm_run<S, V, 256, 1, ANY, BWD>(a, st);
    if (a.D <= 512 * V) return norm_run<S, V, 512, 1, ANY, BWD>(a, st);
    if (a.D <= 1024 * V) return norm_run<S, V, 1024, 1, ANY, BWD>(a, st);
    if (a.D <= 2048 * V) return norm_run<S, V, 1024, 2, ANY, BWD>(a, st);
    if constexpr (V == 4)
        if (a.D > 4096 * V) return norm_run<S, V, 1024, 8, ANY, BWD>(a, st);  // to 32768 float32
    return norm_run<S, V, 1024, 4, ANY, BWD>(a, st);
}

template <typename S, bool BWD>
hipError_t norm_typed(const NormArgs &a, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    bool vec = a.D % V == 0;
    for (const void *p : {a.x, a.y, a.w_post, a.gate, a.w_next, a.dr, a.dh, (const void *)a.r, (const void *)a.h,
                          (const void *)a.dx, (const void *)a.dy, (const void *)a.dgate})
        vec = vec && (uintptr_t)p % 16 == 0;
    return vec ? norm_width<S, false, BWD>(a, st) : norm_width<S, true, BWD>(a, st);
}

}  // namespace

// Blocks of the backward pass, each with rows of one gate row only, and never
// more than rows; every block leaves a row of partial sums.  1024, 512 and 256 of
// them give 16 wavefronts to a CU for 16-bit rows (whose blocks have D / 512
// wavefronts, four for short rows) but for widths of 513 to 1024, blocks of two
// wavefronts and so 8 to a CU; float32 rows have blocks twice as large.
void branch_norm_bwd_plan(int64_t R, int D, int64_t G, int *per_group, int *blocks) {
    const int64_t groups = G == R ? 1 : G;
    const int64_t span = groups ? R / groups : 0;
    const int64_t want = D <= 2048 ? 1024 : D <= 4096 ? 512 : 256;
    int64_t per = (want + groups - 1) / (groups ? groups : 1);
    const int64_t most = D <= 512 ? (span + 15) / 16 : span;  // a block of short rows takes up to 16 at once
    per = per > most ? most : per;
    *per_group = (int)(per < 1 ? 1 : per);
    *blocks = (int)(*per_group * (groups ? groups : 1));
}

hipError_t launch_branch_norm_fwd(const NormArgs &a, int dtype, hipStream_t st) {
    if (!a.R) return hipSuccess;
    if (dtype == CONV_DTYPE_FP32) return norm_typed<float, false>(a, st);
    if (dtype == CONV_DTYPE_FP16) return norm_typed<_Float16, false>(a, st);
    return norm_typed<uint16_t, false>(a, st);
}

hipError_t launch_branch_norm_bwd(const NormArgs &a, int dtype, hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return norm_typed<float, true>(a, st);
    if (dtype == CONV_DTYPE_FP16) return norm_typed<_Float16, true>(a, st);
    return norm_typed<uint16_t, true>(a, st);
}

}  // namespace convlower
