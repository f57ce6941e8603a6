// Short depthwise causal convolution along packed sequences, its gradients
// and its single-token form.
//
//   z[t,c] = bias[c] + sum_j w[c,j] x[t - (W-1) + j, c],   y = act(z)
//
// Two reads and writes per element against 2 W + 4 operations: HBM bound.  A
// thread owns V channels and walks along the tokens of one tile with the last
// W-1 inputs in registers and the next four tokens' loads under way, so x is
// read once but for the W-1 tokens before a tile.  The token index is the same
// for a whole wavefront, so finding sequences costs scalar work only.
// Measured (bf16, W = 4): forward 16384 x 8192 108 us, 4.95 TB/s, which is what
// a large copy reaches; gradients 8192 x 4096 57 + 4 us (41 us at that rate).
#include <algorithm>

#include "mixer_internal.h"

namespace convlower {
namespace {

constexpr int kAhead = 4;  // tokens whose loads are issued together

template <int WT>
__device__ __forceinline__ int width_of(const Conv1dArgs &a) {
    return WT < MIX_CONV1D_MAX_WIDTH ? WT : a.W;
}

// Weights of V channels as w[tap][channel], taps past the width zero.
template <typename S, int V, int WT>
__device__ __forceinline__ void load_taps(const S *w, int c0, int W, float (&wt)[WT][V]) {
#pragma unroll
    for (int j = 0; j < WT; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) wt[j][i] = j < W ? mix_f32(w[(int64_t)(c0 + i) * W + j]) : 0.f;
}

// hist[d-1] = the input d tokens before t in sequence [a, ..), from its state
// or zero before a.
template <typename S, int V, int WT>
__device__ __forceinline__ void load_hist(const Conv1dArgs &A, int n, int64_t a, int64_t t, int c0, int W,
                                          float (&hist)[WT][V]) {
#pragma unroll
    for (int d = 1; d < WT; ++d) {
        const int64_t p = t - d;
#pragma unroll
        for (int i = 0; i < V; ++i) hist[d - 1][i] = 0.f;
        if (d < W) {
            if (p >= a) mix_load<S, V>((const S *)A.x + p * A.xs + c0, hist[d - 1]);
            else if (A.state) {
                const int64_t row = W - 1 + (p - a);  // negative only where cu_seqlens is out of order
                mix_load<S, V>((const S *)A.state + ((int64_t)n * (W - 1) + (row < 0 ? 0 : row)) * A.D + c0, hist[d - 1]);
            }
        }
    }
}

template <int V, int WT>
__device__ __forceinline__ void push(float (&hist)[WT][V], const float (&x)[V]) {
#pragma unroll
    for (int d = WT - 1; d > 0; --d)
#pragma unroll
        for (int i = 0; i < V; ++i) hist[d][i] = hist[d - 1][i];
#pragma unroll
    for (int i = 0; i < V; ++i) hist[0][i] = x[i];
}

// z of one token: taps past the width are left out, not multiplied by zero.
template <int V, int WT>
__device__ __forceinline__ void taps(const float (&wt)[WT][V], const float (&b)[V], const float (&hist)[WT][V],
                                     const float (&x)[V], int W, float (&z)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = b[i];
#pragma unroll
    for (int d = WT - 1; d >= 0; --d) {
        if (d >= W) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            // weight of the input d tokens back
            float w = wt[WT - 1 - d][i];
            if (WT == MIX_CONV1D_MAX_WIDTH) {
#pragma unroll
                for (int j = 0; j < WT; ++j) w = j == W - 1 - d ? wt[j][i] : w;
            }
            z[i] = fmaf(w, d ? hist[d - 1][i] : x[i], z[i]);
        }
    }
}

template <typename S, int V, int WT>
__global__ __launch_bounds__(256) void conv1d_fwd_kernel(Conv1dArgs A) {
    const int W = width_of<WT>(A);
    const int64_t c = ((int64_t)blockIdx.y * 256 + threadIdx.x) * V;
    if (c >= A.D) return;
    const int c0 = (int)c;
    if ((int)blockIdx.x >= A.tiles) {  // the blocks past the tiles: one sequence's last inputs each
        const int n = blockIdx.x - A.tiles;
        int64_t a, e;
        seq_range(A.s, n, &a, &e);
        for (int j = 0; j < W - 1; ++j) {
            const int64_t at = e - a - (W - 1) + j;
            float f[V];
#pragma unroll
            for (int i = 0; i < V; ++i) f[i] = 0.f;
            if (at >= 0) mix_load<S, V>((const S *)A.x + (a + at) * A.xs + c0, f);
            else if (A.state) mix_load<S, V>((const S *)A.state + ((int64_t)n * (W - 1) + (W - 1 + at)) * A.D + c0, f);
            mix_store<S, V>((S *)A.state_out + ((int64_t)n * (W - 1) + j) * A.D + c0, f);
        }
        return;
    }
    float wt[WT][V], b[V], hist[WT][V];
    load_taps<S, V, WT>((const S *)A.w, c0, W, wt);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = A.bias ? mix_f32(((const S *)A.bias)[c0 + i]) : 0.f;
    int64_t t = (int64_t)blockIdx.x * A.tile;
    const int64_t t1 = t + A.tile < A.s.T ? t + A.tile : A.s.T;
    int n = seq_of(A.s, t);
    int64_t a, e;
    seq_range(A.s, n, &a, &e);
    load_hist<S, V, WT>(A, n, a, t, c0, W, hist);
    auto fetch = [&](int64_t u) { return *(const MixVec<S, V> *)((const S *)A.x + (u < t1 ? u : t1 - 1) * A.xs + c0); };
    auto token = [&](int64_t u, const MixVec<S, V> &raw) {
        float x[V], z[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = mix_f32(raw.v[i]);
        taps<V, WT>(wt, b, hist, x, W, z);
        if (A.act == MIX_ACT_SILU)
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] *= mix_sigmoid<S>(z[i]);
        mix_store<S, V>((S *)A.y + u * A.D + c0, z);
        push<V, WT>(hist, x);
    };
    MixVec<S, V> next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = fetch(t + u);
    while (t < t1) {
        if (t >= e && n + 1 < A.s.N) {  // the next sequence that holds a token
            n = seq_of(A.s, t);
            seq_range(A.s, n, &a, &e);
            load_hist<S, V, WT>(A, n, a, t, c0, W, hist);
        }
        const int64_t run = n + 1 < A.s.N && e < t1 ? e : t1;  // to here without another look
        while (t + kAhead <= run) {
            MixVec<S, V> x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) x[u] = next[u];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) next[u] = fetch(t + kAhead + u);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) token(t + u, x[u]);
            t += kAhead;
        }
        if (t < run) {  // fewer than kAhead are left of the run
            for (; t < run; ++t) token(t, fetch(t));
#pragma unroll
            for (int u = 0; u < kAhead; ++u) next[u] = fetch(t + u);
        }
    }
}

// dy of a token, whose inputs before it are in hist, becomes its dz.
template <typename S, int V, int WT>
__device__ __forceinline__ void grad_z(const Conv1dArgs &A, const float (&wt)[WT][V], const float (&b)[V],
                                       const float (&hist)[WT][V], const float (&x)[V], int W, float (&dz)[V]) {
    if (A.act == MIX_ACT_SILU) {
        float z[V];
        taps<V, WT>(wt, b, hist, x, W, z);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float s = mix_sigmoid<S>(z[i]);
            dz[i] *= s * (1.f + z[i] * (1.f - s));
        }
    }
}

// dx[t] = sum_d w[W-1-d] dz[t+d]: a thread walks along its run of tokens (and
// W-1 past it), with the last inputs and the unfinished dx in registers.  A
// block's four wavefronts take four runs of the same channels; their sums for
// dw and dbias meet in LDS, and a row of them goes to `part`.
template <typename S, int V, int WT>
__global__ __launch_bounds__(256) void conv1d_bwd_kernel(Conv1dArgs A) {
    const int W = width_of<WT>(A);
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t c = ((int64_t)blockIdx.y * 64 + lane) * V;
    const bool live = c < A.D;
    const int c0 = live ? (int)c : 0;
    __shared__ float sums[kConvRuns][64 * V];
    float wt[WT][V], b[V], hist[WT][V], x[V], dz[V];
    load_taps<S, V, WT>((const S *)A.w, c0, W, wt);
#pragma unroll
    for (int i = 0; i < V; ++i) b[i] = A.bias ? mix_f32(((const S *)A.bias)[c0 + i]) : 0.f;
    const int blocks = (A.tiles + kConvRuns - 1) / kConvRuns;
    if ((int)blockIdx.x >= blocks) {  // the blocks past those: the state gradients of four sequences each
        const int n = (blockIdx.x - blocks) * kConvRuns + w;
        if (!live || n >= A.s.N) return;
        int64_t a, e;
        seq_range(A.s, n, &a, &e);
        float ds[WT][V];
#pragma unroll
        for (int j = 0; j < WT; ++j)
#pragma unroll
            for (int i = 0; i < V; ++i) ds[j][i] = 0.f;
        load_hist<S, V, WT>(A, n, a, a, c0, W, hist);
#pragma unroll
        for (int p = 0; p < WT - 1; ++p) {  // token a + p reaches the state rows j >= p
            if (p >= W - 1 || a + p >= e) continue;
            mix_load<S, V>((const S *)A.x + (a + p) * A.xs + c0, x);
            mix_load<S, V>((const S *)A.dy + (a + p) * A.dys + c0, dz);
            grad_z<S, V, WT>(A, wt, b, hist, x, W, dz);
            push<V, WT>(hist, x);
#pragma unroll
            for (int j = 0; j < WT - 1; ++j)
                if (j >= p && j < W - 1)  // input a - (W-1) + j meets tap j - p
#pragma unroll
                    for (int i = 0; i < V; ++i) ds[j][i] = fmaf(wt[j - p < 0 ? 0 : j - p][i], dz[i], ds[j][i]);
        }
#pragma unroll
        for (int j = 0; j < WT - 1; ++j) {
            if (j >= W - 1) continue;
            if (A.dstate_out && j >= e - a) {  // a short sequence hands part of its state on
                float f[V];
                mix_load<S, V>((const S *)A.dstate_out + ((int64_t)n * (W - 1) + j - (e - a)) * A.D + c0, f);
#pragma unroll
                for (int i = 0; i < V; ++i) ds[j][i] += f[i];
            }
            mix_store<S, V>((S *)A.dstate + ((int64_t)n * (W - 1) + j) * A.D + c0, ds[j]);
        }
        return;
    }
    float dw[WT][V], db[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        db[i] = 0.f;
#pragma unroll
        for (int j = 0; j < WT; ++j) dw[j][i] = 0.f;
    }
    const int64_t t0 = ((int64_t)blockIdx.x * kConvRuns + w) * A.tile;
    const int64_t t1 = t0 + A.tile < A.s.T ? t0 + A.tile : A.s.T;
    int n = t0 < t1 ? seq_of(A.s, t0) : 0;
    for (int64_t s0 = t0; live && s0 < t1;) {  // the part of the run that lies in one sequence
        int64_t a, e;
        seq_range(A.s, n, &a, &e);
        if (n + 1 == A.s.N && e < t1) e = t1;  // tokens past the last sequence's end belong to it
        const int64_t s1 = e < t1 ? e : t1;
        if (s1 > s0) {
            load_hist<S, V, WT>(A, n, a, s0, c0, W, hist);
            float acc[WT][V];  // acc[d]: dx of token t - d as far as it is summed
#pragma unroll
            for (int d = 0; d < WT; ++d)
#pragma unroll
                for (int i = 0; i < V; ++i) acc[d][i] = 0.f;
            // one token's dz, and the dx that it completes; t >= e: only the latter
            auto token = [&](int64_t t, const MixVec<S, V> &rx, const MixVec<S, V> &ry) {
#pragma unroll
                for (int d = WT - 1; d > 0; --d)
#pragma unroll
                    for (int i = 0; i < V; ++i) acc[d][i] = acc[d - 1][i];
#pragma unroll
                for (int i = 0; i < V; ++i) acc[0][i] = 0.f;
                if (t < e) {
#pragma unroll
                    for (int i = 0; i < V; ++i) x[i] = mix_f32(rx.v[i]), dz[i] = mix_f32(ry.v[i]);
                    grad_z<S, V, WT>(A, wt, b, hist, x, W, dz);
#pragma unroll
                    for (int d = 0; d < WT; ++d) {
                        if (d >= W) continue;
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            float f = wt[WT - 1 - d][i];
                            if (WT == MIX_CONV1D_MAX_WIDTH) {
#pragma unroll
                                for (int j = 0; j < WT; ++j) f = j == W - 1 - d ? wt[j][i] : f;
                            }
                            acc[d][i] = fmaf(f, dz[i], acc[d][i]);
                        }
                    }
                    if (t < s1) {
#pragma unroll
                        for (int i = 0; i < V; ++i) db[i] += dz[i];
#pragma unroll
                        for (int d = 0; d < WT; ++d)  // dw[d]: the tap d tokens back
#pragma unroll
                            for (int i = 0; i < V; ++i)
                                if (d < W) dw[d][i] = fmaf(dz[i], d ? hist[d - 1 < 0 ? 0 : d - 1][i] : x[i], dw[d][i]);
                    }
                    push<V, WT>(hist, x);
                }
                const int64_t o = t - (W - 1);
                if (o >= s0) {
                    float f[V];
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        f[i] = acc[WT - 1][i];
                        if (WT == MIX_CONV1D_MAX_WIDTH)
#pragma unroll
                            for (int d = 0; d < WT; ++d) f[i] = d == W - 1 ? acc[d][i] : f[i];
                    }
                    if (A.dstate_out && o >= e - (W - 1)) {
                        float g[V];
                        mix_load<S, V>((const S *)A.dstate_out + ((int64_t)n * (W - 1) + o - (e - (W - 1))) * A.D + c0,
                                       g);
#pragma unroll
                        for (int i = 0; i < V; ++i) f[i] += g[i];
                    }
                    mix_store<S, V>((S *)A.dx + o * A.D + c0, f);
                }
            };
            const int64_t end = s1 + W - 1, last = (e < A.s.T ? e : A.s.T) - 1;
            MixVec<S, V> nx[kAhead], ny[kAhead];
            auto fetch = [&](int64_t t, MixVec<S, V> &rx, MixVec<S, V> &ry) {
                t = t < last ? t : last;
                rx = *(const MixVec<S, V> *)((const S *)A.x + t * A.xs + c0);
                ry = *(const MixVec<S, V> *)((const S *)A.dy + t * A.dys + c0);
            };
#pragma unroll
            for (int u = 0; u < kAhead; ++u) fetch(s0 + u, nx[u], ny[u]);
            for (int64_t t = s0; t < end; t += kAhead) {
                MixVec<S, V> rx[kAhead], ry[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) rx[u] = nx[u], ry[u] = ny[u];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) fetch(t + kAhead + u, nx[u], ny[u]);
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (t + u < end) token(t + u, rx[u], ry[u]);
            }
            s0 = s1;
        }
        if (++n >= A.s.N) break;
    }
    // the runs' sums, one row of [W + 1][D] a block, in a fixed order
    float *p = A.part + (int64_t)blockIdx.x * (W + 1) * A.D + (int64_t)blockIdx.y * 64 * V;
    const int cols = A.D - (int64_t)blockIdx.y * 64 * V < 64 * V ? (int)(A.D - (int64_t)blockIdx.y * 64 * V) : 64 * V;
#pragma unroll
    for (int d = 0; d <= WT; ++d) {
        if (d < WT && d >= W) continue;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) sums[w][lane * V + i] = d < WT ? dw[d < WT ? d : 0][i] : db[i];
        __syncthreads();
        for (int i = threadIdx.x; i < cols; i += 256)
            p[(int64_t)(d < WT ? d : W) * A.D + i] = (sums[0][i] + sums[1][i]) + (sums[2][i] + sums[3][i]);
    }
}

// The blocks' partial sums in a fixed order: 64 columns of [W+1][D] a block,
// sixteen runs of rows side by side.
template <typename S>
__global__ __launch_bounds__(1024) void conv1d_bwd_sum_kernel(Conv1dArgs A) {
    __shared__ float sum[16][64];
    const int64_t cols = (int64_t)(A.W + 1) * A.D;
    const int lane = threadIdx.x & 63, q = threadIdx.x >> 6, rows = (A.tiles + kConvRuns - 1) / kConvRuns;
    const int64_t i = (int64_t)blockIdx.x * 64 + lane;
    float s = 0.f;
    if (i < cols)
        for (int t = q; t < rows; t += 16) s += A.part[(int64_t)t * cols + i];
    sum[q][lane] = s;
    __syncthreads();
    if (q || i >= cols) return;
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += sum[r][lane];
    const int d = (int)(i / A.D);
    const int64_t c = i - (int64_t)d * A.D;
    if (d < A.W) ((S *)A.dw)[c * A.W + (A.W - 1 - d)] = mix_out<S>(s);
    else if (A.dbias) ((S *)A.dbias)[c] = mix_out<S>(s);
}

template <typename S, int V>
__global__ __launch_bounds__(64) void conv1d_step_kernel(const S *x, int64_t xs, const S *w, const S *bias, S *pool,
                                                         const int32_t *slots, S *y, int P, int D, int W, int act) {
    const int64_t c = ((int64_t)blockIdx.y * 64 + threadIdx.x) * V;
    const int r = blockIdx.x;
    if (c >= D) return;
    const int c0 = (int)c;
    const int slot = slots ? slots[r] : r;
    float z[V], f[V];
    if (slot < 0 || slot >= P) {
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = 0.f;
        mix_store<S, V>(y + (int64_t)r * D + c0, z);
        return;
    }
    S *st = pool + (int64_t)slot * (W - 1) * D + c0;
    MixVec<S, V> line[MIX_CONV1D_MAX_WIDTH];
#pragma unroll
    for (int j = 0; j < MIX_CONV1D_MAX_WIDTH; ++j) {
        if (j < W - 1) line[j] = *(const MixVec<S, V> *)(st + (int64_t)j * D);
        else if (j == W - 1) line[j] = *(const MixVec<S, V> *)(x + r * xs + c0);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) z[i] = bias ? mix_f32(bias[c0 + i]) : 0.f;
#pragma unroll
    for (int j = 0; j < MIX_CONV1D_MAX_WIDTH; ++j)
        if (j < W)
#pragma unroll
            for (int i = 0; i < V; ++i) z[i] = fmaf(mix_f32(w[(int64_t)(c0 + i) * W + j]), mix_f32(line[j].v[i]), z[i]);
#pragma unroll
    for (int j = 1; j < MIX_CONV1D_MAX_WIDTH; ++j)
        if (j < W) *(MixVec<S, V> *)(st + (int64_t)(j - 1) * D) = line[j];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = act == MIX_ACT_SILU ? z[i] * mix_sigmoid<S>(z[i]) : z[i];
    mix_store<S, V>(y + (int64_t)r * D + c0, f);
}

bool aligned16(std::initializer_list<const void *> ps) {
    for (const void *p : ps)
        if ((uintptr_t)p % 16) return false;
    return true;
}

template <typename S, int V>
hipError_t fwd_typed(const Conv1dArgs &a, hipStream_t st) {
    const int cb = (a.D + 256 * V - 1) / (256 * V);
    const int64_t all = (int64_t)a.tiles + (a.state_out && a.W > 1 ? a.s.N : 0);
    if (!all) return hipSuccess;
    if (!grid_fits(all, 256, cb)) return kTooLarge;
    const dim3 grid((unsigned)all, cb);
    switch (a.W) {
        case 2: hipLaunchKernelGGL((conv1d_fwd_kernel<S, V, 2>), grid, dim3(256), 0, st, a); break;
        case 3: hipLaunchKernelGGL((conv1d_fwd_kernel<S, V, 3>), grid, dim3(256), 0, st, a); break;
        case 4: hipLaunchKernelGGL((conv1d_fwd_kernel<S, V, 4>), grid, dim3(256), 0, st, a); break;
        default: hipLaunchKernelGGL((conv1d_fwd_kernel<S, V, 8>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

template <typename S, int V>
hipError_t bwd_typed(const Conv1dArgs &a, hipStream_t st) {
    const int cb = (a.D + 64 * V - 1) / (64 * V);
    const auto blocks = [](int64_t n) { return (n + kConvRuns - 1) / kConvRuns; };
    const int64_t all = blocks(a.tiles) + (a.dstate && a.W > 1 ? blocks(a.s.N) : 0);
    if (!grid_fits(all, 256, cb)) return kTooLarge;
    const dim3 grid((unsigned)all, cb);
    if (all) {
        switch (a.W) {
            case 2: hipLaunchKernelGGL((conv1d_bwd_kernel<S, V, 2>), grid, dim3(256), 0, st, a); break;
            case 3: hipLaunchKernelGGL((conv1d_bwd_kernel<S, V, 3>), grid, dim3(256), 0, st, a); break;
            case 4: hipLaunchKernelGGL((conv1d_bwd_kernel<S, V, 4>), grid, dim3(256), 0, st, a); break;
            default: hipLaunchKernelGGL((conv1d_bwd_kernel<S, V, 8>), grid, dim3(256), 0, st, a);
        }
        if (const hipError_t e = hipGetLastError()) return e;
    }
    const int64_t cols = (int64_t)(a.W + 1) * a.D;
    hipLaunchKernelGGL((conv1d_bwd_sum_kernel<S>), dim3((unsigned)((cols + 63) / 64)), dim3(1024), 0, st, a);
    return hipGetLastError();
}

template <typename S>
hipError_t step_typed(const void *x, int64_t xs, const void *w, const void *bias, void *pool, const int32_t *slots,
                      void *y, int R, int P, int D, int W, int act, hipStream_t st) {
    constexpr int V = 16 / sizeof(S);
    const bool vec = D % V == 0 && xs % V == 0 && aligned16({x, pool, y});
    if (!grid_fits(R, 64, (D + 64 * (vec ? V : 1) - 1) / (64 * (vec ? V : 1)))) return kTooLarge;
    if (vec)
        hipLaunchKernelGGL((conv1d_step_kernel<S, V>), dim3(R, (D + 64 * V - 1) / (64 * V)), dim3(64), 0, st,
                           (const S *)x, xs, (const S *)w, (const S *)bias, (S *)pool, slots, (S *)y, P, D, W, act);
    else
        hipLaunchKernelGGL((conv1d_step_kernel<S, 1>), dim3(R, (D + 63) / 64), dim3(64), 0, st, (const S *)x, xs,
                           (const S *)w, (const S *)bias, (S *)pool, slots, (S *)y, P, D, W, act);
    return hipGetLastError();
}

}  // namespace

// Tokens of a forward tile, and of a backward run: the W-1 tokens before it
// are read again, so long ones, but at least 4096 wavefronts (4 a SIMD), to
// have enough reads under way.
static int run_length(int64_t T, int D) {
    const int64_t waves = (D + 255) / 256;
    int run = 64;
    while (run > 8 && (T + run - 1) / run * waves < 4096) run /= 2;
    return run;
}
int conv1d_bwd_tile(int64_t T, int D) { return run_length(T, D); }

hipError_t launch_conv1d_fwd(Conv1dArgs a, int dtype, hipStream_t st) {
    a.tile = run_length(a.s.T, a.D);
    a.tiles = (int)((a.s.T + a.tile - 1) / a.tile);
    // four channels a thread for 16-bit types too: 64 registers and all 8 wavefronts of a SIMD, against 132 and 3 with
    // eight (16384 x 8192 bf16: 108 us, 4.95 TB/s, against 134 us)
    const bool vec = a.D % 4 == 0 && a.xs % 4 == 0 && aligned16({a.x, a.state, a.y, a.state_out});
    if (dtype == CONV_DTYPE_FP32) return vec ? fwd_typed<float, 4>(a, st) : fwd_typed<float, 1>(a, st);
    if (dtype == CONV_DTYPE_FP16) return vec ? fwd_typed<_Float16, 4>(a, st) : fwd_typed<_Float16, 1>(a, st);
    return vec ? fwd_typed<uint16_t, 4>(a, st) : fwd_typed<uint16_t, 1>(a, st);
}

hipError_t launch_conv1d_bwd(Conv1dArgs a, int dtype, hipStream_t st) {
    a.tile = conv1d_bwd_tile(a.s.T, a.D);
    a.tiles = (int)((a.s.T + a.tile - 1) / a.tile);
    // four channels a thread: with eight, taps, inputs, sums and reads under way take 270 registers
    const bool vec = a.D % 4 == 0 && a.xs % 4 == 0 && a.dys % 4 == 0 &&
                     aligned16({a.x, a.state, a.dy, a.dstate_out, a.dx, a.dstate});
    if (dtype == CONV_DTYPE_FP32) return vec ? bwd_typed<float, 4>(a, st) : bwd_typed<float, 1>(a, st);
    if (dtype == CONV_DTYPE_FP16) return vec ? bwd_typed<_Float16, 4>(a, st) : bwd_typed<_Float16, 1>(a, st);
    return vec ? bwd_typed<uint16_t, 4>(a, st) : bwd_typed<uint16_t, 1>(a, st);
}

hipError_t launch_conv1d_step(const void *x, int64_t xs, const void *w, const void *bias, void *pool,
                              const int32_t *slots, void *y, int R, int P, int D, int W, int act, int dtype,
                              hipStream_t st) {
    if (dtype == CONV_DTYPE_FP32) return step_typed<float>(x, xs, w, bias, pool, slots, y, R, P, D, W, act, st);
    if (dtype == CONV_DTYPE_FP16) return step_typed<_Float16>(x, xs, w, bias, pool, slots, y, R, P, D, W, act, st);
    return step_typed<uint16_t>(x, xs, w, bias, pool, slots, y, R, P, D, W, act, st);
}

}  // namespace convlower
