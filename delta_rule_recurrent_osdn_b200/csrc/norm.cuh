// norm.cuh -- the block norm: what joins a mixer's (or any block's) output f to the residual
// stream x and to the next block, in one pass over the rows of D values:
//   u  = f                                    without w_post
//      = f / rms(f) * w_post                  rms(f) = sqrt(mean(f^2) + eps)
//   u *= act(gate)                            or, gate first, f * act(gate) in place of f above
//   x' = x + scale * u                        (x' = scale * u without x)
//   h  = x' / rms(x') * w_next                from the unrounded x'
// and its gradients, which recompute all of this from the inputs.  With n = v / rms(v), the norm
// n * w has d v = (dn - n * mean(dn * n)) / rms(v), dn = dout * w, and dw = sum over rows dout * n.
//
// A few operations per element: bound by HBM, each input read and each output written once.  A
// row is held in the registers of TPR threads, 8 values each, so one pass suffices; sums over a
// row go by shuffles, and through shared memory when a row takes several warps.
#pragma once

#include "mixer_common.cuh"

namespace osdn {

constexpr int NORM_V = 8;             // values per thread
constexpr int NORM_MAX_D = 1024 * NORM_V;

enum { NORM_ACT_SILU = 0, NORM_ACT_SIGMOID = 1 };

__device__ __forceinline__ float norm_act(float g, int act) {
    return act == NORM_ACT_SILU ? silu_f(g) : sigmoid_f(g);
}
__device__ __forceinline__ float norm_act_grad(float g, int act) {
    if (act == NORM_ACT_SILU) return silu_grad_f(g);
    const float s = sigmoid_f(g);
    return s * (1.f - s);
}

// The 8 values of a row that lane `i` of its TPR threads holds: 8 neighbours when VEC (D a
// multiple of 8 and the rows 16-byte aligned), else every TPR-th, so that a warp's accesses stay
// together in either case.
template <bool VEC, int TPR, typename IO>
__device__ __forceinline__ void norm_load(const IO* __restrict__ p, int i, int D, float* x) {
    if constexpr (VEC) {
        if (i * NORM_V < D) {
            vec_io<NORM_V, IO>::load(p + i * NORM_V, x);
            return;
        }
#pragma unroll
        for (int e = 0; e < NORM_V; ++e) x[e] = 0.f;
    } else {
#pragma unroll
        for (int e = 0; e < NORM_V; ++e)
            x[e] = e * TPR + i < D ? io_traits<IO>::to_f32(p[e * TPR + i]) : 0.f;
    }
}
template <bool VEC, int TPR, typename IO>
__device__ __forceinline__ void norm_store(IO* __restrict__ p, int i, int D, const float* x) {
    if constexpr (VEC) {
        if (i * NORM_V < D) vec_io<NORM_V, IO>::store(p + i * NORM_V, x);
    } else {
#pragma unroll
        for (int e = 0; e < NORM_V; ++e)
            if (e * TPR + i < D) p[e * TPR + i] = io_traits<IO>::from_f32(x[e]);
    }
}

// Sum over the TPR threads of a row.  `red` holds 2 x 32 floats per row slot and alternates by
// `flip`, so one barrier per sum suffices.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float* red, int& flip) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if constexpr (TPR > 32) {
        const int warp = threadIdx.x >> 5;                 // one row per block then
        float* r = red + 32 * flip;
        if ((threadIdx.x & 31) == 0) r[warp] = s;
        __syncthreads();
        s = (threadIdx.x & 31) < TPR / 32 ? r[threadIdx.x & 31] : 0.f;
#pragma unroll
        for (int off = TPR / 64; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
        s = __shfl_sync(0xffffffffu, s, 0);
        flip ^= 1;
    }
    return s;
}

template <bool VEC, int TPR, typename IO>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 128)
norm_fwd_kernel(const IO* __restrict__ f, const IO* __restrict__ x, const IO* __restrict__ gate,
                const float* __restrict__ w_post, const float* __restrict__ w_next, int act,
                int gate_first, float scale, float eps, IO* __restrict__ x_out,
                IO* __restrict__ h, int64_t R, int D) {
    constexpr int ROWS = TPR > 32 ? 1 : 128 / TPR;
    __shared__ float red[64];
    int flip = 0;
    const int i = threadIdx.x % TPR;
    float wp[NORM_V], wn[NORM_V];
    if (w_post) norm_load<VEC, TPR, float>(w_post, i, D, wp);
    if (w_next) norm_load<VEC, TPR, float>(w_next, i, D, wn);
    const float inv_d = 1.f / (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < R; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = r0 + threadIdx.x / TPR;
        const bool live = row < R;
        const int64_t at = (live ? row : R - 1) * D;  // a row that is not there repeats the last
        float u[NORM_V], a[NORM_V], xr[NORM_V];
        norm_load<VEC, TPR, IO>(f + at, i, D, u);
        if (gate) norm_load<VEC, TPR, IO>(gate + at, i, D, a);
        if (x) norm_load<VEC, TPR, IO>(x + at, i, D, xr);
        if (gate) {
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) {
                a[e] = norm_act(a[e], act);
                if (gate_first) u[e] *= a[e];
            }
        }
        if (w_post) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) s = fmaf(u[e], u[e], s);
            const float rs = rsqrtf(fmaf(row_sum<TPR>(s, red, flip), inv_d, eps));
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) u[e] *= rs * wp[e];
        }
#pragma unroll
        for (int e = 0; e < NORM_V; ++e) {
            if (gate && !gate_first) u[e] *= a[e];
            u[e] = x ? fmaf(scale, u[e], xr[e]) : scale * u[e];
        }
        if (x_out && live && OSDN_IN_BOUNDS(row, R)) norm_store<VEC, TPR, IO>(x_out + at, i, D, u);
        if (w_next) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e)
                if (VEC ? i * NORM_V < D : e * TPR + i < D) s = fmaf(u[e], u[e], s);
            const float rs = rsqrtf(fmaf(row_sum<TPR>(s, red, flip), inv_d, eps));
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) u[e] *= rs * wn[e];
            if (live && OSDN_IN_BOUNDS(row, R)) norm_store<VEC, TPR, IO>(h + at, i, D, u);
        }
    }
}

// Gradients.  Each block keeps its threads' sums of dw_post and dw_next over the rows it walks
// in registers, adds its row slots' in shared memory and writes one partial row per weight to
// `part` ([2][gridDim.x][D]); norm_reduce_kernel adds the blocks in a fixed order.
template <bool VEC, int TPR, typename IO>
__global__ void __launch_bounds__(TPR > 32 ? TPR : 128)
norm_bwd_kernel(const IO* __restrict__ f, const IO* __restrict__ x, const IO* __restrict__ gate,
                const float* __restrict__ w_post, const float* __restrict__ w_next, int act,
                int gate_first, float scale, float eps, const IO* __restrict__ dx_out,
                const IO* __restrict__ dh, IO* __restrict__ df, IO* __restrict__ dx,
                IO* __restrict__ dgate, float* __restrict__ part, int64_t R, int D) {
    constexpr int ROWS = TPR > 32 ? 1 : 128 / TPR;
    __shared__ float red[TPR > 32 ? 64 : ROWS * TPR * NORM_V];
    int flip = 0;
    const int i = threadIdx.x % TPR;
    float dwp[NORM_V], dwn[NORM_V];
#pragma unroll
    for (int e = 0; e < NORM_V; ++e) dwp[e] = dwn[e] = 0.f;
    const float inv_d = 1.f / (float)D;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < R; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t row = r0 + threadIdx.x / TPR;
        const bool live = row < R;
        const int64_t at = (live ? row : R - 1) * D;
        float v[NORM_V], a[NORM_V], d[NORM_V], w[NORM_V], xo[NORM_V];
        norm_load<VEC, TPR, IO>(f + at, i, D, v);
        if (gate) norm_load<VEC, TPR, IO>(gate + at, i, D, a);
        if (x) norm_load<VEC, TPR, IO>(x + at, i, D, xo);
        if (dx_out) {
            norm_load<VEC, TPR, IO>(dx_out + at, i, D, d);
        } else {
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) d[e] = 0.f;
        }
        // forward: v = the norm's input, rs its 1 / rms, u = the branch before scale
        float rs = 1.f;
        if (gate && gate_first) {
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) v[e] *= norm_act(a[e], act);
        }
        if (w_post) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) s = fmaf(v[e], v[e], s);
            rs = rsqrtf(fmaf(row_sum<TPR>(s, red, flip), inv_d, eps));
            norm_load<VEC, TPR, float>(w_post, i, D, w);
        } else {
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) w[e] = 1.f;
        }
        if (w_next) {
            float g[NORM_V], s = 0.f;
            norm_load<VEC, TPR, IO>(dh + at, i, D, g);
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) {
                float u = v[e] * rs * w[e];
                if (gate && !gate_first) u *= norm_act(a[e], act);
                u = x ? fmaf(scale, u, xo[e]) : scale * u;
                xo[e] = u;
                if (VEC ? i * NORM_V < D : e * TPR + i < D) s = fmaf(u, u, s);
            }
            const float rn = rsqrtf(fmaf(row_sum<TPR>(s, red, flip), inv_d, eps));
            float wn[NORM_V], dot = 0.f;
            norm_load<VEC, TPR, float>(w_next, i, D, wn);
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) {
                xo[e] *= rn;                                   // n
                if (live) dwn[e] = fmaf(g[e], xo[e], dwn[e]);
                g[e] *= wn[e];                                 // dn
                if (VEC ? i * NORM_V < D : e * TPR + i < D) dot = fmaf(g[e], xo[e], dot);
            }
            dot = row_sum<TPR>(dot, red, flip) * inv_d;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) d[e] += rn * (g[e] - xo[e] * dot);
        }
        if (dx && live && OSDN_IN_BOUNDS(row, R)) norm_store<VEC, TPR, IO>(dx + at, i, D, d);
        float dg[NORM_V];
#pragma unroll
        for (int e = 0; e < NORM_V; ++e) {
            d[e] *= scale;
            if (gate && !gate_first) {
                dg[e] = d[e] * (v[e] * rs * w[e]) * norm_act_grad(a[e], act);
                d[e] *= norm_act(a[e], act);
            }
        }
        if (w_post) {
            float dot = 0.f;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) {
                v[e] *= rs;                                    // n
                if (live) dwp[e] = fmaf(d[e], v[e], dwp[e]);
                d[e] *= w[e];                                  // dn
                if (VEC ? i * NORM_V < D : e * TPR + i < D) dot = fmaf(d[e], v[e], dot);
            }
            dot = row_sum<TPR>(dot, red, flip) * inv_d;
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) d[e] = rs * (d[e] - v[e] * dot);
        }
        if (gate && gate_first) {
            norm_load<VEC, TPR, IO>(f + at, i, D, v);
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) {
                dg[e] = d[e] * v[e] * norm_act_grad(a[e], act);
                d[e] *= norm_act(a[e], act);
            }
        }
        if (live && OSDN_IN_BOUNDS(row, R)) {
            norm_store<VEC, TPR, IO>(df + at, i, D, d);
            if (gate) norm_store<VEC, TPR, IO>(dgate + at, i, D, dg);
        }
    }
    // one partial row per weight and block
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!(k == 0 ? w_post : w_next)) continue;
        float* dw = k == 0 ? dwp : dwn;
        float* out = part + ((int64_t)k * gridDim.x + blockIdx.x) * D;
        if constexpr (ROWS > 1) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < NORM_V; ++e) red[threadIdx.x * NORM_V + e] = dw[e];
            __syncthreads();
            if (threadIdx.x < TPR) {
#pragma unroll
                for (int e = 0; e < NORM_V; ++e) {
                    dw[e] = 0.f;
                    for (int q = 0; q < ROWS; ++q) dw[e] += red[(q * TPR + i) * NORM_V + e];
                }
                norm_store<VEC, TPR, float>(out, i, D, dw);
            }
        } else {
            norm_store<VEC, TPR, float>(out, i, D, dw);
        }
    }
}

// dw[c] = sum over the blocks' partial rows, blockIdx.y = 0: dw_post, 1: dw_next.
constexpr int NORM_RED_WARPS = 8;
__global__ void __launch_bounds__(32 * NORM_RED_WARPS)
norm_reduce_kernel(const float* __restrict__ part, int blocks, int D, float* __restrict__ dw_post,
                   float* __restrict__ dw_next) {
    __shared__ float red[NORM_RED_WARPS][32];
    float* out = blockIdx.y == 0 ? dw_post : dw_next;
    if (!out) return;  // uniform over the block
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < D)
        for (int k = threadIdx.y; k < blocks; k += NORM_RED_WARPS)
            s += part[((int64_t)blockIdx.y * blocks + k) * D + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < D) {
#pragma unroll
        for (int k = 1; k < NORM_RED_WARPS; ++k) s += red[k][threadIdx.x];
        out[c] = s;
    }
}

}  // namespace osdn
