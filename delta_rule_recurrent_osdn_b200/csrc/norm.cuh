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
// Some 20 operations per element and two to four sums over the row: bound by HBM if those stay
// cheap, so a row is held in the registers of TPR threads, sums go by shuffles (and through shared
// memory when a row takes several warps), and the next row's loads are in flight while one is
// worked on.  Forward: 59 us at 16384 bf16 rows of 2048 with residual, gate and both norms (336 MB:
// 51 us at copy speed).  Backward: 47 us at 131,072 rows of 128 with a gate (168 MB: 26 us).  38 of
// them are the kernel, at 66% of the schedulers' slots (47 instructions a value) and with the waits of 5
// warps a scheduler for the rest; then 740 partial rows of weight gradients are added by 4 blocks, a
// chain of 92 loads a warp (13 us with cold caches).  142 us at 16384 rows of 2048 with both norms (537 MB:
// 82 us): 76 instructions a value at 57% of the slots, and four sums across the warps of a row.
// Registers are the limit of the gradient: up to 128, and the forms with the second norm spill for
// fp32 rows (44 bytes and more), wherever D is not a multiple of 8 (112 to 180 bytes) and above 4096
// columns (224 to 344 bytes); without it the fp32 forms, those above 4096 columns and those of
// other D spill 8 to 136 bytes.
#pragma once

#include "mixer_common.cuh"

namespace osdn {

// Values per thread: 16384 rows of 2048, forward 62 us with 16 and 76 with 8, backward 142 with 8
// and 213 with 16, where the registers of both passes' rows leave too few warps (L2 cold).
constexpr int NORM_FWD_V = 16, NORM_BWD_V = 8;
constexpr int NORM_MAX_D = 8192;

enum { NORM_ACT_SILU = 0, NORM_ACT_SIGMOID = 1 };

// The V values of a row that lane `i` of its TPR threads holds: V / 8 times 8 neighbours, TPR * 8
// apart, when VEC (D a multiple of 8: the rows are 16-byte aligned), else every TPR-th; a warp's
// accesses stay together in either case.  Values past D are 0.
template <bool VEC, int TPR, int V, typename IO> struct norm_row {
    raw_io<8, IO> r[V / 8];
    __device__ __forceinline__ void load(const IO* __restrict__ p, int i, int D) {
#pragma unroll
        for (int k = 0; k < V / 8; ++k) {
            const int c = (k * TPR + i) * 8;
            if (c < D) {
                r[k].load(p + c);
            } else {
#pragma unroll
                for (int e = 0; e < raw_io<8, IO>::WORDS; ++e) r[k].w[e] = 0;
            }
        }
    }
    __device__ __forceinline__ void to(float* x) const {
#pragma unroll
        for (int k = 0; k < V / 8; ++k) r[k].to(x + 8 * k);
    }
    static __device__ __forceinline__ void store(IO* __restrict__ p, int i, int D, const float* x) {
#pragma unroll
        for (int k = 0; k < V / 8; ++k) {
            const int c = (k * TPR + i) * 8;
            if (c < D) vec_io<8, IO>::store(p + c, x + 8 * k);
        }
    }
};
template <int TPR, int V, typename IO> struct norm_row<false, TPR, V, IO> {
    IO v[V];
    __device__ __forceinline__ void load(const IO* __restrict__ p, int i, int D) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = e * TPR + i < D ? p[e * TPR + i] : io_traits<IO>::from_f32(0.f);
    }
    __device__ __forceinline__ void to(float* x) const {
#pragma unroll
        for (int e = 0; e < V; ++e) x[e] = io_traits<IO>::to_f32(v[e]);
    }
    static __device__ __forceinline__ void store(IO* __restrict__ p, int i, int D, const float* x) {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e * TPR + i < D) p[e * TPR + i] = io_traits<IO>::from_f32(x[e]);
    }
};

// Sum over the TPR threads of a row.  `red` holds 2 x 32 floats and alternates by `flip`, so one
// barrier per sum suffices.
template <int TPR>
__device__ __forceinline__ float row_sum(float s, float* red, int& flip) {
    constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
    for (int off = W / 2; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if constexpr (TPR > 32) {  // one row per block then
        float* r = red + 32 * flip;
        if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = s;
        __syncthreads();
        s = r[0];
#pragma unroll
        for (int k = 1; k < TPR / 32; ++k) s += r[k];
        flip ^= 1;
    }
    return s;
}

// sum of a[e] * b[e], two at a time
template <int V> __device__ __forceinline__ float norm_dot(const float (&a)[V], const float (&b)[V]) {
    float2 s = make_float2(0.f, 0.f), t = s;
#pragma unroll
    for (int e = 0; e < V; e += 4) {
        s = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), s);
        t = __ffma2_rn(make_float2(a[e + 2], a[e + 3]), make_float2(b[e + 2], b[e + 3]), t);
    }
    return (s.x + s.y) + (t.x + t.y);
}
// x[e] = a[e] * b[e] (* k), two at a time
template <int V> __device__ __forceinline__ void norm_mul(float (&x)[V], const float (&a)[V], const float (&b)[V], float k) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        const float2 t = __fmul2_rn(__fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1])),
                                    make_float2(k, k));
        x[e] = t.x;
        x[e + 1] = t.y;
    }
}
// x[e] = k * a[e] + b[e]
template <int V> __device__ __forceinline__ void norm_axpy(float (&x)[V], float k, const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        const float2 t = __ffma2_rn(make_float2(k, k), make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
        x[e] = t.x;
        x[e + 1] = t.y;
    }
}
template <int V> __device__ __forceinline__ void norm_scale(float (&x)[V], float k) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
        const float2 t = __fmul2_rn(make_float2(k, k), make_float2(x[e], x[e + 1]));
        x[e] = t.x;
        x[e + 1] = t.y;
    }
}

constexpr int norm_threads(int TPR) { return TPR > 32 ? TPR : 128; }
constexpr int norm_rows(int TPR) { return TPR > 32 ? 1 : 128 / TPR; }
// Resident blocks of the backward kernel: 640 threads an SM, 512 with the second norm's registers.
// (131072 rows of 128: 512 threads 50 us, 640 46 us; 8192 rows of 1001 with the second norm: 60
// us, 83 us.)
constexpr int norm_bwd_per_sm(int TPR, bool next) {
    const int threads = norm_threads(TPR);
    return threads >= 512 ? 1 : (next ? 512 : 640) / threads;
}

template <bool VEC, int TPR, typename IO>
__global__ void __launch_bounds__(norm_threads(TPR))
norm_fwd_kernel(const IO* __restrict__ f, const IO* __restrict__ x, const IO* __restrict__ gate,
                const float* __restrict__ w_post, const float* __restrict__ w_next, int act,
                int gate_first, float scale, float eps, IO* __restrict__ x_out,
                IO* __restrict__ h, int64_t R, int D) {
    constexpr int V = NORM_FWD_V;
    using row_t = norm_row<VEC, TPR, V, IO>;
    using wrow_t = norm_row<VEC, TPR, V, float>;
    constexpr int ROWS = norm_rows(TPR);
    __shared__ float red[64];
    int flip = 0;
    const int i = threadIdx.x % TPR;
    const float inv_d = 1.f / (float)D;
    row_t rf, rg, rx;
    auto fetch = [&](int64_t r0) {
        int64_t row = r0 + threadIdx.x / TPR;
        row = row < R ? row : R - 1;  // a row that is not there repeats the last
        rf.load(f + row * D, i, D);
        if (gate) rg.load(gate + row * D, i, D);
        if (x) rx.load(x + row * D, i, D);
    };
    const int64_t hop = (int64_t)gridDim.x * ROWS;
    int64_t r0 = (int64_t)blockIdx.x * ROWS;
    if (r0 < R) fetch(r0);
    for (; r0 < R; r0 += hop) {
        const int64_t row = r0 + threadIdx.x / TPR, at = row * D;
        const bool live = row < R;
        float u[V], a[V], xr[V];
        rf.to(u);
        if (gate) {
            rg.to(a);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float s = sigmoid_f(a[e]);
                a[e] = act == NORM_ACT_SILU ? a[e] * s : s;
            }
        }
        if (x) rx.to(xr);
        if (r0 + hop < R) fetch(r0 + hop);
        if (gate && gate_first) norm_mul(u, u, a, 1.f);
        if (w_post) {
            const float rs = rsqrtf(fmaf(row_sum<TPR>(norm_dot(u, u), red, flip), inv_d, eps));
            wrow_t w;
            float wf[V];
            w.load(w_post, i, D);
            w.to(wf);
            norm_mul(u, u, wf, rs);
        }
        if (gate && !gate_first) norm_mul(u, u, a, 1.f);
        if (x) norm_axpy(u, scale, u, xr);
        else norm_scale(u, scale);
        if (x_out && live && OSDN_IN_BOUNDS(row, R)) row_t::store(x_out + at, i, D, u);
        if (w_next) {
            const float rs = rsqrtf(fmaf(row_sum<TPR>(norm_dot(u, u), red, flip), inv_d, eps));
            wrow_t w;
            float wf[V];
            w.load(w_next, i, D);
            w.to(wf);
            norm_mul(u, u, wf, rs);
            if (live && OSDN_IN_BOUNDS(row, R)) row_t::store(h + at, i, D, u);
        }
    }
}

// Gradients.  Each block keeps its threads' sums of dw_post and dw_next over the rows it walks
// in registers (NEXT: with w_next), adds its row slots' in shared memory and writes one partial row per weight to
// `part` ([2][gridDim.x][D]); norm_reduce_kernel adds the blocks in a fixed order.
template <bool VEC, int TPR, bool NEXT, typename IO>
__global__ void __launch_bounds__(norm_threads(TPR), norm_bwd_per_sm(TPR, NEXT))
norm_bwd_kernel(const IO* __restrict__ f, const IO* __restrict__ x, const IO* __restrict__ gate,
                const float* __restrict__ w_post, const float* __restrict__ w_next, int act,
                int gate_first, float scale, float eps, const IO* __restrict__ dx_out,
                const IO* __restrict__ dh, IO* __restrict__ df, IO* __restrict__ dx,
                IO* __restrict__ dgate, float* __restrict__ part, int64_t R, int D) {
    constexpr int V = NORM_BWD_V;
    using row_t = norm_row<VEC, TPR, V, IO>;
    using wrow_t = norm_row<VEC, TPR, V, float>;
    constexpr int ROWS = norm_rows(TPR);
    __shared__ float red[TPR > 32 ? 64 : norm_threads(TPR) * V];
    int flip = 0;
    const int i = threadIdx.x % TPR;
    float dwp[V], dwn[V];
#pragma unroll
    for (int e = 0; e < V; ++e) dwp[e] = dwn[e] = 0.f;
    const float inv_d = 1.f / (float)D;
    // the next row's loads are in flight while one is worked on, where registers allow it
    constexpr bool AHEAD = TPR < 1024;
    row_t nf, ng, nx, nd, nh;
    auto fetch = [&](int64_t r0) {
        int64_t row = r0 + threadIdx.x / TPR;
        const int64_t at = (row < R ? row : R - 1) * D;  // a row that is not there repeats the last
        nf.load(f + at, i, D);
        if (gate) ng.load(gate + at, i, D);
        if (NEXT && x) nx.load(x + at, i, D);  // x' matters to the second norm alone
        if (dx_out) nd.load(dx_out + at, i, D);
        if (NEXT) nh.load(dh + at, i, D);
    };
    const int64_t hop = (int64_t)gridDim.x * ROWS;
    int64_t r0 = (int64_t)blockIdx.x * ROWS;
    if (AHEAD && r0 < R) fetch(r0);
    for (; r0 < R; r0 += hop) {
        const int64_t row = r0 + threadIdx.x / TPR, at = row * D;
        const bool live = row < R;
        if (!AHEAD) fetch(r0);
        const row_t rf = nf, rg = ng, rx = nx, rd = nd, rh = nh;
        if (AHEAD && r0 + hop < R) fetch(r0 + hop);
        float v[V], s[V], d[V], w[V];  // s: sigmoid of the gate
        rf.to(v);
        if (gate) {
            rg.to(s);
#pragma unroll
            for (int e = 0; e < V; ++e) s[e] = sigmoid_f(s[e]);
        }
        // the gate's factor of element e
        auto factor = [&](const float (&g)[V], int e) { return act == NORM_ACT_SILU ? g[e] * s[e] : s[e]; };
        float rs = 1.f;
        if (gate && gate_first) {
            float g[V];
            rg.to(g);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] *= factor(g, e);
        }
        if (w_post) {
            rs = rsqrtf(fmaf(row_sum<TPR>(norm_dot(v, v), red, flip), inv_d, eps));
            wrow_t wr;
            wr.load(w_post, i, D);
            wr.to(w);
            norm_scale(v, rs);  // the norm's output before its weight
        }
        if (dx_out) {
            rd.to(d);
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) d[e] = 0.f;
        }
        if constexpr (NEXT) {
            float n[V], g[V];
            if (w_post) {
                norm_mul(n, v, w, scale);
            } else {
#pragma unroll
                for (int e = 0; e < V; ++e) n[e] = v[e];
                norm_scale(n, scale);
            }
            if (gate && !gate_first) {
                rg.to(g);
#pragma unroll
                for (int e = 0; e < V; ++e) n[e] *= factor(g, e);
            }
            if (x) {
                rx.to(g);
                norm_axpy(n, 1.f, n, g);
            }
            const float rn = rsqrtf(fmaf(row_sum<TPR>(norm_dot(n, n), red, flip), inv_d, eps));
            norm_scale(n, rn);
            rh.to(g);
            if (live) {
#pragma unroll
                for (int e = 0; e < V; ++e) dwn[e] = fmaf(g[e], n[e], dwn[e]);
            }
            wrow_t wr;
            float wn[V];
            wr.load(w_next, i, D);
            wr.to(wn);
            norm_mul(g, g, wn, 1.f);
            const float dot = row_sum<TPR>(norm_dot(g, n), red, flip) * inv_d;
            norm_axpy(g, -dot, n, g);
            norm_axpy(d, rn, g, d);
        }
        if (dx && live && OSDN_IN_BOUNDS(row, R)) row_t::store(dx + at, i, D, d);
        norm_scale(d, scale);
        // d of the gate: d * (what it multiplies) * act'; act' = s (1 + g (1 - s)) or s (1 - s)
        auto gate_grad = [&](const float (&m)[V]) {
            float g[V], dg[V];
            rg.to(g);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float one = 1.f - s[e];
                const float ds = act == NORM_ACT_SILU ? s[e] * fmaf(g[e], one, 1.f) : s[e] * one;
                dg[e] = d[e] * m[e] * ds;
                d[e] *= factor(g, e);
            }
            if (live && OSDN_IN_BOUNDS(row, R)) row_t::store(dgate + at, i, D, dg);
        };
        if (gate && !gate_first) {
            if (w_post) {
                float m[V];
                norm_mul(m, v, w, 1.f);
                gate_grad(m);
            } else {
                gate_grad(v);
            }
        }
        if (w_post) {
            if (live) {
#pragma unroll
                for (int e = 0; e < V; ++e) dwp[e] = fmaf(d[e], v[e], dwp[e]);
            }
            norm_mul(d, d, w, 1.f);
            const float dot = row_sum<TPR>(norm_dot(d, v), red, flip) * inv_d;
            norm_axpy(d, -dot, v, d);
            norm_scale(d, rs);
        }
        if (gate && gate_first) {
            rf.to(v);
            gate_grad(v);
        }
        if (live && OSDN_IN_BOUNDS(row, R)) row_t::store(df + at, i, D, d);
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
            for (int e = 0; e < V; ++e) red[threadIdx.x * V + e] = dw[e];
            __syncthreads();
            if (threadIdx.x < TPR) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    dw[e] = 0.f;
                    for (int q = 0; q < ROWS; ++q) dw[e] += red[(q * TPR + i) * V + e];
                }
                wrow_t::store(out, i, D, dw);
            }
        } else {
            wrow_t::store(out, i, D, dw);
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
