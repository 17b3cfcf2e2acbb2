// conv.cuh -- the short causal convolution of recurrent layers, one filter per channel:
//   z_t[c] = bias[c] + sum_{w < W} weight[c][w] x_{t - W + 1 + w}[c],   y = z or silu(z),
// where the W - 1 tokens before a sequence are its initial state (or zeros), and its gradient
//   dz = dy act'(z),  dx_p = sum_w weight[w] dz_{p + W - 1 - w},
//   dweight[w] = sum_t dz_t x_{t - W + 1 + w},  dbias = sum_t dz_t.
//
// Every input element is needed W times and every output costs 2 W + a few operations: the
// forward pass is bound by HBM (one read of x, one write of y).  A thread owns V neighbouring
// channels (16 bytes) and walks a strip of consecutive tokens with the last W - 1 inputs in
// registers, so x is read once plus W - 1 rows per strip (which sit in L2).
#pragma once

#include "mixer_common.cuh"

namespace osdn {

constexpr int CONV_THREADS = 128;
template <typename IO> constexpr int CONV_MAX_V = 4;  // channels of a thread
constexpr int CONV_BWD_MAX_V = 2;
constexpr int CONV_UNROLL = 4;  // tokens of a group; the next group's loads are in flight meanwhile

// One row of a sequence at position pos (< 0: a row of the initial state) as fp32.
template <int V, int W, typename IO>
__device__ __forceinline__ void conv_row(const IO* __restrict__ x, const IO* __restrict__ state0,
                                         int n, int64_t a, int64_t pos, int C, int c, float* r) {
    if (pos >= 0) {
        vec_io<V, IO>::load(x + (a + pos) * C + c, r);
    } else if (state0) {
        vec_io<V, IO>::load(state0 + ((int64_t)n * (W - 1) + (W - 1) + pos) * C + c, r);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) r[v] = 0.f;
    }
}

template <int V, int W>
__device__ __forceinline__ void conv_weights(const float* __restrict__ weight,
                                             const float* __restrict__ bias, int c, float (*wt)[V],
                                             float* bs) {
    if constexpr (V > 1 && V * W % 4 == 0) {  // V * W neighbouring floats, 16-byte aligned
        float flat[V * W];
#pragma unroll
        for (int i = 0; i < V * W; i += 4) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(weight + (int64_t)c * W + i));
            flat[i] = f.x; flat[i + 1] = f.y; flat[i + 2] = f.z; flat[i + 3] = f.w;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int w = 0; w < W; ++w) wt[w][v] = flat[v * W + w];
        if (bias) {
            vec_io<V, float>::load(bias + c, bs);
            return;
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int w = 0; w < W; ++w) wt[w][v] = __ldg(weight + (int64_t)(c + v) * W + w);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) bs[v] = bias ? __ldg(bias + c + v) : 0.f;
}

// blockIdx.x: channels; blockIdx.y < strips: a strip of `strip` rows; the blocks behind them
// write one sequence's final state each (the last W - 1 rows of [state0; x], oldest first) and
// check its offsets.
template <int V, int W, typename IO>
__global__ void __launch_bounds__(CONV_THREADS, V * sizeof(IO) == 16 ? 5 : 8)
conv_fwd_kernel(const IO* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, const IO* __restrict__ state0, int silu,
                IO* __restrict__ y, IO* __restrict__ stateT, const int32_t* __restrict__ cu, int N,
                int T, int C, int64_t rows, int strips, int strip) {
    const int c = (blockIdx.x * CONV_THREADS + threadIdx.x) * V;
    if ((int)blockIdx.y >= strips) {
        for (int n = (int)blockIdx.y - strips; n < N; n += (int)gridDim.y - strips) {
            int64_t first, count;
            if (!seq_range(cu, n, N, T, first, count) || !stateT || c >= C) continue;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) {
                float r[V];
                conv_row<V, W>(x, state0, n, first, count - (W - 1) + j, C, c, r);
                if (OSDN_IN_BOUNDS(n, N))
                    vec_io<V, IO>::store(stateT + ((int64_t)n * (W - 1) + j) * C + c, r);
            }
        }
        return;
    }
    if (c >= C) return;
    float wt[W][V], bs[V];
    conv_weights<V, W>(weight, bias, c, wt, bs);
    int64_t row = (int64_t)blockIdx.y * strip;
    const int64_t end = row + strip < rows ? row + strip : rows;
    while (row < end) {
        int n;
        int64_t a, b;
        if (!row_sequence(cu, N, T, row, n, a, b)) { ++row; continue; }
        const int64_t stop = b < end ? b : end;
        float win[W - 1][V];  // the W - 1 inputs before `row`, oldest first
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            conv_row<V, W>(x, state0, n, a, row - a - (W - 1) + j, C, c, win[j]);
        raw_io<V, IO> in[CONV_UNROLL], next[CONV_UNROLL];
#pragma unroll
        for (int u = 0; u < CONV_UNROLL; ++u)
            if (row + u < stop) in[u].load(x + (row + u) * C + c);
#pragma unroll 1
        for (; row < stop; row += CONV_UNROLL) {
#pragma unroll
            for (int u = 0; u < CONV_UNROLL; ++u)
                if (row + CONV_UNROLL + u < stop) next[u].load(x + (row + CONV_UNROLL + u) * C + c);
#pragma unroll
            for (int u = 0; u < CONV_UNROLL; ++u) {
                if (row + u < stop) {
                    float z[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        float s = bs[v];
#pragma unroll
                        for (int w = 0; w < W - 1; ++w) s = fmaf(wt[w][v], win[w][v], s);
                        s = fmaf(wt[W - 1][v], in[u].get(v), s);
                        z[v] = silu ? silu_f(s) : s;
                    }
                    if (OSDN_IN_BOUNDS(row + u, rows))
                        vec_io<V, IO>::store(y + (row + u) * C + c, z);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int w = 0; w + 1 < W - 1; ++w) win[w][v] = win[w + 1][v];
                        win[W - 2][v] = in[u].get(v);
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < CONV_UNROLL; ++u) in[u] = next[u];
        }
        row = stop;
    }
}

// One token per sequence: y from the state and x, the state moved on by one row, in place.
// Bound by HBM for large batches (2 W elements moved per channel), by latency for small ones.
template <int V, int W, typename IO>
__global__ void __launch_bounds__(CONV_THREADS)
conv_step_kernel(const IO* __restrict__ x, const float* __restrict__ weight,
                 const float* __restrict__ bias, IO* __restrict__ state, int silu,
                 IO* __restrict__ y, int N, int C) {
    const int c = (blockIdx.x * CONV_THREADS + threadIdx.x) * V;
    if (c >= C) return;
    for (int n = blockIdx.y; n < N; n += gridDim.y) {
        IO* st = state + (int64_t)n * (W - 1) * C + c;
        float in[W][V], wt[W][V], bs[V], z[V];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) vec_io<V, IO>::load(st + (int64_t)j * C, in[j]);
        vec_io<V, IO>::load(x + (int64_t)n * C + c, in[W - 1]);
        conv_weights<V, W>(weight, bias, c, wt, bs);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = bs[v];
#pragma unroll
            for (int w = 0; w < W; ++w) s = fmaf(wt[w][v], in[w][v], s);
            z[v] = silu ? silu_f(s) : s;
        }
        if (OSDN_IN_BOUNDS(n, N)) {
            vec_io<V, IO>::store(y + (int64_t)n * C + c, z);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) vec_io<V, IO>::store(st + (int64_t)j * C, in[j + 1]);
        }
    }
}

// ---------------------------------------------------------------- backward
// A block is 32 channel lanes (V channels each) x CONV_BWD_STRIPS strips at a time; its partial
// dweight and dbias are summed over the strips it walks in registers, over its rows of threads
// in shared memory, and over the blocks by conv_reduce_kernel, each in a fixed order.
constexpr int CONV_BWD_STRIPS = 8;
constexpr int CONV_BWD_UNROLL = 4;  // tokens loaded before the first is used

template <int V, int W, typename IO, typename GO>
__global__ void __launch_bounds__(32 * CONV_BWD_STRIPS, 3)
conv_bwd_kernel(const IO* __restrict__ x, const float* __restrict__ weight,
                const float* __restrict__ bias, const IO* __restrict__ state0, int silu,
                const GO* __restrict__ dy, const float* __restrict__ dstateT, IO* __restrict__ dx,
                float* __restrict__ dstate0, float* __restrict__ part,
                const int32_t* __restrict__ cu, int N, int T, int C, int64_t rows, int row_blocks,
                int strip) {
    __shared__ float red[CONV_BWD_STRIPS][32][V];
    const int c = (blockIdx.x * 32 + threadIdx.x) * V;
    const bool on = c < C;
    if ((int)blockIdx.y >= row_blocks) {  // offsets of every sequence, and the empty ones' states
        const int per = ((int)gridDim.y - row_blocks) * CONV_BWD_STRIPS;
        for (int n = ((int)blockIdx.y - row_blocks) * CONV_BWD_STRIPS + threadIdx.y; n < N;
             n += per) {
            int64_t first, count;
            if (!seq_range(cu, n, N, T, first, count) || count > 0 || !dstate0 || !on) continue;
            for (int j = 0; j < W - 1; ++j) {
                float r[V];
                const int64_t at = ((int64_t)n * (W - 1) + j) * C + c;
#pragma unroll
                for (int v = 0; v < V; ++v) r[v] = dstateT ? dstateT[at + v] : 0.f;
                if (OSDN_IN_BOUNDS(n, N)) vec_io<V, float>::store(dstate0 + at, r);
            }
        }
        return;
    }
    float wt[W][V], bs[V], dw[W][V], db[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) dw[w][v] = 0.f;
    }
    if (on) {
        conv_weights<V, W>(weight, bias, c, wt, bs);
        const int64_t hop = (int64_t)row_blocks * CONV_BWD_STRIPS * strip;
        for (int64_t s0 = ((int64_t)blockIdx.y * CONV_BWD_STRIPS + threadIdx.y) * strip; s0 < rows;
             s0 += hop) {
            int64_t row = s0;
            const int64_t end = s0 + strip < rows ? s0 + strip : rows;
            while (row < end) {
                int n;
                int64_t a, b;
                if (!row_sequence(cu, N, T, row, n, a, b)) { ++row; continue; }
                const int64_t p0 = row, p1 = b < end ? b : end, len = b - a;
                float win[W][V], dz[W][V];  // x and dz of the last W tokens, oldest first
#pragma unroll
                for (int j = 0; j < W - 1; ++j)
                    conv_row<V, W>(x, state0, n, a, p0 - a - (W - 1) + j, C, c, win[j + 1]);
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) dz[j][v] = 0.f;
                // dz_t from x and dy, then dx_{t - W + 1}, whose last contribution dz_t is
#pragma unroll 1
                for (int64_t t0 = p0; t0 < p1 + W - 1; t0 += CONV_BWD_UNROLL) {
                    raw_io<V, IO> in[CONV_BWD_UNROLL];
                    raw_io<V, GO> g[CONV_BWD_UNROLL];
#pragma unroll
                    for (int u = 0; u < CONV_BWD_UNROLL; ++u)
                        if (t0 + u < p1 + W - 1 && t0 + u < b) {
                            in[u].load(x + (t0 + u) * C + c);
                            g[u].load(dy + (t0 + u) * C + c);
                        }
#pragma unroll
                    for (int u = 0; u < CONV_BWD_UNROLL; ++u) {
                        const int64_t t = t0 + u;
                        if (t >= p1 + W - 1) break;
                        const bool live = t < b;
#pragma unroll
                        for (int v = 0; v < V; ++v) {
#pragma unroll
                            for (int w = 0; w < W - 1; ++w) {
                                win[w][v] = win[w + 1][v];
                                dz[w][v] = dz[w + 1][v];
                            }
                            win[W - 1][v] = live ? in[u].get(v) : 0.f;
                            float d = 0.f;
                            if (live) {
                                d = g[u].get(v);
                                if (silu) {
                                    float z = bs[v];
#pragma unroll
                                    for (int w = 0; w < W; ++w) z = fmaf(wt[w][v], win[w][v], z);
                                    d *= silu_grad_f(z);
                                }
                                if (t < p1) {
                                    db[v] += d;
#pragma unroll
                                    for (int w = 0; w < W; ++w)
                                        dw[w][v] = fmaf(d, win[w][v], dw[w][v]);
                                }
                            }
                            dz[W - 1][v] = d;
                        }
                        const int64_t p = t - (W - 1);  // dz[w] is dz_{p + w}
                        if (p < p0 && (p0 > a || !dstate0)) continue;
                        float r[V];
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            r[v] = 0.f;
#pragma unroll
                            for (int w = 0; w < W; ++w) r[v] = fmaf(wt[W - 1 - w][v], dz[w][v], r[v]);
                        }
                        const int64_t j = p - a - len + (W - 1);  // p's row of the final state
                        if (dstateT && j >= 0) {
                            const float* e = dstateT + ((int64_t)n * (W - 1) + j) * C + c;
#pragma unroll
                            for (int v = 0; v < V; ++v) r[v] += e[v];
                        }
                        if (p >= p0) {
                            if (OSDN_IN_BOUNDS(p, rows)) vec_io<V, IO>::store(dx + p * C + c, r);
                        } else if (OSDN_IN_BOUNDS(n, N)) {
                            vec_io<V, float>::store(
                                dstate0 + ((int64_t)n * (W - 1) + (p - a) + (W - 1)) * C + c, r);
                        }
                    }
                }
                row = p1;
            }
        }
    }
    // [W + 1][C] partial sums of this block
    for (int w = 0; w <= W; ++w) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = db[v];
#pragma unroll
            for (int k = 0; k < W; ++k) s = w == k ? dw[k][v] : s;
            red[threadIdx.y][threadIdx.x][v] = s;
        }
        __syncthreads();
        if (threadIdx.y == 0 && on) {
            float s[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                s[v] = 0.f;
#pragma unroll
                for (int k = 0; k < CONV_BWD_STRIPS; ++k) s[v] += red[k][threadIdx.x][v];
            }
            if (OSDN_IN_BOUNDS(blockIdx.y, row_blocks))
                vec_io<V, float>::store(part + ((int64_t)blockIdx.y * (W + 1) + w) * C + c, s);
        }
        __syncthreads();
    }
}

// dweight[c][w] and dbias[c] from the blocks' partial sums, [row_blocks][W + 1][C]; a warp per
// 32 channels and row w, its block's warps sharing the row blocks.
constexpr int CONV_RED_WARPS = 8;
__global__ void __launch_bounds__(32 * CONV_RED_WARPS)
conv_reduce_kernel(const float* __restrict__ part, int row_blocks, int W, int C,
                   float* __restrict__ dweight, float* __restrict__ dbias) {
    __shared__ float red[CONV_RED_WARPS][32];
    const int c = blockIdx.x * 32 + threadIdx.x, w = blockIdx.y;
    float s = 0.f;
    if (c < C)
        for (int k = threadIdx.y; k < row_blocks; k += CONV_RED_WARPS)
            s += part[((int64_t)k * (W + 1) + w) * C + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < C) {
#pragma unroll
        for (int k = 1; k < CONV_RED_WARPS; ++k) s += red[k][threadIdx.x];
        if (w < W) {
            if (OSDN_IN_BOUNDS((int64_t)c * W + w, (int64_t)C * W)) dweight[(int64_t)c * W + w] = s;
        } else if (dbias) {
            dbias[c] = s;
        }
    }
}

}  // namespace osdn
