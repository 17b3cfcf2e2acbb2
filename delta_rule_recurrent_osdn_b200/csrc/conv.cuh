// conv.cuh -- the short causal convolution of recurrent layers, one filter per channel:
//   z_t[c] = bias[c] + sum_{w < W} weight[c][w] x_{t - W + 1 + w}[c],   y = z or silu(z),
// where the W - 1 tokens before a sequence are its initial state (or zeros), and its gradient
//   dz = dy act'(z),  dx_p = sum_w weight[w] dz_{p + W - 1 - w},
//   dweight[w] = sum_t dz_t x_{t - W + 1 + w},  dbias = sum_t dz_t.
//
// Every input element is needed W times and every output costs 2 W + a few operations (silu: an
// exponential and a quotient).  A thread owns V neighbouring channels, as pairs per instruction,
// and walks a strip of consecutive tokens with the last W - 1 inputs in registers, so x is read
// once plus W - 1 rows per strip (which sit in L2), the next four tokens' loads in flight.
// 31 us at 4 x 4096 tokens of 2048 bf16 channels (134 MB: 20.5 us at copy speed): too few warps wait,
// no unit is full.  14 instructions issued a value take 46% of the schedulers' slots, and of the 11
// cycles between two of a warp's instructions 2.3 are waits for loads, 1.9 for the queue of the special
// functions (silu's exponential and quotient) and 1.9 for fixed latencies, with 5 warps a scheduler.
// The gradient takes 43 us at 8 x 2048 tokens of 1024 channels (101 MB: 15.4 us), 37 of them in the
// kernel: 27 instructions a value take 39% of the slots, and of a warp's 9.8 cycles 3.8 are waits for
// loads.  Its 128 registers leave 16 warps an SM, and with W = 4 some are spilled (24 bytes with bf16
// tokens, 48 with fp32 dy, 120 with fp32 tokens).  The sum of the partial rows takes the rest.
#pragma once

#include "mixer_common.cuh"

namespace osdn {

constexpr int CONV_THREADS = 128;
constexpr int CONV_MAX_C = 1 << 30;  // a channel's number, rounded up to whole blocks, is an int
// Channels of a thread.  With 8 (16 bytes of bf16) the filters, the last inputs and the loads in
// flight leave too few warps: 4 x 4096 tokens of 2048 channels 57 us against 34, the gradient at
// 8 x 2048 of 1024 115 against 47 (L2 cold).
constexpr int CONV_MAX_V = 4;
constexpr int CONV_BWD_MAX_V = 4;
// resident blocks of the forward kernel on an SM, by the bytes of a thread's access
constexpr int conv_per_sm(int bytes) { return bytes == 16 ? 5 : 7; }
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
                                             const float* __restrict__ bias, int c, fvec<V>* wt,
                                             fvec<V>& bs) {
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
            vec_io<V, float>::load(bias + c, bs.x);
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
__global__ void __launch_bounds__(CONV_THREADS, conv_per_sm(V * sizeof(IO)))
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
    fvec<V> wt[W], bs;
    conv_weights<V, W>(weight, bias, c, wt, bs);
    int64_t row = (int64_t)blockIdx.y * strip;
    const int64_t end = row + strip < rows ? row + strip : rows;
    while (row < end) {
        int n;
        int64_t a, b;
        if (!row_sequence(cu, N, T, row, n, a, b)) { ++row; continue; }
        const int64_t stop = b < end ? b : end;
        constexpr int U = CONV_UNROLL;
        fvec<V> win[W - 1 + U];  // the W - 1 inputs before a group of tokens, oldest first, then it
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            conv_row<V, W>(x, state0, n, a, row - a - (W - 1) + j, C, c, win[j].x);
        int left = (int)(stop - row);
        const IO* px = x + row * C + c;
        IO* py = y + row * C + c;
        raw_io<V, IO> in[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (u < left) in[u].load(px + (int64_t)u * C);
#pragma unroll 1
        for (; left > 0; left -= U) {
#pragma unroll
            for (int u = 0; u < U; ++u) in[u].to(win[W - 1 + u].x);
            px += (int64_t)U * C;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (U + u < left) in[u].load(px + (int64_t)u * C);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                fvec<V> z = bs;
#pragma unroll
                for (int w = 0; w < W; ++w) z = fma_v(wt[w], win[u + w], z);
                if (silu) {
#pragma unroll
                    for (int v = 0; v < V; ++v) z[v] = silu_f(z[v]);
                }
                if (u < left && OSDN_IN_BOUNDS(stop - left + u, rows))
                    vec_io<V, IO>::store(py + (int64_t)u * C, z.x);
            }
            py += (int64_t)U * C;
#pragma unroll
            for (int j = 0; j < W - 1; ++j) win[j] = win[U + j];
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
        fvec<V> in[W], wt[W], bs;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) vec_io<V, IO>::load(st + (int64_t)j * C, in[j].x);
        vec_io<V, IO>::load(x + (int64_t)n * C + c, in[W - 1].x);
        conv_weights<V, W>(weight, bias, c, wt, bs);
        fvec<V> z = bs;
#pragma unroll
        for (int w = 0; w < W; ++w) z = fma_v(wt[w], in[w], z);
        if (silu) {
#pragma unroll
            for (int v = 0; v < V; ++v) z[v] = silu_f(z[v]);
        }
        if (OSDN_IN_BOUNDS(n, N)) {
            vec_io<V, IO>::store(y + (int64_t)n * C + c, z.x);
#pragma unroll
            for (int j = 0; j < W - 1; ++j) vec_io<V, IO>::store(st + (int64_t)j * C, in[j + 1].x);
        }
    }
}

// ---------------------------------------------------------------- backward
// A block is 32 channel lanes (V channels each) x CONV_BWD_STRIPS strips at a time; its partial
// dweight and dbias are summed over the strips it walks in registers, over its rows of threads
// in shared memory, and over the blocks by conv_reduce_kernel, each in a fixed order.
constexpr int CONV_BWD_STRIPS = 4, CONV_BWD_PER_SM = 4;
constexpr int CONV_BWD_UNROLL = 4;  // tokens loaded before the first is used

template <int V, int W, typename IO, typename GO>
__global__ void __launch_bounds__(32 * CONV_BWD_STRIPS, CONV_BWD_PER_SM)
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
    fvec<V> wt[W], bs, dw[W], db = zero_v<V>();
#pragma unroll
    for (int w = 0; w < W; ++w) dw[w] = zero_v<V>();
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
                constexpr int U = CONV_BWD_UNROLL;
                // x and dz of the last W - 1 tokens, oldest first, then a group's
                fvec<V> win[W - 1 + U], dz[W - 1 + U];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    conv_row<V, W>(x, state0, n, a, p0 - a - (W - 1) + j, C, c, win[j].x);
                    dz[j] = zero_v<V>();
                }
                // dz_t of token u of a group
                auto grad = [&](int u, const raw_io<V, GO>& g) {
                    fvec<V> d;
                    g.to(d.x);
                    if (silu) {
                        fvec<V> z = bs;
#pragma unroll
                        for (int w = 0; w < W; ++w) z = fma_v(wt[w], win[u + w], z);
#pragma unroll
                        for (int v = 0; v < V; ++v) d[v] *= silu_grad_f(z[v]);
                    }
                    dz[W - 1 + u] = d;
                };
                auto sums = [&](int u) {
                    db = add_v(db, dz[W - 1 + u]);
#pragma unroll
                    for (int w = 0; w < W; ++w) dw[w] = fma_v(dz[W - 1 + u], win[u + w], dw[w]);
                };
                // dx_p, p = t - (W - 1), whose last contribution dz_t is: dz[u + w] is dz_{p + w}
                auto give = [&](int u) {
                    fvec<V> r = zero_v<V>();
#pragma unroll
                    for (int w = 0; w < W; ++w) r = fma_v(wt[W - 1 - w], dz[u + w], r);
                    return r;
                };
                auto shift = [&](int k) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j] = k == 1 ? win[j + 1] : win[j + U];
                        dz[j] = k == 1 ? dz[j + 1] : dz[j + U];
                    }
                };
                // one token near a piece's ends: before its first own dx is complete (t < p0 + W - 1;
                // what is complete there belongs to the initial state or to the piece before), or
                // behind its last token (dz of the next piece's tokens again, 0 behind the sequence)
                auto edge = [&](int64_t t) {
                    const bool live = t < b;
                    win[W - 1] = zero_v<V>();
                    dz[W - 1] = zero_v<V>();
                    if (live) {
                        raw_io<V, IO> i;
                        raw_io<V, GO> g;
                        i.load(x + t * C + c);
                        g.load(dy + t * C + c);
                        i.to(win[W - 1].x);
                        grad(0, g);
                        if (t < p1) sums(0);
                    }
                    const int64_t p = t - (W - 1);
                    if (p >= p0 || (p0 == a && dstate0)) {
                        fvec<V> r = give(0);
                        const int64_t j = p - a - len + (W - 1);  // p's row of the final state
                        if (dstateT && j >= 0) {
                            const float* e = dstateT + ((int64_t)n * (W - 1) + j) * C + c;
#pragma unroll
                            for (int v = 0; v < V; ++v) r[v] += e[v];
                        }
                        if (p >= p0) {
                            if (OSDN_IN_BOUNDS(p, rows)) vec_io<V, IO>::store(dx + p * C + c, r.x);
                        } else if (OSDN_IN_BOUNDS(n, N)) {
                            vec_io<V, float>::store(
                                dstate0 + ((int64_t)n * (W - 1) + (p - a) + (W - 1)) * C + c, r.x);
                        }
                    }
                    shift(1);
                };
                int64_t t = p0;
#pragma unroll 1
                for (; t < p0 + W - 1 && t < p1; ++t) edge(t);
                int groups = (int)((p1 - t) / U);
                raw_io<V, IO> in[U];
                raw_io<V, GO> g[U];
                const IO* px = x + t * C + c;
                const GO* pg = dy + t * C + c;
                IO* po = dx + (t - (W - 1)) * C + c;
                if (groups > 0) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        in[u].load(px + (int64_t)u * C);
                        g[u].load(pg + (int64_t)u * C);
                    }
                }
                t += (int64_t)groups * U;
#pragma unroll 1
                for (; groups > 0; --groups) {
                    px += (int64_t)U * C;
                    pg += (int64_t)U * C;
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        in[u].to(win[W - 1 + u].x);
                        grad(u, g[u]);
                        if (groups > 1) {  // the next group's, in flight from here
                            in[u].load(px + (int64_t)u * C);
                            g[u].load(pg + (int64_t)u * C);
                        }
                        sums(u);
                        const fvec<V> r = give(u);
                        if (OSDN_IN_BOUNDS(p1 - 1, rows)) vec_io<V, IO>::store(po + (int64_t)u * C, r.x);
                    }
                    po += (int64_t)U * C;
                    shift(U);
                }
#pragma unroll 1
                for (; t < p1 + W - 1; ++t) edge(t);
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
