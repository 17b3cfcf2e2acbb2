// mixer_common.cuh -- helpers shared by the layer operators around the token mixer (short
// convolution, selective scan, block norm): vectors of io elements, SiLU, softplus, and the
// sequence that holds a row of a packed batch.
#pragma once

#include <math_constants.h>

#include "common.cuh"

namespace osdn {

// V consecutive io elements <-> fp32 registers, as accesses of up to 16 bytes (V * sizeof(IO)
// bytes, at least 16 at a time where V allows it).  V == 1 makes no assumption on alignment.
template <int V, typename IO> struct vec_io {
    static_assert(V % 4 == 0, "vectors of 4 or 8 elements (2 and 1 below)");
    static __device__ __forceinline__ void load(const IO* p, float* x) {
        if constexpr (V == 8 && sizeof(IO) == 2) {
            const uint4 r = __ldg(reinterpret_cast<const uint4*>(p));
            const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = load4<IO>(p + i);
                x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
            }
        }
    }
    static __device__ __forceinline__ void store(IO* p, const float* x) {
        if constexpr (V == 8 && sizeof(IO) == 2) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t*>(&b);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < V; i += 4)
                store4<IO>(p + i, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
        }
    }
};
template <typename IO> struct vec_io<2, IO> {
    static __device__ __forceinline__ void load(const IO* p, float* x) {
        const float2 v = load2<IO>(p);
        x[0] = v.x; x[1] = v.y;
    }
    static __device__ __forceinline__ void store(IO* p, const float* x) {
        store2<IO>(p, make_float2(x[0], x[1]));
    }
};
template <typename IO> struct vec_io<1, IO> {
    static __device__ __forceinline__ void load(const IO* p, float* x) {
        x[0] = io_traits<IO>::to_f32(*p);
    }
    static __device__ __forceinline__ void store(IO* p, const float* x) {
        *p = io_traits<IO>::from_f32(x[0]);
    }
};

// V consecutive io elements as they lie in memory: loads that are in flight hold half (bf16) the
// registers of their fp32 values.
template <int V, typename IO> struct raw_io {
    static constexpr int WORDS = V * (int)sizeof(IO) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const IO* p) {
        if constexpr (WORDS >= 4) {
#pragma unroll
            for (int i = 0; i < WORDS; i += 4) {
                const uint4 r = __ldg(reinterpret_cast<const uint4*>(p) + i / 4);
                w[i] = r.x; w[i + 1] = r.y; w[i + 2] = r.z; w[i + 3] = r.w;
            }
        } else if constexpr (WORDS == 1) {
            w[0] = __ldg(reinterpret_cast<const unsigned int*>(p));
        } else {
            static_assert(WORDS == 2, "4, 8 or 16 bytes");
            const uint2 r = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = r.x; w[1] = r.y;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(IO) == 4) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
    __device__ __forceinline__ void to(float* x) const {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = get(i);
    }
};
template <typename IO> struct raw_io<1, IO> {
    IO v;
    __device__ __forceinline__ void load(const IO* p) { v = *p; }
    __device__ __forceinline__ float get(int) const { return io_traits<IO>::to_f32(v); }
    __device__ __forceinline__ void to(float* x) const { x[0] = get(0); }
};

// V fp32 values; products and sums two at a time (one instruction per pair).
template <int V> struct fvec {
    float x[V];
    __device__ __forceinline__ float operator[](int i) const { return x[i]; }
    __device__ __forceinline__ float& operator[](int i) { return x[i]; }
};
template <int V> __device__ __forceinline__ fvec<V> fma_v(const fvec<V>& a, const fvec<V>& b, const fvec<V>& c) {
    fvec<V> r;
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = __ffma2_rn(make_float2(a.x[i], a.x[i + 1]), make_float2(b.x[i], b.x[i + 1]),
                                        make_float2(c.x[i], c.x[i + 1]));
            r.x[i] = t.x;
            r.x[i + 1] = t.y;
        }
    } else {
        r.x[0] = fmaf(a.x[0], b.x[0], c.x[0]);
    }
    return r;
}
template <int V> __device__ __forceinline__ fvec<V> add_v(const fvec<V>& a, const fvec<V>& b) {
    fvec<V> r;
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 t = __fadd2_rn(make_float2(a.x[i], a.x[i + 1]), make_float2(b.x[i], b.x[i + 1]));
            r.x[i] = t.x;
            r.x[i + 1] = t.y;
        }
    } else {
        r.x[0] = a.x[0] + b.x[0];
    }
    return r;
}
template <int V> __device__ __forceinline__ fvec<V> zero_v() {
    fvec<V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.x[i] = 0.f;
    return r;
}

// 2^x and 1 / x, each one instruction, good to about 2^-22 (subnormal results are 0).
__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcpf(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + e^-z).  e^-z overflows to inf for z < -88, where the quotient is 0 as it should be.
__device__ __forceinline__ float sigmoid_f(float z) { return rcpf(1.f + ex2f(z * -1.4426950408889634f)); }
__device__ __forceinline__ float silu_f(float z) { return z * sigmoid_f(z); }
// d silu(z) / dz = s (1 + z (1 - s)), s = sigmoid(z)
__device__ __forceinline__ float silu_grad_f(float z) {
    const float s = sigmoid_f(z);
    return s * fmaf(z, 1.f - s, 1.f);
}

// The token step of the scan: softplus(raw) = max(raw, 0) + log(1 + e^-|raw|) (which neither
// overflows nor loses small steps), or raw itself.
__device__ __forceinline__ float scan_step(float raw, int softplus) {
    return softplus ? fmaxf(raw, 0.f) + log1pf(expf(-fabsf(raw))) : raw;
}

__device__ __forceinline__ float warp_sum_f(float x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
}

// The sequence that holds row `row` of the [B * T] token rows, and its token range [a, b).
// Packed offsets are searched by bisection; the range found is checked like seq_range's, so
// offsets that are out of order give false for the rows they do not describe (the caller skips
// the row; the error is recorded where every sequence's offsets are checked).
__device__ __forceinline__ bool row_sequence(const int32_t* __restrict__ cu, int N, int T,
                                             int64_t row, int& n, int64_t& a, int64_t& b) {
    if (cu == nullptr) {
        n = (int)(row / T);
        a = (int64_t)n * T;
        b = a + T;
        return true;
    }
    int lo = 0, hi = N;  // the first n with cu[n + 1] > row
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)__ldg(cu + mid + 1) > row) hi = mid; else lo = mid + 1;
    }
    if (lo >= N) return false;
    n = lo;
    a = __ldg(cu + n);
    b = __ldg(cu + n + 1);
    return a >= 0 && a <= row && row < b && b <= T;
}

// Blocks of `len` tokens of all sequences are numbered so that sequence n's start at
// first / len + n: no two share a number, some have none.  The sequence and the block in it that
// `number` may stand for; false if none (the caller checks the block against the length).
__device__ __forceinline__ bool token_block(const int32_t* __restrict__ cu, int N, int T, int len,
                                            int64_t number, int& n, int& block) {
    int lo = 0, hi = N - 1;  // the last n whose numbers start at or before this one
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int64_t first = cu ? (int64_t)__ldg(cu + mid) : (int64_t)mid * T;
        if (first / len + mid <= number) lo = mid; else hi = mid - 1;
    }
    const int64_t first = cu ? (int64_t)__ldg(cu + lo) : (int64_t)lo * T;
    n = lo;
    block = (int)(number - (first / len + lo));
    return block >= 0;
}

}  // namespace osdn
