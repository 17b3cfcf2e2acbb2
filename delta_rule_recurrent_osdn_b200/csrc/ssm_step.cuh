// ssm_step.cuh -- one token of the selective scan per (sequence, head): the decode path,
//   step = softplus(dt + dt_bias),  S <- exp(step A) S + step x b^T,  y = S c + D x,
// with the state [Dv][Dk] in HBM, read and written once.  Bound by HBM bandwidth: the state is
// 2 x 4 Dk Dv bytes per (sequence, head) and everything else a few hundred.
//
// One CTA of Dv / 8 warps per (sequence, head).  A warp owns 8 state rows, a lane Dk / 32
// neighbouring columns of each; all 8 row loads are issued before the first use.  256 sequences x
// 16 heads of 128 x 128: 83 us, 539 MB at 99% of copy speed.
#pragma once

#include "mixer_common.cuh"

namespace osdn {

template <int DK, int DV, typename IO>
__global__ void __launch_bounds__(DV * 4)
ssm_step_kernel(const IO* __restrict__ x, const float* __restrict__ dt,
                const float* __restrict__ A, const IO* __restrict__ b, const IO* __restrict__ c,
                const float* __restrict__ D, const float* __restrict__ dt_bias, int softplus,
                float* __restrict__ S, IO* __restrict__ y, int64_t NH, int H, int G) {
    constexpr int PL = DK / 32, ROWS = 8, NW = DV / 8;
    const int64_t nh = blockIdx.x;
    const int64_t n = nh / H;
    const int h = (int)(nh - n * H), g = h / (H / G);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* Sh = S + nh * DV * DK + PL * lane;
    float s[ROWS][PL];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float* p = Sh + (int64_t)(warp + NW * i) * DK;
        if constexpr (PL == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            s[i][0] = v.x; s[i][1] = v.y; s[i][2] = v.z; s[i][3] = v.w;
        } else {
            const float2 v = *reinterpret_cast<const float2*>(p);
            s[i][0] = v.x; s[i][1] = v.y;
        }
    }
    float bb[PL], cc[PL];
#pragma unroll
    for (int j = 0; j < PL; j += 2) {
        const float2 u = load2<IO>(b + (n * G + g) * DK + PL * lane + j);
        const float2 w = load2<IO>(c + (n * G + g) * DK + PL * lane + j);
        bb[j] = u.x; bb[j + 1] = u.y;
        cc[j] = w.x; cc[j + 1] = w.y;
    }
    const float step = scan_step(dt[nh] + (dt_bias ? dt_bias[h] : 0.f), softplus);
    const float a = expf(step * A[h]);
    const float skip = D ? D[h] : 0.f;
    // rows warp + NW i: lane i of the first 8 holds row i's x
    const float xr = lane < ROWS ? io_traits<IO>::to_f32(x[nh * DV + warp + NW * lane]) : 0.f;
    float yr = 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float u = step * __shfl_sync(0xffffffffu, xr, i);
        float acc = 0.f;
#pragma unroll
        for (int j = 0; j < PL; ++j) {
            s[i][j] = fmaf(a, s[i][j], u * bb[j]);
            acc = fmaf(s[i][j], cc[j], acc);
        }
        float* p = Sh + (int64_t)(warp + NW * i) * DK;
        if (OSDN_IN_BOUNDS(nh, NH)) {
            if constexpr (PL == 4)
                *reinterpret_cast<float4*>(p) = make_float4(s[i][0], s[i][1], s[i][2], s[i][3]);
            else
                *reinterpret_cast<float2*>(p) = make_float2(s[i][0], s[i][1]);
        }
        acc = warp_sum_f(acc);
        if (lane == i) yr = acc;
    }
    if (lane < ROWS && OSDN_IN_BOUNDS(nh, NH))
        y[nh * DV + warp + NW * lane] = io_traits<IO>::from_f32(fmaf(skip, xr, yr));
}

}  // namespace osdn
