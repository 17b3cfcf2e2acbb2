// ssm_scan.cuh -- the selective state-space scan and its gradient, token by token in fp32.
//
// Per (sequence, head), with step_t = softplus(dt_t + dt_bias), a_t = exp(step_t A):
//   S_t = a_t S_{t-1} + step_t x_t b_t^T,    y_t = S_t c_t + D x_t.
// As a map of three token streams, y = F(c, b, step x) with
//   F(q, k, v)_i = sum_{j <= i} (prod_{j < s <= i} a_s) (q_i . k_j) v_j  + (decayed S_0) q_i,
// and the gradient is the same map three more times:
//   dc = F(dy, x, step b) with the transposed state (forward in time),
//   dx = step F'(b, c, dy) + D dy,  db = step F'(x, dy, c)  with F' = F in reverse time,
//        R_j = k_j v_j^T summed over i >= j with decay prod_{j < s <= i} a_s, carry a_j R_j.
// For the steps: with pos_i = c_i . dc_i and neg_j = b_j . db_j (the head's own share of dc, db),
//   d(log a_t) = sum_{i >= t} pos_i - sum_{j >= t} neg_j + <G, S>,
// the sums running to the end of t's block of SSM_BLOCK tokens and <G, S> taken there between
// the state S and the gradient G that reaches it from later tokens (so nothing is summed over
// more than a block: the two sums nearly cancel over long stretches), and
//   dstep_t = x_t . (dx_t - D dy_t) / step_t + A d(log a_t)   (the quotient is formed unscaled).
//
// One kernel serves all four: a CTA holds 32 rows of the state (DV channels of v) in registers,
// 4 threads a row, each with DQ / 4 columns, and walks the tokens; tiles of q, k, v are staged in
// shared memory, the loads of the tile after the next in flight while one is used.  3 fp32
// operations per state element and token (2 packed FMA-pipe instructions per 2 elements) against
// 16 bytes of shared memory per 8: bound by FMA issue and, for few (sequence, head) pairs, by the
// chain of tokens (a warp alone on its scheduler takes 0.2 us a token).  So when there are few
// chains, sequences are cut into segments that run side by side: a first launch (SEG) makes what
// each segment adds to a zero state, and a segment starts from S_in and those in front of it (in
// its own direction).  7 packed sequences of up to 1000 tokens, 4 heads: 37 us, 209 uncut; the
// gradient 130, 562 uncut.
#pragma once

#include <limits.h>

#include "mixer_common.cuh"

namespace osdn {

constexpr int SSM_TT = 16;        // tokens per staged tile
constexpr int SSM_BV = 32;        // state rows per CTA
constexpr int SSM_THREADS = 128;
constexpr int SSM_BLOCK = 64;     // tokens between two restarts of the step gradient's sums

enum { SSM_FWD = 0, SSM_DC = 1, SSM_DX = 2, SSM_DB = 3 };

struct SsmArgs {
    const float *q, *k, *v;       // streams [rows][heads][.]
    const float *dt, *A, *D, *dt_bias;
    const float *S_in;            // FWD, DC: S0; DX, DB: dST; may be null
    float* out;                   // FWD: y, DX: dx; DC, DB: per head [rows][H][DV]
    float* S_out;                 // FWD: ST, DX: dS0; may be null
    float* ckpt;                  // DC writes, DB reads: S behind each block [slot][H][DV][DQ]
    float* gs;                    // DB: <G, S> behind each block [DV / 32][slot][H]
    float* vk;                    // DC: dy . x per token [H][rows], or null
    float* seg_state;             // SEG writes, the others read: [number][H][DV][DQ]
    float* seg_decay;             // [number][H]
    int seg;                      // tokens of a segment, a multiple of SSM_BLOCK (INT_MAX: none)
    const int32_t* cu;
    int64_t rows;
    int N, T, H, G, softplus;
};

// Blocks of SSM_BLOCK tokens of all sequences are numbered so that sequence n's start at
// first / SSM_BLOCK + n: no two share a number, and rows / SSM_BLOCK + N + 1 numbers suffice.
__host__ __device__ __forceinline__ int64_t ssm_slots(int64_t rows, int64_t N, int block) {
    return rows / block + N + 1;
}

template <int DQ, int DV, int MODE, bool SEG>
__global__ void __launch_bounds__(SSM_THREADS)
ssm_scan_kernel(const SsmArgs p) {
    constexpr bool REV = MODE == SSM_DX || MODE == SSM_DB;   // reverse time
    constexpr bool TRANS = MODE == SSM_DC || MODE == SSM_DB; // state rows are key channels
    constexpr int NF = DQ / 16;                              // float4 per thread and state row
    constexpr int LQ = SSM_TT * DQ / 4 / SSM_THREADS;        // float4 of q (k) a thread stages
    // two tiles: one is worked on while the next is written; gates of 8 tiles at a time
    __shared__ float4 qb[2][SSM_TT][DQ / 4], kb[2][SSM_TT][DQ / 4];
    __shared__ float vb[2][SSM_TT][SSM_BV], ob[2][SSM_TT][SSM_BV];
    __shared__ float ab[2][SSM_THREADS], sb[2][SSM_THREADS];
    __shared__ float part[SSM_THREADS / 32];

    constexpr int NSL = DV / SSM_BV;
    const int slice = blockIdx.x % NSL;
    const int64_t number = blockIdx.x / NSL / p.H;
    const int h = (int)(blockIdx.x / NSL - number * p.H);
    int n, part_of;
    int64_t first, count;
    // every sequence's offsets are checked here, whether or not a number leads to it
    if (number < p.N && !seq_range(p.cu, (int)number, p.N, p.T, first, count) && p.seg == INT_MAX) return;
    if (!token_block(p.cu, p.N, p.T, p.seg, number, n, part_of) ||
        !seq_range(p.cu, n, p.N, p.T, first, count))
        return;
    const int64_t nh = (int64_t)n * p.H + h, seq_first = first;
    const int64_t begin = (int64_t)part_of * p.seg;  // of the segment in its sequence
    if (part_of > 0 && begin >= count) return;       // a number that no segment has
    const int64_t parts = count > 0 ? (count + p.seg - 1) / p.seg : 1;
    // the segment that a direction ends with adds to no other
    if (SEG && part_of == (REV ? 0 : parts - 1)) return;
    const bool ends = part_of == (REV ? 0 : parts - 1);
    first += begin;                                  // all uniform over the CTA
    count = count - begin < p.seg ? count - begin : p.seg;
    const int g = h / (p.H / p.G);
    // heads of the streams: FWD q = c, k = b, v = x; DC q = dy, k = x, v = b; DX q = b, k = c,
    // v = dy; DB q = x, k = dy, v = c.  b and c have G heads, x and dy H.
    const int qh = TRANS ? p.H : p.G, vh = TRANS ? p.G : p.H;
    const int64_t qstride = (int64_t)qh * DQ, vstride = (int64_t)vh * DV;
    const float* q = p.q + (TRANS ? h : g) * DQ;
    const float* k = p.k + (TRANS ? h : g) * DQ;
    const float* v = p.v + (TRANS ? g : h) * DV + slice * SSM_BV;
    const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
    const float skip = !TRANS && p.D ? p.D[h] : 0.f;

    const int tid = threadIdx.x, row = tid >> 2, quarter = tid & 3;
    const int vrow = slice * SSM_BV + row;
    float2 S[2 * NF];
    const int64_t sbase = nh * DV * DQ;
#pragma unroll
    for (int j = 0; j < NF; ++j) {
        const int col = (4 * j + quarter) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        if (!SEG && p.S_in) {
            if constexpr (TRANS) {
                const float* e = p.S_in + sbase + vrow;  // stored [DQ][DV]
                s = make_float4(e[(int64_t)col * DV], e[(int64_t)(col + 1) * DV],
                                e[(int64_t)(col + 2) * DV], e[(int64_t)(col + 3) * DV]);
            } else {
                s = *reinterpret_cast<const float4*>(p.S_in + sbase + (int64_t)vrow * DQ + col);
            }
        }
        S[2 * j] = make_float2(s.x, s.y);
        S[2 * j + 1] = make_float2(s.z, s.w);
    }

    if constexpr (!SEG) {  // the segments in front, in this direction
        for (int64_t e = REV ? parts - 1 : 0; REV ? e > part_of : e < part_of; e += REV ? -1 : 1) {
            const int64_t at = (number - part_of + e) * p.H + h;
            const float d = p.seg_decay[at];
            const float* a = p.seg_state + (at * DV + vrow) * DQ;
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const float4 s = *reinterpret_cast<const float4*>(a + (4 * j + quarter) * 4);
                S[2 * j] = __ffma2_rn(make_float2(d, d), S[2 * j], make_float2(s.x, s.y));
                S[2 * j + 1] = __ffma2_rn(make_float2(d, d), S[2 * j + 1], make_float2(s.z, s.w));
            }
        }
    }
    float whole = 1.f;  // SEG: the decay of all tokens so far
    const int64_t ntile = (count + SSM_TT - 1) / SSM_TT;
    float4 nq[LQ], nk[LQ];
    float nv[4], ndt = 0.f;
    constexpr int GT = SSM_THREADS / SSM_TT;  // tiles of a group of gates
    auto tile_start = [&](int64_t i) { return (REV ? ntile - 1 - i : i) * SSM_TT; };
    auto fetch = [&](int64_t i) {  // tile i's elements of this thread, zeros past the end
        const int64_t t0 = tile_start(i);
#pragma unroll
        for (int e = 0; e < LQ; ++e) {
            const int idx = tid + e * SSM_THREADS, t = idx / (DQ / 4), c4 = idx % (DQ / 4);
            nq[e] = nk[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t0 + t < count) {
                if constexpr (!SEG) nq[e] = load4<float>(q + (first + t0 + t) * qstride + c4 * 4);
                nk[e] = load4<float>(k + (first + t0 + t) * qstride + c4 * 4);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = (tid >> 5) + 4 * e;
            nv[e] = t0 + t < count ? v[(first + t0 + t) * vstride + (tid & 31)] : 0.f;
        }
    };
    auto put = [&](int64_t i) {    // the fetched tile into its buffer
        const int b = (int)(i & 1);
#pragma unroll
        for (int e = 0; e < LQ; ++e) {
            const int idx = tid + e * SSM_THREADS;
            if constexpr (!SEG) qb[b][idx / (DQ / 4)][idx % (DQ / 4)] = nq[e];
            kb[b][idx / (DQ / 4)][idx % (DQ / 4)] = nk[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) vb[b][(tid >> 5) + 4 * e][tid & 31] = nv[e];
    };
    auto fetch_gates = [&](int64_t g) {  // this thread's token of group g
        const int64_t i = g * GT + tid / SSM_TT, t = tile_start(i) + tid % SSM_TT;
        ndt = i < ntile && t < count ? p.dt[(first + t) * p.H + h] : 0.f;
    };
    auto put_gates = [&](int64_t g) {
        const float step = scan_step(ndt + bias, p.softplus);
        sb[g & 1][tid] = step;
        ab[g & 1][tid] = expf(step * A);
    };
    if (ntile > 0) {
        fetch_gates(0);
        fetch(0);
        put_gates(0);
        put(0);
        if (ntile > 1) fetch(1);
        fetch_gates(1);
        __syncthreads();
    }
    for (int64_t i = 0; i < ntile; ++i) {
        const int64_t t0 = tile_start(i);
        const int len = (int)(count - t0 < SSM_TT ? count - t0 : SSM_TT);
        const auto& qs = qb[i & 1];
        const auto& ks = kb[i & 1];
        const auto& vs = vb[i & 1];
        auto& os = ob[i & 1];
        const float* as = ab[(i / GT) & 1] + i % GT * SSM_TT;
        const float* st = sb[(i / GT) & 1] + i % GT * SSM_TT;
        if constexpr (MODE == SSM_DB && !SEG) {
            // entering a block from its end: <G, S>, G = S here (the carried gradient)
            const int64_t e = t0 + len;
            if (e == count || e % SSM_BLOCK == 0) {
                const int64_t slot = seq_first / SSM_BLOCK + n + (begin + e - 1) / SSM_BLOCK;
                const float* cp = p.ckpt + ((slot * p.H + h) * DV + vrow) * DQ;
                float dot = 0.f;
#pragma unroll
                for (int j = 0; j < NF; ++j) {
                    const float4 c4 = *reinterpret_cast<const float4*>(cp + (4 * j + quarter) * 4);
                    dot = fmaf(S[2 * j].x, c4.x, fmaf(S[2 * j].y, c4.y, dot));
                    dot = fmaf(S[2 * j + 1].x, c4.z, fmaf(S[2 * j + 1].y, c4.w, dot));
                }
                dot = warp_sum_f(dot);
                if ((tid & 31) == 0) part[tid >> 5] = dot;
                __syncthreads();
                if (tid == 0) {
                    const int64_t slots = ssm_slots(p.rows, p.N, SSM_BLOCK);
                    if (OSDN_IN_BOUNDS(slot, slots))
                        p.gs[(slice * slots + slot) * p.H + h] = part[0] + part[1] + part[2] + part[3];
                }
                __syncthreads();
            }
        }
        // one token; its output in all 4 threads of the row
        auto token = [&](int t) -> float {
            const float a = as[t], step = st[t];
            const float vraw = vs[t][row];
            const float vv = REV ? vraw : vraw * step;
            const float2 a2 = make_float2(a, a), v2 = make_float2(vv, vv);
            float2 acc0 = make_float2(0.f, 0.f), acc1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int j = 0; j < NF; ++j) {
                const float4 k4 = ks[t][4 * j + quarter], q4 = SEG ? k4 : qs[t][4 * j + quarter];
                const float2 kl = make_float2(k4.x, k4.y), kh = make_float2(k4.z, k4.w);
                if constexpr (REV) {  // the carried state is decayed already
                    S[2 * j] = __ffma2_rn(v2, kl, S[2 * j]);
                    S[2 * j + 1] = __ffma2_rn(v2, kh, S[2 * j + 1]);
                } else {
                    S[2 * j] = __ffma2_rn(a2, S[2 * j], __fmul2_rn(v2, kl));
                    S[2 * j + 1] = __ffma2_rn(a2, S[2 * j + 1], __fmul2_rn(v2, kh));
                }
                if constexpr (!SEG) {
                    acc0 = __ffma2_rn(S[2 * j], make_float2(q4.x, q4.y), acc0);
                    acc1 = __ffma2_rn(S[2 * j + 1], make_float2(q4.z, q4.w), acc1);
                }
                if constexpr (REV) {
                    S[2 * j] = __fmul2_rn(a2, S[2 * j]);
                    S[2 * j + 1] = __fmul2_rn(a2, S[2 * j + 1]);
                }
            }
            return (acc0.x + acc0.y) + (acc1.x + acc1.y);
        };
        auto give = [&](int t, float o) {
            if constexpr (MODE == SSM_DX) o *= st[t];
            os[t][row] = fmaf(skip, vs[t][row], o);
        };
        int u = 0;
        // four tokens at a time, so that their shared-memory reads and the sums over a row's
        // threads overlap; each thread of a row stores one of the four
        for (; u + 4 <= len; u += 4) {
            float o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) o[k] = token(REV ? len - 1 - u - k : u + k);
            if constexpr (SEG) {
                whole *= (as[u] * as[u + 1]) * (as[u + 2] * as[u + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] += __shfl_xor_sync(0xffffffffu, o[k], 1);
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] += __shfl_xor_sync(0xffffffffu, o[k], 2);
                const float mine = quarter == 0 ? o[0] : quarter == 1 ? o[1] : quarter == 2 ? o[2] : o[3];
                give(REV ? len - 1 - u - quarter : u + quarter, mine);
            }
        }
        for (; u < len; ++u) {
            const int t = REV ? len - 1 - u : u;
            float o = token(t);
            if constexpr (SEG) {
                whole *= as[u];
                continue;
            }
            o += __shfl_xor_sync(0xffffffffu, o, 1);
            o += __shfl_xor_sync(0xffffffffu, o, 2);
            if (quarter == 0) give(t, o);
        }
        if constexpr (MODE == SSM_DC && !SEG) {
            const int64_t e = t0 + len;  // S behind a block
            if (e == count || e % SSM_BLOCK == 0) {
                const int64_t slot = seq_first / SSM_BLOCK + n + (begin + e - 1) / SSM_BLOCK;
                float* cp = p.ckpt + ((slot * p.H + h) * DV + vrow) * DQ;
                if (OSDN_IN_BOUNDS(slot, ssm_slots(p.rows, p.N, SSM_BLOCK)))
#pragma unroll
                    for (int j = 0; j < NF; ++j)
                        *reinterpret_cast<float4*>(cp + (4 * j + quarter) * 4) =
                            make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
            }
            if (slice == 0 && p.vk) {  // q . k = dy . x: 8 threads a token
                float dot = 0.f;
#pragma unroll
                for (int c4 = tid & 7; c4 < DQ / 4; c4 += 8) {
                    const float4 x4 = ks[tid >> 3][c4], y4 = qs[tid >> 3][c4];
                    dot += x4.x * y4.x + x4.y * y4.y + x4.z * y4.z + x4.w * y4.w;
                }
                dot += __shfl_xor_sync(0xffffffffu, dot, 1);
                dot += __shfl_xor_sync(0xffffffffu, dot, 2);
                dot += __shfl_xor_sync(0xffffffffu, dot, 4);
                if ((tid & 7) == 0 && (tid >> 3) < len)
                    p.vk[h * p.rows + first + t0 + (tid >> 3)] = dot;
            }
        }
        if (i + 1 < ntile) put(i + 1);
        if (i % GT == GT - 1) {  // the next group's gates, and the loads of the one behind it
            put_gates(i / GT + 1);
            fetch_gates(i / GT + 2);
        }
        if (i + 2 < ntile) fetch(i + 2);
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int t = (tid >> 5) + 4 * e;
            if (!SEG && t < len && OSDN_IN_BOUNDS(first + t0 + t, p.rows)) {
                const int64_t at = ((first + t0 + t) * p.H + h) * DV + slice * SSM_BV + (tid & 31);
                p.out[at] = os[t][tid & 31];
            }
        }
    }
    float* out = SEG ? p.seg_state + (number * p.H + h) * DV * DQ : !TRANS && ends ? p.S_out : nullptr;
    if (!SEG && out) out += sbase;
    if (out && OSDN_IN_BOUNDS(nh, (int64_t)p.N * p.H)) {
#pragma unroll
        for (int j = 0; j < NF; ++j)
            *reinterpret_cast<float4*>(out + (int64_t)vrow * DQ + (4 * j + quarter) * 4) =
                make_float4(S[2 * j].x, S[2 * j].y, S[2 * j + 1].x, S[2 * j + 1].y);
        if (SEG && tid == 0 && slice == 0) p.seg_decay[number * p.H + h] = whole;
    }
}

// The heads' shares of dc and db summed over each group, and per head pos = c . dc and the
// unscaled neg / step = b . db / step.  dch, dbh: [rows][H][DK] fp32, dbh before its factor step.
// A warp per (row, group).
template <int DK>
__global__ void __launch_bounds__(256)
ssm_group_kernel(const float* __restrict__ dch, const float* __restrict__ dbh,
                 const float* __restrict__ b, const float* __restrict__ c, const float* __restrict__ dt,
                 const float* __restrict__ dt_bias, int softplus, float* __restrict__ db,
                 float* __restrict__ dc, float* __restrict__ pos, float* __restrict__ rneg,
                 int64_t rows, int H, int G) {
    constexpr int PL = DK / 32;
    const int lane = threadIdx.x & 31, rep = H / G;
    const int64_t stride = (int64_t)gridDim.x * 8;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < rows * G; u += stride) {
        const int64_t row = u / G;
        const int g = (int)(u - row * G);
        float bb[PL], cc[PL], sb[PL], sc[PL];
#pragma unroll
        for (int j = 0; j < PL; j += 2) {
            const float2 x = load2<float>(b + u * DK + lane * PL + j);
            const float2 y = load2<float>(c + u * DK + lane * PL + j);
            bb[j] = x.x; bb[j + 1] = x.y;
            cc[j] = y.x; cc[j + 1] = y.y;
            sb[j] = sb[j + 1] = sc[j] = sc[j + 1] = 0.f;
        }
        for (int r = 0; r < rep; ++r) {
            const int h = g * rep + r;
            const int64_t at = (row * H + h) * DK + lane * PL;
            const float step = scan_step(dt[row * H + h] + (dt_bias ? dt_bias[h] : 0.f), softplus);
            float dp = 0.f, dn = 0.f;
#pragma unroll
            for (int j = 0; j < PL; j += 2) {
                const float2 x = *reinterpret_cast<const float2*>(dch + at + j);
                const float2 y = *reinterpret_cast<const float2*>(dbh + at + j);
                dp += cc[j] * x.x + cc[j + 1] * x.y;
                dn += bb[j] * y.x + bb[j + 1] * y.y;
                sc[j] += x.x; sc[j + 1] += x.y;
                sb[j] = fmaf(step, y.x, sb[j]);
                sb[j + 1] = fmaf(step, y.y, sb[j + 1]);
            }
            dp = warp_sum_f(dp);
            dn = warp_sum_f(dn);
            if (lane == 0) {
                pos[h * rows + row] = dp;
                rneg[h * rows + row] = dn;
            }
        }
#pragma unroll
        for (int j = 0; j < PL; j += 2) {
            store2<float>(db + u * DK + lane * PL + j, make_float2(sb[j], sb[j + 1]));
            store2<float>(dc + u * DK + lane * PL + j, make_float2(sc[j], sc[j + 1]));
        }
    }
}

// ddt of every token, and per (sequence, head) the sums that dA, dD and ddt_bias are made of.
// Within a block of BLOCK tokens (gs its <G, S> term, nslice shares of it; pos, ri and rn have
// `shares` shares each; rn and wd may be null for 0):
//   d(log a_t) = sum_{i >= t} (pos_i - step_i ri_i) + sum_{j < t} step_j rn_j + gs
//   dstep_t = ri_t + wd_t + rn_t + A d(log a_t)
// The sums that nearly cancel run in 64 bits.  A warp per (block, head); part: the block's sums for dA, dD and ddt_bias, [3][slots][H].
constexpr int SSM_GATE_WARPS = 8;
template <int BLOCK>
__global__ void __launch_bounds__(32 * SSM_GATE_WARPS)
ssm_gate_kernel(const float* __restrict__ pos, const float* __restrict__ ri,
                const float* __restrict__ rn, int shares, const float* __restrict__ wd,
                const float* __restrict__ gs, int nslice, const float* __restrict__ vk,
                const float* __restrict__ dt, const float* __restrict__ A,
                const float* __restrict__ dt_bias, int softplus, float* __restrict__ ddt,
                float* __restrict__ part, const int32_t* __restrict__ cu,
                int N, int T, int H, int64_t rows) {
    constexpr int PT = BLOCK / 32;  // neighbouring tokens of a lane
    const int64_t slots = ssm_slots(rows, N, BLOCK), share = (int64_t)H * rows;
    const int64_t unit = (int64_t)blockIdx.x * SSM_GATE_WARPS + (threadIdx.x >> 5);
    if (unit >= slots * H) return;
    const int lane = threadIdx.x & 31;
    const int64_t slot = unit / H;
    const int h = (int)(unit - slot * H);
    int n, s_of;
    int64_t first = 0, count = 0;
    float sA = 0.f, sD = 0.f, sb = 0.f;
    const bool ok = token_block(cu, N, T, BLOCK, slot, n, s_of) && seq_range(cu, n, N, T, first, count);
    const int64_t t0 = (int64_t)s_of * BLOCK;
    if (ok && t0 < count) {
        const float Ah = A[h], bias = dt_bias ? dt_bias[h] : 0.f;
        float edge = 0.f;
        for (int s = 0; s < nslice; ++s) edge += gs[(s * slots + slot) * H + h];
        float raw[PT], step[PT], r[PT];
        double back[PT], fore[PT], own_b = 0.0, own_f = 0.0;
#pragma unroll
        for (int e = 0; e < PT; ++e) {
            const int64_t t = t0 + lane * PT + e, at = h * rows + first + t;
            const bool live = t < count;
            raw[e] = live ? dt[(first + t) * H + h] + bias : 0.f;
            step[e] = live ? scan_step(raw[e], softplus) : 0.f;
            float ps = 0.f, a = 0.f, b = 0.f;
            for (int s = 0; live && s < shares; ++s) {
                ps += pos[s * share + at];
                a += ri[s * share + at];
                if (rn) b += rn[s * share + at];
            }
            r[e] = a + b + (wd && live ? wd[at] : 0.f);
            back[e] = (double)ps - (double)step[e] * (double)a;
            fore[e] = (double)step[e] * (double)b;
            own_b += back[e];
            own_f += fore[e];
            if (vk && live) sD += vk[at];
        }
        double sum_b = own_b, sum_f = own_f;  // over this lane and the later (earlier) ones
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double o = __shfl_down_sync(0xffffffffu, sum_b, off);
            if (lane + off < 32) sum_b += o;
            const double u = __shfl_up_sync(0xffffffffu, sum_f, off);
            if (lane >= off) sum_f += u;
        }
        double after = sum_b - own_b, before = sum_f - own_f;
        double dla[PT];
#pragma unroll
        for (int e = PT - 1; e >= 0; --e) {
            after += back[e];
            dla[e] = after;
        }
#pragma unroll
        for (int e = 0; e < PT; ++e) {
            dla[e] = (dla[e] + before) + edge;
            before += fore[e];
            const int64_t t = t0 + lane * PT + e;
            if (t < count) {
                float d = fmaf(Ah, (float)dla[e], r[e]);
                if (softplus) d *= 1.f / (1.f + expf(-raw[e]));
                if (OSDN_IN_BOUNDS(first + t, rows)) ddt[(first + t) * H + h] = d;
                sA = fmaf(step[e], (float)dla[e], sA);
                sb += d;
            }
        }
    }
    sA = warp_sum_f(sA);
    sD = warp_sum_f(sD);
    sb = warp_sum_f(sb);
    if (lane == 0) {  // a block that is not there adds 0
        part[slot * H + h] = sA;
        part[(slots + slot) * H + h] = sD;
        part[(2 * slots + slot) * H + h] = sb;
    }
}

// dA, dD, ddt_bias [H]: the blocks' sums, in a fixed order and 64 bits.  blockIdx.x: which of the
// three, blockIdx.y: the head.
__global__ void __launch_bounds__(128)
ssm_param_kernel(const float* __restrict__ part, int64_t slots, int H, float* __restrict__ dA,
                 float* __restrict__ dD, float* __restrict__ ddt_bias) {
    __shared__ double red[4];
    float* out = blockIdx.x == 0 ? dA : blockIdx.x == 1 ? dD : ddt_bias;
    if (!out) return;  // uniform over the block
    double s = 0.0;
    for (int64_t e = threadIdx.x; e < slots; e += 128)
        s += (double)part[(blockIdx.x * slots + e) * H + blockIdx.y];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x == 0) out[blockIdx.y] = (float)((red[0] + red[1]) + (red[2] + red[3]));
}

}  // namespace osdn
