// ssm_tc.cuh -- the selective scan on the sm_100a tensor cores (bf16 tokens): the fused forward
// pass, and the chains of states that the backward pass starts from.
//
// Chunk form, L = 128 tokens, cum_i = sum_{s <= i} step_s A within the chunk (base-2 logs below):
//   G = C B^T                                   [i x j]
//   P_ij = G_ij 2^(cum_i - cum_j) step_j        for j <= i, else 0
//   Y = P X + 2^cum_i (C S^T) + D X             S: the state in front of the chunk
//   S' = 2^cum_L S + sum_j 2^(cum_L - cum_j) step_j x_j b_j^T
// A CTA owns 64 value channels of one (sequence, head) and walks its chunks with the transposed
// state (key channel x value channel) in the registers of one warpgroup.  Four products a chunk,
// all with M = 128 rows: G, C S^T and P X (rows are tokens), and B^T V' (rows are key channels),
// V'_j = 2^(cum_L - cum_j) step_j x_j.
//
// Decays.  cum is kept per sub-block of 16 tokens: an offset l_j inside the sub-block and the
// sub-blocks' bases as two fp32 terms (summed in 64 bits), so differences of far sums lose
// nothing.  Between sub-blocks 2^(cum_i - cum_j) = 2^(cum_i - end_b) 2^(end_b - cum_j), end_b the
// sum at the end of j's sub-block: both factors are at most 1 when A <= 0, the second is one
// value per token and the first one per row and sub-block, so only the 16 x 16 blocks on the
// diagonal take an exponential per element.
//
// Precision.  b, c and x enter products as stored.  V' goes in as two bf16 terms (2^-17 off), so
// states are fp32 results; P and the state in C S^T are rounded once to bf16: their errors reach
// only y, which is rounded to bf16 itself.
//
// Rows past a sequence's end inside its last tile belong to the next sequence: the rows of B, X
// and V' are zeroed in shared memory before a product sums over them.
//
// Warp roles: 0 TMA loads (two stages), 1 MMA issue, 2 the gates (softplus, sums of log decays),
// 4-7 the state, 8-11 V' and the output rows, 12-15 and 16-19 P of even and odd chunks.
// Hand-offs are mbarriers with bounded waits; a role that gives up leaves its loop, the others
// run into their own bounds, and everything in flight is waited for before the CTA leaves.
#pragma once

#include "mixer_common.cuh"
#include "tc_ptx.cuh"

namespace osdn {

constexpr int TCS_L = 128;   // tokens per chunk
constexpr int TCS_BV = 64;   // value channels per CTA

// What a launch of the chain does: the forward pass; the states in front of every chunk (stored
// as bf16 hi / lo images); the same for the gradient's chain, backwards in time.
enum { TCS_FWD = 0, TCS_SAVE = 1, TCS_RSAVE = 2 };

struct TcsArgs {
    const float *dt, *A, *dt_bias;
    const float* D;                // FWD
    const __nv_bfloat16* x;        // FWD: x again, for D x
    const float* S_in;             // S0 (RSAVE: dST), or null
    __nv_bfloat16* y;              // FWD
    float* S_out;                  // ST (RSAVE: dS0), or null
    uint8_t* img;                  // SAVE, RSAVE: images written
    const uint8_t* img_fwd;        // RSAVE: SAVE's images
    float* gs;                     // RSAVE: <G, S> shares [DV / 64 * DQ / 32][slot][H]
    const int32_t* cu;
    int64_t rows;
    int N, T, H, G, softplus, nvt;
    long long limit_ns;
};

template <int DQ, int MODE> struct TcsSmem {
    static constexpr bool OUT = MODE == TCS_FWD;
    static constexpr uint32_t KB = DQ / 64 * 16384, QB = OUT ? KB : 0;
    static constexpr uint32_t Q = 0, K = QB, V = QB + KB, STAGE = V + 16384;
    static constexpr int NVP = OUT ? 1 : 2;           // V' buffers, hi then lo
    static constexpr uint32_t VP = 2 * STAGE;
    static constexpr uint32_t S = VP + NVP * 32768;   // the state as an operand (or image)
    static constexpr uint32_t GATE = S + (OUT ? 16384 : 32768);
    static constexpr uint32_t GATE_BYTES = 1664;
    static constexpr uint32_t BAR = GATE + 2 * GATE_BYTES;
    static constexpr uint32_t TMEM_SLOT = BAR + 176;
    static constexpr size_t BYTES = TMEM_SLOT + 16 + 1024;  // + alignment slack
    static constexpr int THREADS = OUT ? 640 : 384;
    // tensor memory: G / P (two buffers), B^T V', C S^T, P X
    static constexpr uint32_t COL_G = 0, COL_U = OUT ? 256 : 0, COL_Y1 = 320, COL_Y2 = 384;
    static constexpr uint32_t COLS = OUT ? 512 : 64;
};
static_assert(TcsSmem<128, TCS_FWD>::BYTES <= 232448, "shared memory");

// One chunk's gates in shared memory.
struct TcsGate {
    float l[TCS_L];    // sum of log2 decays from the token's sub-block's start, itself included
    float g[TCS_L];    // FWD, SAVE: 2^(end - l) step;  RSAVE: 2^l
    float st[TCS_L];   // step
    float bh[9], bl[9];  // sums in front of each sub-block and behind the last, two terms each
};
static_assert(sizeof(TcsGate) <= TcsSmem<128, TCS_FWD>::GATE_BYTES, "gate arrays");

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values as packed bf16 pairs hi + lo, both rounded to nearest (2^-18 off at most).
__device__ __forceinline__ void split2_rn(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(hi << 16),
                                                   b - __uint_as_float(hi & 0xffff0000u));
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ uint32_t pack2_rn(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Reading half of a chunk's gates (one warp): this lane's tokens 4 lane .. 4 lane + 3.
struct TcsGateIn { float raw[4]; };
__device__ __forceinline__ TcsGateIn tcs_gate_load(const float* __restrict__ dt, int64_t row0,
                                                   int len, int H, int h, int lane) {
    TcsGateIn in;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int t = 4 * lane + e;
        in.raw[e] = t < len ? __ldg(dt + (row0 + t) * H + h) : 0.f;
    }
    return in;
}
template <bool REV>
__device__ __forceinline__ void tcs_gate_store(const TcsGateIn& in, TcsGate* g, int len, float A,
                                               float bias, int softplus, int lane) {
    float st[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const bool live = 4 * lane + e < len;
        st[e] = live ? scan_step(in.raw[e] + bias, softplus) : 0.f;
        // 2^-1e5 is 0 like everything below it; a finite floor keeps differences defined
        float d = live ? st[e] * A * 1.4426950408889634f : 0.f;
        d = d < -1e5f ? -1e5f : d;
        l[e] = e ? l[e - 1] + d : d;
    }
    float own = l[3], pre = 0.f;  // prefix over the 4 lanes of the sub-block
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        const float o = __shfl_up_sync(0xffffffffu, own, off, 4);
        if ((lane & 3) >= off) { own += o; pre += o; }
    }
    const float tot = __shfl_sync(0xffffffffu, own, 3, 4);  // the sub-block's sum
    double base = (double)tot;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, base, off);
        if (lane >= off) base += o;
    }
    if ((lane & 3) == 0) {
        const int b = lane >> 2;
        const float hi = (float)base;
        g->bh[b + 1] = hi;
        g->bl[b + 1] = (float)(base - (double)hi);
        if (b == 0) g->bh[0] = g->bl[0] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float le = pre + l[e];
        g->l[4 * lane + e] = le;
        g->st[4 * lane + e] = st[e];
        g->g[4 * lane + e] = REV ? ex2f(le) : ex2f(tot - le) * st[e];
    }
}

template <int DQ, int MODE>
__global__ void __launch_bounds__(TcsSmem<DQ, MODE>::THREADS, 1)
ssm_tc_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const TcsArgs p) {
    using L = TcsSmem<DQ, MODE>;
    constexpr bool OUT = L::OUT, REV = MODE == TCS_RSAVE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int vt = blockIdx.x % p.nvt;
    const int64_t nh = blockIdx.x / p.nvt;
    const int n = (int)(nh / p.H), h = (int)(nh - (int64_t)n * p.H), g = h / (p.H / p.G);
    int64_t first, count;
    if (!seq_range(p.cu, n, p.N, p.T, first, count)) return;  // uniform over the CTA
    const int nch = (int)((count + TCS_L - 1) / TCS_L);
    const int DV = p.nvt * TCS_BV;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
    uint64_t* full = bars + 0;       // [2] tiles landed
    uint64_t* empty = bars + 2;      // [2] tiles used up (MMA commit)
    uint64_t* gate_full = bars + 4;  // [2]
    uint64_t* g_full = bars + 6;     // [2] G = C B^T
    uint64_t* p_full = bars + 8;     // [2] P written
    uint64_t* vp_full = bars + 10;   // [2] V' written (and dead rows zeroed)
    uint64_t* vp_free = bars + 12;   // [2] V' used up (MMA commit)
    uint64_t* gate_free = bars + 14; // [2] the chunk's gates read by all
    uint64_t* u_full = bars + 16;    // B^T V'
    uint64_t* s_full = bars + 17;    // the state written as an operand, B^T V' read
    uint64_t* y_full = bars + 18;    // C S^T and P X
    uint64_t* y_free = bars + 19;    // ... read
    uint64_t* drain = bars + 20;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::TMEM_SLOT);
    auto gate = [&](int i) { return reinterpret_cast<TcsGate*>(smem + L::GATE + (i & 1) * L::GATE_BYTES); };
    auto stage = [&](int i) { return smem + (i & 1) * L::STAGE; };
    auto chunk_of = [&](int i) { return REV ? nch - 1 - i : i; };
    auto row_of = [&](int i) { return first + (int64_t)chunk_of(i) * TCS_L; };
    auto len_of = [&](int i) -> int {
        const int64_t rem = count - (int64_t)chunk_of(i) * TCS_L;
        return rem < TCS_L ? (int)rem : TCS_L;
    };
    // every lane waits; the warp leaves together
    auto wait = [&](uint64_t* bar, int phase) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_bounded(bar, (uint32_t)phase & 1u, p.limit_ns));
    };

    if (warp == 0) {
        tc::tmem_alloc(tmem_slot, L::COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&gate_full[i], 1);
            mbar_init(&g_full[i], 1);
            mbar_init(&p_full[i], 4);
            mbar_init(&vp_full[i], 4);
            mbar_init(&vp_free[i], 1);
            // FWD: the output rows are the last readers; else V' and the state read them
            mbar_init(&gate_free[i], OUT ? 4 : 8);
        }
        mbar_init(u_full, 1);
        mbar_init(s_full, 4);
        mbar_init(y_full, 1);
        mbar_init(y_free, 4);
        mbar_init(drain, 1);
        tc::fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            int issued = 0;
            for (int i = 0; i < nch; ++i) {
                if (i >= 2 && !mbar_wait_bounded(&empty[i & 1], ((i >> 1) - 1) & 1, p.limit_ns)) break;
                uint8_t* s = stage(i);
                uint64_t* bar = &full[i & 1];
                const int row = (int)row_of(i);
                tc::mbar_expect_tx(bar, L::STAGE);
#pragma unroll
                for (int b = 0; b < DQ / 64; ++b) {
                    if constexpr (OUT) tc::tma_load_3d(s + L::Q + b * 16384, &tm_q, b * 64, g, row, bar);
                    tc::tma_load_3d(s + L::K + b * 16384, &tm_k, b * 64, g, row, bar);
                }
                tc::tma_load_3d(s + L::V, &tm_v, vt * TCS_BV, h, row, bar);
                issued = i + 1;
            }
            // whatever was issued has landed before the CTA may leave
            for (int i = issued > 2 ? issued - 2 : 0; i < issued; ++i)
                mbar_wait_bounded(&full[i & 1], (i >> 1) & 1, p.limit_ns);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        if (lane == 0) {
            constexpr uint32_t ID_G = tc::idesc(1, 0, 0, 128, 128);  // tokens x tokens
            constexpr uint32_t ID_Y = tc::idesc(1, 0, 1, 128, 64);   // tokens x value channels
            constexpr uint32_t ID_U = tc::idesc(1, 1, 1, 128, 64);   // key x value channels
            auto issue_g = [&](int i) {
                const uint32_t q = smem_u32(stage(i) + L::Q), k = smem_u32(stage(i) + L::K);
#pragma unroll
                for (int s = 0; s < DQ / 16; ++s)
                    tc::mma_bf16(tmem + L::COL_G + (i & 1) * 128,
                                 tc::sw128_desc(q + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024),
                                 tc::sw128_desc(k + (s >> 2) * 16384 + (s & 3) * 32, 16, 1024), ID_G,
                                 s != 0);
                tc::mma_commit(&g_full[i & 1]);
            };
            bool ok = true;
            if (OUT && nch > 0) {
                ok = mbar_wait_bounded(&full[0], 0, p.limit_ns);
                if (ok) issue_g(0);
            }
            for (int i = 0; ok && i < nch; ++i) {
                const int s = i & 1, ph = (i >> 1) & 1;
                if (OUT && i + 1 < nch) {
                    if (!(ok = mbar_wait_bounded(&full[s ^ 1], ((i + 1) >> 1) & 1, p.limit_ns))) break;
                    issue_g(i + 1);
                }
                if (!(ok = mbar_wait_bounded(s_full, i & 1, p.limit_ns))) break;
                const uint32_t q = smem_u32(stage(i) + L::Q), k = smem_u32(stage(i) + L::K),
                               v = smem_u32(stage(i) + L::V);
                if constexpr (OUT) {
                    if (i > 0 && !(ok = mbar_wait_bounded(y_free, (i - 1) & 1, p.limit_ns))) break;
                    tc::fence_after_sync();
                    const uint32_t sb = smem_u32(smem + L::S);
#pragma unroll
                    for (int e = 0; e < DQ / 16; ++e)
                        tc::mma_bf16(tmem + L::COL_Y1,
                                     tc::sw128_desc(q + (e >> 2) * 16384 + (e & 3) * 32, 16, 1024),
                                     tc::sw128_desc(sb + e * 2048, 16384, 1024), ID_Y, e != 0);
                }
                // the V' and output warpgroup has seen the tiles land: no wait for `full` here
                if (!(ok = mbar_wait_bounded(&vp_full[i % L::NVP], (i / L::NVP) & 1, p.limit_ns))) break;
                tc::fence_after_sync();
                const uint32_t vp = smem_u32(smem + L::VP + (i % L::NVP) * 32768);
                // (DQ = 64: rows 64..127 read the next tile and are not used)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tc::mma_bf16(tmem + L::COL_U, tc::sw128_desc(k + e * 2048, 16384, 1024),
                                     tc::sw128_desc(vp + t * 16384 + e * 2048, 16384, 1024), ID_U,
                                     (t | e) != 0);
                tc::mma_commit(u_full);
                tc::mma_commit(&vp_free[i % L::NVP]);
                if constexpr (OUT) {
                    if (!(ok = mbar_wait_bounded(&p_full[s], ph, p.limit_ns))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        tc::mma_bf16_ts(tmem + L::COL_Y2, tmem + L::COL_G + s * 128 + 8 * e,
                                        tc::sw128_desc(v + e * 2048, 16384, 1024), ID_Y, e != 0);
                    tc::mma_commit(y_full);
                }
                tc::mma_commit(&empty[s]);
            }
            tc::mma_commit(drain);
            mbar_wait_bounded(drain, 0, p.limit_ns);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ gates
        const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        TcsGateIn in = {};
        if (nch > 0) in = tcs_gate_load(p.dt, row_of(0), len_of(0), p.H, h, lane);
        for (int i = 0; i < nch; ++i) {
            TcsGateIn next = {};
            if (i + 1 < nch) next = tcs_gate_load(p.dt, row_of(i + 1), len_of(i + 1), p.H, h, lane);
            if (i >= 2 && !wait(&gate_free[i & 1], (i >> 1) - 1)) break;
            tcs_gate_store<REV>(in, gate(i), len_of(i), A, bias, p.softplus, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&gate_full[i & 1]);
            in = next;
        }
    } else if (warp >= 4 && warp < 8) {
        // ------------------------------------------------------------ state
        const int r = tid - 128;  // key channel
        const bool on = DQ == 128 || r < DQ;
        float S[TCS_BV];
        const int64_t sbase = (nh * DV + vt * TCS_BV) * DQ + r;  // stored [value][key]
#pragma unroll
        for (int j = 0; j < TCS_BV; ++j) S[j] = on && p.S_in ? p.S_in[sbase + (int64_t)j * DQ] : 0.f;
        uint8_t* so = smem + L::S;
        for (int i = 0; i < nch; ++i) {
            if (!wait(&gate_full[i & 1], i >> 1)) break;
            const float decay = ex2f(gate(i)->bh[8] + gate(i)->bl[8]);
            if (!OUT) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&gate_free[i & 1]);
            }
            if constexpr (OUT) {
                if (on) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = pack2_rn(S[8 * j + 2 * e], S[8 * j + 2 * e + 1]);
                        *reinterpret_cast<uint4*>(so + tc::sw128_off(r, j)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                tc::fence_async_smem();
            } else {
                // images: rows of 128 bytes, hi then lo, as the products read them
                const int64_t slot = first / TCS_L + n + chunk_of(i);
                const int64_t at = ((slot * p.H + h) * p.nvt + vt) * (2 * DQ * 128);
                if constexpr (REV) {  // <G, S> against the forward chain's state
                    float dot = 0.f;
                    if (on) {
                        const uint8_t* f = p.img_fwd + at;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const uint4 a = *reinterpret_cast<const uint4*>(f + tc::sw128_off(r, j));
                            const uint4 b = *reinterpret_cast<const uint4*>(f + DQ * 128 + tc::sw128_off(r, j));
                            const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float x0 = __uint_as_float(aw[e] << 16) + __uint_as_float(bw[e] << 16);
                                const float x1 = __uint_as_float(aw[e] & 0xffff0000u) +
                                                 __uint_as_float(bw[e] & 0xffff0000u);
                                dot = fmaf(S[8 * j + 2 * e], x0, fmaf(S[8 * j + 2 * e + 1], x1, dot));
                            }
                        }
                    }
                    dot = warp_sum_f(dot) * decay;
                    if (on && lane == 0) {
                        const int64_t slots = ssm_slots(p.rows, p.N, TCS_L);
                        if (OSDN_IN_BOUNDS(slot, slots))
                            p.gs[((int64_t)(vt * (DQ / 32) + (warp & 3)) * slots + slot) * p.H + h] = dot;
                    }
                }
                if (on) {
                    if (lane == 0) tc::bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t w[4], x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            split2_rn(S[8 * j + 2 * e], S[8 * j + 2 * e + 1], w[e], x[e]);
                        *reinterpret_cast<uint4*>(so + tc::sw128_off(r, j)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                        *reinterpret_cast<uint4*>(so + 16384 + tc::sw128_off(r, j)) =
                            make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && OSDN_IN_BOUNDS(slot, ssm_slots(p.rows, p.N, TCS_L))) {
                        const uint32_t w0 = (warp & 3) * 4096;
                        tc::bulk_store(p.img + at + w0, so + w0, 4096);
                        tc::bulk_store(p.img + at + DQ * 128 + w0, so + 16384 + w0, 4096);
                        tc::bulk_commit();
                    }
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(s_full);
            if (!wait(u_full, i)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float u[16];
                tc::tmem_ld16(tmem + tlane + L::COL_U + 16 * q, u);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) S[16 * q + e] = fmaf(decay, S[16 * q + e], u[e]);
            }
        }
        if (on && p.S_out && OSDN_IN_BOUNDS(nh, (int64_t)p.N * p.H)) {
#pragma unroll
            for (int j = 0; j < TCS_BV; ++j) p.S_out[sbase + (int64_t)j * DQ] = S[j];
        }
        if (!OUT && lane == 0) tc::bulk_wait_all();
    } else if (warp >= 8 && warp < 12) {
        // ------------------------------------------------------------ V' and output rows
        const int r = tid - 256;  // token of the chunk
        const float skip = OUT && p.D ? p.D[h] : 0.f;
        auto output = [&](int i) -> bool {
            const TcsGate* gt = gate(i);
            const bool live = r < len_of(i);
            const int64_t at = ((row_of(i) + r) * p.H + h) * DV + vt * TCS_BV;
            uint4 xr[8];
            if (p.D && live) {
#pragma unroll
                for (int j = 0; j < 8; ++j) xr[j] = __ldg(reinterpret_cast<const uint4*>(p.x + at) + j);
            }
            if (!wait(y_full, i)) return false;
            tc::fence_after_sync();
            const float rf = ex2f(gt->bh[r >> 4] + gt->l[r] + gt->bl[r >> 4]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float a[16], b[16];
                tc::tmem_ld16(tmem + tlane + L::COL_Y1 + 16 * q, a);
                tc::tmem_ld16(tmem + tlane + L::COL_Y2 + 16 * q, b);
                tc::tmem_ld_wait();
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float y0 = fmaf(rf, a[2 * e], b[2 * e]), y1 = fmaf(rf, a[2 * e + 1], b[2 * e + 1]);
                    if (p.D) {
                        const uint4 xv = xr[2 * q + (e >> 2)];
                        const uint32_t xw = (e & 3) == 0 ? xv.x : (e & 3) == 1 ? xv.y : (e & 3) == 2 ? xv.z : xv.w;
                        y0 = fmaf(skip, __uint_as_float(xw << 16), y0);
                        y1 = fmaf(skip, __uint_as_float(xw & 0xffff0000u), y1);
                    }
                    w[e] = pack2_rn(y0, y1);
                }
                if (live && OSDN_IN_BOUNDS(row_of(i) + r, p.rows)) {
                    uint4* o = reinterpret_cast<uint4*>(p.y + at) + 2 * q;
                    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(y_free);
                mbar_arrive(&gate_free[i & 1]);
            }
            return true;
        };
        bool ok = true;
        for (int i = 0; ok && i < nch; ++i) {
            if (!(ok = wait(&full[i & 1], i >> 1) && wait(&gate_full[i & 1], i >> 1))) break;
            if (i >= L::NVP && !(ok = wait(&vp_free[i % L::NVP], i / L::NVP - 1))) break;
            const TcsGate* gt = gate(i);
            const bool live = r < len_of(i);
            uint8_t* v = stage(i) + L::V;
            uint8_t* vp = smem + L::VP + (i % L::NVP) * 32768;
            const int b = r >> 4;
            // FWD: 2^(cum_L - end_b) 2^(end_b - cum_r) step;  RSAVE: 2^(base_b + l_r)
            const float e = REV ? gt->bh[b] + gt->bl[b]
                                : (gt->bh[8] - gt->bh[b + 1]) + (gt->bl[8] - gt->bl[b + 1]);
            const float w = ex2f(e) * gt->g[r];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t off = tc::sw128_off(r, j);
                uint4 hi = make_uint4(0, 0, 0, 0), lo = hi;
                if (live) {
                    const uint4 x = *reinterpret_cast<const uint4*>(v + off);
                    const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
                    uint32_t hw[4], lw[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        split2_rn(w * __uint_as_float(xw[k] << 16), w * __uint_as_float(xw[k] & 0xffff0000u),
                                  hw[k], lw[k]);
                    hi = make_uint4(hw[0], hw[1], hw[2], hw[3]);
                    lo = make_uint4(lw[0], lw[1], lw[2], lw[3]);
                } else {  // the next sequence's row: 0 x NaN must not reach a sum
                    *reinterpret_cast<uint4*>(v + off) = hi;
#pragma unroll
                    for (int q = 0; q < DQ / 64; ++q)
                        *reinterpret_cast<uint4*>(stage(i) + L::K + q * 16384 + off) = hi;
                }
                *reinterpret_cast<uint4*>(vp + off) = hi;
                *reinterpret_cast<uint4*>(vp + 16384 + off) = lo;
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&vp_full[i % L::NVP]);
                if (!OUT) mbar_arrive(&gate_free[i & 1]);
            }
            if (OUT && i > 0) ok = output(i - 1);
        }
        if (OUT && ok && nch > 0) output(nch - 1);
    } else if (OUT && warp >= 12) {
        // ------------------------------------------------------------ P
        const int wg = (warp - 12) >> 2, wq = warp & 3;
        const int r = 32 * wq + lane, rb = r >> 4;
        for (int i = wg; i < nch; i += 2) {
            if (!wait(&gate_full[i & 1], i >> 1) || !wait(&g_full[wg], i >> 1)) break;
            tc::fence_after_sync();
            const TcsGate* gt = gate(i);
            const float lr = gt->l[r], bh = gt->bh[rb], bl = gt->bl[rb];
            const uint32_t col = tmem + tlane + L::COL_G + wg * 128;
#pragma unroll 1
            for (int b = 0; b < 8; ++b) {
                uint32_t w[8];
                if (b > 2 * wq + 1) {  // past the diagonal for every row of the warp
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[e] = 0;
                } else {
                    float x[16];
                    tc::tmem_ld16(col + 16 * b, x);
                    const float f = ex2f((bh - gt->bh[b + 1]) + (bl - gt->bl[b + 1]) + lr);
                    const float4* gp = reinterpret_cast<const float4*>(gt->g + 16 * b);
                    float wt[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float4 t = gp[e];
                        wt[4 * e] = f * t.x; wt[4 * e + 1] = f * t.y;
                        wt[4 * e + 2] = f * t.z; wt[4 * e + 3] = f * t.w;
                    }
                    if (b >= 2 * wq) {  // the diagonal's sub-blocks
                        const float4* lp = reinterpret_cast<const float4*>(gt->l + 16 * b);
                        const float4* sp = reinterpret_cast<const float4*>(gt->st + 16 * b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 t = lp[e], s = sp[e];
                            const float tv[4] = {t.x, t.y, t.z, t.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int c = 16 * b + 4 * e + k;
                                if (b == rb) wt[4 * e + k] = ex2f(lr - tv[k]) * sv[k];
                                if (c > r) wt[4 * e + k] = 0.f;
                            }
                        }
                    }
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float p0 = x[2 * e] * wt[2 * e], p1 = x[2 * e + 1] * wt[2 * e + 1];
                        if (b >= 2 * wq) {  // a NaN or infinity past the diagonal is left out too
                            if (16 * b + 2 * e > r) p0 = 0.f;
                            if (16 * b + 2 * e + 1 > r) p1 = 0.f;
                        }
                        w[e] = pack2_rn(p0, p1);
                    }
                }
                tc::tmem_st8(col + 8 * b, w);
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[wg]);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, L::COLS);
}

}  // namespace osdn
