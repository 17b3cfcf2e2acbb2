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
// sub-blocks' bases, each summed in 64 bits and kept as two fp32 terms, so differences of far sums
// lose nothing, nor do those of tokens behind one that forgets the state (whose own log decay can
// be thousands: with l_j as one term the weights behind it were 8e-5 off at -1000).  Between sub-blocks 2^(cum_i - cum_j) = 2^(cum_i - end_b) 2^(end_b - cum_j), end_b the
// sum at the end of j's sub-block: both factors are at most 1 when A <= 0, the second is one
// value per token and the first one per row and sub-block, so only the 16 x 16 blocks on the
// diagonal take an exponential per element.
//
// Precision.  b, c and x enter products as stored, P as two bf16 terms (with one, y was 2.35e-3 off in
// L2 norm without D, where rounding y alone gives 1.66e-3; 108 -> 114 us at B=4, T=4096, H=16,
// Dk=Dv=128).  V' goes in as two bf16 terms (each value 2^-17 off at most: ST is 2.5e-6 off; a third
// needs 16 KB of shared memory that the forward pass does not have), three where the state leads to
// gradients of steps (sums over many tokens that nearly cancel), and states are fp32 sums.  The state
// in C S^T is rounded once to bf16: what that adds to y is independent from element to element and at
// most of the size of y's own rounding, 2.35e-3 together where the state makes up all of y.  (A second
// term fits where V' was once it is used up, but lies on the chain from state to state: 133 us.)
//
// Rows past a sequence's end inside its last tile belong to the next sequence: the rows of B, X
// and V' are zeroed in shared memory before a product sums over them.
//
// Warp roles: 0 TMA loads (two tiles each of C, B and X), 1 MMA issue, 2-3 the gates (softplus,
// sums of log decays), 4-7 the state, 8-15 V', 16-19 the output rows, 20-27 P.  (V' by one
// warpgroup is on the chain from one state to the next: 99 against 96 us at B=4, T=4096, H=16,
// Dk=Dv=128, 261 against 246 at T=65,536 with Dv=64, both with P as one term.)
// Bound by the chain: 3.4 us a chunk at 4096 tokens (four products wait for one another
// through shared and tensor memory, with the element-wise work of P, V' and the output rows in
// between), 115 us against 42 for its 274 MB at copy speed.
// Hand-offs are mbarriers with bounded waits; a role that gives up leaves its loop, the others
// run into their own bounds, and everything in flight is waited for before the CTA leaves.
#pragma once

#include <limits.h>

#include "mixer_common.cuh"
#include "tc_ptx.cuh"

namespace osdn {

constexpr int TCS_L = 128;   // tokens per chunk
constexpr int TCS_BV = 64;   // value channels per CTA
constexpr int TCS_GATES = 8; // chunks whose gates are kept: they are made well ahead of their use

// What a launch of the chain does: the forward pass; for the backward pass the states S in front
// of every chunk and, backwards in time over c and dy, the gradients R that reach the states
// behind them, both stored as images of TCS_TERMS bf16 terms (half the CTAs each); what each
// segment of a sequence adds to a zero state, for FWD or (SEG_SAVE, both directions) for SAVE.
enum { TCS_FWD = 0, TCS_SAVE = 1, TCS_SEG = 2, TCS_SEG_SAVE = 3 };
constexpr int TCS_TERMS = 3;

struct TcsArgs {
    const float *dt, *A, *dt_bias;
    const float* D;                // FWD
    const __nv_bfloat16* x;        // FWD: x again, for D x
    const float* S_in;             // S0, or null
    __nv_bfloat16* y;              // FWD
    float* S_out;                  // ST, or null
    uint8_t *img, *img_r;          // SAVE: images of S and R [chunk][H][term][nvt][DQ][64]
    const float* dST;              // SAVE: dST, or null
    float* dS0;                    // SAVE: dS0, or null
    const int32_t* cu;
    int64_t rows;
    float* seg_state;              // SEG writes, FWD reads: [direction][slot][H][nvt][64][DQ]
    float* seg_decay;              // ... and the segment's whole log2 decay [direction][slot][H]
    int seg;                       // tokens of a segment (a multiple of TCS_L; INT_MAX: none)
    int N, T, H, G, softplus, nvt;
};

template <int DQ, int MODE> struct TcsSmem {
    static constexpr bool OUT = MODE == TCS_FWD;
    static constexpr uint32_t KB = DQ / 64 * 16384, QB = OUT ? KB : 0;
    static constexpr uint32_t Q = 0, K = QB, V = QB + KB, STAGE = V + 16384;
    static constexpr bool SEG = MODE == TCS_SEG || MODE == TCS_SEG_SAVE;
    static constexpr bool BOTH = MODE == TCS_SAVE || MODE == TCS_SEG_SAVE;  // directions
    static constexpr int NT = BOTH ? TCS_TERMS : 2;  // bf16 terms of V'
    static constexpr uint32_t VP = 2 * STAGE;
    static constexpr uint32_t S = VP + NT * 16384;    // the state as an operand (or image)
    static constexpr uint32_t GATE = S + (OUT ? 16384 : MODE == TCS_SAVE ? TCS_TERMS * 16384 : 0);
    static constexpr uint32_t GATE_BYTES = 2192;
    static constexpr uint32_t BAR = GATE + TCS_GATES * GATE_BYTES;
    static constexpr uint32_t TMEM_SLOT = BAR + (27 + 2 * TCS_GATES) * 8 + 8;
    static constexpr size_t BYTES = TMEM_SLOT + 16 + 1024;  // + alignment slack
    static constexpr int THREADS = OUT ? 896 : 512;
    static constexpr int VW = 2;            // warpgroups that make V'
    // tensor memory: G / P (two buffers), B^T V' (its terms side by side), C S^T, P X
    static constexpr uint32_t COL_G = 0, COL_U = OUT ? 256 : 0, COL_Y1 = 384, COL_Y2 = 448;
    static constexpr uint32_t COLS = OUT ? 512 : 256;
};
static_assert(TcsSmem<128, TCS_FWD>::BYTES <= 232448 && TcsSmem<128, TCS_SAVE>::BYTES <= 232448,
              "shared memory");

// One chunk's gates in shared memory.
struct TcsGate {
    float l[TCS_L];    // sum of log2 decays from the token's sub-block's start, itself included,
    float l2[TCS_L];   // ... and what l leaves of it
    float g[TCS_L];    // 2^(end - l) step;  backwards in time: 2^l
    float st[TCS_L];   // step
    float bh[9], bl[9];  // sums in front of each sub-block and behind the last, two terms each
    float th[8], tl[8];  // each sub-block's own sum, two terms
};
static_assert(sizeof(TcsGate) <= TcsSmem<128, TCS_FWD>::GATE_BYTES, "gate arrays");

// Two fp32 values as packed bf16 pairs hi + lo, both rounded to nearest (2^-18 off at most).
__device__ __forceinline__ void split2_rn(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    const __nv_bfloat162 l = __floats2bfloat162_rn(a - __uint_as_float(hi << 16),
                                                   b - __uint_as_float(hi & 0xffff0000u));
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// The same in three terms: all 24 bits.
__device__ __forceinline__ void split3_rn(float a, float b, uint32_t& t0, uint32_t& t1, uint32_t& t2) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    t0 = *reinterpret_cast<const uint32_t*>(&h);
    split2_rn(a - __uint_as_float(t0 << 16), b - __uint_as_float(t0 & 0xffff0000u), t1, t2);
}
__device__ __forceinline__ uint32_t pack2_rn(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Bounded wait on an mbarrier phase: at most 2^20 polls, each of which the hardware may hold back
// for up to 2 us, so a wait that cannot end gives up (and records it) within about 2 seconds.
// (A few instructions inline: five roles share the instruction cache.)
__device__ __forceinline__ bool tcs_wait(uint64_t* bar, int phase) {
    const uint32_t a = smem_u32(bar), par = (uint32_t)phase & 1u;
    uint32_t done = 0;
#pragma unroll 1
    for (int n = 0; n < (1 << 20) && !done; ++n)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(a), "r"(par)
            : "memory");
    if (!done) record_status(OSDN_ERR_DEVICE_TIMEOUT);
    return done != 0;
}

// A chunk's gates, by one warp: softplus and the log decays of its tokens, then their sums.
__device__ __forceinline__ void tcs_gates(bool rev, TcsGate* g, const float* __restrict__ dt, int64_t stride,
                                          int len, float A, float bias, int softplus, int lane) {
#pragma unroll
    for (int t = lane; t < TCS_L; t += 32)  // loads in flight together; each lane its own slots
        g->st[t] = t < len ? __ldg(dt + t * stride) : 0.f;
#pragma unroll 1
    for (int t = lane; t < TCS_L; t += 32) {
        float st = 0.f, d = 0.f;
        if (t < len) {
            st = scan_step(g->st[t] + bias, softplus);
            // 2^-1e5 is 0 like everything below it; a finite floor keeps differences defined
            d = st * A * 1.4426950408889634f;
            d = d < -1e5f ? -1e5f : d;
        }
        g->st[t] = st;
        g->l[t] = d;
    }
    __syncwarp();
    // 4 tokens a lane, 4 lanes a sub-block
    const float4 d4 = *reinterpret_cast<const float4*>(g->l + 4 * lane);
    const float4 s4 = *reinterpret_cast<const float4*>(g->st + 4 * lane);
    double l[4] = {d4.x, (double)d4.x + d4.y, 0.0, 0.0};
    l[2] = l[1] + d4.z;
    l[3] = l[2] + d4.w;
    double own = l[3], pre = 0.0;
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, own, off, 4);
        if ((lane & 3) >= off) { own += o; pre += o; }
    }
    const double tot = __shfl_sync(0xffffffffu, own, 3, 4);  // the sub-block's sum
    double base = tot;
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, base, off);
        if (lane >= off) base += o;
    }
    if ((lane & 3) == 0) {
        const int b = lane >> 2;
        const float hi = (float)base, th = (float)tot;
        g->bh[b + 1] = hi;
        g->bl[b + 1] = (float)(base - (double)hi);
        g->th[b] = th;
        g->tl[b] = (float)(tot - (double)th);
        if (b == 0) g->bh[0] = g->bl[0] = 0.f;
    }
    float hi[4], lo[4], w[4];
    const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        l[e] += pre;
        hi[e] = (float)l[e];
        lo[e] = (float)(l[e] - (double)hi[e]);
        w[e] = rev ? ex2f(hi[e]) : ex2f((float)(tot - l[e])) * s[e];
    }
    *reinterpret_cast<float4*>(g->l + 4 * lane) = make_float4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<float4*>(g->l2 + 4 * lane) = make_float4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<float4*>(g->g + 4 * lane) = make_float4(w[0], w[1], w[2], w[3]);
}

// One operand pair's K steps: `n` MMAs, the descriptors' start addresses (16-byte units) moving
// by `da` and `db` per step, and by `ga` and `gb` more after every fourth.  Unrolled: a rolled
// loop took 100 cycles per MMA, this 62.
template <int n>
__device__ __forceinline__ void tcs_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t da,
                                        uint32_t db, uint32_t ga, uint32_t gb) {
#pragma unroll
    for (int e = 0; e < n; ++e)
        tc::mma_bf16(d, a + e * da + (e >> 2) * ga, b + e * db + (e >> 2) * gb, id, e != 0);
}

// Segments.  When there are too few (sequence, head) chains for the machine, sequences are cut into
// segments of p.seg tokens that run side by side: a first launch (SEG, SEG_SAVE) makes what each
// segment adds to a zero state, and a segment of FWD or SAVE builds its initial state from S0 and
// the segments in front of it (backwards: from dST and those behind it).
template <int DQ, int MODE>
__global__ void __launch_bounds__(TcsSmem<DQ, MODE>::THREADS, 1)
ssm_tc_chain_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_v2,
                    const TcsArgs p) {
    using L = TcsSmem<DQ, MODE>;
    constexpr bool OUT = L::OUT;
    // the second half of the grid goes backwards over q and v2 (c and dy)
    const bool rev = L::BOTH && blockIdx.x >= gridDim.x / 2;
    const uint32_t block = rev ? blockIdx.x - gridDim.x / 2 : blockIdx.x;
    const CUtensorMap* map_k = rev ? &tm_q : &tm_k;
    const CUtensorMap* map_v = rev ? &tm_v2 : &tm_v;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int vt = block % p.nvt;
    const int slot = (int)(block / p.nvt / p.H), h = (int)(block / p.nvt - (int64_t)slot * p.H);
    const int g = h / (p.H / p.G);
    int n, seg;
    int64_t first, count;
    // every sequence's offsets are checked here, whether or not a number leads to it
    if (slot < p.N && !seq_range(p.cu, slot, p.N, p.T, first, count) && p.seg == INT_MAX) return;
    if (!token_block(p.cu, p.N, p.T, p.seg, slot, n, seg) || !seq_range(p.cu, n, p.N, p.T, first, count)) return;
    const int64_t start = (int64_t)seg * p.seg;  // of the segment in its sequence
    if (seg > 0 && start >= count) return;       // a number that no segment has
    const bool last = count - start <= p.seg;
    if (L::SEG && (rev ? seg == 0 : last)) return;  // adds to no other segment
    const int base = slot - seg;                 // the sequence's first segment
    const int segs = last ? seg + 1 : (int)((count + p.seg - 1) / p.seg);
    const int64_t half = rev ? p.rows / p.seg + p.N : 0;  // backwards: the second set of numbers
    first += start;                              // all uniform over the CTA
    count = last ? count - start : p.seg;
    const int nch = (int)((count + TCS_L - 1) / TCS_L);
    const int64_t nh = (int64_t)n * p.H + h;
    const int DV = p.nvt * TCS_BV;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
    uint64_t* q_full = bars + 0;     // [2] tiles landed
    uint64_t* k_full = bars + 2;
    uint64_t* v_full = bars + 4;
    uint64_t* q_empty = bars + 6;    // [2] tiles used up (MMA commit)
    uint64_t* k_empty = bars + 8;
    uint64_t* v_empty = bars + 10;
    uint64_t* g_full = bars + 12;    // [2] G = C B^T
    uint64_t* p_full = bars + 14;    // [2] P written
    uint64_t* vp_full = bars + 16;   // V' written (and dead rows zeroed)
    uint64_t* vp_free = bars + 18;   // V' used up (MMA commit)
    uint64_t* u_full = bars + 20;    // B^T V'
    uint64_t* u_free = bars + 21;    // ... read
    uint64_t* s_full = bars + 22;    // FWD: the state written as an operand
    uint64_t* y1_done = bars + 23;   // FWD: ... used up (MMA commit)
    uint64_t* y_full = bars + 24;    // C S^T and P X
    uint64_t* y_free = bars + 25;    // ... read
    uint64_t* drain = bars + 26;
    uint64_t* gate_full = bars + 27;              // [TCS_GATES] the chunk's gates written
    uint64_t* gate_free = gate_full + TCS_GATES;  // [TCS_GATES] ... read by all
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::TMEM_SLOT);
    auto gate = [&](int i) { return reinterpret_cast<TcsGate*>(smem + L::GATE + i % TCS_GATES * L::GATE_BYTES); };
    auto stage = [&](int i) { return smem + (i & 1) * L::STAGE; };
    auto chunk_of = [&](int i) { return rev ? nch - 1 - i : i; };
    auto row_of = [&](int i) { return first + (int64_t)chunk_of(i) * TCS_L; };
    auto len_of = [&](int i) -> int {
        const int64_t rem = count - (int64_t)chunk_of(i) * TCS_L;
        return rem < TCS_L ? (int)rem : TCS_L;
    };
    // every lane waits; the warp leaves together
    auto wait = [&](uint64_t* bar, int phase) -> bool {
        return __all_sync(0xffffffffu, tcs_wait(bar, phase));
    };

    if (warp == 0) {
        tc::tmem_alloc(tmem_slot, L::COLS);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&k_full[i], 1);
            mbar_init(&v_full[i], 1);
            mbar_init(&q_empty[i], 1);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&g_full[i], 1);
            mbar_init(&p_full[i], 8);
            mbar_init(&vp_full[i], 4 * L::VW);
            mbar_init(&vp_free[i], 1);
        }
        for (int i = 0; i < TCS_GATES; ++i) {
            mbar_init(&gate_full[i], 1);
            // FWD: the output rows are the last readers; else V' and the state read them
            mbar_init(&gate_free[i], OUT ? 4 : 4 + 4 * L::VW);
        }
        mbar_init(u_full, 1);
        mbar_init(u_free, 4);
        mbar_init(s_full, 4);
        mbar_init(y1_done, 1);
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

    // FWD: the launch's 7 x 72 registers are shared out 64 + 104 + 2 x 56 + 80 + 2 x 72
    if (warp < 4) {
        if constexpr (OUT) tc::reg_dec<64>();
    if (warp == 0) {
        // ------------------------------------------------------------ TMA
        if (lane == 0) {
            int nq = 0, nk = 0, nv = 0;  // tiles asked for
            for (int i = 0; i < nch; ++i) {
                uint8_t* s = stage(i);
                const int b = i & 1, use = (i >> 1) - 1, row = (int)row_of(i);
                // in the order in which chunk i - 2 gives its tiles back
                if (i >= 2 && !tcs_wait(&k_empty[b], use & 1)) break;
                tc::mbar_expect_tx(&k_full[b], L::KB);
#pragma unroll
                for (int e = 0; e < DQ / 64; ++e)
                    tc::tma_load_3d(s + L::K + e * 16384, map_k, e * 64, g, row, &k_full[b]);
                nk = i + 1;
                if constexpr (OUT) {
                    if (i >= 2 && !tcs_wait(&q_empty[b], use & 1)) break;
                    tc::mbar_expect_tx(&q_full[b], L::QB);
#pragma unroll
                    for (int e = 0; e < DQ / 64; ++e)
                        tc::tma_load_3d(s + L::Q + e * 16384, &tm_q, e * 64, g, row, &q_full[b]);
                    nq = i + 1;
                }
                if (i >= 2 && !tcs_wait(&v_empty[b], use & 1)) break;
                tc::mbar_expect_tx(&v_full[b], 16384);
                tc::tma_load_3d(s + L::V, map_v, vt * TCS_BV, h, row, &v_full[b]);
                nv = i + 1;
            }
            // whatever was asked for has landed before the CTA may leave
            auto landed = [&](uint64_t* bar, int cnt) {
                for (int i = cnt > 2 ? cnt - 2 : 0; i < cnt; ++i)
                    tcs_wait(&bar[i & 1], (i >> 1) & 1);
            };
            landed(k_full, nk);
            landed(q_full, nq);
            landed(v_full, nv);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue
        // per chunk: B^T V', C S^T, the next chunk's G, P X; what a product waits for is ready by
        // the time the one before is issued, so the pipe stays fed
        if (lane == 0) {
            constexpr uint32_t ID_G = tc::idesc(1, 0, 0, 128, 128);  // tokens x tokens
            constexpr uint32_t ID_Y = tc::idesc(1, 0, 1, 128, 64);   // tokens x value channels
            constexpr uint32_t ID_U = tc::idesc(1, 1, 1, 128, 64 * L::NT);  // key x value channels, terms
            auto issue_g = [&](int i) -> bool {
                if (!tcs_wait(&q_full[i & 1], (i >> 1) & 1) ||
                    !tcs_wait(&k_full[i & 1], (i >> 1) & 1))
                    return false;
                const uint32_t q = smem_u32(stage(i) + L::Q), k = smem_u32(stage(i) + L::K);
                tcs_mma<DQ / 16>(tmem + L::COL_G + (i & 1) * 128, tc::sw128_desc(q, 16, 1024),
                                 tc::sw128_desc(k, 16, 1024), ID_G, 2, 2, 1024 - 8, 1024 - 8);
                tc::mma_commit(&g_full[i & 1]);
                return true;
            };
            bool ok = !OUT || nch == 0 || issue_g(0);
            for (int i = 0; ok && i < nch; ++i) {
                const int s = i & 1, ph = (i >> 1) & 1;
                const uint32_t q = smem_u32(stage(i) + L::Q), k = smem_u32(stage(i) + L::K),
                               v = smem_u32(stage(i) + L::V);
                // X has landed before V' is made from it, B before G
                if (!OUT && !(ok = tcs_wait(&k_full[s], ph))) break;
                if (!(ok = tcs_wait(vp_full, i & 1))) break;
                if (i > 0 && !(ok = tcs_wait(u_free, (i - 1) & 1))) break;
                tc::fence_after_sync();
                const uint32_t vp = smem_u32(smem + L::VP);
                // (DQ = 64: rows 64..127 read the next tile and are not used)
                tcs_mma<8>(tmem + L::COL_U, tc::sw128_desc(k, 16384, 1024),
                           tc::sw128_desc(vp, 16384, 1024), ID_U, 128, 128, 0, 0);
                tc::mma_commit(u_full);
                tc::mma_commit(vp_free);
                tc::mma_commit(&k_empty[s]);
                if constexpr (OUT) {
                    if (!(ok = tcs_wait(s_full, i & 1))) break;
                    if (i > 0 && !(ok = tcs_wait(y_free, (i - 1) & 1))) break;
                    tc::fence_after_sync();
                    const uint32_t sb = smem_u32(smem + L::S);
                    tcs_mma<DQ / 16>(tmem + L::COL_Y1, tc::sw128_desc(q, 16, 1024),
                                     tc::sw128_desc(sb, 16384, 1024), ID_Y, 2, 128, 1024 - 8, 0);
                    tc::mma_commit(y1_done);
                    tc::mma_commit(&q_empty[s]);
                    if (i + 1 < nch && !(ok = issue_g(i + 1))) break;
                    if (!(ok = tcs_wait(&p_full[s], ph))) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int e = 0; e < 16; ++e)  // P's leading terms, then the second
                        tc::mma_bf16_ts(tmem + L::COL_Y2, tmem + L::COL_G + s * 128 + 16 * (e & 7) + (e & 8),
                                        tc::sw128_desc(v + (e & 7) * 2048, 16384, 1024), ID_Y, e != 0);
                    tc::mma_commit(y_full);
                }
                tc::mma_commit(&v_empty[s]);
            }
            tc::mma_commit(drain);
            tcs_wait(drain, 0);
        }
    } else {
        // ------------------------------------------------------------ gates, every other chunk
        const float A = p.A[h], bias = p.dt_bias ? p.dt_bias[h] : 0.f;
        for (int i = warp - 2; i < nch; i += 2) {
            if (i >= TCS_GATES && !wait(&gate_free[i % TCS_GATES], i / TCS_GATES - 1)) break;
            tcs_gates(rev, gate(i), p.dt + row_of(i) * p.H + h, p.H, len_of(i), A, bias, p.softplus, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&gate_full[i % TCS_GATES]);
        }
    }
    } else if (warp < 8) {
        if constexpr (OUT) tc::reg_inc<104>();
        // ------------------------------------------------------------ state
        const int r = tid - 128;  // key channel
        const bool on = DQ == 128 || r < DQ;
        float S[TCS_BV];
        const int64_t sbase = (nh * DV + vt * TCS_BV) * DQ + r;  // stored [value][key]
        const float* s_in = L::SEG ? nullptr : rev ? p.dST : p.S_in;
#pragma unroll
        for (int j = 0; j < TCS_BV; ++j)
            S[j] = on && s_in ? s_in[sbase + (int64_t)j * DQ] : 0.f;
        if constexpr (!L::SEG) {  // the segments in front, the nearest last
            for (int e = rev ? base + segs - 1 : base; on && e != slot; e += rev ? -1 : 1) {
                const int64_t at = (half + e) * p.H + h;
                const float d = ex2f(p.seg_decay[at]);
                const float* a = p.seg_state + (at * p.nvt + vt) * (TCS_BV * DQ) + r;
#pragma unroll
                for (int j = 0; j < TCS_BV; ++j) S[j] = fmaf(d, S[j], a[j * DQ]);
            }
        }
        float total = 0.f;  // SEG: log2 decay so far
        uint8_t* so = smem + L::S;
        for (int i = 0; i < nch; ++i) {
            if (!wait(&gate_full[i % TCS_GATES], i / TCS_GATES)) break;
            // all that is needed of the slot, before it is given back
            const float log_decay = gate(i)->bh[8] + gate(i)->bl[8];
            const float decay = ex2f(log_decay);
            if constexpr (L::SEG) total += log_decay;
            if (!OUT) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&gate_free[i % TCS_GATES]);
            }
            if constexpr (OUT) {
                if (i > 0 && !wait(y1_done, i - 1)) break;
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
                __syncwarp();
                if (lane == 0) mbar_arrive(s_full);
            } else if constexpr (!L::SEG) {
                // images: rows of 128 bytes as the products read them, the terms one after another
                const int64_t cs = first / TCS_L + n + chunk_of(i);
                if (on) {
                    if (lane == 0) tc::bulk_wait_read_all();
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            split3_rn(S[8 * j + 2 * e], S[8 * j + 2 * e + 1], t0[e], t1[e], t2[e]);
                        uint4* o = reinterpret_cast<uint4*>(so + tc::sw128_off(r, j));
                        o[0] = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                        o[1024] = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                        o[2048] = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                    }
                    tc::fence_async_smem();
                    __syncwarp();
                    if (lane == 0 && OSDN_IN_BOUNDS(cs, ssm_slots(p.rows, p.N, TCS_L))) {
                        const uint32_t w0 = (warp & 3) * 4096;
                        uint8_t* im = (rev ? p.img_r : p.img) + w0 +
                                      ((cs * p.H + h) * (TCS_TERMS * p.nvt) + vt) * (DQ * 128);
#pragma unroll
                        for (int t = 0; t < TCS_TERMS; ++t)
                            tc::bulk_store(im + t * p.nvt * (DQ * 128), so + t * 16384 + w0, 4096);
                        tc::bulk_commit();
                    }
                }
            }
            if (!wait(u_full, i)) break;
            tc::fence_after_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float u[L::NT][16];
#pragma unroll
                for (int t = 0; t < L::NT; ++t)
                    tc::tmem_ld16(tmem + tlane + L::COL_U + 64 * t + 16 * q, u[t]);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; e += 2) {
                    float2 a = make_float2(u[0][e], u[0][e + 1]);
                    float2 b = make_float2(u[1][e], u[1][e + 1]);
                    if constexpr (L::NT == 3) b = __fadd2_rn(b, make_float2(u[2][e], u[2][e + 1]));
                    const float2 t = __ffma2_rn(make_float2(decay, decay),
                                                make_float2(S[16 * q + e], S[16 * q + e + 1]),
                                                __fadd2_rn(a, b));
                    S[16 * q + e] = t.x;
                    S[16 * q + e + 1] = t.y;
                }
            }
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(u_free);
        }
        if constexpr (L::SEG) {
            const int64_t at = (half + slot) * p.H + h;
            if (on && OSDN_IN_BOUNDS(slot, p.rows / p.seg + p.N)) {
#pragma unroll
                for (int j = 0; j < TCS_BV; ++j)
                    p.seg_state[(at * p.nvt + vt) * (TCS_BV * DQ) + j * DQ + r] = S[j];
                if (r == 0 && vt == 0) p.seg_decay[at] = total;
            }
        } else {
            float* s_out = rev ? p.dS0 : p.S_out;
            if (on && s_out && (rev ? seg == 0 : last) && OSDN_IN_BOUNDS(nh, (int64_t)p.N * p.H)) {
#pragma unroll
                for (int j = 0; j < TCS_BV; ++j) s_out[sbase + (int64_t)j * DQ] = S[j];
            }
        }
        if (!OUT && lane == 0) tc::bulk_wait_all();
    } else if (warp < 8 + 4 * L::VW) {
        if constexpr (OUT) tc::reg_dec<56>();
        // ------------------------------------------------------------ V'
        const int r = tid & 127, b = r >> 4;  // token of the chunk
        constexpr int NJ = 8 / L::VW;         // 8-channel groups of a thread
        const int j0 = (warp - 8) / 4 * NJ;
        for (int i = 0; i < nch; ++i) {
            if (!wait(&gate_full[i % TCS_GATES], i / TCS_GATES) || !wait(&v_full[i & 1], i >> 1)) break;
            const TcsGate* gt = gate(i);
            // 2^(cum_L - end_b) 2^(end_b - cum_r) step;  backwards: 2^(base_b + l_r)
            const float e = rev ? gt->bh[b] + gt->bl[b]
                                : (gt->bh[8] - gt->bh[b + 1]) + (gt->bl[8] - gt->bl[b + 1]);
            const float w = ex2f(e) * gt->g[r];
            const float2 w2 = make_float2(w, w);
            uint8_t* v = stage(i) + L::V;
            uint8_t* vp = smem + L::VP;
            const bool live = r < len_of(i);
            if (len_of(i) < TCS_L && !wait(&k_full[i & 1], i >> 1)) break;
            if (!live) {  // the next sequence's row: 0 x NaN must not reach a sum
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int j = j0; j < j0 + NJ; ++j) {
                    const uint32_t off = tc::sw128_off(r, j);
                    *reinterpret_cast<uint4*>(v + off) = z;
#pragma unroll
                    for (int q = 0; q < DQ / 64; ++q)
                        *reinterpret_cast<uint4*>(stage(i) + L::K + q * 16384 + off) = z;
                }
            }
            uint4 x[NJ];
#pragma unroll
            for (int j = 0; j < NJ; ++j) x[j] = *reinterpret_cast<const uint4*>(v + tc::sw128_off(r, j0 + j));
            if (i > 0 && !wait(vp_free, i - 1)) break;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint32_t xw[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
                uint32_t t0[4], t1[4], t2[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 t = __fmul2_rn(w2, make_float2(__uint_as_float(xw[k] << 16),
                                                                __uint_as_float(xw[k] & 0xffff0000u)));
                    if constexpr (L::NT == 3) split3_rn(t.x, t.y, t0[k], t1[k], t2[k]);
                    else split2_rn(t.x, t.y, t0[k], t1[k]);
                    if (!live) t0[k] = t1[k] = t2[k] = 0;
                }
                uint4* o = reinterpret_cast<uint4*>(vp + tc::sw128_off(r, j0 + j));
                o[0] = make_uint4(t0[0], t0[1], t0[2], t0[3]);
                o[1024] = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                if constexpr (L::NT == 3) o[2048] = make_uint4(t2[0], t2[1], t2[2], t2[3]);
            }
            tc::fence_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(vp_full);
                if (!OUT) mbar_arrive(&gate_free[i % TCS_GATES]);
            }
        }
    } else if constexpr (OUT) {
    if (warp < 20) {
        tc::reg_inc<80>();
        // ------------------------------------------------------------ output rows
        const int r = tid & 127;  // token of the chunk
        const float skip = p.D ? p.D[h] : 0.f;
        auto output = [&](int i) -> bool {
            const TcsGate* gt = gate(i);
            const bool live = r < len_of(i);
            const int64_t at = ((row_of(i) + r) * p.H + h) * DV + vt * TCS_BV;
            const bool add = p.D && live;
            uint4 xr[8];  // in flight while the products are waited for
#pragma unroll
            for (int j = 0; j < 8; ++j)
                xr[j] = add ? __ldg(reinterpret_cast<const uint4*>(p.x + at) + j) : make_uint4(0, 0, 0, 0);
            const float rf = ex2f(gt->bh[r >> 4] + gt->l[r] + gt->bl[r >> 4]);
            if (!wait(y_full, i)) return false;
            tc::fence_after_sync();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float a[16], b[16];
                tc::tmem_ld16(tmem + tlane + L::COL_Y1 + 16 * q, a);
                tc::tmem_ld16(tmem + tlane + L::COL_Y2 + 16 * q, b);
                tc::tmem_ld_wait();
                if (q == 3) {  // all read: the next products may overwrite them
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(y_free);
                        mbar_arrive(&gate_free[i % TCS_GATES]);
                    }
                }
                const uint32_t xw[8] = {xr[2 * q].x, xr[2 * q].y, xr[2 * q].z, xr[2 * q].w,
                                        xr[2 * q + 1].x, xr[2 * q + 1].y, xr[2 * q + 1].z, xr[2 * q + 1].w};
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 y = __ffma2_rn(
                        make_float2(skip, skip),
                        make_float2(__uint_as_float(xw[e] << 16), __uint_as_float(xw[e] & 0xffff0000u)),
                        __ffma2_rn(make_float2(rf, rf), make_float2(a[2 * e], a[2 * e + 1]),
                                   make_float2(b[2 * e], b[2 * e + 1])));
                    w[e] = pack2_rn(y.x, y.y);
                }
                if (live && OSDN_IN_BOUNDS(row_of(i) + r, p.rows)) {
                    uint4* o = reinterpret_cast<uint4*>(p.y + at) + 2 * q;
                    o[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    o[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
                __syncwarp();
            }
            return true;
        };
        for (int i = 0; i < nch; ++i)
            if (!wait(&gate_full[i % TCS_GATES], i / TCS_GATES) || !output(i)) break;
    } else {
        // ------------------------------------------------------------ P
        // two warpgroups share P's columns by sub-blocks; P's 16 columns of sub-block b lie over their
        // own scores, packed: the leading terms over the first half, the second over the other
        const int wg = (warp - 20) >> 2, wq = warp & 3;
        const int r = 32 * wq + lane, rb = r >> 4;
        for (int i = 0; i < nch; ++i) {
            if (!wait(&gate_full[i % TCS_GATES], i / TCS_GATES)) break;
            const TcsGate* gt = gate(i);
            const float lr = gt->l[r], bh = gt->bh[rb], bl = gt->bl[rb];
            if (!wait(&g_full[i & 1], i >> 1)) break;
            tc::fence_after_sync();
            const uint32_t col = tmem + tlane + L::COL_G + (i & 1) * 128;
            float x[16];
            uint32_t w[16];  // two terms
#pragma unroll 1
            for (int k = 0; k < wq; ++k) {  // sub-blocks in front of every row of the warp
                const int b = 2 * k + wg;
                tc::tmem_ld16(col + 16 * b, x);
                const float f = ex2f((bh - gt->bh[b + 1]) + (bl - gt->bl[b + 1]) + lr);
                const float4* gp = reinterpret_cast<const float4*>(gt->g + 16 * b);
                float4 g4[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) g4[e] = gp[e];
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f2 = make_float2(f, f);
                    const float2 t = __fmul2_rn(__fmul2_rn(f2, make_float2(g4[e].x, g4[e].y)),
                                                make_float2(x[4 * e], x[4 * e + 1]));
                    const float2 u = __fmul2_rn(__fmul2_rn(f2, make_float2(g4[e].z, g4[e].w)),
                                                make_float2(x[4 * e + 2], x[4 * e + 3]));
                    split2_rn(t.x, t.y, w[2 * e], w[8 + 2 * e]);
                    split2_rn(u.x, u.y, w[2 * e + 1], w[8 + 2 * e + 1]);
                }
                tc::tmem_st8(col + 16 * b, w);
                tc::tmem_st8(col + 16 * b + 8, w + 8);
            }
            {  // the sub-blocks on the diagonal: wg = 0: of the first 16 rows, wg = 1: of the others
                const int b = 2 * wq + wg;
                tc::tmem_ld16(col + 16 * b, x);
                // cum_r - cum_j: l_r - l_j where the sub-block is the row's own, (its sum - l_j) + l_r
                // where it is the one in front
                const bool own = rb == b;
                const float dh = own ? lr : gt->th[b], dl = own ? gt->l2[r] : gt->tl[b];
                const float rest = own ? 0.f : lr;
                const float4* lp = reinterpret_cast<const float4*>(gt->l + 16 * b);
                const float4* mp = reinterpret_cast<const float4*>(gt->l2 + 16 * b);
                const float4* sp = reinterpret_cast<const float4*>(gt->st + 16 * b);
                const int c0 = 16 * b;
                float wt[16];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float4 l4 = lp[e], m4 = mp[e], s4 = sp[e];
                    wt[4 * e] = ex2f((dh - l4.x) + (dl - m4.x) + rest) * s4.x;
                    wt[4 * e + 1] = ex2f((dh - l4.y) + (dl - m4.y) + rest) * s4.y;
                    wt[4 * e + 2] = ex2f((dh - l4.z) + (dl - m4.z) + rest) * s4.z;
                    wt[4 * e + 3] = ex2f((dh - l4.w) + (dl - m4.w) + rest) * s4.w;
                }
                tc::tmem_ld_wait();
                // what lies past the diagonal is left out, infinities and NaN too
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    split2_rn(c0 + 2 * e > r ? 0.f : x[2 * e] * wt[2 * e],
                              c0 + 2 * e + 1 > r ? 0.f : x[2 * e + 1] * wt[2 * e + 1], w[e], w[8 + e]);
                __syncwarp();
                tc::tmem_st8(col + 16 * b, w);
                tc::tmem_st8(col + 16 * b + 8, w + 8);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e] = 0;
#pragma unroll 1
            for (int k = wq + 1; k < 4; ++k) {
                tc::tmem_st8(col + 16 * (2 * k + wg), w);
                tc::tmem_st8(col + 16 * (2 * k + wg) + 8, w);
            }
            tc::tmem_st_wait();
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[i & 1]);
        }
    }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 0) tc::tmem_dealloc(tmem, L::COLS);
}

}  // namespace osdn
