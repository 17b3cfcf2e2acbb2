// ssm_tc_bwd.cuh -- the selective scan's gradient on the sm_100a tensor cores (bf16 tokens): one
// CTA per chunk of 128 tokens and head, after the chains of ssm_tc.cuh have stored the state S in
// front of every chunk and the gradient R that reaches the state behind it.
//
// With L_ij = 2^(cum_i - cum_j) for i >= j (0 otherwise), all within the chunk:
//   dx_j = step_j [ sum_i (b_j.c_i) L_ij dy_i + 2^(cum_L - cum_j) R b_j ] + D dy_j
//   db_j = step_j [ sum_i (x_j.dy_i) L_ij c_i + 2^(cum_L - cum_j) R^T x_j ]
//   dc_i = sum_j (dy_i.x_j) L_ij step_j b_j + 2^cum_i S^T dy_i
// and for the steps, with W_ij = (c_i.b_j)(dy_i.x_j) L_ij in fp32:
//   pos_i = sum_{j < i} W_ij step_j + 2^cum_i c_i.(S^T dy_i),   ri_j = sum_{i > j} W_ij,
//   rn_j = 2^(cum_L - cum_j) b_j.(R^T x_j)
//   d(log a_t) = sum_{i >= t} (pos_i - step_i ri_i) + sum_{j < t} step_j rn_j + 2^cum_L <R, S>
//   dstep_t = ri_t + W_tt + rn_t + A d(log a_t)   (sums over the chunk; see ssm_gate_kernel)
// The pairs inside the chunk enter both sums as one and the same W_ij, summed over rows by each
// thread and over columns across them, so what cancels between the sums does so to fp32 (two
// evaluations of W, each good to 2^-22, left dA wrong by up to 1e-5); what crosses the chunk's
// ends is summed without cancelling.
// Rounding: the weighted scores go into a product as two bf16 terms (with one, dx, db and dc were
// 2.3e-3 off in L2 norm, where rounding the results alone gives 1.66e-3); S and R as three bf16
// terms where pos and rn are made from them (with two, dA was up to 1e-5 off), as two in R b_j.
//
// Nine products a chunk: three of scores (x.dy in both orientations: P X-like products read the
// weighted scores as rows), three with the states, three with the weighted scores.  Tensor
// memory holds two score tiles and two accumulators, and dc takes the place of the first scores
// once they are used up; the state products go in first, are scaled by their rows' decays in
// place, and the weighted scores accumulate on top.
//
// Warps 0-15: element-wise work, thread = row, the four warpgroups taking every fourth 16-column
// sub-block of scores and a quarter of the outputs' columns; warp 16: loads and MMAs; 17: gates.
// The images' terms pass through two slots of shared memory, each loaded again once used up.
// 340M layer (B=8, T=2048, H=8, 128 x 128): 131 us for 361 MB read and 81 written, seven rounds
// of CTAs at 19 us each (16 with one term of the weighted scores and two in <R, S>).  A CTA's products, its element-wise work and its stores follow one
// another, and shared memory (four tiles, two terms) leaves room for one CTA on an SM.
#pragma once

#include <stddef.h>

#include "ssm_tc.cuh"

namespace osdn {

struct TcgArgs {
    const float *dt, *A, *dt_bias, *D;
    const uint8_t *img, *img_r;    // S in front of each chunk, R behind it
    __nv_bfloat16* dx;
    __nv_bfloat16 *db, *dc;        // G == H: written; else null
    float *dbh, *dch;              // G < H: the heads' shares [rows][H][DK]
    float *pos, *ri, *rn;          // [4][H][rows], a share from each warpgroup
    float* gs;                     // 2^cum_L <R, S> [16][slots][H], a share from each warp
    float* vk;                     // dy . x [H][rows], or null
    float* wd;                     // W_tt [H][rows]
    const int32_t* cu;
    int64_t rows, slots;
    int N, T, H, G, softplus, round;  // round: CTAs that run at a time
};

template <int DK, int DV> struct TcgSmem {
    static constexpr uint32_t TK = DK / 64 * 16384, TV = DV / 64 * 16384;
    static constexpr uint32_t X = 0, DY = TV, B = 2 * TV, C = 2 * TV + TK, IMG = 2 * TV + 2 * TK;
    static constexpr uint32_t IMG_ONE = DK * 128, TERM = DV / 64 * IMG_ONE;
    static constexpr uint32_t GATE = IMG + 2 * TERM;
    static constexpr uint32_t ROWSUM = GATE + 2704;  // [4 row quarters][128] shares of sum_j W_ij step_j
    static constexpr uint32_t BAR = ROWSUM + 4 * TCS_L * 4;
    static constexpr uint32_t TMEM_SLOT = BAR + 20 * 8;
    static constexpr size_t BYTES = TMEM_SLOT + 16 + 1024;
    static constexpr int THREADS = 576;
};
static_assert(TcgSmem<128, 128>::BYTES <= 232448, "shared memory");

// The chunk's gates: TcsGate's arrays of the forward orientation, and 2^l of the other.
struct TcgGate {
    float r[TCS_L];
    TcsGate f;
};
static_assert(sizeof(TcgGate) <= 2704, "gate arrays");
static_assert(offsetof(TcgGate, f) % 16 == 0 && offsetof(TcsGate, g) % 16 == 0 &&
                  offsetof(TcsGate, st) % 16 == 0 && offsetof(TcsGate, l2) % 16 == 0 && TcsSmem<128, TCS_FWD>::GATE_BYTES % 16 == 0,
              "the arrays are read 16 bytes at a time");

// K steps of a product: n MMAs, start addresses moving by da / db (16-byte units) per step and by
// ga / gb more after every fourth; `acc`: add to the accumulator from the first step on.
template <int n>
__device__ __forceinline__ void tcg_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t da,
                                        uint32_t db, uint32_t ga, uint32_t gb, bool acc) {
#pragma unroll
    for (int e = 0; e < n; ++e)
        tc::mma_bf16(d, a + e * da + (e >> 2) * ga, b + e * db + (e >> 2) * gb, id, acc || e != 0);
}

template <int DK, int DV>
__global__ void __launch_bounds__(TcgSmem<DK, DV>::THREADS, 1)
ssm_tc_grad_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_dy,
                   const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_c,
                   const TcgArgs p) {
    using L = TcgSmem<DK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_align1024(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t slot = blockIdx.x / p.H;
    const int h = (int)(blockIdx.x - slot * p.H), g = h / (p.H / p.G);
    int n, chunk;
    int64_t first, count;
    if (!token_block(p.cu, p.N, p.T, TCS_L, slot, n, chunk) ||
        !seq_range(p.cu, n, p.N, p.T, first, count))
        return;
    const int64_t start = (int64_t)chunk * TCS_L;
    if (start >= count) return;  // a number that no chunk has; all uniform over the CTA
    const int64_t row0 = first + start;
    const int len = count - start < TCS_L ? (int)(count - start) : TCS_L;

    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR);
    uint64_t* tiles = bars + 0;    // x, dy, b, c landed
    uint64_t* img0 = bars + 1;     // slots 0 and 1: a term landed
    uint64_t* img1 = bars + 14;
    uint64_t* use0 = bars + 15;    // ... used up (MMA commit)
    uint64_t* use1 = bars + 8;
    uint64_t* gates = bars + 2;
    uint64_t* zeroed = bars + 3;   // dead rows of a short chunk
    uint64_t* sc1 = bars + 4;      // scores [j][i]
    uint64_t* in1 = bars + 5;      // R products
    uint64_t* ew1 = bars + 6;      // weighted scores and scaled R products written
    uint64_t* acc1 = bars + 7;     // dx, db complete
    uint64_t* sc2 = bars + 9;      // scores [i][j]
    uint64_t* in2 = bars + 10;     // S product
    uint64_t* ew2 = bars + 11;
    uint64_t* acc2 = bars + 12;    // dc complete
    uint64_t* drain = bars + 13;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::TMEM_SLOT);
    TcgGate* gt = reinterpret_cast<TcgGate*>(smem + L::GATE);
    auto wait = [&](uint64_t* bar, int phase) -> bool {
        return __all_sync(0xffffffffu, tcs_wait(bar, phase));
    };

    if (warp == 16) {
        tc::tmem_alloc(tmem_slot, 512);
        tc::tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 16; ++i) {
            uint64_t* b = bars + i;
            mbar_init(b, b == zeroed || b == ew1 || b == ew2 ? 16 : 1);
        }
        tc::fence_mbar_init();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t T0 = 0, T1 = 128, A0 = 256, A1 = 384;  // score tiles, accumulators

    if (warp == 16) {
        // ------------------------------------------------------------ loads and MMAs
        if (lane == 0) {
            const int64_t at = (slot * p.H + h) * (int64_t)(TCS_TERMS * L::TERM);
            const uint8_t *im = p.img + at, *imr = p.img_r + at;
            auto load_term = [&](int s, const uint8_t* src) {
                uint64_t* bar = s ? img1 : img0;
                tc::mbar_expect_tx(bar, L::TERM);
                tc::bulk_load(smem + L::IMG + s * L::TERM, src, L::TERM, bar);
            };
            tc::mbar_expect_tx(tiles, 2 * L::TV + 2 * L::TK);
#pragma unroll
            for (int e = 0; e < DK / 64; ++e) {
                tc::tma_load_3d(smem + L::B + e * 16384, &tm_b, e * 64, g, (int)row0, tiles);
                tc::tma_load_3d(smem + L::C + e * 16384, &tm_c, e * 64, g, (int)row0, tiles);
            }
#pragma unroll
            for (int e = 0; e < DV / 64; ++e) {
                tc::tma_load_3d(smem + L::X + e * 16384, &tm_x, e * 64, h, (int)row0, tiles);
                tc::tma_load_3d(smem + L::DY + e * 16384, &tm_dy, e * 64, h, (int)row0, tiles);
            }
            load_term(0, imr);
            load_term(1, imr + L::TERM);
            // What the CTA that follows here about a round later will load, into L2 meanwhile: its
            // first loads then do not wait for HBM.  Asked for once this CTA's own loads (all but
            // one term) are under way, which would stand in line behind it: 226 us at the 340M
            // shape (the whole gradient), 243 when asked for at the start, 230 without.
            const int64_t ahead = (int64_t)blockIdx.x + p.round, aslot = ahead / p.H;
            const int ah = (int)(ahead - aslot * p.H), ag = ah / (p.H / p.G);
            int an, achunk;
            int64_t ar = -1;
            if (aslot < p.slots && token_block(p.cu, p.N, p.T, TCS_L, aslot, an, achunk))
                ar = (p.cu ? (int64_t)__ldg(p.cu + an) : (int64_t)an * p.T) + (int64_t)achunk * TCS_L;
            if (ar >= p.rows) ar = -1;
            const int64_t aat = (aslot * p.H + ah) * (int64_t)(TCS_TERMS * L::TERM);
            int n0 = 1, n1 = 1;  // terms asked for
            constexpr uint32_t ID_S = tc::idesc(1, 0, 0, 128, 128);   // scores
            constexpr uint32_t ID_KK = tc::idesc(1, 0, 0, 128, DK);   // rows x key channels, K-major
            constexpr uint32_t ID_MV = tc::idesc(1, 0, 1, 128, DV);   // rows x value channels, MN-major
            constexpr uint32_t ID_MK = tc::idesc(1, 0, 1, 128, DK);
            const uint32_t ax = smem_u32(smem + L::X), ady = smem_u32(smem + L::DY),
                           ab = smem_u32(smem + L::B), ac = smem_u32(smem + L::C),
                           ai = smem_u32(smem + L::IMG);
            auto kd = [](uint32_t a) { return tc::sw128_desc(a, 16, 1024); };
            auto scores = [&](uint32_t t, uint32_t a, uint32_t b, auto steps) {
                tcg_mma<decltype(steps)::value>(tmem + t, kd(a), kd(b), ID_S, 2, 2, 1024 - 8, 1024 - 8,
                                                false);
            };
            using NK = std::integral_constant<int, DK / 16>;
            using NV = std::integral_constant<int, DV / 16>;
            // a [tokens][value channels] times the state's [key][value] in slot s
            auto state_k = [&](uint32_t d, uint32_t a, int s, bool acc) {
                tcg_mma<DV / 16>(tmem + d, kd(a), kd(ai + s * L::TERM), ID_KK, 2, 2, 1024 - 8,
                                 (L::IMG_ONE >> 4) - 8, acc);
            };
            // weighted scores, two terms, times a token tile, added
            auto weighted = [&](uint32_t d, uint32_t s, uint32_t b, uint32_t id) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    tc::mma_bf16_ts(tmem + d, tmem + s + 16 * (e & 7) + (e & 8),
                                    tc::sw128_desc(b + (e & 7) * 2048, 16384, 1024), id, 1);
            };
            // R b_j, R's term in slot s: key channels summed, [key][value] read MN-major
            auto state_v = [&](int s, bool acc) {
                tcg_mma<DK / 16>(tmem + A0, kd(ab), tc::sw128_desc(ai + s * L::TERM, L::IMG_ONE, 1024),
                                 ID_MV, 2, 128, 1024 - 8, 0, acc);
            };
            bool ok = tcs_wait(tiles, 0) && (len == TCS_L || tcs_wait(zeroed, 0));
            if (ok) {
                scores(T0, ab, ac, NK{});   // b_j . c_i
                scores(T1, ax, ady, NV{});  // x_j . dy_i
                tc::mma_commit(sc1);
                ok = tcs_wait(img0, 0);
            }
            if (ok) {
                state_v(0, false);          // R b_j
                state_k(A1, ax, 0, false);  // R^T x_j
                tc::mma_commit(use0);
                ok = tcs_wait(img1, 0);
            }
            if (ok) {
                state_v(1, true);
                state_k(A1, ax, 1, true);
                tc::mma_commit(use1);
                ok = tcs_wait(use0, 0);
            }
            if (ok) {
                load_term(0, imr + 2 * L::TERM);
                n0 = 2;
                ok = tcs_wait(use1, 0);
            }
            if (ok) {
                load_term(1, im);
                n1 = 2;
                ok = tcs_wait(img0, 1);
            }
            if (ok) {
                state_k(A1, ax, 0, true);
                tc::mma_commit(in1);
                ok = tcs_wait(in1, 0);
            }
            if (ok) {
                load_term(0, im + L::TERM);
                n0 = 3;
                if (ar >= 0) {
#pragma unroll
                    for (int e = 0; e < DK / 64; ++e) {
                        tc::tma_prefetch_3d(&tm_b, e * 64, ag, (int)ar);
                        tc::tma_prefetch_3d(&tm_c, e * 64, ag, (int)ar);
                    }
#pragma unroll
                    for (int e = 0; e < DV / 64; ++e) {
                        tc::tma_prefetch_3d(&tm_x, e * 64, ah, (int)ar);
                        tc::tma_prefetch_3d(&tm_dy, e * 64, ah, (int)ar);
                    }
                }
                ok = tcs_wait(ew1, 0);
            }
            if (ok) {
                tc::fence_after_sync();
                weighted(A0, T0, ady, ID_MV);
                weighted(A1, T1, ac, ID_MK);
                tc::mma_commit(acc1);
                ok = tcs_wait(acc1, 0);  // T0 and T1 used up: nothing orders products with
            }                            // different accumulators but a wait
            if (ok) {
                tc::fence_after_sync();
                scores(T1, ady, ax, NV{});  // dy_i . x_j
                tc::mma_commit(sc2);
                ok = tcs_wait(img1, 1);
            }
            if (ok) {
                state_k(T0, ady, 1, false);  // S^T dy_i
                tc::mma_commit(use1);
                ok = tcs_wait(use1, 1);
            }
            if (ok) {
                load_term(1, im + 2 * L::TERM);
                n1 = 3;
                if (ar >= 0) {
                    tc::bulk_prefetch(p.img_r + aat, TCS_TERMS * L::TERM);
                    tc::bulk_prefetch(p.img + aat, TCS_TERMS * L::TERM);
                }
                ok = tcs_wait(img0, 2);
            }
            if (ok) {
                state_k(T0, ady, 0, true);
                ok = tcs_wait(img1, 2);
            }
            if (ok) {
                state_k(T0, ady, 1, true);
                tc::mma_commit(in2);
                ok = tcs_wait(ew2, 0);
            }
            if (ok) {
                tc::fence_after_sync();
                weighted(T0, T1, ab, ID_MK);
                tc::mma_commit(acc2);
            }
            tc::mma_commit(drain);
            tcs_wait(drain, 0);
            tcs_wait(tiles, 0);             // nothing in flight when the CTA leaves
            tcs_wait(img0, n0 - 1);
            tcs_wait(img1, n1 - 1);
        }
    } else if (warp == 17) {
        tcs_gates(false, &gt->f, p.dt + row0 * p.H + h, p.H, len, p.A[h], p.dt_bias ? p.dt_bias[h] : 0.f,
                         p.softplus, lane);
        __syncwarp();
#pragma unroll
        for (int t = lane; t < TCS_L; t += 32) gt->r[t] = ex2f(gt->f.l[t]);
        __syncwarp();
        if (lane == 0) mbar_arrive(gates);
    } else {
        const int wg = warp >> 2, wq = warp & 3;
        const int r = 32 * wq + lane, rb = r >> 4;
        const uint32_t tl = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const bool live = r < len;
        const int64_t row = row0 + r;
        const TcsGate* f = &gt->f;
        // 16 bytes (8 channels from ch on) of this thread's row of a token tile
        auto tile16 = [&](uint32_t tile, int ch) {
            return *reinterpret_cast<const uint4*>(smem + tile + (ch >> 6) * 16384 +
                                                   tc::sw128_off(r, (ch & 63) >> 3));
        };
        // 32 channels (64 bytes) of each of the warp's rows, packed in w: four lanes exchange their
        // quarters, so that a store covers 64 bytes of 8 rows instead of 16 of 32
        auto store_rows = [&](__nv_bfloat16* base, int64_t stride, uint32_t (&w)[16]) {
            const bool odd1 = lane & 1, odd2 = lane & 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // quarters 0 <-> 1 and 2 <-> 3 with the neighbour
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    const uint32_t t = __shfl_xor_sync(0xffffffffu, odd1 ? w[4 * q + e] : w[4 * q + 4 + e], 1);
                    if (odd1) w[4 * q + e] = t; else w[4 * q + 4 + e] = t;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // 0 <-> 2 and 1 <-> 3 with the pair next to it
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t t = __shfl_xor_sync(0xffffffffu, odd2 ? w[4 * q + e] : w[4 * q + 8 + e], 2);
                    if (odd2) w[4 * q + e] = t; else w[4 * q + 8 + e] = t;
                }
            }
            const int r4 = 32 * wq + (lane & ~3);  // w[4 k ..]: this lane's quarter of row r4 + k
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (r4 + k < len && OSDN_IN_BOUNDS(row0 + r4 + k, p.rows))
                    *reinterpret_cast<uint4*>(base + (row0 + r4 + k) * stride + 8 * (lane & 3)) =
                        make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        };
        // this warpgroup's quarter of rows of W channels (all heads: stride H * W)
        auto put_bf16 = [&](__nv_bfloat16* base, auto width, uint32_t (&w)[16]) {
            constexpr int W = decltype(width)::value;
            __nv_bfloat16* o = base + wg * (W / 4);
            if constexpr (W == 128) {
                store_rows(o, (int64_t)p.H * W, w);
            } else if (live && OSDN_IN_BOUNDS(row, p.rows)) {
                uint4* e = reinterpret_cast<uint4*>(o + row * p.H * W);
                e[0] = make_uint4(w[0], w[1], w[2], w[3]);
                e[1] = make_uint4(w[4], w[5], w[6], w[7]);
            }
            __syncwarp();
        };
        auto arrive = [&](uint64_t* bar) {
            tc::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
        };
        // every warp that reads the tiles waits for the copies itself
        bool ok = wait(tiles, 0);
        if (ok && len < TCS_L) {     // rows of the next sequence: 0 x NaN must not reach a sum
            if (!live && wg == 0) {
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                for (int t = 0; t < (int)(L::IMG / 16384); ++t)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        *reinterpret_cast<uint4*>(smem + t * 16384 + tc::sw128_off(r, j)) = z;
            }
            tc::fence_async_smem();
            arrive(zeroed);
        }
        ok = ok && wait(gates, 0) && wait(sc1, 0);
        // Sums of a token are stored once a phase's results are handed over: a store can wait for
        // those of the outputs in front of it.
        const bool mine = (rb & 3) == wg;  // this thread has its row's diagonal element
        float diag = 0.f, ri = 0.f, rn = 0.f;
        // l_r, two terms; from behind token r to the end of its sub-block
        const float lr = f->l[r], lr2 = f->l2[r], to_end = (f->th[rb] - lr) + (f->tl[rb] - lr2);
        if (ok) {
            tc::fence_after_sync();
            // ---- scores [j][i], i >= j: 2^(cum_i - cum_j) = 2^l_i 2^(base_b - cum_j)
            const float sj = f->st[r];
            float* rowsum = reinterpret_cast<float*>(smem + L::ROWSUM) + wq * TCS_L;
#pragma unroll 1
            for (int b = wg; b < 8; b += 4) {
                uint32_t w1[16], w2[16];  // the leading terms, then the second
                if (b < 2 * wq) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w1[e] = w2[e] = 0;
                    if (lane < 16) rowsum[16 * b + lane] = 0.f;
                } else {
                    float s1[16], s2[16], wt[16];
                    tc::tmem_ld16(tl + T0 + 16 * b, s1);
                    tc::tmem_ld16(tl + T1 + 16 * b, s2);
                    if (b <= 2 * wq + 1) {  // the row's own sub-block, or the one behind
                        const float dh = b == rb ? lr : 0.f, dl = b == rb ? lr2 : 0.f;
                        const float rest = b == rb ? 0.f : to_end;
                        const float4* lp = reinterpret_cast<const float4*>(f->l + 16 * b);
                        const float4* mp = reinterpret_cast<const float4*>(f->l2 + 16 * b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 l4 = lp[e], m4 = mp[e];
                            const int c = 16 * b + 4 * e;
                            wt[4 * e] = c < r ? 0.f : ex2f((l4.x - dh) + (m4.x - dl) + rest);
                            wt[4 * e + 1] = c + 1 < r ? 0.f : ex2f((l4.y - dh) + (m4.y - dl) + rest);
                            wt[4 * e + 2] = c + 2 < r ? 0.f : ex2f((l4.z - dh) + (m4.z - dl) + rest);
                            wt[4 * e + 3] = c + 3 < r ? 0.f : ex2f((l4.w - dh) + (m4.w - dl) + rest);
                        }
                    } else {
                        const float fr =
                            ex2f((f->bh[b] - f->bh[rb + 1]) + (f->bl[b] - f->bl[rb + 1]) + to_end);
                        const float4* gp = reinterpret_cast<const float4*>(gt->r + 16 * b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 g4 = gp[e];
                            wt[4 * e] = fr * g4.x; wt[4 * e + 1] = fr * g4.y;
                            wt[4 * e + 2] = fr * g4.z; wt[4 * e + 3] = fr * g4.w;
                        }
                    }
                    tc::tmem_ld_wait();
                    const int own = b == rb ? r & 15 : -1;  // the diagonal's column
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 t = make_float2(wt[2 * e], wt[2 * e + 1]);
                        const float2 u = __fmul2_rn(t, make_float2(s1[2 * e], s1[2 * e + 1]));
                        const float2 v = __fmul2_rn(t, make_float2(s2[2 * e], s2[2 * e + 1]));
                        split2_rn(u.x, u.y, w1[e], w1[8 + e]);
                        split2_rn(v.x, v.y, w2[e], w2[8 + e]);
                        float2 x = __fmul2_rn(u, make_float2(s2[2 * e], s2[2 * e + 1]));  // W
                        if (own == 2 * e) { diag = x.x; x.x = 0.f; }
                        if (own == 2 * e + 1) { diag = x.y; x.y = 0.f; }
                        ri += x.x;
                        ri += x.y;
                        s1[2 * e] = sj * x.x;
                        s1[2 * e + 1] = sj * x.y;
                    }
                    __syncwarp();
                    // 16 columns summed over the warp's 32 rows: each step halves the columns a
                    // lane keeps and doubles the rows that they stand for
#pragma unroll
                    for (int half = 8; half > 0; half >>= 1) {
                        const bool up = lane & (2 * half);
#pragma unroll
                        for (int e = 0; e < half; ++e) {
                            const float send = up ? s1[e] : s1[e + half];
                            const float keep = up ? s1[e + half] : s1[e];
                            s1[e] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * half);
                        }
                    }
                    const float sum = s1[0] + __shfl_xor_sync(0xffffffffu, s1[0], 1);
                    if (!(lane & 1)) rowsum[16 * b + (lane >> 1)] = sum;
                }
                tc::tmem_st8(tl + T0 + 16 * b, w1);
                tc::tmem_st8(tl + T0 + 16 * b + 8, w1 + 8);
                tc::tmem_st8(tl + T1 + 16 * b, w2);
                tc::tmem_st8(tl + T1 + 16 * b + 8, w2 + 8);
            }
        }
        ok = ok && wait(in1, 0);
        const float st = f->st[r];
        if (ok) {
            tc::fence_after_sync();
            // ---- R products scaled by 2^(cum_L - cum_j) in place
            const float e1 = ex2f((f->bh[8] - f->bh[rb + 1]) + (f->bl[8] - f->bl[rb + 1]) + to_end);
            const float2 e2 = make_float2(e1, e1);
#pragma unroll 1
            for (int q = 0; q < DV / 64; ++q) {
                const int c = wg * (DV / 4) + 16 * q;
                float v[16];
                tc::tmem_ld16(tl + A0 + c, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= e1;
                tc::tmem_st16(tl + A0 + c, v);
            }
#pragma unroll 1
            for (int q = 0; q < DK / 64; ++q) {
                const int c = wg * (DK / 4) + 16 * q;
                float v[16];
                tc::tmem_ld16(tl + A1 + c, v);
                const uint4 u0 = tile16(L::B, c), u1 = tile16(L::B, c + 8);
                const uint32_t bw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 t = __fmul2_rn(e2, make_float2(v[2 * e], v[2 * e + 1]));
                    rn = fmaf(t.x, __uint_as_float(bw[e] << 16), rn);
                    rn = fmaf(t.y, __uint_as_float(bw[e] & 0xffff0000u), rn);
                    v[2 * e] = t.x;
                    v[2 * e + 1] = t.y;
                }
                tc::tmem_st16(tl + A1 + c, v);
            }
            tc::tmem_st_wait();
            arrive(ew1);
            if (live && OSDN_IN_BOUNDS(row, p.rows)) {
                const int64_t at = h * p.rows + row, share = (wg * (int64_t)p.H) * p.rows;
                p.ri[share + at] = ri;
                p.rn[share + at] = rn;
                if (mine) p.wd[at] = diag;
            }
        }
        // ---- 2^cum_L <R, S> from all three terms (where states hardly decay it is most of the step
        // gradient: with two terms dA was 3.5e-6 off there), in L2 by now
        if (ok) {
            float dot = 0.f;
            const int64_t at = (slot * p.H + h) * (int64_t)(TCS_TERMS * L::TERM);
            const uint4* a = reinterpret_cast<const uint4*>(p.img_r + at);
            const uint4* b = reinterpret_cast<const uint4*>(p.img + at);
            constexpr int NB = L::TERM / 16;
            // the lower and the upper halves of word k, their terms added from the smallest on
            auto lo = [](const uint4 (&t)[3], int k) {
                const uint32_t w[3] = {(&t[0].x)[k], (&t[1].x)[k], (&t[2].x)[k]};
                return __uint_as_float(w[0] << 16) + (__uint_as_float(w[1] << 16) + __uint_as_float(w[2] << 16));
            };
            auto hi = [](const uint4 (&t)[3], int k) {
                const uint32_t w[3] = {(&t[0].x)[k], (&t[1].x)[k], (&t[2].x)[k]};
                return __uint_as_float(w[0] & 0xffff0000u) +
                       (__uint_as_float(w[1] & 0xffff0000u) + __uint_as_float(w[2] & 0xffff0000u));
            };
#pragma unroll 2
            for (int e = tid; e < NB; e += 512) {
                const uint4 x[3] = {__ldg(a + e), __ldg(a + NB + e), __ldg(a + 2 * NB + e)};
                const uint4 y[3] = {__ldg(b + e), __ldg(b + NB + e), __ldg(b + 2 * NB + e)};
#pragma unroll
                for (int k = 0; k < 4; ++k) dot = fmaf(hi(x, k), hi(y, k), fmaf(lo(x, k), lo(y, k), dot));
            }
            dot = warp_sum_f(dot);
            if (lane == 0 && OSDN_IN_BOUNDS(slot, p.slots))
                p.gs[(warp * p.slots + slot) * p.H + h] = dot * ex2f(f->bh[8] + f->bl[8]);
            ok = wait(acc1, 0);
        }
        if (ok) {
            tc::fence_after_sync();
            // ---- dx and db
            const float skip = p.D ? p.D[h] : 0.f;
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < DV / 64; ++q) {
                const int c = wg * (DV / 4) + 16 * q;
                float v[16];
                tc::tmem_ld16(tl + A0 + c, v);
                const uint4 u0 = tile16(L::DY, c), u1 = tile16(L::DY, c + 8);
                const uint32_t yw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[8 * q + e] = pack2_rn(fmaf(st, v[2 * e], skip * __uint_as_float(yw[e] << 16)),
                                            fmaf(st, v[2 * e + 1], skip * __uint_as_float(yw[e] & 0xffff0000u)));
            }
            put_bf16(p.dx + (int64_t)h * DV, std::integral_constant<int, DV>{}, w);
        }
        // this warpgroup's quarter of a head's rows of db or dc, each value times k
        auto give = [&](__nv_bfloat16* o16, float* o32, uint32_t acc, float k) {
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < DK / 64; ++q) {
                const int c = wg * (DK / 4) + 16 * q;
                float v[16];
                tc::tmem_ld16(tl + acc + c, v);
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= k;
                if (o16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) w[8 * q + e] = pack2_rn(v[2 * e], v[2 * e + 1]);
                } else if (live && OSDN_IN_BOUNDS(row, p.rows)) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        *reinterpret_cast<float4*>(o32 + (row * p.H + h) * DK + c + 4 * e) =
                            make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
                __syncwarp();
            }
            if (o16) put_bf16(o16 + (int64_t)h * DK, std::integral_constant<int, DK>{}, w);
        };
        if (ok) {
            give(p.db, p.dbh, A1, st);
            ok = wait(sc2, 0);
        }
        float pos = 0.f;
        if (ok && wg == 0 && (ok = wait(ew1, 0))) {  // every quarter's shares are written
            const float* rowsum = reinterpret_cast<const float*>(smem + L::ROWSUM) + r;
            pos = (rowsum[0] + rowsum[TCS_L]) + (rowsum[2 * TCS_L] + rowsum[3 * TCS_L]);
        }
        if (ok) {
            tc::fence_after_sync();
            // ---- scores [i][j], j <= i
#pragma unroll 1
            for (int b = wg; b < 8; b += 4) {
                uint32_t w2[16];
                if (b > 2 * wq + 1) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) w2[e] = 0;
                } else {
                    float s2[16], wt[16];
                    tc::tmem_ld16(tl + T1 + 16 * b, s2);
                    if (b >= 2 * wq) {
                        const float dh = b == rb ? lr : f->th[b], dl = b == rb ? lr2 : f->tl[b];
                        const float rest = b == rb ? 0.f : lr;
                        const float4* lp = reinterpret_cast<const float4*>(f->l + 16 * b);
                        const float4* mp = reinterpret_cast<const float4*>(f->l2 + 16 * b);
                        const float4* sp = reinterpret_cast<const float4*>(f->st + 16 * b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 l4 = lp[e], m4 = mp[e], s4 = sp[e];
                            const int c = 16 * b + 4 * e;
                            wt[4 * e] = c > r ? 0.f : ex2f((dh - l4.x) + (dl - m4.x) + rest) * s4.x;
                            wt[4 * e + 1] = c + 1 > r ? 0.f : ex2f((dh - l4.y) + (dl - m4.y) + rest) * s4.y;
                            wt[4 * e + 2] = c + 2 > r ? 0.f : ex2f((dh - l4.z) + (dl - m4.z) + rest) * s4.z;
                            wt[4 * e + 3] = c + 3 > r ? 0.f : ex2f((dh - l4.w) + (dl - m4.w) + rest) * s4.w;
                        }
                    } else {
                        const float fr = ex2f((f->bh[rb] - f->bh[b + 1]) + (f->bl[rb] - f->bl[b + 1]) + lr);
                        const float4* gp = reinterpret_cast<const float4*>(f->g + 16 * b);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 g4 = gp[e];
                            wt[4 * e] = fr * g4.x; wt[4 * e + 1] = fr * g4.y;
                            wt[4 * e + 2] = fr * g4.z; wt[4 * e + 3] = fr * g4.w;
                        }
                    }
                    tc::tmem_ld_wait();
                    const int own = b == rb ? r & 15 : -1;
#pragma unroll
                    for (int e = 0; e < 16; ++e) diag = e == own ? s2[e] : diag;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 v = __fmul2_rn(make_float2(wt[2 * e], wt[2 * e + 1]),
                                                    make_float2(s2[2 * e], s2[2 * e + 1]));
                        split2_rn(v.x, v.y, w2[e], w2[8 + e]);
                    }
                }
                tc::tmem_st8(tl + T1 + 16 * b, w2);
                tc::tmem_st8(tl + T1 + 16 * b + 8, w2 + 8);
            }
            ok = wait(in2, 0);
        }
        if (ok) {
            tc::fence_after_sync();
            // ---- the S product scaled by 2^cum_i in place
            const float e1 = ex2f(f->bh[rb] + lr + f->bl[rb]);
            const float2 e2 = make_float2(e1, e1);
#pragma unroll 1
            for (int q = 0; q < DK / 64; ++q) {
                const int c = wg * (DK / 4) + 16 * q;
                float v[16];
                tc::tmem_ld16(tl + T0 + c, v);
                const uint4 u0 = tile16(L::C, c), u1 = tile16(L::C, c + 8);
                const uint32_t cw[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
                tc::tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 t = __fmul2_rn(e2, make_float2(v[2 * e], v[2 * e + 1]));
                    pos = fmaf(t.x, __uint_as_float(cw[e] << 16), pos);
                    pos = fmaf(t.y, __uint_as_float(cw[e] & 0xffff0000u), pos);
                    v[2 * e] = t.x;
                    v[2 * e + 1] = t.y;
                }
                tc::tmem_st16(tl + T0 + c, v);
            }
            tc::tmem_st_wait();
            arrive(ew2);
            if (live && OSDN_IN_BOUNDS(row, p.rows)) {
                p.pos[(wg * p.H + h) * p.rows + row] = pos;
                if (mine && p.vk) p.vk[h * p.rows + row] = diag;  // dy . x
            }
            ok = wait(acc2, 0);
        }
        if (ok) {
            tc::fence_after_sync();
            give(p.dc, p.dch, T0, 1.f);
        }
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 16) tc::tmem_dealloc(tmem, 512);
}

// db and dc of the groups: the heads' fp32 shares summed in order, rounded once.  8 channels a
// thread; n = rows * G * DK / 8.
__global__ void __launch_bounds__(256)
ssm_group_sum_kernel(const float* __restrict__ dbh, const float* __restrict__ dch,
                     __nv_bfloat16* __restrict__ db, __nv_bfloat16* __restrict__ dc, int64_t n, int rep,
                     int DK) {
    const int64_t stride = (int64_t)gridDim.x * 256;
    const int v = DK / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += stride) {
        const int64_t at = (i / v) * rep * DK + (i % v) * 8;
        float s[8], t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = t[e] = 0.f;
        for (int r = 0; r < rep; ++r) {
            float a[8], b[8];
            vec_io<8, float>::load(dbh + at + (int64_t)r * DK, a);
            vec_io<8, float>::load(dch + at + (int64_t)r * DK, b);
#pragma unroll
            for (int e = 0; e < 8; ++e) { s[e] += a[e]; t[e] += b[e]; }
        }
        vec_io<8, __nv_bfloat16>::store(db + i * 8, s);
        vec_io<8, __nv_bfloat16>::store(dc + i * 8, t);
    }
}

}  // namespace osdn
