// mixer_lib.cu -- libosdn: host side of the layer operators around the token mixer (short
// convolution, selective scan, block norm), declared in include/osdn.h.
//
// As in osdn_lib.cu: the host code validates arguments, picks a kernel for the sizes and dtype
// and enqueues it on the caller's stream; it never allocates and never synchronizes.
#include <cuda_runtime.h>
#include <stdint.h>

#include "osdn.h"
#include "common.cuh"
#include "host_util.cuh"
#include "conv.cuh"
#include "norm.cuh"
#include "ssm_step.cuh"
#include "ssm_scan.cuh"
#include "ssm_tc.cuh"
#include "ssm_tc_bwd.cuh"

namespace osdn {

bool take_mixer_status(int* value) {
    const int zero = 0;
    if (cudaMemcpyFromSymbol(value, g_device_status, sizeof(int)) != cudaSuccess) return false;
    return *value == 0 ||
           cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) == cudaSuccess;
}

namespace {

struct Buf { const void* p; size_t bytes; };

// Alignment of every buffer, and that no written buffer overlaps any other.
osdn_status_t check_buffers(const Buf* in, int n_in, const Buf* out, int n_out) {
    for (int i = 0; i < n_in; ++i)
        if (in[i].p && !aligned16(in[i].p)) return OSDN_ERR_ALIGNMENT;
    for (int i = 0; i < n_out; ++i)
        if (out[i].p && !aligned16(out[i].p)) return OSDN_ERR_ALIGNMENT;
    for (int i = 0; i < n_out; ++i) {
        for (int j = 0; j < n_in; ++j)
            if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return OSDN_ERR_INVALID_ARG;
        for (int j = i + 1; j < n_out; ++j)
            if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return OSDN_ERR_INVALID_ARG;
    }
    return OSDN_OK;
}

osdn_status_t check_tokens(const int32_t* cu, int32_t num_seqs, int32_t B, int32_t T,
                           osdn_dtype_t io, int64_t* rows, int64_t* N) {
    if (io != OSDN_BF16 && io != OSDN_F32) return OSDN_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || num_seqs < 0) return OSDN_ERR_INVALID_ARG;
    if (cu && B != 1) return OSDN_ERR_INVALID_ARG;
    *rows = (int64_t)B * T;
    *N = cu ? num_seqs : B;
    // without a sequence there is nothing that packed rows could belong to
    if (cu && num_seqs == 0 && T > 0) return OSDN_ERR_INVALID_ARG;
    if (*rows >= (int64_t(1) << 31)) return OSDN_ERR_UNSUPPORTED;
    return OSDN_OK;
}

osdn_status_t check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return OSDN_OK;
    if (!ws || have < need) return OSDN_ERR_INVALID_ARG;
    return (reinterpret_cast<uintptr_t>(ws) & 255u) ? OSDN_ERR_ALIGNMENT : OSDN_OK;
}

// Runs f(constant V, constant W) for the channels of a thread and the filter length: the widest V
// of MAX, MAX / 2, .. 2 that divides C (rows stay aligned to V elements then), else 1.
template <int MAX, typename F> osdn_status_t conv_dispatch(int C, int W, F f) {
    if constexpr (MAX > 1)
        if (C % MAX != 0) return conv_dispatch<MAX / 2>(C, W, f);
    using v = std::integral_constant<int, MAX>;
    switch (W) {
        case 2: return f(v{}, std::integral_constant<int, 2>{});
        case 3: return f(v{}, std::integral_constant<int, 3>{});
        default: return f(v{}, std::integral_constant<int, 4>{});
    }
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tokens of a strip, so that `per_sm` blocks on each of 148 SMs (a constant, so that the backward
// workspace's size does not need a device), `gx` blocks side by side per strip, share the rows in
// whole rounds: no round is left half empty.  At most `most` tokens, and 8 at least (a strip
// re-reads the W - 1 tokens before it).
int64_t conv_strip(int64_t rows, int64_t gx, int per_sm, int64_t most) {
    const int64_t side = 148LL * per_sm / gx, lanes = side < 1 ? 1 : side;
    const int64_t rounds = ceil_div(ceil_div(rows, lanes), most);
    const int64_t strip = ceil_div(rows, lanes * (rounds < 1 ? 1 : rounds));
    return strip < 8 ? 8 : strip;
}

template <typename IO>
osdn_status_t launch_conv_fwd(const void* x, const float* weight, const float* bias,
                              const void* state0, int silu, void* y, void* stateT,
                              const int32_t* cu, int N, int T, int C, int W, int64_t rows,
                              cudaStream_t stream) {
    return conv_dispatch<CONV_MAX_V>(C, W, [&](auto v, auto w) -> osdn_status_t {
        constexpr int V = decltype(v)::value, WW = decltype(w)::value;
        const int64_t gx = ceil_div(C, (int64_t)V * CONV_THREADS);
        int64_t strip = conv_strip(rows, gx, conv_per_sm(V * sizeof(IO)), 64);
        const int64_t least = ceil_div(rows, 32768);
        strip = strip < least ? least : strip;
        const int64_t strips = ceil_div(rows, strip);
        const int64_t tail = cu || stateT ? (N < 4096 ? N : 4096) : 0;
        if (gx > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
        if (strips + tail == 0) return OSDN_OK;
        conv_fwd_kernel<V, WW, IO><<<dim3((unsigned)gx, (unsigned)(strips + tail)),
                                     dim3(CONV_THREADS), 0, stream>>>(
            static_cast<const IO*>(x), weight, bias, static_cast<const IO*>(state0), silu,
            static_cast<IO*>(y), static_cast<IO*>(stateT), cu, N, T, C, rows, (int)strips,
            (int)strip);
        return launch_status();
    });
}

template <typename IO>
osdn_status_t launch_conv_step(const void* x, const float* weight, const float* bias, void* state,
                               int silu, void* y, int N, int C, int W, cudaStream_t stream) {
    return conv_dispatch<CONV_MAX_V>(C, W, [&](auto v, auto w) -> osdn_status_t {
        constexpr int V = decltype(v)::value, WW = decltype(w)::value;
        const int64_t gx = ceil_div(C, (int64_t)V * CONV_THREADS);
        conv_step_kernel<V, WW, IO><<<dim3((unsigned)gx, (unsigned)(N < 32768 ? N : 32768)),
                                      dim3(CONV_THREADS), 0, stream>>>(
            static_cast<const IO*>(x), weight, bias, static_cast<IO*>(state), silu,
            static_cast<IO*>(y), N, C);
        return launch_status();
    });
}

// How the backward pass splits the rows: strips of `strip` tokens, CONV_BWD_STRIPS of them a
// block at a time, row_blocks blocks per group of channels.
struct ConvBwdPlan { int64_t gx; int strip, row_blocks; };
ConvBwdPlan conv_bwd_plan(int64_t rows, int C) {
    ConvBwdPlan pl;
    int V = CONV_BWD_MAX_V;  // as conv_dispatch picks it
    while (C % V != 0) V /= 2;
    pl.gx = ceil_div(C, 32 * V);
    pl.strip = (int)conv_strip(rows, pl.gx, CONV_BWD_PER_SM * CONV_BWD_STRIPS, 128);
    const int64_t need = ceil_div(rows, CONV_BWD_STRIPS * pl.strip);
    const int64_t side = 148LL * CONV_BWD_PER_SM / pl.gx, most = side < 1 ? 1 : side;
    pl.row_blocks = (int)(need < 1 ? 1 : need > most ? most : need);
    return pl;
}

template <typename IO, typename GO>
osdn_status_t launch_conv_bwd(const void* x, const float* weight, const float* bias,
                              const void* state0, int silu, const void* dy, const float* dstateT,
                              void* dx, float* dweight, float* dbias, float* dstate0, float* part,
                              const int32_t* cu, int N, int T, int C, int W, int64_t rows,
                              cudaStream_t stream) {
    const ConvBwdPlan pl = conv_bwd_plan(rows, C);
    const int64_t tail = cu || dstate0 ? ceil_div(N < 4096 ? N : 4096, CONV_BWD_STRIPS) : 0;
    const osdn_status_t st = conv_dispatch<CONV_BWD_MAX_V>(C, W, [&](auto v, auto w) -> osdn_status_t {
        constexpr int V = decltype(v)::value, WW = decltype(w)::value;
        conv_bwd_kernel<V, WW, IO, GO>
            <<<dim3((unsigned)pl.gx, (unsigned)(pl.row_blocks + tail)), dim3(32, CONV_BWD_STRIPS), 0,
               stream>>>(static_cast<const IO*>(x), weight, bias, static_cast<const IO*>(state0), silu,
                         static_cast<const GO*>(dy), dstateT, static_cast<IO*>(dx), dstate0, part, cu, N,
                         T, C, rows, pl.row_blocks, pl.strip);
        return launch_status();
    });
    if (st != OSDN_OK) return st;
    conv_reduce_kernel<<<dim3((unsigned)ceil_div(C, 32), (unsigned)(W + 1)),
                         dim3(32, CONV_RED_WARPS), 0, stream>>>(part, pl.row_blocks, W, C, dweight,
                                                                dbias);
    return launch_status();
}

// ---------------------------------------------------------------- block norm
// Runs f(constant VEC, constant TPR) for rows of D values: TPR threads of V values each, the
// smallest power of two that holds a row.
template <int V, int TPR = 4, typename F> osdn_status_t norm_dispatch(int D, F f) {
    using tpr = std::integral_constant<int, TPR>;
    if constexpr (TPR * V < NORM_MAX_D)
        if (D > TPR * V) return norm_dispatch<V, 2 * TPR>(D, f);
    return D % 8 == 0 ? f(std::true_type{}, tpr{}) : f(std::false_type{}, tpr{});
}

// Blocks of the backward pass (each leaves one partial row of dw_post and dw_next): as many as
// are resident on 148 SMs (a constant, so that the workspace's size does not need a device), or
// one per set of rows.
int64_t norm_bwd_blocks(int64_t R, int D, bool next) {
    int tpr = 4;
    while (tpr * NORM_BWD_V < D) tpr *= 2;
    const int64_t most = 148LL * norm_bwd_per_sm(tpr, next), have = ceil_div(R, norm_rows(tpr));
    return have < most ? have : most;
}

// ---------------------------------------------------------------- selective scan
// How the fp32 scan cuts sequences into segments (see ssm_scan.cuh): tokens of one (INT_MAX: no
// cuts), how many numbers they take, and the bytes they need.  About 4 CTAs for each of 148 SMs (a
// constant, so that the workspace's size does not need a device), of 128 tokens at least, and only
// where a sequence gives two: the first launch re-reads k and v and costs about 2/3 of a token's
// time per token.
struct SsmSegments { int seg; int64_t slots; size_t state, decay, bytes; };
SsmSegments ssm_f32_segments(int64_t rows, int64_t N, int64_t T, int H, int Dk, int Dv) {
    SsmSegments s = {INT_MAX, N, 0, 0, 0};
    const int64_t most = Dk > Dv ? Dk : Dv;  // rows of the state, in either orientation
    const int64_t len = ceil_div(ceil_div(rows * H * (most / SSM_BV), 4 * 148), SSM_BLOCK) * SSM_BLOCK;
    const int64_t tokens = len < 128 ? 128 : len;
    if (2 * tokens <= T && tokens < INT_MAX) {
        s.seg = (int)tokens;
        s.slots = rows / tokens + N;
        s.decay = up256((size_t)s.slots * H * Dv * Dk * 4);
        s.bytes = s.decay + up256((size_t)s.slots * H * 4);
    }
    return s;
}

template <int MODE, bool SEG>
osdn_status_t launch_ssm_scan_one(const SsmArgs& a, int64_t slots, int DQ, int DV, cudaStream_t stream) {
    const int64_t ctas = slots * a.H * (DV / SSM_BV);
    if (ctas == 0) return OSDN_OK;
    if (ctas > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ctas), block(SSM_THREADS);
    if (DQ == 128 && DV == 128)
        ssm_scan_kernel<128, 128, MODE, SEG><<<grid, block, 0, stream>>>(a);
    else if (DQ == 128)
        ssm_scan_kernel<128, 64, MODE, SEG><<<grid, block, 0, stream>>>(a);
    else if (DV == 128)
        ssm_scan_kernel<64, 128, MODE, SEG><<<grid, block, 0, stream>>>(a);
    else
        ssm_scan_kernel<64, 64, MODE, SEG><<<grid, block, 0, stream>>>(a);
    return launch_status();
}

// One scan of a mode, its segments' launch first.  ws: the segments' workspace.
template <int MODE>
osdn_status_t launch_ssm_scan(SsmArgs a, const SsmSegments& sg, uint8_t* ws, int DQ, int DV,
                              cudaStream_t stream) {
    a.seg = sg.seg;
    if (sg.seg != INT_MAX) {
        a.seg_state = reinterpret_cast<float*>(ws + sg.state);
        a.seg_decay = reinterpret_cast<float*>(ws + sg.decay);
        const osdn_status_t st = launch_ssm_scan_one<MODE, true>(a, sg.slots, DQ, DV, stream);
        if (st != OSDN_OK) return st;
    }
    return launch_ssm_scan_one<MODE, false>(a, sg.slots, DQ, DV, stream);
}

// 3-D bf16 view [rows][heads][D] of a token tensor; boxes of 64 channels x 1 head x 128 tokens,
// 128-byte swizzle.
bool make_chunk_map(CUtensorMap* m, const void* base, int D, int heads, int64_t rows) {
    EncodeTiledFn enc = tensor_map_encoder();
    if (!enc || rows <= 0) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2};
    cuuint32_t box[3] = {64, 1, TCS_L};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// How the forward pass cuts sequences into segments: tokens of one (INT_MAX: no cuts), how many
// numbers they take, and the bytes they need.  148 SMs (a constant, so that the workspace's size
// does not need a device) take one CTA each.
//   Equal sequences: as many segments each as keep every CTA on an SM of its own, if a sequence
//   still gives 4 chunks to a segment: the first launch re-reads b and x and costs about half
//   a chunk's time per chunk (16 heads, Dv=64: 65,536 tokens 267 us, 1403 uncut; 2048 tokens 35, 53
//   uncut).
//   Packed sequences (more than one: a single one has all T tokens, whether offsets say so or not),
//   whose lengths the host does not know: twice the tokens that an even split
//   of the whole would give a CTA, so only sequences far above the average are cut (16 heads,
//   Dv=64: 300 + 9000 + 200 tokens 96 us, 205 uncut; six of up to 4096 tokens 78, 100 uncut; eight
//   of 1024, none of them cut, 43, and 37 without the first launch).
//   The backward pass's chains go both ways (dirs 2), a CTA each, and their first launch costs
//   more (three terms of V'): three segments of 8 chunks at least (B=1, T=7112, H=16, Dv=64: 266
//   us uncut, 225 in four; two segments at T=2048: 96 uncut, 103 cut), and packed sequences stay
//   whole (six of up to 4096 tokens, H=16: 242, cut 279; a few long ones with few heads lose by it: two
//   of 16,384 tokens with H=2 317, cut 172).
SsmSegments ssm_segments(bool packed, int64_t rows, int64_t N, int64_t T, int H, int Dk, int Dv,
                         int dirs) {
    const int64_t nvt = dirs * Dv / TCS_BV, chunks = ceil_div(packed ? rows : T, TCS_L), sms = 148;
    SsmSegments s = {INT_MAX, N, 0, 0, 0};
    int64_t len = chunks;
    if (packed && dirs == 1) {
        len = 2 * ceil_div(chunks * H * nvt, sms);
        len = len < 4 ? 4 : len;
    } else if (!packed && N * H * nvt > 0) {
        const int64_t most = chunks / (4 * dirs), fit = sms / (N * H * nvt);
        const int64_t segs = fit < most ? fit : most;
        if (segs > dirs) len = ceil_div(chunks, segs);
    }
    if (len < chunks && len * TCS_L < INT_MAX) {
        s.seg = (int)(len * TCS_L);
        s.slots = rows / s.seg + N;
        s.state = 0;
        s.decay = up256((size_t)dirs * s.slots * H * Dv * Dk * 4);
        s.bytes = s.decay + up256((size_t)dirs * s.slots * H * 4);
    }
    return s;
}

// q, k: [rows][G][DQ], v, v2: [rows][H][nvt * 64] (v2: dy, for both directions).  slots: the
// segments' numbers, or the sequences'.
template <int DQ, int MODE>
osdn_status_t launch_tc_chain(const void* q, const void* k, const void* v, const void* v2,
                              const TcsArgs& a, int64_t slots, cudaStream_t stream) {
    using L = TcsSmem<DQ, MODE>;
    const int64_t ctas = slots * a.H * a.nvt * (L::BOTH ? 2 : 1);
    if (ctas == 0) return OSDN_OK;
    if (ctas > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    CUtensorMap mq, mk, mv, mv2;
    if (!make_chunk_map(&mk, k, DQ, a.G, a.rows) || !make_chunk_map(&mv, v, a.nvt * TCS_BV, a.H, a.rows) ||
        !make_chunk_map(&mq, q, DQ, a.G, a.rows) || !make_chunk_map(&mv2, v2, a.nvt * TCS_BV, a.H, a.rows))
        return OSDN_ERR_CUDA;
    auto kern = ssm_tc_chain_kernel<DQ, MODE>;
    if (!set_smem(kern, L::BYTES)) return OSDN_ERR_CUDA;
    kern<<<dim3((unsigned)ctas), dim3(L::THREADS), L::BYTES, stream>>>(mq, mk, mv, mv2, a);
    return launch_status();
}

template <int DQ>
osdn_status_t launch_tc_fwd(const void* q, const void* k, const void* v, const TcsArgs& a,
                            int64_t slots, cudaStream_t stream) {
    if (a.seg != INT_MAX) {
        const osdn_status_t st = launch_tc_chain<DQ, TCS_SEG>(q, k, v, v, a, slots, stream);
        if (st != OSDN_OK) return st;
    }
    return launch_tc_chain<DQ, TCS_FWD>(q, k, v, v, a, slots, stream);
}

osdn_status_t check_ssm(int32_t H, int32_t G, int32_t Dk, int32_t Dv) {
    if (H < 1 || G < 1 || H % G != 0) return OSDN_ERR_INVALID_ARG;
    if ((Dk != 64 && Dk != 128) || (Dv != 64 && Dv != 128)) return OSDN_ERR_UNSUPPORTED;
    return H > 65535 ? OSDN_ERR_UNSUPPORTED : OSDN_OK;
}

SsmSegments ssm_bwd_segments(int64_t rows, int64_t N, int64_t T, int H, int Dk, int Dv) {
    return ssm_segments(rows != N * T, rows, N, T, H, Dk, Dv, 2);
}

// Workspace of osdn_ssm_bwd, each part rounded up to 256 bytes.  fp32 tokens: the heads' dc and
// db, the state behind each block of SSM_BLOCK tokens.  bf16 tokens: the states in front of and
// the gradients behind each chunk as images of bf16 terms, the heads' dc and db when heads share
// rows of b and c.  Both: the sums that the step gradient is made of.
struct SsmBwdWorkspace {
    size_t seg, dch, dbh, ckpt, ckpt_r, gs, pos, ri, rn, wd, vk, part, total;
};
SsmBwdWorkspace ssm_bwd_workspace(int64_t rows, int64_t N, int64_t T, int32_t H, int32_t G,
                                  int32_t Dk, int32_t Dv, osdn_dtype_t io) {
    SsmBwdWorkspace w;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += up256(bytes);
        return at;
    };
    const bool tc = io == OSDN_BF16;
    const size_t th = (size_t)rows * H, slots = (size_t)ssm_slots(rows, N, tc ? TCS_L : SSM_BLOCK);
    const size_t heads = !tc || G < H ? th * Dk * 4 : 0, shares = tc ? 4 : 1;
    const size_t image = slots * H * Dk * Dv * (tc ? TCS_TERMS * 2 : 4);
    w.seg = take((tc ? ssm_bwd_segments(rows, N, T, H, Dk, Dv)
                     : ssm_f32_segments(rows, N, T, H, Dk, Dv)).bytes);
    w.dch = take(heads);
    w.dbh = take(heads);
    w.ckpt = take(image);
    w.ckpt_r = take(tc ? image : 0);
    w.gs = take(slots * H * (tc ? 16 : Dk / SSM_BV) * 4);
    w.pos = take(shares * th * 4);
    w.ri = take(shares * th * 4);
    w.rn = take(tc ? shares * th * 4 : 0);
    w.wd = take(tc ? th * 4 : 0);
    w.vk = take(th * 4);
    w.part = take((size_t)3 * slots * H * 4);
    w.total = off;
    return w;
}

struct SsmBwdCall {
    const void* x; const float *dt, *A; const void *b, *c; const float *D, *dt_bias; int softplus;
    const float* S0; const void* dy; const float* dST; void* dx; float *ddt, *dA; void *db, *dc;
    float *dD, *ddt_bias, *dS0; const int32_t* cu; int64_t N; int T, H, G, Dk, Dv; int64_t rows;
    uint8_t* ws; cudaStream_t stream;
};

// ddt of every token, then dA, dD and ddt_bias.
template <int BLOCK>
osdn_status_t launch_ssm_gates(const SsmBwdCall& k, const SsmBwdWorkspace& w, const float* rn,
                               const float* wd, int shares, int nslice) {
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(k.ws + at); };
    const int64_t slots = ssm_slots(k.rows, k.N, BLOCK), units = slots * k.H;
    const int64_t blocks = ceil_div(units, SSM_GATE_WARPS);
    if (blocks > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    if (k.N > 0) {
        ssm_gate_kernel<BLOCK><<<dim3((unsigned)blocks), dim3(32 * SSM_GATE_WARPS), 0, k.stream>>>(
            f32(w.pos), f32(w.ri), rn, shares, wd, f32(w.gs), nslice, k.dD ? f32(w.vk) : nullptr, k.dt, k.A,
            k.dt_bias, k.softplus, k.ddt, f32(w.part), k.cu, (int)k.N, k.T, k.H, k.rows);
        const osdn_status_t st = launch_status();
        if (st != OSDN_OK) return st;
    }
    ssm_param_kernel<<<dim3(3, k.H), 128, 0, k.stream>>>(f32(w.part), k.N > 0 ? slots : 0, k.H, k.dA,
                                                         k.dD, k.ddt_bias);
    return launch_status();
}

// fp32 tokens, and calls without tokens: three scans token by token.
osdn_status_t launch_ssm_bwd_f32(const SsmBwdCall& k) {
    const SsmBwdWorkspace w = ssm_bwd_workspace(k.rows, k.N, k.T, k.H, k.G, k.Dk, k.Dv, OSDN_F32);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(k.ws + at); };
    SsmArgs a = {};
    a.dt = k.dt; a.A = k.A; a.D = k.D; a.dt_bias = k.dt_bias; a.softplus = k.softplus;
    a.cu = k.cu; a.rows = k.rows; a.N = (int)k.N; a.T = k.T; a.H = k.H; a.G = k.G;
    a.ckpt = f32(w.ckpt);
    a.gs = f32(w.gs);
    const float *x = static_cast<const float*>(k.x), *b = static_cast<const float*>(k.b),
                *c = static_cast<const float*>(k.c), *dy = static_cast<const float*>(k.dy);
    SsmArgs dcp = a, dxp = a, dbp = a;
    dcp.q = dy; dcp.k = x; dcp.v = b; dcp.S_in = k.S0; dcp.out = f32(w.dch);
    dcp.vk = k.dD ? f32(w.vk) : nullptr;
    dxp.q = b; dxp.k = c; dxp.v = dy; dxp.S_in = k.dST; dxp.out = static_cast<float*>(k.dx); dxp.S_out = k.dS0;
    dbp.q = x; dbp.k = dy; dbp.v = c; dbp.S_in = k.dST; dbp.out = f32(w.dbh);
    const SsmSegments sg = ssm_f32_segments(k.rows, k.N, k.T, k.H, k.Dk, k.Dv);
    osdn_status_t st = launch_ssm_scan<SSM_DC>(dcp, sg, k.ws + w.seg, k.Dv, k.Dk, k.stream);
    if (st == OSDN_OK) st = launch_ssm_scan<SSM_DX>(dxp, sg, k.ws + w.seg, k.Dk, k.Dv, k.stream);
    if (st == OSDN_OK) st = launch_ssm_scan<SSM_DB>(dbp, sg, k.ws + w.seg, k.Dv, k.Dk, k.stream);
    if (st != OSDN_OK) return st;
    if (k.rows > 0) {
        const int64_t need = ceil_div(k.rows * k.G, 8), cap = 16LL * sm_count();
        const dim3 grid((unsigned)(need < cap ? need : cap));
        auto kern = k.Dk == 128 ? ssm_group_kernel<128> : ssm_group_kernel<64>;
        kern<<<grid, 256, 0, k.stream>>>(f32(w.dch), f32(w.dbh), b, c, k.dt, k.dt_bias, k.softplus,
                                         static_cast<float*>(k.db), static_cast<float*>(k.dc),
                                         f32(w.pos), f32(w.ri), k.rows, k.H, k.G);
        st = launch_status();
        if (st != OSDN_OK) return st;
    }
    return launch_ssm_gates<SSM_BLOCK>(k, w, nullptr, nullptr, 1, k.Dk / SSM_BV);
}

// bf16 tokens: the chains of states in both directions, then all chunks at once.
template <int DK, int DV> osdn_status_t launch_ssm_bwd_tc(const SsmBwdCall& k) {
    using bf16 = __nv_bfloat16;
    const SsmBwdWorkspace w = ssm_bwd_workspace(k.rows, k.N, k.T, k.H, k.G, DK, DV, OSDN_BF16);
    auto f32 = [&](size_t at) { return reinterpret_cast<float*>(k.ws + at); };
    TcsArgs a = {};
    a.dt = k.dt; a.A = k.A; a.dt_bias = k.dt_bias; a.softplus = k.softplus; a.cu = k.cu;
    a.rows = k.rows; a.N = (int)k.N; a.T = k.T; a.H = k.H; a.G = k.G; a.nvt = DV / TCS_BV;
    const SsmSegments sg = ssm_bwd_segments(k.rows, k.N, k.T, k.H, DK, DV);
    a.seg = sg.seg;
    a.seg_state = f32(w.seg + sg.state); a.seg_decay = f32(w.seg + sg.decay);
    a.S_in = k.S0; a.img = k.ws + w.ckpt; a.img_r = k.ws + w.ckpt_r;
    a.dST = k.dST; a.dS0 = k.dS0;
    osdn_status_t st = OSDN_OK;
    if (a.seg != INT_MAX)
        st = launch_tc_chain<DK, TCS_SEG_SAVE>(k.c, k.b, k.x, k.dy, a, sg.slots, k.stream);
    if (st == OSDN_OK)
        st = launch_tc_chain<DK, TCS_SAVE>(k.c, k.b, k.x, k.dy, a, sg.slots, k.stream);
    if (st != OSDN_OK) return st;
    TcgArgs g = {};
    g.dt = k.dt; g.A = k.A; g.dt_bias = k.dt_bias; g.D = k.D; g.softplus = k.softplus;
    g.img = k.ws + w.ckpt; g.img_r = k.ws + w.ckpt_r; g.dx = static_cast<bf16*>(k.dx);
    if (k.G == k.H) {
        g.db = static_cast<bf16*>(k.db);
        g.dc = static_cast<bf16*>(k.dc);
    } else {
        g.dbh = f32(w.dbh);
        g.dch = f32(w.dch);
    }
    g.pos = f32(w.pos); g.ri = f32(w.ri); g.rn = f32(w.rn); g.gs = f32(w.gs); g.wd = f32(w.wd); g.vk = k.dD ? f32(w.vk) : nullptr;
    g.cu = k.cu; g.rows = k.rows; g.N = (int)k.N; g.T = k.T; g.H = k.H; g.G = k.G;
    g.slots = ssm_slots(k.rows, k.N, TCS_L);
    g.round = sm_count();
    if (g.slots * k.H > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    using L = TcgSmem<DK, DV>;
    CUtensorMap mx, my, mb, mc;
    if (!make_chunk_map(&mx, k.x, DV, k.H, k.rows) || !make_chunk_map(&my, k.dy, DV, k.H, k.rows) ||
        !make_chunk_map(&mb, k.b, DK, k.G, k.rows) || !make_chunk_map(&mc, k.c, DK, k.G, k.rows))
        return OSDN_ERR_CUDA;
    auto kern = ssm_tc_grad_kernel<DK, DV>;
    if (!set_smem(kern, L::BYTES)) return OSDN_ERR_CUDA;
    kern<<<dim3((unsigned)(g.slots * k.H)), dim3(L::THREADS), L::BYTES, k.stream>>>(mx, my, mb, mc, g);
    st = launch_status();
    if (st != OSDN_OK) return st;
    if (k.G < k.H) {
        const int64_t n = k.rows * k.G * DK / 8, need = ceil_div(n, 256), cap = 16LL * sm_count();
        ssm_group_sum_kernel<<<dim3((unsigned)(need < cap ? need : cap)), 256, 0, k.stream>>>(
            f32(w.dbh), f32(w.dch), static_cast<bf16*>(k.db), static_cast<bf16*>(k.dc), n, k.H / k.G, DK);
        st = launch_status();
        if (st != OSDN_OK) return st;
    }
    return launch_ssm_gates<TCS_L>(k, w, g.rn, g.wd, 4, 16);
}

}  // namespace
}  // namespace osdn

using namespace osdn;

extern "C" {

// ---------------------------------------------------------------- short causal convolution
osdn_status_t osdn_conv_fwd(const void* x, const float* weight, const float* bias,
                            const void* state0, int32_t silu, void* y, void* stateT,
                            const int32_t* cu_seqlens, int32_t num_seqs, int32_t B, int32_t T,
                            int32_t C, int32_t W, osdn_dtype_t io, void* stream) {
    int64_t rows, N;
    osdn_status_t st = check_tokens(cu_seqlens, num_seqs, B, T, io, &rows, &N);
    if (st != OSDN_OK) return st;
    if (C < 1 || (silu != 0 && silu != 1)) return OSDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || C > CONV_MAX_C) return OSDN_ERR_UNSUPPORTED;
    if (!weight || (rows > 0 && (!x || !y))) return OSDN_ERR_INVALID_ARG;
    const size_t es = io_size(io), xb = (size_t)rows * C * es, sb = (size_t)N * (W - 1) * C * es;
    const Buf in[] = {{x, xb}, {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {state0, sb},
                      {cu_seqlens, ((size_t)N + 1) * 4}};
    const Buf out[] = {{y, xb}, {stateT, sb}};
    st = check_buffers(in, 5, out, 2);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (io == OSDN_BF16)
        return launch_conv_fwd<__nv_bfloat16>(x, weight, bias, state0, silu, y, stateT, cu_seqlens,
                                              (int)N, T, C, W, rows, s);
    return launch_conv_fwd<float>(x, weight, bias, state0, silu, y, stateT, cu_seqlens, (int)N, T, C,
                                  W, rows, s);
}

osdn_status_t osdn_conv_step(const void* x, const float* weight, const float* bias, void* state,
                             int32_t silu, void* y, int32_t N, int32_t C, int32_t W,
                             osdn_dtype_t io, void* stream) {
    if (io != OSDN_BF16 && io != OSDN_F32) return OSDN_ERR_INVALID_ARG;
    if (N < 0 || C < 1 || (silu != 0 && silu != 1)) return OSDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || C > CONV_MAX_C) return OSDN_ERR_UNSUPPORTED;
    if (N == 0) return OSDN_OK;
    if (!x || !weight || !state || !y) return OSDN_ERR_INVALID_ARG;
    const size_t xb = (size_t)N * C * io_size(io);
    const Buf in[] = {{x, xb}, {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}};
    const Buf out[] = {{y, xb}, {state, xb * (W - 1)}};
    const osdn_status_t st = check_buffers(in, 3, out, 2);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (io == OSDN_BF16)
        return launch_conv_step<__nv_bfloat16>(x, weight, bias, state, silu, y, N, C, W, s);
    return launch_conv_step<float>(x, weight, bias, state, silu, y, N, C, W, s);
}

size_t osdn_conv_bwd_workspace_bytes(int32_t B, int32_t T, int32_t C, int32_t W) {
    if (B < 0 || T < 0 || C < 1 || C > CONV_MAX_C || W < 2 || W > 4) return 0;
    return up256((size_t)conv_bwd_plan((int64_t)B * T, C).row_blocks * (W + 1) * C * 4);
}

osdn_status_t osdn_conv_bwd(const void* x, const float* weight, const float* bias,
                            const void* state0, int32_t silu, const void* dy, osdn_dtype_t dy_io,
                            const float* dstateT, void* dx, float* dweight, float* dbias,
                            float* dstate0, const int32_t* cu_seqlens, int32_t num_seqs, int32_t B,
                            int32_t T, int32_t C, int32_t W, osdn_dtype_t io, void* workspace,
                            size_t workspace_bytes, void* stream) {
    int64_t rows, N;
    osdn_status_t st = check_tokens(cu_seqlens, num_seqs, B, T, io, &rows, &N);
    if (st != OSDN_OK) return st;
    if (C < 1 || (silu != 0 && silu != 1) || (dy_io != OSDN_F32 && dy_io != io))
        return OSDN_ERR_INVALID_ARG;
    if (W < 2 || W > 4 || C > CONV_MAX_C) return OSDN_ERR_UNSUPPORTED;
    if (!weight || !dweight || (rows > 0 && (!x || !dy || !dx))) return OSDN_ERR_INVALID_ARG;
    const size_t need = osdn_conv_bwd_workspace_bytes(B, T, C, W);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != OSDN_OK) return st;
    const size_t es = io_size(io), xb = (size_t)rows * C * es, sb = (size_t)N * (W - 1) * C;
    const Buf in[] = {{x, xb}, {weight, (size_t)C * W * 4}, {bias, (size_t)C * 4}, {state0, sb * es},
                      {dy, (size_t)rows * C * io_size(dy_io)}, {dstateT, sb * 4},
                      {cu_seqlens, ((size_t)N + 1) * 4}};
    const Buf out[] = {{dx, xb}, {dweight, (size_t)C * W * 4}, {dbias, (size_t)C * 4},
                       {dstate0, sb * 4}, {workspace, need}};
    st = check_buffers(in, 7, out, 5);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    if (io == OSDN_F32)
        return launch_conv_bwd<float, float>(x, weight, bias, state0, silu, dy, dstateT, dx, dweight,
                                             dbias, dstate0, part, cu_seqlens, (int)N, T, C, W, rows,
                                             s);
    if (dy_io == OSDN_F32)
        return launch_conv_bwd<__nv_bfloat16, float>(x, weight, bias, state0, silu, dy, dstateT, dx,
                                                     dweight, dbias, dstate0, part, cu_seqlens,
                                                     (int)N, T, C, W, rows, s);
    return launch_conv_bwd<__nv_bfloat16, __nv_bfloat16>(x, weight, bias, state0, silu, dy, dstateT,
                                                         dx, dweight, dbias, dstate0, part,
                                                         cu_seqlens, (int)N, T, C, W, rows, s);
}

// ---------------------------------------------------------------- selective scan
osdn_status_t osdn_ssm_fwd(const void* x, const float* dt, const float* A, const void* b,
                           const void* c, const float* D, const float* dt_bias, int32_t softplus,
                           const float* S0, void* y, float* ST, const int32_t* cu_seqlens,
                           int32_t num_seqs, int32_t B, int32_t T, int32_t H, int32_t G, int32_t Dk,
                           int32_t Dv, osdn_dtype_t io, void* workspace, size_t workspace_bytes,
                           void* stream) {
    int64_t rows, N;
    osdn_status_t st = check_tokens(cu_seqlens, num_seqs, B, T, io, &rows, &N);
    if (st == OSDN_OK) st = check_ssm(H, G, Dk, Dv);
    if (st != OSDN_OK) return st;
    if (softplus != 0 && softplus != 1) return OSDN_ERR_INVALID_ARG;
    if (!A || (rows > 0 && (!x || !dt || !b || !c || !y))) return OSDN_ERR_INVALID_ARG;
    const size_t need =
        osdn_ssm_fwd_workspace_bytes(cu_seqlens ? num_seqs : 0, B, T, H, Dk, Dv, io);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != OSDN_OK) return st;
    const size_t es = io_size(io), xb = (size_t)rows * H * Dv * es, gb = (size_t)rows * G * Dk * es,
                 sb = (size_t)N * H * Dv * Dk * 4, hb = (size_t)H * 4;
    const Buf in[] = {{x, xb}, {dt, rows * hb}, {A, hb}, {b, gb}, {c, gb}, {D, hb}, {dt_bias, hb},
                      {S0, sb}, {cu_seqlens, ((size_t)N + 1) * 4}};
    const Buf out[] = {{y, xb}, {ST, sb}, {need ? workspace : nullptr, need}};
    st = check_buffers(in, 9, out, 3);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // bf16 tokens run on the tensor cores; fp32 ones, and calls without tokens (states pass
    // through), token by token
    if (io == OSDN_BF16 && rows > 0) {
        TcsArgs t = {};
        t.dt = dt; t.A = A; t.dt_bias = dt_bias; t.D = D; t.x = static_cast<const __nv_bfloat16*>(x);
        t.S_in = S0; t.y = static_cast<__nv_bfloat16*>(y); t.S_out = ST; t.cu = cu_seqlens;
        t.rows = rows; t.N = (int)N; t.T = T; t.H = H; t.G = G; t.softplus = softplus;
        t.nvt = Dv / TCS_BV;
        const SsmSegments sg = ssm_segments(rows != N * T, rows, N, T, H, Dk, Dv, 1);
        t.seg = sg.seg;
        t.seg_state = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sg.state);
        t.seg_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sg.decay);
        return Dk == 128 ? launch_tc_fwd<128>(c, b, x, t, sg.slots, s)
                         : launch_tc_fwd<64>(c, b, x, t, sg.slots, s);
    }
    SsmArgs a = {};
    a.q = static_cast<const float*>(c); a.k = static_cast<const float*>(b);
    a.v = static_cast<const float*>(x); a.out = static_cast<float*>(y);
    a.dt = dt; a.A = A; a.D = D; a.dt_bias = dt_bias; a.S_in = S0; a.S_out = ST; a.cu = cu_seqlens;
    a.rows = rows; a.N = (int)N; a.T = T; a.H = H; a.G = G; a.softplus = softplus;
    return launch_ssm_scan<SSM_FWD>(a, ssm_f32_segments(rows, N, T, H, Dk, Dv),
                                    static_cast<uint8_t*>(workspace), Dk, Dv, s);
}

size_t osdn_ssm_fwd_workspace_bytes(int32_t num_seqs, int32_t B, int32_t T, int32_t H, int32_t Dk,
                                    int32_t Dv, osdn_dtype_t io) {
    if (B < 0 || T < 0 || H < 1 || num_seqs < 0 || (Dk != 64 && Dk != 128) ||
        (Dv != 64 && Dv != 128) || (io != OSDN_BF16 && io != OSDN_F32) || (int64_t)B * T == 0)
        return 0;
    const int64_t rows = (int64_t)B * T, N = num_seqs > 0 ? num_seqs : B;
    return io == OSDN_BF16 ? ssm_segments(rows != N * T, rows, N, T, H, Dk, Dv, 1).bytes
                           : ssm_f32_segments(rows, N, T, H, Dk, Dv).bytes;
}

osdn_status_t osdn_ssm_step(const void* x, const float* dt, const float* A, const void* b,
                            const void* c, const float* D, const float* dt_bias, int32_t softplus,
                            float* S, void* y, int32_t N, int32_t H, int32_t G, int32_t Dk,
                            int32_t Dv, osdn_dtype_t io, void* stream) {
    if (io != OSDN_BF16 && io != OSDN_F32) return OSDN_ERR_INVALID_ARG;
    if (N < 0 || (softplus != 0 && softplus != 1)) return OSDN_ERR_INVALID_ARG;
    osdn_status_t st = check_ssm(H, G, Dk, Dv);
    if (st != OSDN_OK) return st;
    const int64_t nh = (int64_t)N * H;
    if (nh == 0) return OSDN_OK;
    if (nh > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    if (!x || !dt || !A || !b || !c || !S || !y) return OSDN_ERR_INVALID_ARG;
    const size_t es = io_size(io), xb = (size_t)nh * Dv * es, gb = (size_t)N * G * Dk * es,
                 hb = (size_t)H * 4;
    const Buf in[] = {{x, xb}, {dt, N * hb}, {A, hb}, {b, gb}, {c, gb}, {D, hb}, {dt_bias, hb}};
    const Buf out[] = {{y, xb}, {S, (size_t)nh * Dv * Dk * 4}};
    st = check_buffers(in, 7, out, 2);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto launch = [&](auto dk, auto dv, auto zero) {
        using IO = decltype(zero);
        constexpr int DK = decltype(dk)::value, DV = decltype(dv)::value;
        ssm_step_kernel<DK, DV, IO><<<dim3((unsigned)nh), dim3(DV * 4), 0, s>>>(
            static_cast<const IO*>(x), dt, A, static_cast<const IO*>(b), static_cast<const IO*>(c), D,
            dt_bias, softplus, S, static_cast<IO*>(y), nh, H, G);
        return launch_status();
    };
    auto dims = [&](auto zero) {
        using c64 = std::integral_constant<int, 64>;
        using c128 = std::integral_constant<int, 128>;
        if (Dk == 128)
            return Dv == 128 ? launch(c128{}, c128{}, zero) : launch(c128{}, c64{}, zero);
        return Dv == 128 ? launch(c64{}, c128{}, zero) : launch(c64{}, c64{}, zero);
    };
    return io == OSDN_BF16 ? dims(__nv_bfloat16{}) : dims(0.f);
}

size_t osdn_ssm_bwd_workspace_bytes(int32_t num_seqs, int32_t B, int32_t T, int32_t H, int32_t Dk,
                                    int32_t Dv, osdn_dtype_t io) {
    if (B < 0 || T < 0 || H < 1 || num_seqs < 0 || (Dk != 64 && Dk != 128) ||
        (Dv != 64 && Dv != 128) || (io != OSDN_BF16 && io != OSDN_F32))
        return 0;
    // enough for heads that share rows of b and c, and for a call without tokens
    const int64_t rows = (int64_t)B * T, N = num_seqs > 0 ? num_seqs : B;
    return ssm_bwd_workspace(rows, N, T, H, 1, Dk, Dv, rows > 0 ? io : OSDN_F32).total;
}

osdn_status_t osdn_ssm_bwd(const void* x, const float* dt, const float* A, const void* b,
                           const void* c, const float* D, const float* dt_bias, int32_t softplus,
                           const float* S0, const void* dy, const float* dST, void* dx, float* ddt,
                           float* dA, void* db, void* dc, float* dD, float* ddt_bias, float* dS0,
                           const int32_t* cu_seqlens, int32_t num_seqs, int32_t B, int32_t T,
                           int32_t H, int32_t G, int32_t Dk, int32_t Dv, osdn_dtype_t io,
                           void* workspace, size_t workspace_bytes, void* stream) {
    int64_t rows, N;
    osdn_status_t st = check_tokens(cu_seqlens, num_seqs, B, T, io, &rows, &N);
    if (st == OSDN_OK) st = check_ssm(H, G, Dk, Dv);
    if (st != OSDN_OK) return st;
    if (softplus != 0 && softplus != 1) return OSDN_ERR_INVALID_ARG;
    if (!A || !dA || (rows > 0 && (!x || !dt || !b || !c || !dy || !dx || !ddt || !db || !dc)))
        return OSDN_ERR_INVALID_ARG;
    const osdn_dtype_t path = rows > 0 ? io : OSDN_F32;
    const size_t need = ssm_bwd_workspace(rows, N, T, H, G, Dk, Dv, path).total;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != OSDN_OK) return st;
    if (N * H > 0x7fffffff) return OSDN_ERR_UNSUPPORTED;
    const size_t es = io_size(io), xb = (size_t)rows * H * Dv * es, gb = (size_t)rows * G * Dk * es,
                 sb = (size_t)N * H * Dv * Dk * 4, hb = (size_t)H * 4;
    const Buf in[] = {{x, xb}, {dt, rows * hb}, {A, hb}, {b, gb}, {c, gb}, {D, hb}, {dt_bias, hb},
                      {S0, sb}, {dy, xb}, {dST, sb}, {cu_seqlens, ((size_t)N + 1) * 4}};
    const Buf out[] = {{dx, xb}, {ddt, rows * hb}, {dA, hb}, {db, gb}, {dc, gb}, {dD, hb},
                       {ddt_bias, hb}, {dS0, sb}, {workspace, need}};
    st = check_buffers(in, 11, out, 9);
    if (st != OSDN_OK) return st;
    const SsmBwdCall k = {x, dt, A, b, c, D, dt_bias, softplus, S0, dy, dST, dx, ddt, dA, db, dc, dD,
                          ddt_bias, dS0, cu_seqlens, N, T, H, G, Dk, Dv, rows,
                          static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)};
    if (path == OSDN_F32) return launch_ssm_bwd_f32(k);
    if (Dk == 128) return Dv == 128 ? launch_ssm_bwd_tc<128, 128>(k) : launch_ssm_bwd_tc<128, 64>(k);
    return Dv == 128 ? launch_ssm_bwd_tc<64, 128>(k) : launch_ssm_bwd_tc<64, 64>(k);
}

// ---------------------------------------------------------------- block norm
osdn_status_t osdn_norm_fwd(const void* f, const void* x, const void* gate, const float* w_post,
                            const float* w_next, int32_t gate_act, int32_t gate_first, float scale,
                            float eps, void* x_out, void* h, int64_t R, int32_t D, osdn_dtype_t io,
                            void* stream) {
    if (io != OSDN_BF16 && io != OSDN_F32) return OSDN_ERR_INVALID_ARG;
    if (R < 0 || D < 1 || (gate_act != 0 && gate_act != 1) || (gate_first != 0 && gate_first != 1))
        return OSDN_ERR_INVALID_ARG;
    if (D > NORM_MAX_D) return OSDN_ERR_UNSUPPORTED;
    if (R == 0) return OSDN_OK;
    if (!f || (w_next ? !h : h || !x_out)) return OSDN_ERR_INVALID_ARG;
    const size_t rb = (size_t)R * D * io_size(io), wb = (size_t)D * 4;
    const Buf in[] = {{f, rb}, {x, rb}, {gate, rb}, {w_post, wb}, {w_next, wb}};
    const Buf out[] = {{x_out, rb}, {h, rb}};
    const osdn_status_t st = check_buffers(in, 5, out, 2);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto go = [&](auto zero) {
        using IO = decltype(zero);
        return norm_dispatch<NORM_FWD_V>(D, [&](auto vec, auto tpr) {
            constexpr int TPR = decltype(tpr)::value;
            // 512 threads an SM that walk the rows with the next one's loads in flight
            const int64_t need = ceil_div(R, norm_rows(TPR)), cap = (int64_t)(512 / norm_threads(TPR)) * sm_count();
            norm_fwd_kernel<decltype(vec)::value, TPR, IO>
                <<<dim3((unsigned)(need < cap ? need : cap)), dim3(norm_threads(TPR)), 0, s>>>(
                    static_cast<const IO*>(f), static_cast<const IO*>(x),
                    static_cast<const IO*>(gate), w_post, w_next, gate_act, gate_first, scale, eps,
                    static_cast<IO*>(x_out), static_cast<IO*>(h), R, D);
            return launch_status();
        });
    };
    return io == OSDN_BF16 ? go(__nv_bfloat16{}) : go(0.f);
}

size_t osdn_norm_bwd_workspace_bytes(int64_t R, int32_t D) {
    if (R < 0 || D < 1 || D > NORM_MAX_D) return 0;
    return up256((size_t)2 * norm_bwd_blocks(R, D, false) * D * 4);  // the larger of the two
}

osdn_status_t osdn_norm_bwd(const void* f, const void* x, const void* gate, const float* w_post,
                            const float* w_next, int32_t gate_act, int32_t gate_first, float scale,
                            float eps, const void* dx_out, const void* dh, void* df, void* dx,
                            void* dgate, float* dw_post, float* dw_next, int64_t R, int32_t D,
                            osdn_dtype_t io, void* workspace, size_t workspace_bytes,
                            void* stream) {
    if (io != OSDN_BF16 && io != OSDN_F32) return OSDN_ERR_INVALID_ARG;
    if (R < 0 || D < 1 || (gate_act != 0 && gate_act != 1) || (gate_first != 0 && gate_first != 1))
        return OSDN_ERR_INVALID_ARG;
    if (D > NORM_MAX_D) return OSDN_ERR_UNSUPPORTED;
    if ((w_post != nullptr) != (dw_post != nullptr) || (w_next != nullptr) != (dw_next != nullptr))
        return OSDN_ERR_INVALID_ARG;
    if (R > 0 && (!f || !df || (!dx_out && !dh) || (w_next != nullptr) != (dh != nullptr) ||
                  (gate != nullptr) != (dgate != nullptr) || (!x && dx)))
        return OSDN_ERR_INVALID_ARG;
    const size_t need = osdn_norm_bwd_workspace_bytes(R, D);
    osdn_status_t st = check_workspace(workspace, workspace_bytes, need);
    if (st != OSDN_OK) return st;
    const size_t rb = (size_t)R * D * io_size(io), wb = (size_t)D * 4;
    const Buf in[] = {{f, rb}, {x, rb}, {gate, rb}, {w_post, wb}, {w_next, wb}, {dx_out, rb}, {dh, rb}};
    const Buf out[] = {{df, rb}, {dx, rb}, {dgate, rb}, {dw_post, wb}, {dw_next, wb},
                       {workspace, need}};
    st = check_buffers(in, 7, out, 6);
    if (st != OSDN_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* part = static_cast<float*>(workspace);
    const int64_t blocks = norm_bwd_blocks(R, D, w_next != nullptr);
    if (blocks > 0) {
        auto go = [&](auto zero) {
            using IO = decltype(zero);
            return norm_dispatch<NORM_BWD_V>(D, [&](auto vec, auto tpr) {
                constexpr int TPR = decltype(tpr)::value;
                auto kern = w_next ? norm_bwd_kernel<decltype(vec)::value, TPR, true, IO>
                                   : norm_bwd_kernel<decltype(vec)::value, TPR, false, IO>;
                kern<<<dim3((unsigned)blocks), dim3(norm_threads(TPR)), 0, s>>>(
                    static_cast<const IO*>(f), static_cast<const IO*>(x), static_cast<const IO*>(gate),
                    w_post, w_next, gate_act, gate_first, scale, eps, static_cast<const IO*>(dx_out),
                    static_cast<const IO*>(dh), static_cast<IO*>(df), static_cast<IO*>(dx),
                    static_cast<IO*>(dgate), part, R, D);
                return launch_status();
            });
        };
        st = io == OSDN_BF16 ? go(__nv_bfloat16{}) : go(0.f);
        if (st != OSDN_OK) return st;
    }
    if (!dw_post && !dw_next) return OSDN_OK;
    norm_reduce_kernel<<<dim3((unsigned)ceil_div(D, 32), 2), dim3(32, NORM_RED_WARPS), 0, s>>>(
        part, (int)blocks, D, dw_post, dw_next);
    return launch_status();
}

}  // extern "C"
