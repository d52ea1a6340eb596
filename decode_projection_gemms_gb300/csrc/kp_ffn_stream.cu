// Forward products for few tokens, where the cost is reading the weights once:
//     y[m, n] = round( sum_k x[m, k] W[n, k] )                      (plain)
//     h[m, n] = round( act(sum_k x[m, k] Wg[n, k]) * sum_k x[m, k] Wu[n, k] )   (gated)
// over bf16 / fp16 operands or over microscaled 4-bit ones.
//
// The MMA's 128 rows are rows of the weights, its columns the tokens (16 .. 128 a
// tile, further tiles along the grid's y axis read the weights from L2). The
// 16-bit gated form has 64 rows of Wg and the same 64 of Wu in one MMA, the 4-bit
// one 128 of each in two accumulators. A feature tile's K range is split over the
// C CTAs of a cluster; their fp32 partial tiles go through L2, or up to 8 tokens
// through distributed shared memory, and the cluster sums them in rank order, so
// the result does not depend on timing; the sums of a gate and of its factor meet
// in one thread there. A K block is 128 bytes of a row (64 16-bit or 256 4-bit
// columns), in boxes of 8 or 16 KB; a 4-bit stage also brings its scale tiles,
// which tcgen05.cp lays into the stage's own TMEM columns (their last readers
// finished before the stage was refilled).
//
// Bound: HBM plus about 5 us that do not grow with the weights (launch, tensor memory,
// the first copies' latency, the two-step sum): with cold weights in a graph, T = 1, K =
// 7168 reads F = 256 (7.3 MB) in 7.2 us, F = 1408 (40 MB) in 10.9, F = 2048 (58.7 MB) in
// 13.1 (4.5 TB/s, of 6.8 measured), F = 4096 (117 MB) in 21.2 (5.5 TB/s); in 4 bits N =
// 4096 (15.7 MB) in 7.4. That part is not a floor: the projection's kernels read the
// same 58.7 MB in 10.7 us (CUDA cores, one token) and 11.4 (tcgen05, two tokens).
//
// Up to 8 tokens the 4-bit forms also quantise x themselves: warps 2 .. 5 turn a
// stage's 256 columns of two tokens each into the operand and scale tile that a copy
// would have brought (T = 1, N = 4096, K = 7168: 7.4 us on the device against 8.0 with a
// launch for x, 12 us against 20 from Python, which then allocates nothing but y).
//
// Warp 0: copies; warp 1: TMEM and MMA; warps 2 .. 5: x in 4 bits (few tokens),
// epilogue; all six reduce.
#include <algorithm>
#include <mutex>

#include "kp_mx4.cuh"

namespace kp {

namespace {

constexpr int kThreads = 192;
constexpr int kRows = 128;                 // rows of an MMA
constexpr int kMaxTok = 128;               // tokens per tile
constexpr int kMaxStages = 10;
constexpr int kFewTok = 8;                 // tokens up to which a call needs no workspace
constexpr size_t kBarBytes = 256;
constexpr size_t kMaxSmem = 227 * 1024;
// What a CTA takes for its stages: half an SM, so that clusters of eight fill the
// GPU. With all of an SM's shared memory each, 15 such clusters fit where two to
// an SM makes 36 (T = 1, F = 2048, K = 7168, cold weights: 24.6 us against 13.1).
constexpr size_t kSmem = 113 * 1024;

struct StreamParams {
    const uint8_t *sa, *sb, *sx;   // 4-bit: scale tiles
    int kt_n;                      // 128-column scale tiles per row tile
    uint16_t *y;
    float *g, *u;   // optional: both products' sums, [M, N]
    int64_t ldy;
    float *ws;                     // partial tiles; few tokens: shared memory instead
    const void *x;                 // 4-bit, few tokens: x in 16 bits, quantised here
    int64_t ldx;
    int x_vec;                     // its rows start on 16 bytes
    int *err;
    int few;                       // partial tiles stay in shared memory
    int M, N, K, Mpad, KB, C, stages, n_tiles, act, dtype, vec4;
    uint32_t idesc, tmem_cols, stage_bytes, sf_col;
};

// What a CTA holds of the weights: 128 rows of W (plain); 64 rows of Wg and the
// same 64 of Wu in one MMA (16-bit gated); 128 and 128 with an accumulator each
// (4-bit gated: a scale tile is 128 rows of one matrix).
template <bool kMx4, bool kGated>
struct Shape {
    static constexpr int acc = kMx4 && kGated ? 2 : 1;            // accumulators
    static constexpr int feat = kGated && !kMx4 ? 64 : 128;       // features per tile
    static constexpr uint32_t w_bytes = acc * kRows * 128;        // a K block of the weights
    static constexpr uint32_t sc_bytes = kMx4 ? (acc + 1) * 1024 : 0;
    static constexpr uint32_t sf_cols = kMx4 ? 8 * (acc + 1) : 0; // TMEM columns of a stage's scales
    static __host__ __device__ uint32_t off_sc(int Mpad) { return w_bytes + static_cast<uint32_t>(Mpad) * 128; }
    static __host__ __device__ uint32_t stage_bytes(int Mpad) { return off_sc(Mpad) + sc_bytes; }
};

template <bool kMx4, bool kGated>
__global__ void __launch_bounds__(kThreads, 1)
    ffn_stream_kernel(const __grid_constant__ CUtensorMap tma, const __grid_constant__ CUtensorMap tmb,
                      const __grid_constant__ CUtensorMap tmx, const StreamParams p) {
    using L = Shape<kMx4, kGated>;
    constexpr int kAcc = L::acc;
    constexpr int kPart = kAcc * kRows;   // fp32 sums per token of a partial tile
    extern __shared__ uint8_t fs_smem_raw[];
    const uint32_t raw = smem_u32(fs_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = fs_smem_raw + (base - raw);
    const int S = p.stages;
    uint64_t *full = reinterpret_cast<uint64_t *>(gbase + static_cast<size_t>(S) * p.stage_bytes);
    uint64_t *empty = full + S;
    uint64_t *accf = empty + S;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(accf + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int C = p.C;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int tile = static_cast<int>(blockIdx.x) / C;
    const int m0 = static_cast<int>(blockIdx.y) * p.Mpad;
    const int Mloc = min(p.M - m0, p.Mpad);
    const int kb0 = static_cast<int>(static_cast<long long>(p.KB) * rank / C);
    const int kb1 = static_cast<int>(static_cast<long long>(p.KB) * (rank + 1) / C);
    const int n_st = kb1 - kb0;
    const int pre = n_st < S ? n_st : S;
    const uint32_t xbytes = static_cast<uint32_t>(p.Mpad) * 128;
    constexpr int kCols = kMx4 ? 128 : 64;   // map columns (bytes or elements) per K block
    const bool quantises = kMx4 && p.x != nullptr;

    // scale tiles that exist of K block kb (two but at the end of K)
    auto sc_tiles = [&](int kb) { return min(2, p.kt_n - 2 * kb); };
    auto issue_w = [&](int s, int stage) {
        const uint64_t pol = policy_evict_first();
        const int kb = kb0 + s;
        const uint32_t st = base + stage * p.stage_bytes;
        const uint32_t bar = smem_u32(full + stage);
        const uint32_t scb = kMx4 ? 512u * static_cast<uint32_t>(sc_tiles(kb)) : 0u;
        mbar_expect_tx(bar, L::w_bytes + scb * kAcc + (quantises ? 0u : xbytes + scb));
        tma_load_2d(st, &tma, bar, kb * kCols, tile * L::feat, pol);
        if constexpr (kGated) tma_load_2d(st + L::w_bytes / 2, &tmb, bar, kb * kCols, tile * L::feat, pol);
        if constexpr (kMx4) {
            const size_t off = (static_cast<size_t>(tile) * p.kt_n + 2 * kb) * 512;
            const uint32_t sc = st + L::off_sc(p.Mpad);
            bulk_load(sc, p.sa + off, scb, bar);
            if constexpr (kAcc == 2) bulk_load(sc + 1024, p.sb + off, scb, bar);
        }
    };
    auto issue_x = [&](int s, int stage) {
        const int kb = kb0 + s;
        const uint32_t st = base + stage * p.stage_bytes;
        const uint32_t bar = smem_u32(full + stage);
        tma_load_2d(st + L::w_bytes, &tmx, bar, kb * kCols, m0, policy_evict_last());
        if constexpr (kMx4) {
            const size_t off = (static_cast<size_t>(m0 >> 7) * p.kt_n + 2 * kb) * 512;
            bulk_load(st + L::off_sc(p.Mpad) + kAcc * 1024, p.sx + off,
                      512u * static_cast<uint32_t>(sc_tiles(kb)), bar);
        }
    };

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            // the copies, and the warps that quantise a token
            mbar_init(smem_u32(full + s), quantises ? 1 + static_cast<uint32_t>(min(Mloc, 4)) : 1u);
            mbar_init(smem_u32(empty + s), 1);
        }
        mbar_init(smem_u32(accf), 1);
        *abort_flag = 0;
        fence_mbar_init();
        // the weights do not depend on the kernel before: they start at once
        for (int s = 0; s < pre; ++s) issue_w(s, s);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), p.tmem_cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        const bool mine = elect_one();
        pdl_wait();   // x (quantised by the kernel before, when there is one)
        if (mine && !quantises)
            for (int s = 0; s < pre; ++s) issue_x(s, s);
        int stage = 0;
        uint32_t phase = 0;
        for (int s = pre; s < n_st; ++s) {
            mbar_wait_bounded(smem_u32(empty + stage), phase, abort_flag, p.err, DEV_TIMEOUT_EMPTY);
            if (mine) {
                issue_w(s, stage);
                if (!quantises) issue_x(s, stage);
            }
            if (++stage == S) stage = 0, phase ^= 1;
        }
        // every copy has landed before this CTA leaves, also where another warp's wait
        // runs out after this one's last copy is issued
        for (int s = n_st > S ? n_st - S : 0; s < n_st; ++s)
            ffn_drain_wait(smem_u32(full + (s % S)), static_cast<uint32_t>((s / S) & 1));
        __syncwarp();
    } else if (warp == 1) {
        const bool mine = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        for (int s = 0; s < n_st; ++s) {
            mbar_wait_bounded(smem_u32(full + stage), phase, abort_flag, p.err, DEV_TIMEOUT_FULL);
            tc_fence_after();
            if (mine) {
                const uint32_t st = base + stage * p.stage_bytes;
                const uint64_t ad = desc_kmajor(st);
                const uint64_t bd = desc_kmajor(st + L::w_bytes);
                if constexpr (kMx4) {
                    const int kb = kb0 + s;
                    const uint32_t sf = tmem + p.sf_col + static_cast<uint32_t>(stage) * L::sf_cols;
                    const uint64_t sc = desc_scales(st + L::off_sc(p.Mpad));
                    for (int j = 0; j < sc_tiles(kb); ++j)
#pragma unroll
                        for (int o = 0; o <= kAcc; ++o)   // weights, tokens
                            tmem_cp_scales(sf + 8 * o + 4 * j, sc + 64 * o + 32 * j);
                    // 64 columns a step; steps past K are left out (their scales are not loaded)
                    const int steps = min(4, (p.K - kb * 256 + 63) >> 6);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        if (kk >= steps) break;
                        const uint32_t id = idesc_sf(p.idesc, (kk & 1) * 2);
                        const uint32_t sfk = sf + 4 * (kk >> 1);
#pragma unroll
                        for (int a = 0; a < kAcc; ++a)
                            umma_mxf4(tmem + a * p.Mpad, ad + (a * kRows * 128 >> 4) + 2 * kk, bd + 2 * kk, id,
                                      sfk + 8 * a, sfk + 8 * kAcc, (s > 0 || kk > 0) ? 1u : 0u);
                    }
                } else {
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_bf16(tmem, ad + 2 * kk, bd + 2 * kk, p.idesc, (s > 0 || kk > 0) ? 1u : 0u);
                }
                umma_commit(smem_u32(empty + stage));
            }
            if (++stage == S) stage = 0, phase ^= 1;
        }
        if (mine) umma_commit(smem_u32(accf));
        __syncwarp();
    } else {
        if constexpr (kMx4) {
            if (quantises) {
                // Warp 2 + w has tokens w and w + 4 of every stage, eight rows of 256
                // columns loaded at a time. It sees every round of every buffer, so it
                // is never two phases behind the barrier that it waits on.
                auto run = [&](auto zero) {
                    using T = decltype(zero);
                    const int w = warp - 2;
                    const int lg = w + 4 < Mloc ? 1 : 0;     // log2 of its tokens
                    const int units = w < Mloc ? n_st << lg : 0;
                    int stage = 0;
                    uint32_t phase = 1;   // of a buffer's round before: passes at once in the first
                    for (int u0 = 0; u0 < units; u0 += 8) {
                        Eight<T> e[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int u = min(u0 + i, units - 1);
                            const T *row = static_cast<const T *>(p.x) + (m0 + w + 4 * (u & lg)) * p.ldx;
                            const int c = (kb0 + (u >> lg)) * 256 + lane * 8;
                            if (p.x_vec && c + 8 <= p.K)
                                e[i].load_full(row + c);
                            else
                                e[i].load(row, c, p.K);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (u0 + i >= units) break;
                            const int r = w + 4 * ((u0 + i) & lg);
                            mbar_wait_bounded(smem_u32(empty + stage), phase, abort_flag, p.err, DEV_TIMEOUT_EMPTY);
                            uint8_t *x8 = gbase + static_cast<size_t>(stage) * p.stage_bytes + L::w_bytes;
                            uint8_t *sc = gbase + static_cast<size_t>(stage) * p.stage_bytes + L::off_sc(p.Mpad) + kAcc * 1024;
                            uint32_t b;
                            const uint32_t q = quantize8(e[i], b);
                            // row r of the 128-byte swizzled operand, lane r of the scale tile
                            *reinterpret_cast<uint32_t *>(x8 + r * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4) = q;
                            if ((lane & 3) == 0)
                                sc[(lane >> 4) * 512 + r * 16 + ((lane >> 2) & 3)] = static_cast<uint8_t>(b);
                            if (((u0 + i) & lg) == lg) {   // the warp's last token of the stage
                                // the tensor cores read it through the asynchronous proxy
                                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                                __syncwarp();
                                if (lane == 0) mbar_arrive(smem_u32(full + stage));
                                if (++stage == S) stage = 0, phase ^= 1;
                            }
                        }
                    }
                };
                if (p.dtype == KP_FP16)
                    run(__half());
                else
                    run(__nv_bfloat16());
            }
        }
        // accumulators -> this CTA's partial tile [token][kPart], 128 bytes a warp
        // and token: in L2, or for few tokens or one CTA in the stage memory, which
        // is free once the last MMA has completed
        const int q = warp & 3;
        const int row = q * 32 + lane;
        mbar_wait_bounded(smem_u32(accf), 0, abort_flag, p.err, DEV_TIMEOUT_ACC_FULL);
        tc_fence_after();
        const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16);
        float *part = p.few ? reinterpret_cast<float *>(gbase)
                            : p.ws + ((static_cast<size_t>(blockIdx.y) * p.n_tiles + tile) * C + rank) *
                                         static_cast<size_t>(kPart) * p.Mpad;
        for (int c0 = 0; c0 < Mloc; c0 += 16) {
            uint32_t v[kAcc][16];
#pragma unroll
            for (int a = 0; a < kAcc; ++a) tmem_ld16(taddr + a * p.Mpad + c0, v[a]);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (c0 + i < Mloc)
#pragma unroll
                    for (int a = 0; a < kAcc; ++a)
                        part[(c0 + i) * kPart + a * kRows + row] = __uint_as_float(v[a][i]);
        }
        tc_fence_before();
    }

    // every partial tile of the cluster is written and visible after this
    __syncwarp();
    if (C > 1)
        cluster_sync_all();
    else
        __syncthreads();
    {
        const size_t stride = static_cast<size_t>(kPart) * p.Mpad;
        const float *parts = p.ws + (static_cast<size_t>(blockIdx.y) * p.n_tiles + tile) * C * stride;
        // A lane takes four features of a token, CTA r of the cluster every C-th
        // group of tokens, kDeep groups at a time so that their sums are read
        // together.
        constexpr int kLanes = L::feat / 4;              // lanes per token: 16 or 32
        constexpr int kTok = kThreads / kLanes;          // tokens of a group
        constexpr int kDeep = kGated ? 2 : 4;
        const int f = 4 * (threadIdx.x % kLanes);
        const int n = tile * L::feat + f;
        for (int mb = rank * kTok + threadIdx.x / kLanes; mb < Mloc; mb += kTok * C * kDeep) {
            float va[kDeep][4], vb[kDeep][4];
#pragma unroll
            for (int d = 0; d < kDeep; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i) va[d][i] = vb[d][i] = 0.f;
            auto add = [](const float4 a, float(&v)[4]) { v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w; };
#pragma unroll 4
            for (int r = 0; r < C; ++r)   // in rank order
#pragma unroll
                for (int d = 0; d < kDeep; ++d) {
                    // past the end: the last token again, so that no branch parts the loads
                    const int at = min(mb + d * kTok * C, Mloc - 1) * kPart + f;
                    if (p.few) {
                        const uint32_t src = mapa_shared(base, static_cast<uint32_t>(r)) + 4u * static_cast<uint32_t>(at);
                        add(ld_dsmem_f4(src), va[d]);
                        if constexpr (kGated) add(ld_dsmem_f4(src + 4u * L::feat), vb[d]);
                    } else {
                        const float4 *src = reinterpret_cast<const float4 *>(parts + r * stride + at);
                        add(__ldcg(src), va[d]);
                        if constexpr (kGated) add(__ldcg(src + L::feat / 4), vb[d]);
                    }
                }
#pragma unroll
            for (int d = 0; d < kDeep; ++d) {
                const int64_t om = m0 + mb + d * kTok * C;
                if (om - m0 >= Mloc) continue;
                auto put = [&](uint16_t *dst, int64_t ld, const float(&v)[4]) {
                    uint16_t *o = dst + om * ld + n;
                    const uint32_t lo = elem_round(v[0], p.dtype) | static_cast<uint32_t>(elem_round(v[1], p.dtype)) << 16;
                    const uint32_t hi = elem_round(v[2], p.dtype) | static_cast<uint32_t>(elem_round(v[3], p.dtype)) << 16;
                    if (p.vec4 && n + 4 <= p.N) {
                        *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
                    } else {
                        if (n < p.N) o[0] = static_cast<uint16_t>(lo);
                        if (n + 1 < p.N) o[1] = static_cast<uint16_t>(lo >> 16);
                        if (n + 2 < p.N) o[2] = static_cast<uint16_t>(hi);
                        if (n + 3 < p.N) o[3] = static_cast<uint16_t>(hi >> 16);
                    }
                };
                auto put_sums = [&](float *dst, const float(&v)[4]) {
                    float *o = dst + om * p.N + n;
                    if (p.N % 4 == 0 && n + 4 <= p.N) {
                        *reinterpret_cast<float4 *>(o) = make_float4(v[0], v[1], v[2], v[3]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n + i < p.N) o[i] = v[i];
                    }
                };
                if constexpr (kGated) {
                    float h[4];
                    ffn_gate(va[d], vb[d], p.act, h);
                    put(p.y, p.ldy, h);
                    if (!kMx4 && p.g) {
                        put_sums(p.g, va[d]);
                        put_sums(p.u, vb[d]);
                    }
                } else {
                    put(p.y, p.ldy, va[d]);
                }
            }
        }
    }
    __syncwarp();
    if (C > 1 && p.few) cluster_sync_all();   // the peers have read this CTA's partial tile
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, p.tmem_cols);
}

// ---- launch plan ----------------------------------------------------------------

struct Plan {
    int Mpad, mt, tiles, KB, C, stages;
    int acc, feat;
    bool few;   // partial tiles in shared memory
    uint32_t stage_bytes, sf_cols, tmem_cols;
};

template <bool kMx4, bool kGated>
void shape_of(Plan &q) {
    using L = Shape<kMx4, kGated>;
    q.acc = L::acc;
    q.feat = L::feat;
    q.sf_cols = L::sf_cols;
    q.stage_bytes = L::stage_bytes(q.Mpad);
}

Plan make_plan(bool mx4, bool gated, int M, int N, int K, int sms) {
    Plan q;
    q.Mpad = std::min((M + 15) / 16 * 16, kMaxTok);
    if (mx4)
        gated ? shape_of<true, true>(q) : shape_of<true, false>(q);
    else
        shape_of<false, true>(q);
    q.mt = (M + q.Mpad - 1) / q.Mpad;
    q.tiles = (N + q.feat - 1) / q.feat;
    q.KB = mx4 ? (K + 255) / 256 : (K + 63) / 64;
    // The cluster grows while each CTA keeps two K blocks and the grid stays below
    // what was measured to help, with weights that the L2 does not hold: 1.7 CTAs per SM
    // in 16 bits (T = 1, K = 7168, gated: F = 2048 C = 8 13.1 us, 4 13.4, 2 16.0; F = 1408
    // 10.9, 11.4, 15.3; F = 256 7.2, 9.4, 14.4), one in 4 bits (x quantised before, 16 x
    // 4096 x 7168: C = 8 8.5 us, 4 7.7, 2 8.8), and for C = 8 in 4 bits the 15 clusters
    // that fit at one CTA per SM (16 x 1408: C = 8 6.7, 4 6.8; 16 x 2048: 7.3, 7.0). Two
    // blocks: 77 x 4099 x 2050 in 4 bits (nine) C = 8 8.9, 4 6.7, 2 8.1.
    const int64_t grid = static_cast<int64_t>(q.tiles) * q.mt;
    const int most = mx4 ? sms : sms * 17 / 10;
    q.C = 1;
    while (q.C < 8 && q.KB >= 4 * q.C && grid * q.C * 2 <= (mx4 && q.C == 4 ? sms * 4 / 5 : most)) q.C *= 2;
    const uint32_t acc = static_cast<uint32_t>(q.acc) * q.Mpad;
    int st = static_cast<int>((kSmem - 1024 - kBarBytes) / q.stage_bytes);
    st = std::min(st, kMaxStages);
    if (mx4) st = std::min(st, static_cast<int>((512 - acc) / q.sf_cols));
    st = std::min(st, (q.KB + q.C - 1) / q.C);
    // partial tiles in the stage memory
    q.few = q.C == 1 || M <= kFewTok;
    if (q.few)
        st = std::max<int>(st, (static_cast<size_t>(q.acc) * kRows * 4 * q.Mpad + q.stage_bytes - 1) / q.stage_bytes);
    q.stages = st;
    q.tmem_cols = 32;
    while (q.tmem_cols < acc + q.sf_cols * st) q.tmem_cols <<= 1;
    return q;
}

std::mutex g_mu;
bool g_ready[64];   // devices whose kernels have their shared memory raised

}  // namespace

// Least-squares fits of 720 measured products (16 <= M <= 1536, 256 <= N <= 4096,
// 512 <= K <= 7168), off by 5 to 13 % on average: rounds of CTAs over the SMs, each
// with its K blocks and its share of the tokens' sums.
float ffn_stream_us(bool mx4, bool gated, int M, int N, int K, int sms) {
    const Plan q = make_plan(mx4, gated, M, N, K, sms);
    const float tok = static_cast<float>(q.Mpad) / kMaxTok;
    const int per_sm = mx4 && gated && q.Mpad > 64 ? 1 : 2;   // TMEM: scales and two accumulators
    const float r = static_cast<float>((static_cast<int64_t>(q.tiles) * q.mt * q.C + sms * per_sm - 1) / (sms * per_sm));
    const float kb = static_cast<float>((q.KB + q.C - 1) / q.C);
    if (!mx4) return 4.5f + r * (-0.2f + 0.38f * kb + tok * (2.6f + 2.f / q.C));
    return gated ? 2.3f + r * (1.4f + 0.48f * kb + tok * (5.4f + 1.2f / q.C))
                 : -5.f + r * (8.7f + 0.38f * kb + tok * (2.6f + 0.8f / q.C));
}

bool ffn_stream_quantises(int M) { return M <= kFewTok; }

size_t ffn_stream_scratch(bool mx4, bool gated, int M, int N, int K, int sms) {
    const Plan q = make_plan(mx4, gated, M, N, K, sms);
    if (q.few) return 0;
    return static_cast<size_t>(q.mt) * q.tiles * q.C * q.acc * kRows * q.Mpad * sizeof(float);
}

cudaError_t ffn_stream_launch(const FfnArgs &a, const FfnDev &d, cudaStream_t s) {
    const Plan q = make_plan(a.mx4, a.gated, a.M, a.N, a.K, d.sms);
    if (!q.few && !a.ws) return cudaErrorInvalidValue;
    const bool quantises = a.mx4 && a.x;
    if (quantises && a.M > kFewTok) return cudaErrorInvalidValue;
    using Fn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, StreamParams);
    static const Fn kernels[] = {ffn_stream_kernel<false, true>, ffn_stream_kernel<true, false>,
                                 ffn_stream_kernel<true, true>};   // 16-bit gated, 4-bit, 4-bit gated
    if (!a.mx4 && !a.gated) return cudaErrorInvalidValue;          // skinny_gemm's work
    cudaError_t e = cudaSuccess;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (d.dev >= 64 || !g_ready[d.dev]) {
            for (Fn f : kernels)
                if (e == cudaSuccess)
                    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMaxSmem));
            if (e != cudaSuccess) return e;
            if (d.dev < 64) g_ready[d.dev] = true;
        }
    }
    StreamParams p = {};
    p.sa = a.qa.scales;
    p.sb = a.qb.scales;
    p.sx = a.qx.scales;
    p.kt_n = static_cast<int>(mx4_ktiles(a.K));
    p.y = static_cast<uint16_t *>(a.y);
    p.g = a.g;
    p.u = a.u;
    p.ldy = a.ldy;
    p.ws = a.ws;
    p.few = q.few;
    if (quantises) {
        p.x = a.x;
        p.ldx = a.ldx;
        p.x_vec = (reinterpret_cast<uintptr_t>(a.x) & 15) == 0 && a.ldx % 8 == 0;
    }
    p.err = a.err;
    p.M = a.M;
    p.N = a.N;
    p.K = a.K;
    p.Mpad = q.Mpad;
    p.KB = q.KB;
    p.C = q.C;
    p.stages = q.stages;
    p.n_tiles = q.tiles;
    p.act = a.act;
    p.dtype = a.dtype;
    p.vec4 = a.ldy % 4 == 0 && (reinterpret_cast<uintptr_t>(a.y) & 7) == 0;   // 8-byte stores of y's rows
    p.idesc = a.mx4 ? idesc_mxf4(kRows, q.Mpad) : idesc_f16(a.dtype, kRows, q.Mpad);
    p.tmem_cols = q.tmem_cols;
    p.stage_bytes = q.stage_bytes;
    p.sf_col = static_cast<uint32_t>(q.acc * q.Mpad);

    CUtensorMap ma, mb, mx;
    if (a.mx4) {
        const int64_t pitch = mx4_pitch(a.K);
        e = ffn_tensor_map(&ma, a.qa.codes, a.N, pitch, pitch, kRows, 128, kMapU8);
        if (e == cudaSuccess && a.gated) e = ffn_tensor_map(&mb, a.qb.codes, a.N, pitch, pitch, kRows, 128, kMapU8);
        if (quantises)
            mx = ma;
        else if (e == cudaSuccess)
            e = ffn_tensor_map(&mx, a.qx.codes, a.M, pitch, pitch, q.Mpad, 128, kMapU8);
    } else {
        e = ffn_tensor_map(&ma, a.Wa, a.N, a.K, a.lda, q.feat, 64, a.dtype);
        if (e == cudaSuccess && a.gated) e = ffn_tensor_map(&mb, a.Wb, a.N, a.K, a.ldb, q.feat, 64, a.dtype);
        if (e == cudaSuccess) e = ffn_tensor_map(&mx, a.x, a.M, a.K, a.ldx, q.Mpad, 64, a.dtype);
    }
    if (e != cudaSuccess) return e;
    if (!a.gated) mb = ma;

    size_t smem = 0;
    e = ffn_smem_for_tmem(d.dev, q.tmem_cols, static_cast<size_t>(q.stages) * q.stage_bytes + 1024 + kBarBytes, &smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(q.tiles * q.C), static_cast<unsigned>(q.mt), 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(q.C);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernels[a.mx4 ? 1 + a.gated : 0], ma, mb, mx, p);
}

}  // namespace kp
