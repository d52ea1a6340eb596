// Tile kernel of the feed-forward operators: D[m, n] = sum_k A[m, k] B[n, k] with
// fp32 accumulation, for many tokens (forward) and for the backward pass, where
// the tensor cores are the bound.
//
// Two CTAs of a cluster (an SM pair) compute one 256 x nt tile (nt up to 256) with
// tcgen05.mma.cta_group::2: each holds 128 rows of A, half of B's nt rows, and
// the accumulator rows of its own A, so an operand byte in shared memory feeds
// twice the products that it would in a tile of one CTA. The leader's warp 1
// issues every MMA; both CTAs' copies complete on the leader's barriers, and
// tcgen05.commit returns stages and accumulators to both. Clusters are
// persistent: a cluster takes items c, c + n, ... of the tile list, whose order
// keeps a band of row tiles together so that their operands stay in L2.
// D[m, n] = sum_k A[m, k] B[n, k], D row-major.
//
// Forms:
//   gated    B's halves are nt/2 rows of Wg (CTA 0) and the same ones of Wu (CTA
//            1): a thread of the epilogue finds the gate in accumulator column c
//            and its factor in column nt/2 + c;
//   backward one list of the tiles of dx and of both weights' gradients (T = 333, F =
//            1416, K = 2048: 20 us, as two launches 30). dx is two products into one
//            accumulator (dG Wg, then dU Wu), Wg and Wu read as they lie, N
//            contiguous (the MMA's transposed operand); the weights' gradients are
//            dG^T x and dU^T x, both operands with K (the tokens) strided. dx's items,
//            the longest, come first; clusters without one take weight tiles for as
//            long. Where even so dx would end last, its contraction is split over
//            clusters, whose fp32 partial sums a second kernel adds in order;
//   4-bit    kind::mxf4; scale tiles go to TMEM columns of their stage. The
//            accumulator and the scales fill the tensor memory, so these have
//            one accumulator, the 16-bit forms two.
//
// Bound: the tensor cores, which are busy 87 % of the time in the gated form (4003 x
// 2048 x 7168, 128 to 130 us, 1.81 to 1.84 PFLOP/s: the measured library rate is 1.88),
// 90 % in the backward pass and 52 % in 4 bits (4096 x 4096 x 7168, the product alone,
// 47 us, 5.1 PFLOP/s; there four rounds of tiles hold 3.4 rounds of work, and the
// accumulator's way out takes 9 %).
//
// Warp 0: copies; warp 1: TMEM, MMA (leader); warps 2 .. 9: epilogue.
#include <algorithm>
#include <mutex>

#include "kp_ffn.cuh"

namespace kp {

namespace {

constexpr int kThreads = 320;
constexpr int kTile = 256;                // rows of D per cluster; columns at most
constexpr uint32_t kHalf = 128 * 128;     // bytes of 128 rows of a K block (128 bytes of K)
constexpr int kBand = 16;                 // row tiles kept together in the tile order (8: backward 1.5 % slower)
constexpr size_t kMaxSmem = 227 * 1024;
constexpr size_t kBarBytes = 256;

// 16-bit forms' outputs leave through shared memory, 32 rows of 64 columns a warp at
// a time, in copies of whole lines (gated 4003 x 2048 x 7168: 127 us, with stores of
// 32 bytes from each lane to a row of its own 130). In 4 bits the stage that this
// memory costs is worth more (4096 x 4096 x 7168: 51.6 us, with stores 50.1).
// Outputs whose rows do not start on 16 bytes pass through it in both cases, 16
// columns at a time in rows of kOutPitch bytes.
constexpr uint32_t kOutPitch = 48;
constexpr uint32_t out_box(bool mx4) { return mx4 ? 32 * kOutPitch : 32 * 128; }
constexpr uint32_t out_bytes(bool mx4) { return 8 * out_box(mx4); }
// Operand halves and, in 4 bits, pairs of scale tiles (one of A, up to two of B); as
// many stages as fit.
constexpr uint32_t stage_bytes(bool mx4) { return 2 * kHalf + (mx4 ? 3 * 1024 : 0); }
constexpr int stages(bool mx4) {
    return static_cast<int>((kMaxSmem - 1024 - kBarBytes - out_bytes(mx4)) / stage_bytes(mx4));
}

struct TileMaps {
    CUtensorMap a0, a1, b0, b1, sa, sb0, sb1;
    CUtensorMap aw0, aw1, bw;   // backward: operands of the weights' gradients
    CUtensorMap y[3];           // outputs: gated, of the tile's two halves; backward, dx, dWg, dWu
    CUtensorMap g, u;           // gated: the two products in fp32
};

// The tiles of one output shape.
struct TileSet {
    int M, N;             // of the output
    int tiles_m, tiles_n;
    int nt;               // accumulator columns of a tile (gated: of both products)
    int KB;               // K blocks
    uint32_t idesc;
};

struct TileParams {
    TileSet set[2];       // 0: the forward output or dx; 1: the weights' gradients, twice
    uint16_t *y[3];
    float *g, *u;
    int64_t ldy;
    float *ws;
    const float *scale;   // backward: factor of every sum (none: 1)
    int *err;
    int K;
    int items;            // of set 0: tiles, times the parts of a split contraction
    int splits;
    int w_items, w_first; // of set 1; those a cluster without an own last item of set 0 takes meanwhile
    int KB1;              // K blocks of dx's first product
    int kt_n;             // 4-bit: scale tiles per row tile
    int act, dtype, vec, vec_gu;
    int pairs;            // y's rows start on 4 bytes
    int copy_out;         // y's rows allow copies from shared memory (16-byte starts and lengths)
};

// ---- cta_group::2 forms ----------------------------------------------------------
__device__ __forceinline__ void pair_load(uint32_t dst, const void *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void pair_commit(uint32_t bar) {   // the same barrier in both CTAs
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ void pair_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void pair_mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa,
                                              uint32_t sb, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
        : "memory");
}
__device__ __forceinline__ void pair_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ void remote_arrive(uint32_t bar) {   // shared::cluster address
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Operand stored with M / N contiguous, 128-byte swizzle: 64-element groups
// 8 KB apart (64 K rows of 128 bytes), 8 K rows 1 KB apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
    return elem_round(a, dtype) | static_cast<uint32_t>(elem_round(b, dtype)) << 16;
}

// Up to 32 consecutive outputs of one row (pairs), in stores of 32 bytes (vec 2) or
// 16 (1); 8 columns at a time at the row's end.
__device__ __forceinline__ void put_row32(uint16_t *dst, const uint32_t (&w)[16], int left, int vec) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int more = left - 16 * i;
        const uint32_t *x = w + 8 * i;
        uint16_t *d = dst + 16 * i;
        if (vec == 2 && more >= 16) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(d), "r"(x[0]), "r"(x[1]),
                         "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                         : "memory");
        } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (more >= 8 * k + 8) {
                    reinterpret_cast<uint4 *>(d)[k] = make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (8 * k + j < more) d[8 * k + j] = static_cast<uint16_t>(x[4 * k + j / 2] >> (16 * (j & 1)));
                }
            }
        }
    }
}

// The same for rows that do not start on 16 bytes, by a whole warp (a lane a row):
// through shared memory, so that a store covers 4 rows of 32 bytes (two columns a
// lane, where rows start on 4 bytes) or 2 instead of 2 bytes in each of 32 rows
// (16-bit gated 1536 x 700 x 1024: 11.1 us against 19.0).
__device__ __forceinline__ void put_odd_rows32(uint16_t *dst, int64_t ld, const uint32_t (&w)[16], int left, int rows,
                                               uint32_t box, int lane, bool pairs) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int cols = left - 16 * h;
        if (cols <= 0) break;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t *x = w + 8 * h + 4 * i;
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + lane * kOutPitch + 16 * i), "r"(x[0]),
                         "r"(x[1]), "r"(x[2]), "r"(x[3])
                         : "memory");
        }
        __syncwarp();
        uint16_t *d = dst + 16 * h;
        if (pairs) {
            const int c = 2 * (lane & 7);
#pragma unroll
            for (int r = lane >> 3; r < 32; r += 4) {
                uint32_t two;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(two) : "r"(box + r * kOutPitch + 2 * c) : "memory");
                if (r >= rows || c >= cols) continue;
                if (c + 1 < cols)
                    *reinterpret_cast<uint32_t *>(d + r * ld + c) = two;
                else
                    d[r * ld + c] = static_cast<uint16_t>(two);
            }
        } else {
            const int c = lane & 15;
#pragma unroll 4
            for (int r = lane >> 4; r < 32; r += 2) {
                uint16_t one;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(one) : "r"(box + r * kOutPitch + 2 * c) : "memory");
                if (r < rows && c < cols) d[r * ld + c] = one;
            }
        }
    }
}

// The same into a row of a warp's box in shared memory: 16-byte pieces 4 k .. 4 k + 3,
// as far as the row goes; rows of 128 bytes are swizzled.
__device__ __forceinline__ void put_box32(uint32_t row, const uint32_t (&w)[16], int k, int lane, uint32_t pitch) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t piece = static_cast<uint32_t>(4 * k + i);
        if (piece * 16 >= pitch) break;
        const uint32_t at = row + (pitch == 128 ? (piece ^ (static_cast<uint32_t>(lane) & 7u)) : piece) * 16;
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[4 * i]), "r"(w[4 * i + 1]),
                     "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
    }
}

// 32 fp32 sums into a swizzled row of a warp's box.
__device__ __forceinline__ void put_box_sums32(uint32_t row, const float (&v)[32], int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(row + ((i ^ (lane & 7)) << 4)), "f"(v[4 * i]),
                     "f"(v[4 * i + 1]), "f"(v[4 * i + 2]), "f"(v[4 * i + 3])
                     : "memory");
}

// Outputs of a tile's columns that the first four epilogue warps take.
__host__ __device__ constexpr int first_half(int out_n) { return (out_n / 2 + 31) & ~31; }

// Up to 32 consecutive fp32 sums of one row.
__device__ __forceinline__ void put_sums32(float *dst, const float (&v)[32], int left, int vec) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (vec && 4 * i + 4 <= left) {
            reinterpret_cast<float4 *>(dst)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (4 * i + k < left) dst[4 * i + k] = v[4 * i + k];
        }
    }
}

template <int kForm>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    ffn_tile_kernel(const __grid_constant__ TileMaps tm, const TileParams p) {
    constexpr bool kMx4 = kForm == TILE_MX4 || kForm == TILE_MX4_GATED;
    constexpr bool kGated = kForm == TILE_GATED || kForm == TILE_MX4_GATED;
    constexpr bool kBwd = kForm == TILE_BACKWARD;
    constexpr uint32_t kStage = stage_bytes(kMx4);
    constexpr int kStages = stages(kMx4);
    constexpr int kAccs = kMx4 ? 1 : 2;
    constexpr int kCols = kMx4 ? 128 : 64;      // map columns per K block, K-major operands
    constexpr uint32_t kSfCol = 256, kSfStage = 24;   // 4-bit: scale columns (A 8, B 16 a stage)
    const int sb_tiles = kGated ? 2 : p.set[0].nt >> 7;   // 4 bits: row tiles of B's scales

    extern __shared__ uint8_t ft_smem_raw[];
    const uint32_t raw = smem_u32(ft_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = ft_smem_raw + (base - raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(gbase + kStages * kStage + out_bytes(kMx4));
    uint64_t *empty = full + kStages;
    uint64_t *accf = empty + kStages;
    uint64_t *acce = accf + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acce + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int cid = static_cast<int>(blockIdx.x) >> 1;
    const int nclu = static_cast<int>(gridDim.x) >> 1;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(full + s), 1);
            mbar_init(smem_u32(empty + s), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(accf + i), 1);
            mbar_init(smem_u32(acce + i), 16);   // eight epilogue warps of each CTA
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync_all();   // barriers of both CTAs exist
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    struct Item {
        int set;              // 1: a tile of a weight's gradient, z which
        int z, split, m0, n0, kb0, kb1;
        int half_n, out_n;    // rows of B per CTA, outputs along N
    };
    // The i-th item of this cluster; false when there is none.
    auto get = [&](int i, Item &it) {
        int j = cid + i * nclu;
        it.set = 0;
        if constexpr (kBwd) {
            // items of set 0 in rounds; `last` clusters have one more than the others,
            // which take up to w_first weight tiles each before the common rounds
            const int last = p.items % nclu;
            const int mine0 = p.items / nclu + (cid < last);
            if (i >= mine0) {
                i -= mine0;
                const int idle = nclu - last;
                const int early = last ? min(p.w_first * idle, p.w_items) : 0;
                const int own = cid >= last && early > cid - last ? (early - (cid - last) + idle - 1) / idle : 0;
                j = i < own ? cid - last + i * idle : early + cid + (i - own) * nclu;
                if (j >= p.w_items) return false;
                it.set = 1;
            }
        } else if (j >= p.items) {
            return false;
        }
        const TileSet &t = p.set[kBwd ? it.set : 0];
        const int tiles = t.tiles_m * t.tiles_n;
        const int part = j / tiles;      // set 0: of the contraction; set 1: which weight
        j -= part * tiles;
        it.z = it.set ? part : 0;
        it.split = it.set ? 0 : part;
        const int splits = it.set ? 1 : p.splits;
        // bands of kBand row tiles, column tiles within a band, rows innermost
        const int band = j / (kBand * t.tiles_n);
        const int r = j - band * kBand * t.tiles_n;
        const int h = min(kBand, t.tiles_m - band * kBand);
        it.half_n = t.nt / 2;
        it.out_n = kGated ? it.half_n : t.nt;
        it.m0 = (band * kBand + r % h) * kTile;
        it.n0 = r / h * it.out_n;
        it.kb0 = static_cast<int>(static_cast<long long>(t.KB) * it.split / splits);
        it.kb1 = static_cast<int>(static_cast<long long>(t.KB) * (it.split + 1) / splits);
        return true;
    };

    if (warp == 0) {
        {
            const bool mine = elect_one();
            pdl_wait();
            const uint32_t full0 = mapa_shared(smem_u32(full), 0);   // the leader's barriers
            int stage = 0;
            uint32_t phase = 1;   // a fresh barrier passes a wait for the phase before its first
            Item it;
            for (int i = 0; get(i, it); ++i) {
                const int m = it.m0 + rank * 128;
                const uint32_t tx =
                    2 * (kHalf + static_cast<uint32_t>(it.half_n) * 128 + (kMx4 ? 1024u * (1 + sb_tiles) : 0u));
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    mbar_wait_bounded(smem_u32(empty + stage), phase, abort_flag, p.err, DEV_TIMEOUT_EMPTY);
                    const uint32_t st = base + stage * kStage;
                    const uint32_t bar = full0 + 8 * stage;
                    if (rank == 0 && mine) mbar_expect_tx(smem_u32(full + stage), tx);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                    if (!mine) continue;
                    const int n = it.n0 + (kGated ? 0 : rank * it.half_n);
                    if constexpr (kBwd) {
                        const bool second = !it.set && kb >= p.KB1;
                        const int k = second ? kb - p.KB1 : kb;
                        if (it.set) {
                            const CUtensorMap *ma = it.z ? &tm.aw1 : &tm.aw0;
                            pair_load(st, ma, bar, m, k * 64);
                            pair_load(st + 8192, ma, bar, m + 64, k * 64);
                        } else {
                            pair_load(st, second ? &tm.a1 : &tm.a0, bar, k * 64, m);
                        }
                        const CUtensorMap *mb = it.set ? &tm.bw : second ? &tm.b1 : &tm.b0;
                        pair_load(st + kHalf, mb, bar, n, k * 64);
                        if (it.half_n > 64) pair_load(st + kHalf + 8192, mb, bar, n + 64, k * 64);
                    } else {
                        pair_load(st, &tm.a0, bar, kb * kCols, m);
                        pair_load(st + kHalf, kGated && rank ? &tm.b1 : &tm.b0, bar, kb * kCols, n);
                    }
                    if constexpr (kMx4) {
                        // the scales of this CTA's A rows and of all of B's rows
                        const uint32_t sc = st + 2 * kHalf;
                        pair_load(sc, &tm.sa, bar, 0, (m >> 7) * p.kt_n + 2 * kb);
                        const int nt = it.n0 >> 7;
                        for (int t = 0; t < sb_tiles; ++t)
                            pair_load(sc + 1024 * (1 + t), kGated && t ? &tm.sb1 : &tm.sb0, bar, 0,
                                      (kGated ? nt : nt + t) * p.kt_n + 2 * kb);
                    }
                }
            }
            // Every copy of this CTA has landed, and every MMA that reads its
            // shared memory has completed, before it leaves: each stage's last
            // round was returned (a stage without a round passes at once). After a
            // wait that ran out MMAs are issued, and their stages returned, without
            // their copies: the leader, which the other CTA does not leave before,
            // waits for those of both as well (the same parity: that of the last round).
            for (int t = 0; t < kStages; ++t) {
                ffn_drain_wait(smem_u32(empty + stage), phase);
                if (rank == 0) ffn_drain_wait(smem_u32(full + stage), phase);
                if (++stage == kStages) stage = 0, phase ^= 1;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const bool mine = elect_one();
            // The tensor cores keep next to no MMAs queued, so what this thread
            // does between two stages is time lost. Stage and phase are counted
            // on, and the next stage is waited for before the last MMA of this one
            // is issued; in 4 bits before the first, since its scales' way to TMEM
            // then passes under all four (4096 x 4096 x 7168: after 3, 2, 1 and 0 MMAs
            // 51.0, 48.1, 45.9 and 44.8 us; 16-bit gated 126.6, 126.5, 126.4, 127.8).
            // Two stages ahead cost more than it gave.
            constexpr int kBefore = kMx4 ? 0 : 3;
            int stage = 0, as = 0;
            uint32_t phase = 0, aphase = 1;
            auto prepare = [&](int s, uint32_t ph) {
                mbar_wait_bounded(smem_u32(full + s), ph, abort_flag, p.err, DEV_TIMEOUT_FULL);
                tc_fence_after();
                if constexpr (kMx4) {
                    // columns of a stage, four a tile: A's tiles 0 and 1 of the block, then
                    // for either B's row tiles
                    const uint32_t sf = tmem + kSfCol + static_cast<uint32_t>(s) * kSfStage;
                    const uint64_t sc = desc_scales(base + s * kStage + 2 * kHalf);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (!mine) break;
                        pair_cp_scales(sf + 4 * j, sc + 32 * j);
                        pair_cp_scales(sf + 8 + 8 * j, sc + 64 + 32 * j);
                        if (sb_tiles > 1) pair_cp_scales(sf + 12 + 8 * j, sc + 128 + 32 * j);
                    }
                }
            };
            Item it, next;
            bool more_items = get(0, it);
            if (more_items) prepare(0, 0);
            for (int i = 0; more_items; ++i, it = next) {
                more_items = get(i + 1, next);
                const bool a_mn = kBwd && it.set;
                const uint32_t idesc = p.set[kBwd ? it.set : 0].idesc;
                mbar_wait_bounded(smem_u32(acce + as), aphase, abort_flag, p.err, DEV_TIMEOUT_ACC_EMPTY);
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(as) * 256;
                for (int kb = it.kb0; kb < it.kb1; ++kb) {
                    const uint32_t st = base + stage * kStage;
                    const uint64_t ad = a_mn ? desc_mn(st) : desc_kmajor(st);
                    const uint64_t bd = kBwd ? desc_mn(st + kHalf) : desc_kmajor(st + kHalf);
                    const uint32_t sf = tmem + kSfCol + static_cast<uint32_t>(stage) * kSfStage;
                    const uint32_t bar = smem_u32(empty + stage);
                    // 64 4-bit columns a step, and steps past K are left out (their
                    // scales belong to other rows); 16 16-bit ones, 32 bytes of a row
                    // or 16 rows of 128 bytes on
                    const int steps = kMx4 ? min(4, (p.K - kb * 256 + 63) >> 6) : 4;
                    auto mma = [&](int kk) {
                        if (!mine) return;
                        const uint32_t more = kb > it.kb0 || kk > 0;
                        if constexpr (kMx4)
                            pair_mma_mxf4(d, ad + 2 * kk, bd + 2 * kk, idesc_sf(idesc, (kk & 1) * 2),
                                          sf + 4 * (kk >> 1), sf + 8 + 8 * (kk >> 1), more);
                        else
                            pair_mma_f16(d, ad + kk * (a_mn ? 128 : 2), bd + kk * (kBwd ? 128 : 2), idesc, more);
                    };
#pragma unroll
                    for (int kk = 0; kk < kBefore; ++kk) mma(kk);
                    if (++stage == kStages) stage = 0, phase ^= 1;
                    if (kb + 1 < it.kb1 || more_items) prepare(stage, phase);
#pragma unroll
                    for (int kk = kBefore; kk < 4; ++kk)
                        if (kk < steps) mma(kk);
                    if (mine) pair_commit(bar);
                }
                if (mine) pair_commit(smem_u32(accf + as));
                if (++as == kAccs) as = 0, aphase ^= 1;
            }
        }
        __syncwarp();
    } else {
        // Two warps for each quarter of the accumulator's rows, each with half of
        // the tile's outputs. A warp reads all of its sums into registers and gives
        // the accumulator back before it computes or stores anything.
        const int q = warp & 3;
        const int half = warp >= 6;
        const uint32_t box = base + kStages * kStage + static_cast<uint32_t>(warp - 2) * out_box(kMx4);
        auto take_box = [&]() {   // the last copy has read it
            if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            __syncwarp();
        };
        auto send_box = [&](const CUtensorMap *map, int n, int m) {   // rows and columns past the output's are left out
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0)
                asm volatile(
                    "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];\n\t"
                    "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
                    "r"(n), "r"(m), "r"(box)
                    : "memory");
        };
        const float scale = kBwd && p.scale ? __ldg(p.scale) : 1.f;   // a power of two
        int as = 0;
        uint32_t aphase = 0;
        Item it;
        for (int i = 0; get(i, it); ++i) {
            const int span = first_half(it.out_n);
            const uint32_t pitch = kGated ? 2u * static_cast<uint32_t>(half ? it.out_n - span : span) : 128u;   // of the box's rows
            const int M = p.set[kBwd ? it.set : 0].M, N = p.set[kBwd ? it.set : 0].N;
            mbar_wait_bounded(smem_u32(accf + as), aphase, abort_flag, p.err, DEV_TIMEOUT_ACC_FULL);
            tc_fence_after();
            const uint32_t t = tmem + static_cast<uint32_t>(as) * 256 + (static_cast<uint32_t>(q * 32) << 16) + half * span;
            uint32_t v[4][32];   // gated: 0 and 1 the gates, 2 and 3 their factors
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(t + (kGated && c >= 2 ? it.half_n - 64 : 0) + 32 * c, v[c]);
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive(mapa_shared(smem_u32(acce + as), 0));
            if (++as == kAccs) as = 0, aphase ^= 1;
            const int m_first = it.m0 + rank * 128 + q * 32;
            if (m_first >= M) continue;
            const int64_t m = m_first + lane;
#pragma unroll
            for (int pair = 0; pair < (kGated ? 1 : 2); ++pair) {   // 64 columns at a time
                const int at = half * span + 64 * pair;              // within the tile
                const int n = it.n0 + at;
                const int left = min(N - n, (half ? it.out_n : span) - at);
                if (left <= 0) break;
                const bool copy_out = kBwd ? it.set || p.splits == 1 : !kMx4 && p.copy_out;
                if (kForm == TILE_GATED && p.g) {
                    // g and u through the box as well, 32 columns at a time (2046 x 3216 x 328:
                    // 25.7 us, with stores of 16 bytes from each lane 32.8; three boxes a
                    // warp for two stages less 23.5, but 4096 x 2048 x 7168 131.7 -> 158)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {   // two pieces of g, two of u
                        const int c = 32 * (k & 1);
                        if (c >= left) continue;
                        float a[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] = __uint_as_float(v[k][j]);
                        if (copy_out && (half ? it.out_n : span) - at >= c + 32) {
                            take_box();
                            put_box_sums32(box + lane * 128, a, lane);
                            send_box(k < 2 ? &tm.g : &tm.u, n + c, m_first);
                        } else if (m < M) {
                            put_sums32((k < 2 ? p.g : p.u) + m * N + n + c, a, left - c, p.vec_gu);
                        }
                    }
                }
                if (copy_out) take_box();
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if (32 * k >= left) break;
                    const int c = 2 * pair + k;
                    float a[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) a[j] = __uint_as_float(v[c][j]);
                    if constexpr (kBwd)
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] *= scale;
                    if constexpr (kGated) {
                        float b[32], h[32];
#pragma unroll
                        for (int j = 0; j < 32; ++j) b[j] = __uint_as_float(v[2 + k][j]);
                        ffn_gate(a, b, p.act, h);
#pragma unroll
                        for (int j = 0; j < 32; ++j) a[j] = h[j];
                    }
                    if (kBwd && !copy_out) {
                        if (m < M)
                            put_sums32(p.ws + (static_cast<int64_t>(it.split) * M + m) * N + n + 32 * k, a,
                                       left - 32 * k, 1);
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) w[j] = pack2(a[2 * j], a[2 * j + 1], p.dtype);
                        uint16_t *y = p.y[0] + n + 32 * k;
                        if (kBwd || copy_out) {
                            put_box32(box + lane * pitch, w, k, lane, pitch);
                        } else if (p.vec) {
                            if (m < M) put_row32(y + m * p.ldy, w, left - 32 * k, p.vec);
                        } else {
                            put_odd_rows32(y + m_first * p.ldy, p.ldy, w, left - 32 * k, M - m_first, box, lane, p.pairs);
                        }
                    }
                }
                if (copy_out) send_box(&tm.y[kGated ? half : it.set ? 1 + it.z : 0], n, m_first);
            }
        }
        if (!kMx4 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync_all();   // the peer is done with this CTA's barriers and memory
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Partial sums [S][M][N] added in order and rounded.
__global__ void __launch_bounds__(256) join_kernel(const float *ws, int64_t n, int splits, uint16_t *y, int dtype) {
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
         i += static_cast<int64_t>(gridDim.x) * 1024) {
        float4 s = *reinterpret_cast<const float4 *>(ws + i);
        for (int k = 1; k < splits; ++k) {
            const float4 v = *reinterpret_cast<const float4 *>(ws + k * n + i);
            s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        *reinterpret_cast<uint2 *>(y + i) = make_uint2(pack2(s.x, s.y, dtype), pack2(s.z, s.w, dtype));
    }
}

int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

// Accumulator columns of a forward tile: those whose rounds of tiles over the SM
// pairs cost least, a tile costing its columns' K blocks and about six K blocks of
// fixed work. 4-bit tiles start at whole scale tiles of 128 rows (a gated one holds
// one of each weight): the MMA reads B's scales from a multiple of four TMEM columns.
// Gated 4003 x 2048 x 7168 (256 tiles of 256 columns on 76 SM pairs, or 304 of 224):
// 141 us with 256 columns, 130 with 224.
int tile_columns(int form, int64_t M, int64_t N, int KB, int sms) {
    const bool gated = form == TILE_GATED || form == TILE_MX4_GATED;
    const int step = form == TILE_GATED ? 32 : form == TILE_MX4_GATED ? 256 : 128;
    int best = 256;
    int64_t least = -1;
    for (int nt = 256; nt >= (step > 64 ? step : 64); nt -= step) {
        const int64_t tiles = static_cast<int64_t>(cdiv(M, kTile)) * cdiv(N, gated ? nt / 2 : nt);
        const int64_t cost = (tiles + sms / 2 - 1) / (sms / 2) * (static_cast<int64_t>(nt) * KB + 256 * 6);
        if (least < 0 || cost < least) least = cost, best = nt;
    }
    return best;
}

// The backward list: columns of dx's and of the weight gradients' tiles (256, or 128
// for more and shorter items; B with N contiguous comes in boxes of 64), parts that
// dx's contraction is split into, and the weight tiles that take as long as the last
// item of dx. Chosen by the longest cluster's work, in K blocks of a 256-column tile:
// a 128-column one takes 0.65 (its loads bind), an item's start and end four, the
// kernel that joins a split dx twelve.
struct BackwardPlan {
    int nt[2], tiles_m[2], tiles_n[2], KB[2];
    int splits, w_first;
    int64_t items, w_items;
};

BackwardPlan backward_plan(int T, int F, int K, int sms) {
    const int P = sms / 2;
    BackwardPlan best = {};
    float least = -1.f;
    for (int pick = 0; pick < 4; ++pick) {
        BackwardPlan q = {};
        q.nt[0] = pick & 1 ? 128 : 256;
        q.nt[1] = pick & 2 ? 128 : 256;
        q.KB[0] = 2 * cdiv(F, 64);
        q.KB[1] = cdiv(T, 64);
        q.tiles_m[0] = cdiv(T, kTile);
        q.tiles_m[1] = cdiv(F, kTile);
        for (int i = 0; i < 2; ++i) q.tiles_n[i] = cdiv(K, q.nt[i]);
        const int64_t tiles = static_cast<int64_t>(q.tiles_m[0]) * q.tiles_n[0];
        q.w_items = 2ll * q.tiles_m[1] * q.tiles_n[1];
        const float w = q.KB[1] * (q.nt[1] == 128 ? 0.65f : 1.f) + 4.f;
        for (q.splits = 1; q.splits <= 8; ++q.splits) {
            if (q.splits > 1 && (q.KB[0] / q.splits < 8 || tiles * q.splits > P)) break;
            q.items = tiles * q.splits;
            const float x = (q.KB[0] + q.splits - 1) / q.splits * (q.nt[0] == 128 ? 0.65f : 1.f) + 4.f;
            const int64_t rounds = q.items / P, last = q.items % P;
            q.w_first = last ? static_cast<int>(x / w + 0.5f) : 0;
            const int64_t early = last ? std::min<int64_t>(q.w_first * (P - last), q.w_items) : 0;
            const int64_t early_rounds = early ? (early + P - last - 1) / (P - last) : 0;
            const float cost = rounds * x + std::max(last ? x : 0.f, early_rounds * w) +
                               static_cast<float>((q.w_items - early + P - 1) / P) * w + (q.splits > 1 ? 12.f : 0.f);
            if (least < 0 || cost < least) least = cost, best = q;
        }
    }
    return best;
}

std::mutex g_mu;
bool g_ready[64];   // devices whose kernels have their shared memory raised

}  // namespace

// By estimates of both kernels' times, from rounds of 256-column tiles and K blocks
// for this one (in 16 bits a tenth more, which the choice was best with). Over 300
// sizes in 16 bits and 240 in 4, plain and gated, the choice is 0.9, 0.6 and 0.5 %
// slower than the better of the two on average; each is up to 2.5 times as fast as
// the other (4 bits, K = 7168: 64 x 256 6.6 us streamed, 16 in tiles; 1024 x 4096 30
// against 17).
bool ffn_use_tile(bool mx4, bool gated, int M, int N, int K, int sms) {
    const int64_t tiles = static_cast<int64_t>(cdiv(M, kTile)) * cdiv(N, gated ? 128 : 256);
    const float waves = static_cast<float>((tiles + sms / 2 - 1) / (sms / 2));
    const float kb = static_cast<float>(cdiv(K, mx4 ? 256 : 64));
    const float us = !mx4    ? 1.1f * (3.7f + waves * (2.7f + 0.21f * kb))
                     : gated ? 5.3f + waves * (2.1f + 0.34f * kb)
                             : 2.4f + waves * (3.7f + 0.34f * kb);
    // (the other kernel has its token tiles of 128 on the grid's y axis)
    return M > 65535 * 128 || us < ffn_stream_us(mx4, gated, M, N, K, sms);
}

size_t ffn_backward_scratch(int T, int F, int K, int sms) {
    const int s = backward_plan(T, F, K, sms).splits;
    return s > 1 ? static_cast<size_t>(s) * T * K * sizeof(float) : 0;
}

cudaError_t ffn_tile_launch(const FfnTileArgs &a, const FfnDev &d, cudaStream_t s) {
    const bool mx4 = a.form == TILE_MX4 || a.form == TILE_MX4_GATED;
    const bool gated = a.form == TILE_GATED || a.form == TILE_MX4_GATED;
    const bool backward = a.form == TILE_BACKWARD;
    using Fn = void (*)(TileMaps, TileParams);
    static const Fn kernels[] = {ffn_tile_kernel<TILE_GATED>, ffn_tile_kernel<TILE_MX4_GATED>,
                                 ffn_tile_kernel<TILE_MX4>, ffn_tile_kernel<TILE_BACKWARD>};
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
    TileParams p = {};
    p.y[0] = static_cast<uint16_t *>(a.y0);
    p.y[1] = static_cast<uint16_t *>(a.y1);
    p.y[2] = static_cast<uint16_t *>(a.y2);
    p.g = a.g;
    p.u = a.u;
    p.ldy = a.ldy;
    p.ws = a.ws;
    p.scale = a.scale;
    p.err = a.err;
    p.K = a.K;
    p.splits = 1;
    int64_t items = 0, w_items = 0;
    if (backward) {
        const BackwardPlan q = backward_plan(a.M, a.N, a.K, d.sms);
        for (int i = 0; i < 2; ++i)
            p.set[i] = {i ? a.N : a.M, a.K, q.tiles_m[i], q.tiles_n[i], q.nt[i], q.KB[i],
                        idesc_f16(a.dtype, 256, q.nt[i], i == 1, true)};
        items = q.items;
        w_items = q.w_items;
        p.splits = q.splits;
        p.w_first = q.w_first;
        p.KB1 = q.KB[0] / 2;
    } else {
        TileSet &t = p.set[0];
        t.M = a.M;
        t.N = a.N;
        t.KB = mx4 ? cdiv(a.K, 256) : cdiv(a.K, 64);
        t.nt = tile_columns(a.form, a.M, a.N, t.KB, d.sms);
        t.tiles_m = cdiv(a.M, kTile);
        t.tiles_n = cdiv(a.N, gated ? t.nt / 2 : t.nt);
        t.idesc = mx4 ? idesc_mxf4(256, t.nt) : idesc_f16(a.dtype, 256, t.nt);
        items = static_cast<int64_t>(t.tiles_m) * t.tiles_n;
    }
    if (items + w_items > (1 << 30) || (p.splits > 1 && !a.ws)) return cudaErrorInvalidValue;
    p.items = static_cast<int>(items);
    p.w_items = static_cast<int>(w_items);
    p.kt_n = static_cast<int>(mx4_ktiles(a.K));
    p.act = a.act;
    p.dtype = a.dtype;
    // the widest store that every row's 32-column pieces allow: of y, and of g and u
    // (stride N, 16-byte aligned)
    const uintptr_t starts = reinterpret_cast<uintptr_t>(a.y0) | static_cast<uintptr_t>(a.ldy * 2);
    p.vec = starts % 32 == 0 ? 2 : starts % 16 == 0 ? 1 : 0;
    p.pairs = starts % 4 == 0;
    p.vec_gu = a.N % 4 == 0;

    TileMaps tm = {};
    auto map = [&](CUtensorMap *m, const void *ptr, int64_t rows, int64_t cols, int64_t ld, int box_rows, int box_cols,
                   int type, bool swizzle = true) {
        if (e == cudaSuccess) e = ffn_tensor_map(m, ptr, rows, cols, ld, box_rows, box_cols, type, swizzle);
    };
    if (mx4) {
        const int64_t pitch = mx4_pitch(a.K);
        map(&tm.a0, a.qa.codes, a.M, pitch, pitch, 128, 128, kMapU8);
        map(&tm.b0, a.qb0.codes, a.N, pitch, pitch, p.set[0].nt / 2, 128, kMapU8);
        if (gated) map(&tm.b1, a.qb1.codes, a.N, pitch, pitch, p.set[0].nt / 2, 128, kMapU8);
        auto scales = [&](CUtensorMap *m, const Mx4Mat &q, int rows) {
            if (e == cudaSuccess)
                e = ffn_scale_map(m, q.scales, static_cast<int64_t>(cdiv(rows, 128)) * p.kt_n);
        };
        scales(&tm.sa, a.qa, a.M);
        scales(&tm.sb0, a.qb0, a.N);
        if (gated) scales(&tm.sb1, a.qb1, a.N);
    } else if (a.form == TILE_GATED) {
        map(&tm.a0, a.A0, a.M, a.K, a.lda, 128, 64, a.dtype);
        map(&tm.b0, a.B0, a.N, a.K, a.ldb0, p.set[0].nt / 2, 64, a.dtype);
        map(&tm.b1, a.B1, a.N, a.K, a.ldb1, p.set[0].nt / 2, 64, a.dtype);
    } else {
        map(&tm.a0, a.A0, a.M, a.N, a.lda, 128, 64, a.dtype);
        map(&tm.a1, a.A1, a.M, a.N, a.lda, 128, 64, a.dtype);
        map(&tm.b0, a.B0, a.N, a.K, a.ldb0, 64, 64, a.dtype);
        map(&tm.b1, a.B1, a.N, a.K, a.ldb1, 64, 64, a.dtype);
        map(&tm.aw0, a.A0, a.M, a.N, a.lda, 64, 64, a.dtype);
        map(&tm.aw1, a.A1, a.M, a.N, a.lda, 64, 64, a.dtype);
        map(&tm.bw, a.X, a.M, a.K, a.ldx, 64, 64, a.dtype);
        if (p.splits == 1) map(&tm.y[0], a.y0, a.M, a.K, a.ldy, 32, 64, a.dtype);
        map(&tm.y[1], a.y1, a.N, a.K, a.ldy, 32, 64, a.dtype);
        map(&tm.y[2], a.y2, a.N, a.K, a.ldy, 32, 64, a.dtype);
    }
    // whole 16-byte pieces only: a copy's last piece reaches past a row end within one
    p.copy_out = a.form == TILE_GATED && p.vec != 0 && a.N % 8 == 0;
    if (p.copy_out) {
        const int out_n = p.set[0].nt / 2;
        const int first = first_half(out_n);
        map(&tm.y[0], a.y0, a.M, a.N, a.ldy, 32, first, a.dtype, first == 64);
        if (out_n > first) map(&tm.y[1], a.y0, a.M, a.N, a.ldy, 32, out_n - first, a.dtype, out_n - first == 64);
        if (a.g) {
            map(&tm.g, a.g, a.M, a.N, a.N, 32, 32, kMapF32);
            map(&tm.u, a.u, a.M, a.N, a.N, 32, 32, kMapF32);
        }
    }
    if (e != cudaSuccess) return e;

    size_t smem = 0;
    if ((e = ffn_smem_for_tmem(d.dev, 512, stages(mx4) * stage_bytes(mx4) + out_bytes(mx4) + 1024 + kBarBytes, &smem)) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * static_cast<unsigned>(std::min(p.items + p.w_items, d.sms / 2)), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pdl ? 1 : 0;
    if ((e = cudaLaunchKernelEx(&cfg, kernels[a.form], tm, p)) != cudaSuccess) return e;
    if (p.splits > 1) {
        const int64_t n = static_cast<int64_t>(a.M) * a.K;
        const int blocks = static_cast<int>(std::min<int64_t>((n / 4 + 255) / 256, static_cast<int64_t>(d.sms) * 8));
        join_kernel<<<blocks, 256, 0, s>>>(a.ws, n, p.splits, p.y[0], a.dtype);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace kp
