// Products grouped by expert: out[n, m] = sum_k A[m, k] B[n, k] with fp32 accumulation,
// where n runs over an expert's rows (the weights' gradients: over features) and m along
// a row of the output.
//
// The features lie on the MMA's 256 rows and the tokens on its columns, so that a
// tile is as wide as its expert has rows, in steps of 32: ragged sizes cost little, and
// with a row or two an expert the kernel streams weights. Two CTAs of a cluster (an SM
// pair) compute one 256 x nt tile (nt up to 256) with tcgen05.mma.cta_group::2: each
// holds 128 rows of A, half of B's nt rows and the accumulator of its own A. The
// leader's warp 1 issues every MMA; both CTAs' copies complete on the leader's barriers,
// and tcgen05.commit returns stages and accumulators to both. Clusters are persistent: a
// cluster takes items c, c + n, ... of a list that every CTA reads off the experts'
// offsets in device memory; the host knows only how many rows there may be.
//
//   PLAIN   A = W_e (K contiguous), B = rows of x.
//   GATED   A = 64 rows of Wg_e and the same ones of Wu_e per CTA: gates are in
//           accumulator lanes 0 .. 63 and their factors in lanes 64 .. 127, and the warps
//           that read them swap halves through shared memory.
//   BACKWARD  one list of the tiles of dx and of the weights' gradients.
//           dx: A = W_e read along its rows (the MMA's transposed operand), B = rows of
//           the output's gradient; two products into one accumulator for the gated block.
//           dW: A = x, B = the output's gradient, both transposed, contracted over the
//           expert's rows. The block of 64 that an expert's rows end in also brings rows
//           of others: MMA steps of 16 past the end are left out, and in the step that
//           the end is in, warp 10 of both CTAs clears the others' rows first.
//
// An accumulator's lanes are columns of the output: it is read in 8 x 8 fragments, which
// stmatrix lays down transposed in a warp's box, and leaves in pieces of 64 bytes of eight
// rows a store (with two columns of two rows a store, swapped between lanes, a 256 x 256
// tile took 13000 cycles on its way out, as long as 25 K blocks).
//
// Bound: HBM with few rows an expert (gated, one row on each of 8 experts, 2048 x 7168: 75 us,
// 6.2 TB/s), the tensor cores with many (gated, 16384 rows on 32 experts, 2048 x 7168: 612 us, 1.57
// PFLOP/s, tensor pipe active 82 %; dx and dW of 1024 rows on each of 16, 2048 x 4096: 316 us, 1.74).
// Rows that do not start on 128 bytes lie in two lines each and take 1.2 to 1.6 times as long.
//
// Warp 0: copies; warp 1: TMEM, MMA (leader); warps 2 .. 9: epilogue; warp 10: BACKWARD.
#include <algorithm>
#include <mutex>

#include "kp_moe.cuh"

namespace kp {

namespace {

constexpr int kThreads = 320, kThreadsBack = 352;
constexpr int kTile = 256;                // rows of A per cluster; of B at most
constexpr uint32_t kHalf = 128 * 128;     // bytes of 128 rows of a K block (128 bytes of K)
constexpr size_t kMaxSmem = 227 * 1024;
constexpr int kMaxStages = 12;
constexpr uint32_t kBox = 2048;           // of a warp on an accumulator's way out
constexpr size_t kBarBytes = (3 * kMaxStages + 4) * 8 + 16;

struct GroupedMaps {
    CUtensorMap a0, a1, b0, b1;   // W (gated: Wg, Wu; dx: of either product), rows of x or of the gradients
    CUtensorMap ax, bw0, bw1;     // dW: x, the gradients
};

struct GroupedParams {
    const int32_t *offsets;
    uint16_t *y[3];       // y, h or dx; dW0, dW1
    float *g, *u;
    int64_t ldy;
    const float *scale;
    int *err;
    int R, E, N;
    int M;                // columns of the outputs
    int tiles_m;          // tiles along them
    int cap;              // rows of B in a tile that a stage has room for (dW: not)
    int box;              // rows of a copy of B (dW: 64)
    int KB, K;            // K blocks and columns of the contraction (dx: of one product; dW: not)
    int products;         // dx: into one accumulator; dW: outputs
    int tiles_n, nt, KBw; // dW: tiles along the features, their width, about how many K blocks
    int stages;
    uint32_t stage_bytes, idesc;
    int act, dtype;
    int vec[2];           // the output's (dW's) rows start on 16 (2) or 4 (1) bytes
};

__device__ __forceinline__ void pair_load2(uint32_t dst, const void *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
__device__ __forceinline__ void pair_load3(uint32_t dst, const void *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// On a barrier of this CTA.
__device__ __forceinline__ void own_load2(uint32_t dst, const void *map, uint32_t bar, int c0, int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
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
__device__ __forceinline__ void pair_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}
// Behind writes to this CTA's shared memory that a thread of either CTA hands to its MMAs,
// on that thread's barrier (shared::cluster address). Cluster scope on both sides, since
// they may be two CTAs: one that ends at the CTA orders nothing between them. (890 cycles
// instead of 40, while the stages before it are still in the MMAs' queue.)
__device__ __forceinline__ void remote_arrive_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// The other side: once the phase has been waited for.
__device__ __forceinline__ void acquire_cluster(uint32_t bar, uint32_t parity) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%0], %1;\n\t}" ::"r"(bar),
        "r"(parity)
        : "memory");
}
// An arrival that no write has to be seen behind. (A releasing arrival waits for the
// stores before it: an epilogue that gives its accumulator back after a tile's stores, or a
// copying warp at every stage, then lags behind by their latency.)
__device__ __forceinline__ void remote_arrive_relaxed(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Operand stored with M / N contiguous, 128-byte swizzle: 64-element groups 8 KB apart
// (64 K rows of 128 bytes), 8 K rows 1 KB apart.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

// 16 accumulator lanes x 32 columns. A thread gets, of every eight columns c, lanes t / 4
// (0, 1) and t / 4 + 8 (2, 3) at columns 2 (t % 4) and the one behind it: the fragments
// that stmatrix takes.
__device__ __forceinline__ void tmem_ld16x32(uint32_t taddr, uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}
// Four 8 x 8 fragments, transposed: thread t's address is row t % 8 of fragment t / 8.
__device__ __forceinline__ void store_fragments(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}
__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
    if (dtype == KP_FP16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// A warp's box in shared memory: rows of 32 elements (64 bytes), whose 16-byte pieces are
// permuted so that neither fragments nor rows meet in a bank.
__device__ __forceinline__ uint32_t box_at(uint32_t box, int n, int piece) {
    return box + n * 64 + ((piece ^ ((n >> 1) & 3)) << 4);
}
// Its first `rows` rows to rows of the output from dst on, columns m .. m + 31 below M;
// vec 2: rows of 16-byte pieces, 1: of 4-byte ones, 0: of single elements.
template <int N>
__device__ __forceinline__ void put_box(uint16_t *dst, int64_t ld, uint32_t box, int m, int M, int rows, int lane,
                                        int vec) {
    __syncwarp();
    if (vec == 2) {
        const int c = m + 8 * (lane & 3);
        uint16_t *d = dst + (lane >> 2) * ld + c;
#pragma unroll
        for (int i = 0; i < N / 8; ++i) {
            const int n = (lane >> 2) + 8 * i;
            uint32_t w[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "r"(box_at(box, n, lane & 3))
                         : "memory");
            if (n < rows) {
                if (c + 8 <= M) {
                    *reinterpret_cast<uint4 *>(d) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (c + k < M) d[k] = static_cast<uint16_t>(w[k >> 1] >> (16 * (k & 1)));
                }
            }
            d += 8 * ld;
        }
    } else if (vec == 1) {
        const int c = m + 2 * (lane & 15);
        uint16_t *d = dst + (lane >> 4) * ld + c;
#pragma unroll 4
        for (int n = lane >> 4; n < N; n += 2, d += 2 * ld) {
            uint32_t w;
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(w)
                         : "r"(box_at(box, n, (lane & 15) >> 2) + 4 * (lane & 3))
                         : "memory");
            if (n >= rows) break;
            if (c + 2 <= M)
                *reinterpret_cast<uint32_t *>(d) = w;
            else if (c < M)
                *d = static_cast<uint16_t>(w);
        }
    } else {
        uint16_t *d = dst + m + lane;
#pragma unroll 4
        for (int n = 0; n < N; ++n, d += ld) {
            uint16_t w;
            asm volatile("ld.shared.u16 %0, [%1];"
                         : "=h"(w)
                         : "r"(box_at(box, n, lane >> 3) + 2 * (lane & 7))
                         : "memory");
            if (n >= rows) break;
            if (m + lane < M) *d = w;
        }
    }
    __syncwarp();   // the box is free
}

// Widths that tiles of rows are cut to.
constexpr int kCaps = 7;
__host__ __device__ constexpr int cap_of(int i) { return kTile - 32 * i; }
// SM cycles of a tile: its K blocks, each bound by its MMAs or by the copies of its operands
// (about 70 bytes a cycle reach an SM), the accumulator's way out where that is longer, and
// what neither hides.
__host__ __device__ __forceinline__ float tile_cycles(float nt, float kb) {
    const float block = fmaxf(2.f * nt, (16384.f + 64.f * nt) / 70.f);
    return fmaxf(kb * block, 800.f + 18.f * nt) + 1500.f;
}

// Limit of a wait that `blocks` K blocks of the CTA's own products may lie behind: 1 s, and
// 4 us a block, which takes 0.2 to 0.6 of one. (An expert's 2^29 rows contracted by one
// cluster are 2^23 blocks, 2.2 s.)
__device__ __forceinline__ uint64_t wait_limit_ns(uint64_t blocks) { return 1000000000ull + 4000ull * blocks; }

template <int kForm>
__global__ void __launch_bounds__(kForm == GROUPED_BACKWARD ? kThreadsBack : kThreads, 1) __cluster_dims__(2, 1, 1)
    grouped_kernel(const __grid_constant__ GroupedMaps tm, const GroupedParams p) {
    constexpr bool kGated = kForm == GROUPED_GATED;
    constexpr bool kBack = kForm == GROUPED_BACKWARD;

    extern __shared__ uint8_t gt_smem_raw[];
    const uint32_t raw = smem_u32(gt_smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t *gbase = gt_smem_raw + (base - raw);
    const int S = p.stages;
    const uint32_t boxes0 = base + S * p.stage_bytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(gbase + S * p.stage_bytes + 8 * kBox);
    uint64_t *empty = full + kMaxStages;
    uint64_t *ends = empty + kMaxStages;      // dW: copies of a block that an expert's rows end in
    uint64_t *accf = ends + kMaxStages;
    uint64_t *acce = accf + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acce + 2);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int32_t *first = reinterpret_cast<int32_t *>(tmem_slot + 4);   // [E] of each expert's rows,
    int32_t *count = first + p.E;                                  // [E] how many,
    int32_t *tiles = count + p.E;                                  // [E + 1] tiles of the experts before

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int cid = static_cast<int>(blockIdx.x) >> 1;
    const int nclu = static_cast<int>(gridDim.x) >> 1;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(smem_u32(full + s), kBack ? 2 : 1);
            mbar_init(smem_u32(empty + s), 1);
            mbar_init(smem_u32(ends + s), 1);
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
    if (warp == 2) {   // the experts' rows, and the sums of their tiles
        // Whatever the offsets hold, the rows lie within [0, R) and no two experts
        // have the same: an expert's begin at the largest number up to its own. The loads go
        // first: in the scan they were waited for one by one (1024 experts: 2 us more).
#pragma unroll 8
        for (int e = lane; e <= p.E; e += 32) tiles[e] = min(max(__ldg(p.offsets + e), 0), p.R);
        __syncwarp();
        int most = 0, all = 0;
        int n[kCaps] = {};
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int f = max(e <= p.E ? tiles[e] : 0, most);
            int next = e < p.E ? tiles[e + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) f = max(f, __shfl_up_sync(0xFFFFFFFFu, f, d));
            next = max(next, f);
            most = __shfl_sync(0xFFFFFFFFu, next, 31);
            const int c = e < p.E ? next - f : 0;
            all += c;
#pragma unroll
            for (int i = 0; i < kCaps; ++i) n[i] += (c + cap_of(i) - 1) / cap_of(i);
            if (e < p.E) {
                first[e] = f;
                count[e] = c;
            }
        }
        // The width that tiles of rows are cut to: the one whose rounds of tiles over the
        // clusters take least. (Gated, 1021 rows on 12 experts, 331 features: 18 us with 256
        // columns, 11 with 64; 4003 rows on 8 experts, 1000 x 1416: 16.2 with 256, 19.7 with 128.)
        int cap = p.cap;
        if (cap > cap_of(kCaps - 1)) {   // a lane a width
            const float rows = static_cast<float>(__reduce_add_sync(0xFFFFFFFFu, all)) * p.tiles_m;
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < kCaps; ++i) {
                const int v = __reduce_add_sync(0xFFFFFFFFu, n[i]);
                if (lane == i) t = static_cast<float>(v) * p.tiles_m;
            }
            const float one = tile_cycles(__fdividef(rows, fmaxf(t, 1.f)), static_cast<float>(p.KB * (kBack ? p.products : 1)));
            float cost = ceilf(__fdividef(t, nclu)) * one;
            if constexpr (kBack) {
                const float w = static_cast<float>(p.E * p.products) * (p.tiles_m * p.tiles_n);
                const float one_w = tile_cycles(p.nt, static_cast<float>(p.KBw));
                cost = fmaxf(one, __fdividef(t * one + w * one_w, nclu) + (t + w > nclu ? 0.5f * one_w : 0.f));
            }
            // (positive floats order like their bits; the wider one where they are about equal)
            cost = lane < kCaps && kTile - 32 * lane <= p.cap ? cost * (1.f + 0.004f * lane) : 3e38f;
            const uint32_t least = __reduce_min_sync(0xFFFFFFFFu, __float_as_uint(cost));
            cap = kTile - 32 * (__ffs(__ballot_sync(0xFFFFFFFFu, __float_as_uint(cost) == least)) - 1);
        }
        __syncwarp();   // `tiles` held the offsets
        int run = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int t = e < p.E ? (count[e] + cap - 1) / cap : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int o = __shfl_up_sync(0xFFFFFFFFu, t, d);
                if (lane >= d) t += o;
            }
            if (e < p.E) tiles[e + 1] = run + t;
            run += __shfl_sync(0xFFFFFFFFu, t, 31);
        }
        if (lane == 0) tiles[0] = 0;
    }
    tc_fence_before();
    __syncthreads();
    __syncwarp();
    cluster_sync_all();   // barriers of both CTAs exist
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();   // the kernel before may still write gradients and their scale; nothing above reads them

    struct Item {
        int e, z;             // expert; 0: y, h or dx; 1, 2: a weight's gradient
        int m0, n0, rows;     // first row of A, first row of B, rows of B that count
        int nt, kb;           // MMA columns, K blocks
    };
    // The i-th item of this cluster, e at or behind `it`'s last but for the gradients of
    // the weights; false when there is none. By whole warps, 32 experts at a time. (Experts
    // with one row, 256 of 256 x 512: 16.9 us, 29 with an expert at a time; 1024 of 64 x 64: 29, 56.)
    auto get = [&](int i, Item &it) {
        int j = cid + i * nclu;
        const int t = j / p.tiles_m;
        if (t < tiles[p.E]) {
            for (int past = 32; past == 32; it.e += past)
                past = __popc(__ballot_sync(0xFFFFFFFFu, it.e + lane < p.E && tiles[it.e + lane + 1] <= t));
            const int n = tiles[it.e + 1] - tiles[it.e];
            const int l = j - tiles[it.e] * p.tiles_m;
            const int c = count[it.e];
            const int per = ((c + n - 1) / n + 31) & ~31;   // rows of a tile, about even; `cap` at most,
                                                             // so that the last one has some
            it.z = 0;
            it.m0 = l / n * (kGated ? 128 : kTile);
            it.n0 = l % n * per;
            it.rows = min(c - it.n0, per);
            it.nt = (it.rows + 31) & ~31;
            it.kb = p.KB * (kBack ? p.products : 1);
            return true;
        }
        if constexpr (kBack) {
            j -= tiles[p.E] * p.tiles_m;
            const int per = p.tiles_m * p.tiles_n;
            it.e = j / (per * p.products);
            if (it.e >= p.E) return false;
            j -= it.e * per * p.products;
            it.z = 1 + j / per;
            j -= (it.z - 1) * per;
            it.m0 = j % p.tiles_m * kTile;
            it.n0 = j / p.tiles_m * p.nt;
            it.rows = min(p.N - it.n0, p.nt);
            it.nt = p.nt;
            it.kb = (count[it.e] + 63) >> 6;
            return true;
        }
        return false;
    };

    if (warp == 0) {
        const bool mine = elect_one();
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);   // the leader's barriers
        int stage = 0;
        uint32_t phase = 1;   // a fresh barrier passes a wait for the phase before its first
        uint32_t own_used = 0, own_odd = 0;   // of `ends`, a bit a stage: in use, an odd number of times
        Item it = {};
        for (int i = 0; get(i, it); ++i) {
            const int row0 = first[it.e];
            const int half = it.nt >> 1;
            const bool dw = kBack && it.z;
            const int box = dw ? 64 : p.box;
            const int boxes = (half + box - 1) / box;
            const uint32_t bytes = kHalf + static_cast<uint32_t>(boxes * box) * 128u;
            const bool left = dw && (count[it.e] & 15);          // an end within an MMA's 16 rows
            for (int kb = 0; kb < it.kb; ++kb) {
                mbar_wait_bounded(smem_u32(empty + stage), phase, abort_flag, p.err, DEV_TIMEOUT_EMPTY);
                const uint32_t st = base + stage * p.stage_bytes;
                const uint32_t bar = full0 + 8 * stage;
                const int s = stage;
                if (++stage == S) stage = 0, phase ^= 1;
                const bool last = left && kb == it.kb - 1;
                if (last) own_used |= 1u << s, own_odd ^= 1u << s;
                if (!mine) continue;
                const int m = it.m0 + rank * (kGated ? 64 : 128);
                if (last) {   // on a barrier of this CTA's, which warp 10 waits for
                    const uint32_t own = smem_u32(ends + s);
                    const int n = it.n0 + rank * half, r = row0 + kb * 64;
                    mbar_expect_tx(own, bytes);
                    own_load2(st, &tm.ax, own, m, r);
                    own_load2(st + 8192, &tm.ax, own, m + 64, r);
                    for (int b = 0; b < boxes; ++b)
                        own_load2(st + kHalf + b * 8192, it.z == 2 ? &tm.bw1 : &tm.bw0, own, n + b * 64, r);
                    continue;
                }
                if (rank == 0)
                    mbar_expect_tx(smem_u32(full + s), 2 * bytes);
                else if (kBack)
                    remote_arrive_relaxed(bar);
                if (dw) {
                    const int n = it.n0 + rank * half, r = row0 + kb * 64;
                    pair_load2(st, &tm.ax, bar, m, r);
                    pair_load2(st + 8192, &tm.ax, bar, m + 64, r);
                    for (int b = 0; b < boxes; ++b)
                        pair_load2(st + kHalf + b * 8192, it.z == 2 ? &tm.bw1 : &tm.bw0, bar, n + b * 64, r);
                } else {
                    const bool second = kBack && kb >= p.KB;
                    const int k = (second ? kb - p.KB : kb) * 64;
                    const CUtensorMap *ma = second ? &tm.a1 : &tm.a0;
                    if constexpr (kGated) {
                        pair_load3(st, &tm.a0, bar, k, m, it.e);
                        pair_load3(st + 8192, &tm.a1, bar, k, m, it.e);
                    } else if constexpr (kBack) {
                        pair_load3(st, ma, bar, m, k, it.e);
                        pair_load3(st + 8192, ma, bar, m + 64, k, it.e);
                    } else {
                        pair_load3(st, ma, bar, k, m, it.e);
                    }
                    const int n = row0 + it.n0 + rank * half;
                    const CUtensorMap *mb = second ? &tm.b1 : &tm.b0;
                    for (int b = 0; b < boxes; ++b) pair_load2(st + kHalf + b * box * 128, mb, bar, k, n + b * box);
                }
            }
        }
        // Every copy of this CTA has landed, and every MMA that reads its shared memory
        // has completed, before it leaves: each stage's last round was returned (a stage
        // without a round passes at once). After a wait that ran out MMAs are issued, and
        // their stages returned, without their copies: the leader, which the other CTA
        // does not leave before, waits for those of both as well.
        for (int t = 0; t < S; ++t) {
            ffn_drain_wait(smem_u32(empty + stage), phase);
            if (rank == 0) ffn_drain_wait(smem_u32(full + stage), phase);
            if (kBack && (own_used >> stage & 1)) ffn_drain_wait(smem_u32(ends + stage), (own_odd >> stage & 1) ^ 1);
            if (++stage == S) stage = 0, phase ^= 1;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            // As in the tile kernel of the feed-forward operators: the next stage is
            // waited for before the last MMA of this one is issued.
            const bool mine = elect_one();
            int stage = 0, as = 0;
            uint32_t phase = 0, aphase = 1;
            auto prepare = [&](int s, uint32_t ph) {
                mbar_wait_bounded(smem_u32(full + s), ph, abort_flag, p.err, DEV_TIMEOUT_FULL);
                tc_fence_after();
            };
            // the next item with a contraction
            auto find = [&](int &i, Item &it) {
                while (get(i, it)) {
                    if (it.kb) return true;
                    ++i;
                }
                return false;
            };
            Item it = {}, next;
            int i = 0;
            bool more_items = find(i, it);
            if (more_items) prepare(0, 0);
            while (more_items) {
                next = it;
                const bool dw = kBack && it.z;
                const uint32_t idesc = p.idesc | static_cast<uint32_t>(it.nt >> 3) << 17 | (dw ? 1u << 16 : 0u);
                const int depth = dw ? count[it.e] : p.K;
                const uint32_t bstep = dw ? 128 : 2;
                const int clear = dw && (depth & 15) ? it.kb - 1 : -1;   // warp 10 clears rows in this block
                mbar_wait_bounded(smem_u32(acce + as), aphase, abort_flag, p.err, DEV_TIMEOUT_ACC_EMPTY);
                tc_fence_after();
                const uint32_t d = tmem + static_cast<uint32_t>(as) * 256;
                for (int kb = 0; kb < it.kb; ++kb) {
                    const uint32_t st = base + stage * p.stage_bytes;
                    const uint64_t ad = kBack ? desc_mn(st) : desc_kmajor(st);
                    const uint64_t bd = dw ? desc_mn(st + kHalf) : desc_kmajor(st + kHalf);
                    const uint32_t bar = smem_u32(empty + stage);
                    // (here and not in every block's wait: dx and dW of 512 rows on each of 16 180.4
                    // us instead of 182.4; those rows reach the asynchronous proxy by warp 10's fence)
                    if (kBack && __builtin_expect(kb == clear, 0)) {
                        acquire_cluster(smem_u32(full + stage), phase);
                        tc_fence_after();
                    }
                    const int at = kBack && !dw && kb >= p.KB ? kb - p.KB : kb;
                    const int steps = min(4, (depth - at * 64 + 15) >> 4);
                    auto mma = [&](int kk) {
                        if (mine)
                            pair_mma(d, ad + kk * (kBack ? 128 : 2), bd + kk * bstep, idesc, kb > 0 || kk > 0);
                    };
#pragma unroll
                    for (int kk = 0; kk < 3; ++kk)
                        if (kk < steps) mma(kk);
                    if (kb == 0) {   // found while those run
                        ++i;
                        more_items = find(i, next);
                    }
                    if (++stage == S) stage = 0, phase ^= 1;
                    if (kb + 1 < it.kb || more_items) prepare(stage, phase);
                    if (steps > 3) mma(3);
                    if (mine) pair_commit(bar);
                }
                if (mine) pair_commit(smem_u32(accf + as));
                if (++as == 2) as = 0, aphase ^= 1;
                it = next;
            }
        }
        __syncwarp();
    } else if (warp < 10) {
        // Two warps for each quarter of the accumulator's lanes, every other 32 columns each.
        const int q = warp & 3;
        const int half = warp >= 6;
        const float scale = p.scale ? __ldg(p.scale) : 1.f;   // a power of two
        int as = 0;
        uint32_t aphase = 0;
        const uint32_t box = boxes0 + static_cast<uint32_t>(warp - 2) * kBox;
        const uint32_t other = boxes0 + static_cast<uint32_t>((warp - 2) ^ 2) * kBox;   // gated: the partner's
        Item it = {};
        for (int i = 0; get(i, it); ++i) {
            const int m = it.m0 + (kGated ? rank * 64 + (q & 1) * 32 : rank * 128 + q * 32);
            const bool dw = kBack && it.z;
            const int64_t ldy = dw ? p.M : p.ldy;
            const int vec = p.vec[dw];
            uint16_t *dst = p.y[kBack ? it.z : 0] +
                            (dw ? static_cast<int64_t>(it.e) * p.N + it.n0 : static_cast<int64_t>(first[it.e] + it.n0)) * ldy;
            if (kBack && it.kb == 0) {   // an expert without rows
                const uint32_t zero[4] = {};
                for (int c = 0; c < 4; ++c) store_fragments(box_at(box, 8 * c + (lane & 7), lane >> 3), zero);
                for (int c = 32 * half; c < it.rows; c += 64)
                    put_box<32>(dst + c * ldy, ldy, box, m, p.M, it.rows - c, lane, vec);
                continue;
            }
            mbar_wait_bounded(smem_u32(accf + as), aphase, abort_flag, p.err, DEV_TIMEOUT_ACC_FULL,
                              wait_limit_ns(it.kb));
            tc_fence_after();
            const uint32_t t = tmem + static_cast<uint32_t>(as) * 256 + (static_cast<uint32_t>(q * 32) << 16);
            for (int c = 32 * half; c < it.nt; c += 64) {
                uint32_t v[2][16];   // lanes 0 .. 15 and 16 .. 31
                tmem_ld16x32(t + c, v[0]);
                tmem_ld16x32(t + c + (16u << 16), v[1]);
                tmem_ld_wait();
                if constexpr (kGated) {
                    // Partner q ^ 2 has the factors of these gates: this warp takes the first
                    // 16 of the 32 rows, the other the last.
                    float a[16], b[16], h[16];   // eight of accumulator lanes 0 .. 15, eight of 16 .. 31
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int g = i >> 1, x = 4 * (i & 1);
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(box + i * 512 + lane * 16),
                                     "r"(q < 2 ? v[g][8 + x] : v[g][x]), "r"(q < 2 ? v[g][9 + x] : v[g][1 + x]),
                                     "r"(q < 2 ? v[g][10 + x] : v[g][2 + x]), "r"(q < 2 ? v[g][11 + x] : v[g][3 + x])
                                     : "memory");
                    }
                    named_bar_sync(1 + 2 * half + (q & 1), 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int g = i >> 1, x = 4 * (i & 1);
                        float got[4];
                        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                     : "=f"(got[0]), "=f"(got[1]), "=f"(got[2]), "=f"(got[3])
                                     : "r"(other + i * 512 + lane * 16)
                                     : "memory");
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float own = __uint_as_float(q < 2 ? v[g][x + k] : v[g][8 + x + k]);
                            a[8 * g + x + k] = q < 2 ? own : got[k];
                            b[8 * g + x + k] = q < 2 ? got[k] : own;
                        }
                    }
                    named_bar_sync(1 + 2 * half + (q & 1), 64);   // both have read
                    const int n = c + (q < 2 ? 0 : 16);
                    const int rows = it.rows - n;
                    if (p.g) {
                        const int64_t at = static_cast<int64_t>(first[it.e] + it.n0 + n) * p.M + m + (lane >> 2);
#pragma unroll
                        for (int g = 0; g < 2; ++g)
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const int r = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1), mo = 16 * g + 8 * ((i >> 1) & 1);
                                if (r < rows && m + mo + (lane >> 2) < p.M) {
                                    p.g[at + static_cast<int64_t>(r) * p.M + mo] = a[8 * g + i];
                                    p.u[at + static_cast<int64_t>(r) * p.M + mo] = b[8 * g + i];
                                }
                            }
                    }
                    ffn_gate(a, b, p.act, h);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            r[k] = pack2(h[8 * (k >> 1) + 4 * i + 2 * (k & 1)], h[8 * (k >> 1) + 4 * i + 2 * (k & 1) + 1],
                                         p.dtype);
                        store_fragments(box_at(box, 8 * i + (lane & 7), lane >> 3), r);
                    }
                    put_box<16>(dst + n * ldy, ldy, box, m, p.M, rows, lane, vec);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t r[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            r[k] = pack2(__uint_as_float(v[k >> 1][4 * i + 2 * (k & 1)]) * scale,
                                         __uint_as_float(v[k >> 1][4 * i + 2 * (k & 1) + 1]) * scale, p.dtype);
                        store_fragments(box_at(box, 8 * i + (lane & 7), lane >> 3), r);
                    }
                    put_box<32>(dst + c * ldy, ldy, box, m, p.M, it.rows - c, lane, vec);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) remote_arrive_relaxed(mapa_shared(smem_u32(acce + as), 0));
            if (++as == 2) as = 0, aphase ^= 1;
        }
        __syncwarp();
    } else if constexpr (kBack) {
        // Rows of others behind an expert's last one, within the MMA step that it is in.
        const uint32_t full0 = mapa_shared(smem_u32(full), 0);
        uint32_t seen = 0;   // phases of `ends`, a bit a stage
        int end = 0;         // the stage behind the last one of the item before
        uint64_t behind = 0; // K blocks since the last wait
        Item it = {};
        for (int i = 0; get(i, it); ++i) {
            const int left = count[it.e] & 15;
            end = (end + it.kb) % S;
            behind += it.kb + 8;   // and an item's way out
            if (!it.z || !it.kb || !left) continue;
            const int s = end ? end - 1 : S - 1;
            // (this warp has nothing to do while dx is computed)
            mbar_wait_bounded(smem_u32(ends + s), (seen >> s) & 1, abort_flag, p.err, DEV_TIMEOUT_FULL,
                              wait_limit_ns(behind));
            behind = 0;
            seen ^= 1u << s;
            const int r0 = count[it.e] & 63, n = 16 - left;      // K rows r0 .. r0 + n - 1 of every 8 KB group
            const int groups = 2 + (it.nt >> 7);
            for (int gr = 0; gr < groups; ++gr) {
                const uint32_t to = base + s * p.stage_bytes + gr * 8192 + r0 * 128;
#pragma unroll
                for (int x = lane; x < 15 * 8; x += 32)
                    if (x < n * 8) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to + x * 16), "r"(0) : "memory");
            }
            // the tensor cores read them through the asynchronous proxy
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) remote_arrive_release(full0 + 8 * s);
        }
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

int cdiv(int64_t a, int64_t b) { return static_cast<int>((a + b - 1) / b); }

std::mutex g_mu;
bool g_ready[64];   // devices whose kernels have their shared memory raised

}  // namespace

cudaError_t grouped_launch(const GroupedArgs &a, const FfnDev &d, cudaStream_t s) {
    using Fn = void (*)(GroupedMaps, GroupedParams);
    static const Fn kernels[] = {grouped_kernel<GROUPED_PLAIN>, grouped_kernel<GROUPED_GATED>,
                                 grouped_kernel<GROUPED_BACKWARD>};
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
    const bool gated = a.form == GROUPED_GATED, back = a.form == GROUPED_BACKWARD;
    GroupedParams p = {};
    p.offsets = a.offsets;
    p.y[0] = static_cast<uint16_t *>(a.y);
    p.y[1] = static_cast<uint16_t *>(a.dw0);
    p.y[2] = static_cast<uint16_t *>(a.dw1);
    p.g = a.g;
    p.u = a.u;
    p.ldy = a.ldy;
    p.scale = a.scale;
    p.err = a.err;
    p.R = a.R;
    p.E = a.E;
    p.N = a.N;
    p.M = back ? a.K : a.N;
    p.tiles_m = cdiv(p.M, gated ? 128 : kTile);
    p.products = back && a.d1 ? 2 : 1;
    p.K = back ? a.N : a.K;
    p.KB = cdiv(p.K, 64);
    p.act = a.act;
    p.dtype = a.dtype;
    auto starts = [](const void *y, int64_t ld) {
        const uintptr_t v = reinterpret_cast<uintptr_t>(y) | static_cast<uintptr_t>(ld * 2);
        return v % 16 == 0 ? 2 : v % 4 == 0 ? 1 : 0;
    };
    p.vec[0] = starts(a.y, a.ldy);
    p.vec[1] = starts(a.dw0, a.K);
    p.idesc = idesc_f16(a.dtype, 256, 0, back);
    // Copies of rows: in as few pieces as do not bring many of other experts. (Gated, one row on
    // each of 64 experts, 1024 x 2048: 51.5 us with 16 rows a copy, 53.8 with 64; 512 on each of 8,
    // 2048 x 4096: 88.2 with 16, 86.2 with 64; from 8 to 256 rows all three within 4 %, as runs are.)
    const int used = std::min(a.E, a.R), mean = a.R / used;
    p.cap = a.R < kTile ? (a.R + 31) / 32 * 32 : kTile;
    p.box = std::min(mean >= 128 ? 64 : mean >= 32 ? 32 : 16, p.cap / 2);
    int half = cdiv(p.cap / 2, p.box) * p.box;   // rows of B that a CTA holds at most
    int64_t items = (static_cast<int64_t>(a.R) / std::min(p.cap, cap_of(kCaps - 1)) + used) * p.tiles_m;
    if (back) {
        // the weights' gradients in tiles of 256 or 128 features, by rounds times a tile's cycles
        p.KBw = cdiv(a.R, 64ll * a.E);
        auto cost = [&](int nt) {
            const float tiles = static_cast<float>(a.E) * (p.products * p.tiles_m) * cdiv(a.N, nt);
            return std::max(1.f, tiles / (d.sms / 2)) * tile_cycles(nt, static_cast<float>(p.KBw));
        };
        p.nt = cost(128) < cost(kTile) ? 128 : kTile;
        p.tiles_n = cdiv(a.N, p.nt);
        half = std::max(half, p.nt / 2);
        items += static_cast<int64_t>(a.E) * p.tiles_m * p.tiles_n * p.products;
    }
    if (items > (1 << 30)) return cudaErrorInvalidValue;
    p.stage_bytes = kHalf + static_cast<uint32_t>(half) * 128;
    const size_t fixed = 1024 + 8 * kBox + kBarBytes + (3 * static_cast<size_t>(a.E) + 1) * sizeof(int32_t);
    p.stages = std::min<int>(kMaxStages, static_cast<int>((kMaxSmem - fixed) / p.stage_bytes));

    GroupedMaps tm = {};
    auto experts = [&](CUtensorMap *m, const MoeMat &w, int box_rows) {
        if (e == cudaSuccess) e = ffn_tensor_map3(m, w.p, a.E, a.N, a.K, w.ld, w.se, box_rows, a.dtype);
    };
    auto rows = [&](CUtensorMap *m, const void *ptr, int cols, int64_t ld, int box_rows) {
        if (e == cudaSuccess) e = ffn_tensor_map(m, ptr, a.R, cols, ld, box_rows, 64, a.dtype);
    };
    experts(&tm.a0, a.w0, gated || back ? 64 : 128);
    if (gated || p.products == 2) experts(&tm.a1, a.w1, 64);
    if (back) {
        rows(&tm.b0, a.d0, a.N, a.ldd, p.box);
        rows(&tm.bw0, a.d0, a.N, a.ldd, 64);
        if (p.products == 2) {
            rows(&tm.b1, a.d1, a.N, a.ldd, p.box);
            rows(&tm.bw1, a.d1, a.N, a.ldd, 64);
        }
        rows(&tm.ax, a.x, a.K, a.ldx, 64);
    } else {
        rows(&tm.b0, a.x, a.K, a.ldx, p.box);
    }
    if (e != cudaSuccess) return e;
    size_t smem = 0;
    if ((e = ffn_smem_for_tmem(d.dev, 512, fixed + static_cast<size_t>(p.stages) * p.stage_bytes, &smem)) != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2u * static_cast<unsigned>(std::min<int64_t>(items, d.sms / 2)), 1, 1);
    cfg.blockDim = dim3(back ? kThreadsBack : kThreads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernels[a.form], tm, p);
}

}  // namespace kp
