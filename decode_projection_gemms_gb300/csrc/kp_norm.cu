// Layer norm of rows and its gradients:
//     xhat = (x - mean) rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps), y = round(xhat w + b)
//     dx = rstd (g - mean(g) - xhat mean(g xhat)), g = dy w;  dw = sum_t dy xhat, db = sum_t dy
// (without centring: mean and mean(g) are 0, root-mean-square norm).
//
// A row is read once and stays in the registers of a team of warps, so that the squares are
// summed around the mean that was found first: no difference of two large sums. The gradients
// start from x - mean too: x rstd - mean rstd is a rounding of mean rstd off for a whole row
// (rows of 1e5 +- 1 in fp32: 8e-4 on every xhat, which adds up in dw). All sums are fp32.
// Backward, a block takes rows b, b + blocks, ... and a thread keeps the same columns, whose
// dw and db it adds up in registers; the blocks' sums go to a workspace and a second kernel
// adds them in order, so nothing depends on timing.
//
// Bound: HBM forward (8192 x 7168 bf16: 39 us, 6.0 TB/s; 16384 x 4096 6.5). Backward the
// instructions, about 30 an element of which a row's sums and addresses are 10, and the wait for
// the row's sums: 84 us, 4.2 TB/s. What it took to get there from 139: rows ahead through shared
// memory, a block's teams' sums joined in it (a block's sums cost as much memory as four rows), the
// two sums of a row halved between the lanes, the next row's statistics read beforehand.
#include <algorithm>
#include <type_traits>

#include "kp_norm.cuh"

namespace kp {

namespace {

constexpr int kPieces = 4;   // 8 elements each, of a thread at most

// Eight elements of a row as they lie in memory. A 16-bit one is widened only where a
// product needs it in fp32 beside another fp32 number: products and sums of two of them
// take the mixed-precision FMA, whose product is exact and which rounds once, as on the
// widened values.
template <typename T>
struct Piece {
    static constexpr bool k16 = sizeof(T) == 2;
    static constexpr int D = std::is_same<T, __half>::value ? KP_FP16 : KP_BF16;
    static constexpr int kWords = 2 * sizeof(T);
    uint32_t w[kWords];
    __device__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ void load_whole(const void *p) {   // 16-byte aligned
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 a = static_cast<const uint4 *>(p)[i];
            w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
        }
    }
    __device__ void load(const T *row, int c, int K, bool whole) {   // zeros past K
        if (whole) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row + c) + i);
                w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
            }
        } else if constexpr (!k16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = c + i < K ? __float_as_uint(__ldg(reinterpret_cast<const float *>(row) + c + i)) : 0u;
        } else {
            const uint16_t *h = reinterpret_cast<const uint16_t *>(row) + c;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = (c + 2 * i < K ? __ldg(h + 2 * i) : 0u) |
                       (c + 2 * i + 1 < K ? static_cast<uint32_t>(__ldg(h + 2 * i + 1)) << 16 : 0u);
        }
    }
    __device__ float operator[](int j) const {
        if constexpr (!k16)
            return __uint_as_float(w[j]);
        else
            return j & 1 ? elem_hi<D>(w[j >> 1]) : elem_lo<D>(w[j >> 1]);
    }
    // element j times element j of b, plus c
    __device__ float mul_add(int j, const Piece &b, float c) const {
        if constexpr (!k16) return fmaf((*this)[j], b[j], c);
        return mix(w[j >> 1], b.w[j >> 1], j & 1, c);
    }
    // element j plus c
    __device__ float add(int j, float c) const {
        if constexpr (!k16) return (*this)[j] + c;
        return mix(w[j >> 1], D == KP_FP16 ? 0x3C003C00u : 0x3F803F80u, j & 1, c);
    }
    static __device__ float mix(uint32_t a, uint32_t b, bool hi, float c) {
        float r;
        if constexpr (D == KP_FP16) {
            if (hi)
                asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\tfma.rn.f32.f16 %0, h, n, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(c));
            else
                asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\tfma.rn.f32.f16 %0, l, m, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(c));
        } else {
            if (hi)
                asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\tfma.rn.f32.bf16 %0, h, n, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(c));
            else
                asm("{\n\t.reg .b16 l, h, m, n;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 {m, n}, %2;\n\tfma.rn.f32.bf16 %0, l, m, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(c));
        }
        return r;
    }
};

// Eight results, rounded, into columns c .. of a row, those below K.
template <typename T>
__device__ __forceinline__ void store8(T *row, int c, int K, bool whole, const float (&f)[8]) {
    if constexpr (sizeof(T) == 4) {
        if (whole) {
            reinterpret_cast<float4 *>(row + c)[0] = make_float4(f[0], f[1], f[2], f[3]);
            reinterpret_cast<float4 *>(row + c)[1] = make_float4(f[4], f[5], f[6], f[7]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < K) row[c + i] = f[i];
        }
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (Piece<T>::D == KP_FP16) {
                const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
                w[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        uint16_t *to = reinterpret_cast<uint16_t *>(row) + c;
        if (whole) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i < K) to[i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Sums over a team of W warps, the same in every thread, always in the same order. `turn`
// picks one of two buffers, so that one barrier a sum is enough. kBar: a named barrier of the
// team's own (its number + 1), else the block's.
template <int W, bool kBar>
__device__ __forceinline__ void team_barrier(int team) {
    if constexpr (kBar)
        named_bar_sync(1 + team, 32 * W);
    else
        __syncthreads();
}
template <int W>
__device__ __forceinline__ void team_sum(float &v, float (&sh)[2][W], int &turn) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if constexpr (W > 1) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) sh[turn][(threadIdx.x >> 5) % W] = v;
        team_barrier<W, false>(0);
        v = sh[turn][lane % W];
#pragma unroll
        for (int d = W / 2; d; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        turn ^= 1;
    }
}
// Two of them at a time, each in half of the lanes after the first exchange.
template <int W>
__device__ __forceinline__ void team_sum2(float (&v)[2], float (&sh)[2][2][W], int &turn, int team) {
    const int lane = threadIdx.x & 31;
    const bool upper = lane & 16;
    float mine = upper ? v[1] : v[0];
    mine += __shfl_xor_sync(0xFFFFFFFFu, upper ? v[0] : v[1], 16);
#pragma unroll
    for (int d = 8; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
    if constexpr (W > 1) {
        if ((lane & 15) == 0) sh[turn][upper][(threadIdx.x >> 5) % W] = mine;
        team_barrier<W, true>(team);
        constexpr int H = W < 16 ? W : 16;
        mine = sh[turn][upper][lane % H];
        if constexpr (W == 32) mine += sh[turn][upper][16 + lane % 16];
#pragma unroll
        for (int d = H / 2; d; d >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, d);
        turn ^= 1;
    }
    v[0] = __shfl_sync(0xFFFFFFFFu, mine, 0);
    v[1] = __shfl_sync(0xFFFFFFFFu, mine, 16);
}

struct NormParams {
    const void *x, *w, *b, *dy;
    void *y;                  // y or dx
    float *mean, *rstd;
    float *part;              // backward: [blocks][2][K], dw's and db's sums
    int64_t ldx, ldy, lddy;
    int T, K, center, vec;    // vec: all rows start on 16 bytes and K is a multiple of 8
    int bias;                 // backward: db is wanted
    float eps;
};

// Forward: W warps a row; a single one: four rows a block.
template <int W>
constexpr int rows_of() { return W == 1 ? 4 : 1; }
// Backward: teams of a block, 16 warps in all, so that few blocks hold a sum of every column.
__host__ __device__ constexpr int teams_of(int W) { return W < 16 ? 16 / W : 1; }

// Blocks of an SM, for 16-bit rows: as many as their packed pieces leave registers for.
template <typename T, int W>
constexpr int forward_blocks() { return (sizeof(T) == 4 ? 32 : 40) / (W * rows_of<W>()) > 0 ? (sizeof(T) == 4 ? 32 : 40) / (W * rows_of<W>()) : 1; }

// kVec: all rows start on 16 bytes and K is a multiple of 8.
template <typename T, int W, int P, bool kVec>
__global__ void __launch_bounds__(32 * W * rows_of<W>(), forward_blocks<T, W>()) norm_kernel(const NormParams p) {
    __shared__ float sh[2][W];
    const int lane = W == 1 ? threadIdx.x & 31 : threadIdx.x;
    const int64_t t = static_cast<int64_t>(blockIdx.x) * rows_of<W>() + (W == 1 ? threadIdx.x >> 5 : 0);
    if (W == 1 && t >= p.T) return;
    const T *x = static_cast<const T *>(p.x) + t * p.ldx;
    int turn = 0;
    Piece<T> v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * 32 * W + lane) * 8;
        if (c < p.K)
            v[i].load(x, c, p.K, kVec);
        else
            v[i].zero();
    }
    float mean = 0.f, sum = 0.f;
    if (p.center) {
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = v[i].add(j, sum);   // zeros past K
        team_sum<W>(sum, sh, turn);
        mean = sum / static_cast<float>(p.K);
    }
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * 32 * W + lane) * 8;
        if (c >= p.K) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = v[i].add(j, -mean);
            if (kVec || c + j < p.K) sum = fmaf(d, d, sum);
        }
    }
    team_sum<W>(sum, sh, turn);
    const float rstd = 1.f / sqrtf(sum / static_cast<float>(p.K) + p.eps);
    if (lane == 0) {
        if (p.mean) p.mean[t] = mean;
        if (p.rstd) p.rstd[t] = rstd;
    }
    const T *w = static_cast<const T *>(p.w), *b = static_cast<const T *>(p.b);
    T *y = static_cast<T *>(p.y) + t * p.ldy;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int c = (i * 32 * W + lane) * 8;
        if (c >= p.K) break;
        Piece<T> wp, bp;
        wp.load(w, c, p.K, kVec);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i].add(j, -mean) * rstd * wp[j];
        if (b) {
            bp.load(b, c, p.K, kVec);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = bp.add(j, f[j]);
        }
        store8(y, c, p.K, kVec, f);
    }
}

// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the last N groups have landed
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows ahead of the one at hand. A thread copies the pieces of x and dy that it will read
// itself, so its own wait is all they need, and reads them twice, around the row's two
// sums: held in registers they would halve the blocks on an SM.
constexpr int kAhead = 2;

// kRing: rows come through shared memory; without it (rows that do not start on 16 bytes)
// they are read from global memory twice.
template <typename T, int W, int P, bool kRing>
__global__ void __launch_bounds__(32 * W * teams_of(W), 32 / (W * teams_of(W)))
    norm_backward_kernel(const NormParams p) {
    constexpr int kTeams = teams_of(W);
    constexpr int kLanes = 32 * W;
    constexpr int kBytes = 8 * sizeof(T);   // of a piece
    extern __shared__ uint8_t ring[];
    __shared__ float sh[kTeams][2][2][W];
    const int lane = threadIdx.x % kLanes;
    const int team = threadIdx.x / kLanes;
    float dw[P][8] = {}, db[P][8] = {};
    int turn = 0;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kTeams + team;
    // piece i of x (0) or dy (1) in buffer s
    auto at = [&](int s, int which, int i) {
        return ((((s * kTeams + team) * 2 + which) * P + i) * kLanes + lane) * kBytes;
    };
    // the next row to fetch, and this thread's first piece of it
    int64_t ahead = first;
    const T *xa = static_cast<const T *>(p.x) + first * p.ldx + lane * 8, *da = static_cast<const T *>(p.dy) + first * p.lddy + lane * 8;
    const int64_t xstep = step * p.ldx, dstep = step * p.lddy, ystep = step * p.ldy;
    const uint32_t ring0 = smem_u32(ring);
    auto fetch = [&](int s) {
        if (ahead < p.T) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if ((i * kLanes + lane) * 8 >= p.K) break;
#pragma unroll
                for (int b = 0; b < kBytes; b += 16) {
                    copy16(ring0 + at(s, 0, i) + b, reinterpret_cast<const char *>(xa + i * kLanes * 8) + b);
                    copy16(ring0 + at(s, 1, i) + b, reinterpret_cast<const char *>(da + i * kLanes * 8) + b);
                }
            }
        }
        ahead += step;
        xa += xstep;
        da += dstep;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kRing)
        for (int s = 0; s < kAhead; ++s) fetch(s);
    int s = 0;
    T *dx = static_cast<T *>(p.y) + first * p.ldy;
    // a row's statistics are read while the one before it is at hand
    float next_rstd = first < p.T ? __ldg(p.rstd + first) : 0.f;
    float next_mean = p.center && first < p.T ? __ldg(p.mean + first) : 0.f;
    for (int64_t t = first; t < p.T; t += step, dx += ystep) {
        const T *x = static_cast<const T *>(p.x) + t * p.ldx, *dy = static_cast<const T *>(p.dy) + t * p.lddy;   // (no ring)
        const float rstd = next_rstd, mean = next_mean;
        if (t + step < p.T) {
            next_rstd = __ldg(p.rstd + t + step);
            if (p.center) next_mean = __ldg(p.mean + t + step);
        }
        if constexpr (kRing) {
            fetch(s ? s - 1 : kAhead);   // the buffer of the row before
            copies_wait<kAhead>();
        }
        // x and dy of piece i
        auto piece = [&](int i, int c, Piece<T> &xp, Piece<T> &dp) {
            if constexpr (kRing) {
                xp.load_whole(ring + at(s, 0, i));
                dp.load_whole(ring + at(s, 1, i));
            } else {
                xp.load(x, c, p.K, false);
                dp.load(dy, c, p.K, false);
            }
        };
        float sum[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * kLanes + lane) * 8;
            if (c >= p.K) break;
            Piece<T> xp, dp, wp;
            piece(i, c, xp, dp);
            wp.load(static_cast<const T *>(p.w), c, p.K, kRing);
            // (x is widened here: with the mixed-precision sum 8192 x 12288 bf16 takes 174 us instead of 162)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (!kRing && c + j >= p.K) break;
                const float xh = (xp[j] - mean) * rstd, g = dp.mul_add(j, wp, 0.f);
                dw[i][j] = fmaf(dp[j], xh, dw[i][j]);
                sum[0] += g;
                sum[1] = fmaf(g, xh, sum[1]);
            }
            if (p.bias)
#pragma unroll
                for (int j = 0; j < 8; ++j) db[i][j] = dp.add(j, db[i][j]);   // zeros past K
        }
        team_sum2<W>(sum, sh[team], turn, team);
        // rstd (g - a - xhat m), with xhat m = (x - mean) (rstd m)
        const float a = p.center ? sum[0] / static_cast<float>(p.K) : 0.f;
        const float slope = -rstd * (sum[1] / static_cast<float>(p.K));
#pragma unroll
        for (int i = 0; i < P; ++i) {
            const int c = (i * kLanes + lane) * 8;
            if (c >= p.K) break;
            Piece<T> xp, dp, wp;
            piece(i, c, xp, dp);
            wp.load(static_cast<const T *>(p.w), c, p.K, kRing);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = fmaf(xp[j] - mean, slope, dp.mul_add(j, wp, -a)) * rstd;
            store8(dx, c, p.K, kRing, f);
        }
        if (++s == kAhead + 1) s = 0;
    }
    if constexpr (kRing) copies_wait<0>();
    // the block's sums: of its teams, in order
    float *part = p.part + static_cast<int64_t>(blockIdx.x) * 2 * p.K;
    float *all = reinterpret_cast<float *>(ring);   // [kTeams][P * 8][kLanes]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (which && !p.bias) break;
        if constexpr (kTeams > 1) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) all[(team * P * 8 + i * 8 + j) * kLanes + lane] = which ? db[i][j] : dw[i][j];
            __syncthreads();
            for (int k = threadIdx.x; k < P * 8 * kLanes; k += kLanes * kTeams) {
                const int c = (k / (8 * kLanes) * kLanes + k % kLanes) * 8 + k / kLanes % 8;
                float v = 0.f;
#pragma unroll
                for (int q = 0; q < kTeams; ++q) v += all[q * P * 8 * kLanes + k];
                if (c < p.K) part[which * p.K + c] = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int c = (i * kLanes + lane) * 8;
                const float(&v)[8] = which ? db[i] : dw[i];
                if (kRing && c < p.K) {   // K is a multiple of 8
                    reinterpret_cast<float4 *>(part + which * p.K + c)[0] = make_float4(v[0], v[1], v[2], v[3]);
                    reinterpret_cast<float4 *>(part + which * p.K + c)[1] = make_float4(v[4], v[5], v[6], v[7]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (c + j < p.K) part[which * p.K + c + j] = v[j];
                }
            }
        }
    }
}

// dw and db: the blocks' sums added in order; a lane two columns of [dw, db], warps (32 at
// most) the blocks by turns.
__global__ void norm_join_kernel(const float *__restrict__ part, int blocks, int K, int columns, void *dw, void *db,
                                 int dtype) {
    __shared__ float2 sh[32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x) >> 5;
    const int c = (static_cast<int>(blockIdx.x) * 32 + lane) * 2;
    float2 v = make_float2(0.f, 0.f);
    if (c < columns) {   // (2 K is even)
#pragma unroll 8
        for (int b = warp; b < blocks; b += warps) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(part + static_cast<int64_t>(b) * 2 * K + c));
            v.x += a.x, v.y += a.y;
        }
    }
    sh[warp][lane] = v;
    __syncthreads();
    if (warp) return;
    v = make_float2(0.f, 0.f);
    for (int w = 0; w < warps; ++w) v.x += sh[w][lane].x, v.y += sh[w][lane].y;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (c + k >= columns) break;
        void *to = c + k < K ? dw : db;
        const int at = c + k < K ? c + k : c + k - K;
        const float f = k ? v.y : v.x;
        if (dtype == KP_FP32)
            static_cast<float *>(to)[at] = f;
        else
            static_cast<uint16_t *>(to)[at] = elem_round(f, dtype);
    }
}

// Warps of a team and pieces of a thread for K columns.
struct Shape {
    int W, P;
};
Shape shape_of(int K) {
    const int pieces = (K + 7) / 8;
    if (pieces <= 32) return {1, 1};
    if (pieces <= 64) return {1, 2};
    Shape s = {1, kPieces};
    while (s.W * 32 * kPieces < pieces) s.W *= 2;
    return s;
}
// Backward: two pieces at most, since a thread also holds their columns' sums. With 32 warps
// of 64 registers an SM 8192 x 7168 takes 106 us, with four pieces and 16 warps 129.
Shape backward_shape(int K) {
    const int pieces = (K + 7) / 8;
    if (pieces <= 32) return {1, 1};
    Shape s = {1, 2};
    while (s.W * 64 < pieces) s.W *= 2;
    return s;
}

using Fn = void (*)(NormParams);

// Kernel: 0 and 1 forward (whole pieces), 2 and 3 backward (through the ring).
template <typename T, int W, int P, int kKernel>
Fn kernel() {
    if constexpr (kKernel < 2)
        return norm_kernel<T, W, P, kKernel == 1>;
    else
        return norm_backward_kernel<T, W, P, kKernel == 3>;
}
template <typename T, int kKernel>
Fn kernel_of(const Shape &s) {
    if (s.W == 1) return s.P == 1 ? kernel<T, 1, 1, kKernel>() : s.P == 2 ? kernel<T, 1, 2, kKernel>() : kernel<T, 1, kPieces, kKernel>();
    switch (s.W) {
    case 2: return kernel<T, 2, kPieces, kKernel>();
    case 4: return kernel<T, 4, kPieces, kKernel>();
    case 8: return kernel<T, 8, kPieces, kKernel>();
    default: return kernel<T, 16, kPieces, kKernel>();
    }
}
template <typename T, int kKernel>
Fn backward_kernel_of(const Shape &s) {
    if (s.W == 1) return s.P == 1 ? kernel<T, 1, 1, kKernel>() : kernel<T, 1, 2, kKernel>();
    switch (s.W) {
    case 2: return kernel<T, 2, 2, kKernel>();
    case 4: return kernel<T, 4, 2, kKernel>();
    case 8: return kernel<T, 8, 2, kKernel>();
    case 16: return kernel<T, 16, 2, kKernel>();
    default: return kernel<T, 32, 2, kKernel>();
    }
}
template <typename T>
Fn pick(const Shape &s, int kernel) {
    return kernel == 0   ? kernel_of<T, 0>(s)
           : kernel == 1 ? kernel_of<T, 1>(s)
           : kernel == 2 ? backward_kernel_of<T, 2>(s)
                         : backward_kernel_of<T, 3>(s);
}
Fn pick(const Shape &s, int dtype, int kernel) {
    return dtype == KP_FP32   ? pick<float>(s, kernel)
           : dtype == KP_FP16 ? pick<__half>(s, kernel)
                              : pick<__nv_bfloat16>(s, kernel);
}

// Blocks of the backward kernel: 32 warps an SM, or as many as their rings leave room for.
int backward_blocks(int T, const Shape &s, size_t ring, int sms) {
    const int teams = teams_of(s.W);
    const int per_sm = std::min(32 / (s.W * teams), std::max<int>(1, static_cast<int>(220 * 1024 / (ring + 4096))));
    return static_cast<int>(std::min<int64_t>((static_cast<int64_t>(T) + teams - 1) / teams, static_cast<int64_t>(sms) * per_sm));
}

bool starts16(const void *p, int64_t ld, int es) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld * es)) & 15) == 0;
}

}  // namespace

size_t norm_backward_scratch(int T, int K, int sms) {
    return static_cast<size_t>(backward_blocks(T, backward_shape(K), 0, sms)) * 2 * K * sizeof(float);
}

cudaError_t norm_launch(const NormArgs &a, cudaStream_t s) {
    const int es = a.dtype == KP_FP32 ? 4 : 2;
    const Shape sh = shape_of(a.K);
    NormParams p = {};
    p.x = a.x;
    p.w = a.w;
    p.b = a.b;
    p.y = a.y;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.ldx = a.ldx;
    p.ldy = a.ldy;
    p.T = a.T;
    p.K = a.K;
    p.center = a.center;
    p.eps = a.eps;
    p.vec = a.K % 8 == 0 && starts16(a.x, a.ldx, es) && starts16(a.y, a.ldy, es) && starts16(a.w, 0, es) && starts16(a.b, 0, es);
    const int rows = sh.W == 1 ? 4 : 1;
    const Fn f = pick(sh, a.dtype, p.vec);
    f<<<static_cast<unsigned>((static_cast<int64_t>(a.T) + rows - 1) / rows), 32 * sh.W * rows, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t norm_backward_launch(const NormArgs &a, const FfnDev &d, cudaStream_t s) {
    const int es = a.dtype == KP_FP32 ? 4 : 2;
    const Shape sh = backward_shape(a.K);
    NormParams p = {};
    p.x = a.x;
    p.w = a.w;
    p.dy = a.dy;
    p.y = a.y;
    p.mean = a.mean;
    p.rstd = a.rstd;
    p.part = a.part;
    p.ldx = a.ldx;
    p.ldy = a.ldy;
    p.lddy = a.lddy;
    p.T = a.T;
    p.K = a.K;
    p.center = a.center;
    p.bias = a.dbias != nullptr;
    const int threads = 32 * sh.W * teams_of(sh.W);
    // (fp32 rows of more than 8192 columns have no room for a ring: 4096 x 16384 559 us, bf16 103)
    const size_t ring = static_cast<size_t>(kAhead + 1) * 2 * sh.P * threads * 8 * es;
    const size_t sums = static_cast<size_t>(sh.P) * 8 * threads * sizeof(float);   // (no more than a ring)
    const bool vec = a.K % 8 == 0 && starts16(a.x, a.ldx, es) && starts16(a.y, a.ldy, es) && starts16(a.dy, a.lddy, es) &&
                     starts16(a.w, 0, es) && ring <= 200 * 1024;
    const int blocks = backward_blocks(a.T, sh, vec ? ring : 0, d.sms);
    const Fn f = pick(sh, a.dtype, vec ? 3 : 2);
    const size_t smem = vec ? ring : sums;
    if (smem > 40 * 1024) {   // 48 KB with what the kernel declares itself
        const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    f<<<blocks, threads, smem, s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int columns = a.dbias ? 2 * a.K : a.K;
    norm_join_kernel<<<(columns + 63) / 64, 32 * std::min(32, (blocks + 3) / 4), 0, s>>>(a.part, blocks, a.K, columns, a.dw,
                                                                                        a.dbias, a.dtype);
    return cudaGetLastError();
}

}  // namespace kp
