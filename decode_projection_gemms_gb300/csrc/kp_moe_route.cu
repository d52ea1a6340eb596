// Router of the mixture-of-experts operators: each token's top-k experts, the weights
// of their outputs, and the order that puts the chosen (token, slot) pairs expert by
// expert, tokens ascending within each.
//
// A warp a token: a lane holds experts lane, lane + 32, ...; a choice is a maximum over
// the warp of keys that order like the logits, then a minimum over the experts that
// have it. The order is a counting sort: every block of kTokens tokens counts its
// choices by expert, the counts of the blocks before it are summed, and a pair's row is
// its expert's first row, plus those of the blocks before, plus the pairs before it
// within the block. Counts are whole numbers, so nothing depends on timing.
//
// Bound: latency for few tokens (one: 4.3 us, in one block that does everything; up to
// kAllTokens), instructions for many: 16384 tokens, top 8 of 256, sigmoid and bias, fp32 36 us (23
// without bias), of which the choice 31 (74 % of the issue slots; of its 1000 instructions a token
// a third are the sigmoids); gradient 6. The bytes would take 8.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "kp_moe.cuh"

namespace kp {

namespace {

constexpr int kThreads = 256;    // of the gradient's blocks
constexpr int kTokens = 16;      // of a block
constexpr int kChoosers = 32 * kTokens, kPlacers = 128;   // threads of a block that chooses, that places
constexpr int kScanExperts = 8;  // of a block that sums counts
constexpr int kSumBlocks = 32;   // whose counts a block that places sums itself (512 x 256, top 8: 10.9 us, summed before)
// Of the one block that does everything. Up to 64 tokens, since a call from the host then takes 11
// us instead of 19 (a launch and a workspace less); on the device alone it is behind from 32 on
// (64 experts, top 6: 5.7 us, 4.9 in several blocks; 64 tokens 7.5 and 5.2; 256 experts, top 8 10.7
// and 7.3; 1024, top 32 77 and 34, which the host does not hide).
constexpr int kAllThreads = 1024, kAllTokens = 64;

struct RouteParams {
    MoeRouteArgs a;
    int blocks;
    int32_t *counts;   // [blocks][E]: choices of a block, then of the blocks before it
    int32_t *totals;   // [E]
};

// A logit in fp32: NaN counts as minus infinity, plus infinity as the largest finite number.
__device__ __forceinline__ float logit_of(const void *p, int64_t i, int dtype) {
    const float v = dtype == KP_FP32 ? __ldg(static_cast<const float *>(p) + i)
                                     : elem_widen(__ldg(static_cast<const uint16_t *>(p) + i), dtype);
    return v != v ? -INFINITY : fminf(v, 3.402823466e38f);
}
// Bits that order like the value; 0 for minus infinity and NaN, which are not chosen.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);   // -0 like 0
    if (!(v > -INFINITY)) return 0;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));
    if (!(v > -INFINITY)) return 0;
    return b >> 63 ? ~b : b | 1ull << 63;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t v) { return __reduce_max_sync(0xFFFFFFFFu, v); }
__device__ __forceinline__ uint64_t warp_max(uint64_t v) {
    const uint32_t hi = warp_max(static_cast<uint32_t>(v >> 32));
    const uint32_t lo = warp_max(static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
    return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

// The k largest of the warp's keys (lane holds experts lane + 32 i), ties to the lowest
// expert: lane j gets the j-th one's expert (-1: there is none) and, with kGap, whether
// two of the k + 1 largest are nearer than fp32 sums of a score and a bias are exact.
// A lane has its two best ready, and looks for more when both are taken; what is taken
// lies above the last choice, so nothing is marked.
template <int NV, typename Key, bool kGap>
__device__ __forceinline__ int choose(const Key (&key)[NV], int k, int lane, bool &close) {
    int mine = -1;
    float last = 0.f;
    close = false;
    Key best = 0, next = 0;   // of this lane, 0: none; and their experts
    int at = lane, at_next = lane;
    auto put = [&](Key x, int e) {   // e ascending
        if (x > best)
            next = best, at_next = at, best = x, at = e;
        else if (x > next)
            next = x, at_next = e;
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) put(key[i], lane + 32 * i);
    for (int j = 0; j < k + (kGap ? 1 : 0); ++j) {
        const Key top = warp_max(best);
        if (top == 0) break;
        const int e = static_cast<int>(
            __reduce_min_sync(0xFFFFFFFFu, best == top ? static_cast<uint32_t>(at) : 0xFFFFFFFFu));
        if constexpr (kGap) {
            const float v = value_of(top);
            close = close || (j && last - v <= 2e-6f * fmaxf(1.f, fabsf(v)));
            last = v;
        }
        if (j < k && lane == j) mine = e;
        if (at == e && best == top) {
            best = next, at = at_next, next = 0;
            if (NV > 2 && best == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int x = lane + 32 * i;
                    if (key[i] < top || (key[i] == top && x > e)) put(key[i], x);
                }
            }
        }
    }
    return mine;
}

// The choice by sigmoid plus bias in 64 bits, for the few tokens that fp32 leaves open.
template <int NV>
__device__ __noinline__ int choose_exactly(const void *logits, int64_t row, const float *bias, int E, int k, int dtype,
                                            int lane) {
    uint64_t key[NV];
    bool close;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        const float v = e < E ? logit_of(logits, row + e, dtype) : -INFINITY;
        key[i] = v > -INFINITY ? order_key(1.0 / (1.0 + exp(-static_cast<double>(v))) + static_cast<double>(__ldg(bias + e)))
                               : 0;
    }
    return choose<NV, uint64_t, false>(key, k, lane, close);
}

// Experts and weights of a token; lane j < k gets the j-th.
template <int NV, bool kBias>
__device__ __forceinline__ void route_token(const MoeRouteArgs &a, int64_t t, int lane, int &id, float &w) {
    const int64_t row = t * a.ld;
    uint32_t key[NV];
    bool close;
    float x[NV];
    if (a.dtype == KP_FP32) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            x[i] = lane + 32 * i < a.E ? __ldg(static_cast<const float *>(a.logits) + row + lane + 32 * i) : -INFINITY;
    } else {
        uint16_t h[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            h[i] = lane + 32 * i < a.E ? __ldg(static_cast<const uint16_t *>(a.logits) + row + lane + 32 * i) : 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = lane + 32 * i < a.E ? elem_widen(h[i], a.dtype) : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 32 * i;
        const float v = x[i];
        key[i] = order_key(fminf(v, 3.402823466e38f));
        if (v != v) key[i] = 0;
        // By sigmoid plus bias: fp32 keys decide, off by less than 1e-6 (the exponential's
        // argument is rounded by at most 2^-24 |v|, a quarter of which reaches the score);
        // but where two of them lie so near each other that fp32 does not, the token is
        // chosen again in 64 bits (one in 2000 of 16384 tokens with 256 experts).
        if (kBias && e < a.E) {
            const uint32_t biased = order_key(__fdividef(1.f, 1.f + __expf(-v)) + __ldg(a.bias + e));
            key[i] = key[i] ? biased : 0;
        }
    }
    id = choose<NV, uint32_t, kBias>(key, a.k, lane, close);
    if (kBias && close) id = choose_exactly<NV>(a.logits, row, a.bias, a.E, a.k, a.dtype, lane);
    const float l = id >= 0 ? logit_of(a.logits, row + id, a.dtype) : -INFINITY;
    // the largest chosen logit
    const uint32_t most = warp_max(order_key(l));
    if (most == 0) {
        w = 0.f;
        return;
    }
    const float top = value_of(most);
    float s = 0.f;
    if (id >= 0) {
        if (a.score == KP_SCORE_SIGMOID) {
            // all scores times e^m, m = max(0, -top), so that they do not vanish together
            const float m = fmaxf(0.f, -top);
            s = 1.f / (expf(-m) + expf(-l - m));
        } else {
            s = expf(l - top);
        }
    }
    float sum = s;
#pragma unroll
    for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
    w = s / sum;
}

// Exclusive sums of n <= kMoeMaxExperts whole numbers in shared memory, by a block of kT
// threads; returns the sum of all.
template <int kT>
__device__ int block_scan(int32_t *v, int n, int32_t *sums) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int per = (n + kT - 1) / kT, at = threadIdx.x * per;
    int mine = 0;
    for (int i = 0; i < per; ++i)
        if (at + i < n) mine += v[at + i];
    int run = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, run, d);
        if (lane >= d) run += o;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kT / 32; ++i) {
        if (i < warp) before += sums[i];
        all += sums[i];
    }
    run += before - mine;
    for (int i = 0; i < per; ++i)
        if (at + i < n) {
            const int x = v[at + i];
            v[at + i] = run;
            run += x;
        }
    __syncthreads();
    return all;
}

// Rows of a block's choices: base[e] holds the first row of expert e for this block.
// Slots are taken kT at a time in order; cnt [kT / 32][E].
template <int kT>
__device__ void place(const RouteParams &p, int64_t first, int n, int32_t *base, int32_t *cnt) {
    const int E = p.a.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int s0 = 0; s0 < n; s0 += kT) {
        const int warps = min((n - s0 + 31) >> 5, kT / 32);
        for (int i = threadIdx.x; i < warps * E; i += kT) cnt[i] = 0;
        __syncthreads();
        const int i = s0 + threadIdx.x;
        const int e = i < n ? p.a.ids[first + i] : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
        const int before = __popc(same & ((1u << lane) - 1));
        if (e >= 0 && before == 0) cnt[warp * E + e] = __popc(same);
        __syncthreads();
        for (int x = threadIdx.x; x < E; x += kT) {
            int run = base[x];
            for (int q = 0; q < warps; ++q) {
                const int c = cnt[q * E + x];
                cnt[q * E + x] = run;
                run += c;
            }
            base[x] = run;
        }
        __syncthreads();
        if (i < n) {
            int r = -1;
            if (e >= 0) {
                r = cnt[warp * E + e] + before;
                p.a.order[r] = static_cast<int32_t>(first + i);
            }
            p.a.position[first + i] = r;
        }
        __syncthreads();
    }
}

extern __shared__ int32_t route_smem[];

// kAll: one block, which does everything.
template <int NV, bool kBias, bool kAll>
__global__ void __launch_bounds__(kAll ? kAllThreads : kChoosers, kAll || NV > 8 ? 1 : 3)
    route_kernel(const RouteParams p) {
    constexpr int kT = kAll ? kAllThreads : kChoosers;
    const MoeRouteArgs &a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int32_t *hist = route_smem;
    if (!kAll) pdl_trigger();   // the next kernel waits for this one all the same
    for (int i = threadIdx.x; i < a.E; i += kT) hist[i] = 0;
    __syncthreads();
    const int t0 = kAll ? 0 : static_cast<int>(blockIdx.x) * kTokens;
    const int t1 = kAll ? a.T : min(t0 + kTokens, a.T);
    for (int t = t0 + warp; t < t1; t += kT / 32) {
        int id;
        float w;
        route_token<NV, kBias>(a, t, lane, id, w);
        if (lane < a.k) {
            a.ids[static_cast<int64_t>(t) * a.k + lane] = id;
            a.weights[static_cast<int64_t>(t) * a.k + lane] = w;
            if (id >= 0) atomicAdd(hist + id, 1);
        }
    }
    __syncthreads();
    if constexpr (!kAll) {
        for (int i = threadIdx.x; i < a.E; i += kT) p.counts[static_cast<int64_t>(blockIdx.x) * a.E + i] = hist[i];
    } else {
        int32_t *sums = hist + a.E, *cnt = sums + kT / 32;
        const int rows = block_scan<kT>(hist, a.E, sums);
        for (int i = threadIdx.x; i < a.E; i += kT) a.offsets[i] = hist[i];
        if (threadIdx.x == 0) a.offsets[a.E] = rows;
        for (int i = rows + threadIdx.x; i < a.T * a.k; i += kT) a.order[i] = -1;
        __syncthreads();   // offsets are written from hist, which the placing moves on
        place<kT>(p, 0, a.T * a.k, hist, cnt);
    }
}

// counts[b][e] -> sum of counts[0 .. b)[e]: a block for eight experts, a warp's lanes
// eight experts by four runs of blocks.
__global__ void __launch_bounds__(1024) route_scan_kernel(const RouteParams p) {
    constexpr int kRuns = 1024 / kScanExperts;
    __shared__ int32_t part[kRuns][kScanExperts];
    const int E = p.a.E, x = threadIdx.x % kScanExperts, y = threadIdx.x / kScanExperts;
    const int e = blockIdx.x * kScanExperts + x;
    const int per = (p.blocks + kRuns - 1) / kRuns, b0 = y * per, b1 = min(b0 + per, p.blocks);
    int32_t *const at = p.counts + e;
    int sum = 0;
    if (e < E) {
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += at[static_cast<int64_t>(b) * E];
    }
    part[y][x] = sum;
    __syncthreads();
    if (threadIdx.x < 32 * kScanExperts) {   // a warp an expert: sums of the runs before each
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        int v[kRuns / 32], mine = 0;
#pragma unroll
        for (int i = 0; i < kRuns / 32; ++i) v[i] = part[lane * (kRuns / 32) + i][w], mine += v[i];
        int run = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, run, d);
            if (lane >= d) run += o;
        }
        if (lane == 31 && blockIdx.x * kScanExperts + w < E) p.totals[blockIdx.x * kScanExperts + w] = run;
        run -= mine;
#pragma unroll
        for (int i = 0; i < kRuns / 32; ++i) {
            part[lane * (kRuns / 32) + i][w] = run;
            run += v[i];
        }
    }
    __syncthreads();
    if (e < E) {
        int run = part[y][x];
#pragma unroll 8
        for (int b = b0; b < b1; ++b) {
            const int c = at[static_cast<int64_t>(b) * E];
            at[static_cast<int64_t>(b) * E] = run;
            run += c;
        }
    }
}

// kSum: sums the few blocks' counts itself.
template <bool kSum>
__global__ void __launch_bounds__(kPlacers) route_place_kernel(const RouteParams p) {
    const MoeRouteArgs &a = p.a;
    int32_t *base = route_smem, *sums = base + a.E, *cnt = sums + kPlacers / 32;
    pdl_wait();
    for (int i = threadIdx.x; i < a.E; i += kPlacers) {
        if constexpr (kSum) {
            int all = 0, before = 0;
#pragma unroll 16
            for (int b = 0; b < p.blocks; ++b) {
                const int c = p.counts[static_cast<int64_t>(b) * a.E + i];
                all += c;
                before += b < static_cast<int>(blockIdx.x) ? c : 0;
            }
            base[i] = all;
            cnt[i] = before;   // (as many as experts: the placing clears it)
        } else {
            base[i] = p.totals[i];
        }
    }
    __syncthreads();
    const int rows = block_scan<kPlacers>(base, a.E, sums);
    if (blockIdx.x == 0) {
        for (int i = threadIdx.x; i < a.E; i += kPlacers) a.offsets[i] = base[i];
        if (threadIdx.x == 0) a.offsets[a.E] = rows;
    }
    const int64_t slots = static_cast<int64_t>(a.T) * a.k;
    for (int64_t i = rows + static_cast<int64_t>(blockIdx.x) * kPlacers + threadIdx.x; i < slots;
         i += static_cast<int64_t>(gridDim.x) * kPlacers)
        a.order[i] = -1;
    __syncthreads();   // offsets are written from base, which the placing moves on
    for (int i = threadIdx.x; i < a.E; i += kPlacers)
        base[i] += kSum ? cnt[i] : p.counts[static_cast<int64_t>(blockIdx.x) * a.E + i];
    __syncthreads();
    const int t0 = static_cast<int>(blockIdx.x) * kTokens;
    place<kPlacers>(p, static_cast<int64_t>(t0) * a.k, min(kTokens, a.T - t0) * a.k, base, cnt);
}

// dlogits: a warp a token. With w the weights and d = dw - sum_j w_j dw_j a chosen
// expert gets w d (softmax) or w d (1 - s) (sigmoid); the others get 0.
__global__ void __launch_bounds__(kThreads)
    route_backward_kernel(const float *__restrict__ dweights, const void *__restrict__ logits, int64_t ld,
                          const int32_t *__restrict__ ids, const float *__restrict__ weights, void *__restrict__ dlogits,
                          int64_t ldd, int T, int E, int k, int score, int dtype) {
    const int lane = threadIdx.x & 31;
    const int es = dtype == KP_FP32 ? 4 : 2;
    for (int64_t t = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; t < T;
         t += (static_cast<int64_t>(gridDim.x) * kThreads) >> 5) {
        int id = -1;
        float w = 0.f, dw = 0.f;
        if (lane < k) {
            id = __ldg(ids + t * k + lane);
            if (id >= E) id = -1;
            w = id >= 0 ? __ldg(weights + t * k + lane) : 0.f;
            dw = id >= 0 ? __ldg(dweights + t * k + lane) : 0.f;
        }
        float sum = w * dw;
#pragma unroll
        for (int i = 16; i; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        float d = w * (dw - sum);
        if (score == KP_SCORE_SIGMOID && id >= 0) d *= 1.f / (1.f + expf(logit_of(logits, t * ld + id, dtype)));   // 1 - s
        // zeros in the row, then the chosen experts' over them
        const int64_t at = t * ldd;
        char *out = static_cast<char *>(dlogits) + at * es;
        const int bytes = E * es;
        int head = static_cast<int>(-reinterpret_cast<intptr_t>(out) & 15);
        head = min(head, bytes);
        const int body = (bytes - head) >> 4;
        for (int i = lane; i < body; i += 32) reinterpret_cast<uint4 *>(out + head)[i] = make_uint4(0, 0, 0, 0);
        const int edge = bytes - 16 * body;   // bytes before and behind
        for (int i = lane * 2; i < edge; i += 64)
            *reinterpret_cast<uint16_t *>(out + (i < head ? i : 16 * body + i)) = 0;
        __syncwarp();
        if (id >= 0) {
            if (dtype == KP_FP32)
                static_cast<float *>(dlogits)[at + id] = d;
            else
                static_cast<uint16_t *>(dlogits)[at + id] = elem_round(d, dtype);
        }
    }
}

// Shared memory of a block that places `slots` choices: base, the scan's sums, and each
// warp's counts by expert.
size_t place_smem(int threads, int E, int64_t slots) {
    const int warps = static_cast<int>(std::min<int64_t>((slots + 31) / 32, threads / 32));
    return (static_cast<size_t>(E) * (1 + warps) + threads / 32) * sizeof(int32_t);
}

std::mutex g_mu;
bool g_ready[64];   // devices whose kernels of one block have their shared memory raised

int blocks_of(int T) { return T <= kAllTokens ? 1 : (T + kTokens - 1) / kTokens; }

}  // namespace

size_t moe_route_scratch(int T, int E) {
    const int b = blocks_of(T);
    return b > 1 ? (static_cast<size_t>(b) + 1) * E * sizeof(int32_t) : 0;
}

cudaError_t moe_route_launch(const MoeRouteArgs &a, const FfnDev &d, cudaStream_t s) {
    using Fn = void (*)(RouteParams);
    auto pick = [](auto all, bool bias, int v) -> Fn {   // of 32 << v experts
        constexpr bool kAll = decltype(all)::value;
        static const Fn kernels[2][6] = {
            {route_kernel<1, false, kAll>, route_kernel<2, false, kAll>, route_kernel<4, false, kAll>,
             route_kernel<8, false, kAll>, route_kernel<16, false, kAll>, route_kernel<32, false, kAll>},
            {route_kernel<1, true, kAll>, route_kernel<2, true, kAll>, route_kernel<4, true, kAll>,
             route_kernel<8, true, kAll>, route_kernel<16, true, kAll>, route_kernel<32, true, kAll>}};
        return kernels[bias][v];
    };
    const bool bias = a.bias != nullptr;
    int v = 0;
    while (32 << v < a.E) ++v;
    RouteParams p;
    p.a = a;
    p.blocks = blocks_of(a.T);
    p.counts = static_cast<int32_t *>(a.work);
    p.totals = p.blocks > 1 ? p.counts + static_cast<int64_t>(p.blocks) * a.E : nullptr;
    if (p.blocks == 1) {
        const size_t smem = place_smem(kAllThreads, a.E, static_cast<int64_t>(a.T) * a.k);
        if (smem > 48 * 1024) {
            // once, to the most that a kernel may need: a limit set for this call would be
            // lowered by a call with fewer tokens on another thread before this one's launch
            std::lock_guard<std::mutex> lk(g_mu);
            if (d.dev >= 64 || !g_ready[d.dev]) {
                for (int i = 0; 32 << i <= kMoeMaxExperts; ++i) {
                    const size_t most = place_smem(kAllThreads, 32 << i, kAllTokens * kMoeMaxTopK);
                    for (const bool b : {false, true}) {
                        if (most <= 48 * 1024) continue;
                        const cudaError_t e = cudaFuncSetAttribute(pick(std::true_type(), b, i), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                   static_cast<int>(most));
                        if (e != cudaSuccess) return e;
                    }
                }
                if (d.dev < 64) g_ready[d.dev] = true;
            }
        }
        pick(std::true_type(), bias, v)<<<1, kAllThreads, smem, s>>>(p);
        return cudaGetLastError();
    }
    pick(std::false_type(), bias, v)<<<p.blocks, kChoosers, a.E * sizeof(int32_t), s>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const size_t smem = place_smem(kPlacers, a.E, static_cast<int64_t>(kTokens) * a.k);
    if (p.blocks > kSumBlocks) {
        route_scan_kernel<<<(a.E + kScanExperts - 1) / kScanExperts, 1024, 0, s>>>(p);
        route_place_kernel<false><<<p.blocks, kPlacers, smem, s>>>(p);
        return cudaGetLastError();
    }
    // Launched programmatically behind the choice, whose few blocks leave room beside them (in
    // front of many blocks it takes their place while it waits: 16384 x 256 38 -> 46 us).
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.blocks), 1, 1);
    cfg.blockDim = dim3(kPlacers, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_place_kernel<true>, p);
}

cudaError_t moe_route_backward_launch(const float *dweights, const void *logits, int64_t ld, const int32_t *ids,
                                      const float *weights, void *dlogits, int64_t ldd, int T, int E, int k,
                                      int score, int dtype, const FfnDev &d, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(T) + kThreads / 32 - 1) / (kThreads / 32);
    route_backward_kernel<<<static_cast<int>(std::min<int64_t>(blocks, static_cast<int64_t>(d.sms) * 8)), kThreads, 0, s>>>(
        dweights, logits, ld, ids, weights, dlogits, ldd, T, E, k, score, dtype);
    return cudaGetLastError();
}

}  // namespace kp
