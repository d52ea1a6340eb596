// The rows' way to their experts and back: copies of tokens' rows in expert order, and
// weighted sums of the experts' rows of a token, with their gradients.
//
// Nothing is reused but a token's row, so all of them are bound by HBM (8192 tokens, 4
// slots, K = 4096, bf16: 335 MB in 61 us there and in 58 back; 604 MB in 97 for the gradients of the
// way back). A thread takes 16 bytes of a token for all of its slots.
#include <algorithm>

#include "kp_moe.cuh"

namespace kp {

namespace {

constexpr int kThreads = 256;

// Eight elements of a 16-bit row from c on, zeros past K.
struct Piece {
    uint4 v;
    __device__ void load(const uint16_t *row, int c, int K, bool vec) {
        if (vec) {
            v = __ldg(reinterpret_cast<const uint4 *>(row + c));
            return;
        }
        uint16_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = c + i < K ? row[c + i] : 0;
        v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
    }
    __device__ void store(uint16_t *row, int c, int K, bool vec) const {
        if (vec) {
            *reinterpret_cast<uint4 *>(row + c) = v;
            return;
        }
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < K) row[c + i] = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
    }
    __device__ void widen(float (&f)[8], int dtype) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = elem_widen(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))), dtype);
    }
    __device__ void round(const float (&f)[8], int dtype) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = elem_round(f[2 * i], dtype) | static_cast<uint32_t>(elem_round(f[2 * i + 1], dtype)) << 16;
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// position holds rows within [0, T k) or -1; anything else is taken for -1.
__device__ __forceinline__ int row_at(const int32_t *position, int64_t slot, int64_t slots) {
    const int r = __ldg(position + slot);
    return r < slots ? r : -1;
}

__global__ void __launch_bounds__(kThreads)
    dispatch_kernel(const uint16_t *__restrict__ x, int64_t ldx, const int32_t *__restrict__ position,
                    uint16_t *__restrict__ rows, int64_t ldr, int T, int k, int K, int vec) {
    const int chunks = (K + 7) >> 3;
    const int64_t total = static_cast<int64_t>(T) * chunks, slots = static_cast<int64_t>(T) * k;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / chunks;
        const int c = static_cast<int>(i - t * chunks) * 8;
        Piece v;
        v.load(x + t * ldx, c, K, vec);
        for (int s = 0; s < k; ++s) {
            const int r = row_at(position, t * k + s, slots);
            if (r >= 0) v.store(rows + r * ldr, c, K, vec);
        }
    }
}

__global__ void __launch_bounds__(kThreads)
    combine_kernel(const uint16_t *__restrict__ rows, int64_t ldr, const float *__restrict__ weights,
                   const int32_t *__restrict__ position, uint16_t *__restrict__ y, int64_t ldy, int T, int k, int K,
                   int dtype, int vec) {
    const int chunks = (K + 7) >> 3;
    const int64_t total = static_cast<int64_t>(T) * chunks, slots = static_cast<int64_t>(T) * k;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / chunks;
        const int c = static_cast<int>(i - t * chunks) * 8;
        float sum[8] = {};
        for (int s = 0; s < k; ++s) {
            const int64_t slot = t * k + s;
            const int r = row_at(position, slot, slots);
            if (r < 0) continue;
            const float w = weights ? __ldg(weights + slot) : 1.f;
            Piece v;
            v.load(rows + r * ldr, c, K, vec);
            float f[8];
            v.widen(f, dtype);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] = fmaf(w, f[j], sum[j]);
        }
        Piece out;
        out.round(sum, dtype);
        out.store(y + t * ldy, c, K, vec);
    }
}

// A warp a slot: its row's gradient and the dot product of the output's gradient with
// the row, which is the weight's. Two pieces of both rows at a time (with one, 2048 tokens, 2
// slots, K = 7168: 31.7 us instead of 26.9; 8192 tokens, 8 slots, K = 4096, on the other hand, 174
// instead of 184).
__global__ void __launch_bounds__(kThreads)
    combine_backward_kernel(const uint16_t *__restrict__ dy, int64_t lddy, const uint16_t *__restrict__ rows,
                            int64_t ldr, const float *__restrict__ weights, const int32_t *__restrict__ position,
                            uint16_t *__restrict__ drows, int64_t lddr, float *__restrict__ dweights, int T, int k,
                            int K, int dtype, int vec) {
    const int64_t slots = static_cast<int64_t>(T) * k;
    const int lane = threadIdx.x & 31;
    for (int64_t slot = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 5; slot < slots;
         slot += (static_cast<int64_t>(gridDim.x) * kThreads) >> 5) {
        const int r = row_at(position, slot, slots);
        float dot = 0.f;
        if (r >= 0) {
            const int64_t t = slot / k;
            const float w = __ldg(weights + slot);
            for (int c0 = lane * 8; c0 < K; c0 += 512) {   // two pieces of both rows on their way
                Piece a[2], b[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = c0 + 256 * i;
                    if (c >= K) break;
                    a[i].load(dy + t * lddy, c, K, vec);
                    b[i].load(rows + r * ldr, c, K, vec);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = c0 + 256 * i;
                    if (c >= K) break;
                    float fa[8], fb[8];
                    a[i].widen(fa, dtype);
                    b[i].widen(fb, dtype);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        dot = fmaf(fa[j], fb[j], dot);
                        fa[j] *= w;
                    }
                    a[i].round(fa, dtype);
                    a[i].store(drows + r * lddr, c, K, vec);
                }
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, m);
        }
        if (lane == 0) dweights[slot] = dot;
    }
}

bool rows16(const void *p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; }

int grid_for(int64_t threads, int sms) {
    return static_cast<int>(std::min<int64_t>((threads + kThreads - 1) / kThreads, static_cast<int64_t>(sms) * 8));
}

}  // namespace

cudaError_t moe_dispatch_launch(const void *x, int64_t ldx, const int32_t *position, void *rows, int64_t ldr, int T,
                                int k, int K, const FfnDev &d, cudaStream_t s) {
    const int vec = K % 8 == 0 && rows16(x, ldx) && rows16(rows, ldr);
    dispatch_kernel<<<grid_for(static_cast<int64_t>(T) * ((K + 7) / 8), d.sms), kThreads, 0, s>>>(
        static_cast<const uint16_t *>(x), ldx, position, static_cast<uint16_t *>(rows), ldr, T, k, K, vec);
    return cudaGetLastError();
}

cudaError_t moe_combine_launch(const void *rows, int64_t ldr, const float *weights, const int32_t *position, void *y,
                               int64_t ldy, int T, int k, int K, int dtype, const FfnDev &d, cudaStream_t s) {
    const int vec = K % 8 == 0 && rows16(y, ldy) && rows16(rows, ldr);
    combine_kernel<<<grid_for(static_cast<int64_t>(T) * ((K + 7) / 8), d.sms), kThreads, 0, s>>>(
        static_cast<const uint16_t *>(rows), ldr, weights, position, static_cast<uint16_t *>(y), ldy, T, k, K, dtype,
        vec);
    return cudaGetLastError();
}

cudaError_t moe_combine_backward_launch(const void *dy, int64_t lddy, const void *rows, int64_t ldr,
                                        const float *weights, const int32_t *position, void *drows, int64_t lddr,
                                        float *dweights, int T, int k, int K, int dtype, const FfnDev &d,
                                        cudaStream_t s) {
    const int vec = K % 8 == 0 && rows16(dy, lddy) && rows16(rows, ldr) && rows16(drows, lddr);
    combine_backward_kernel<<<grid_for(static_cast<int64_t>(T) * k * 32, d.sms), kThreads, 0, s>>>(
        static_cast<const uint16_t *>(dy), lddy, static_cast<const uint16_t *>(rows), ldr, weights, position,
        static_cast<uint16_t *>(drows), lddr, dweights, T, k, K, dtype, vec);
    return cudaGetLastError();
}

}  // namespace kp
