// Gradients of the gated block's two products, element by element:
//     dU = dh act(g),   dG = dh u act'(g).
// Three matrices read and two written, nothing reused: bound by HBM (T = 4003, F =
// 2048: 115 MB in 17 us). A thread takes eight columns. They are
// rounded to 16 bits because the tensor cores of the three products behind them
// read 16-bit operands; everything before that rounding is fp32, g and u included:
// with those saved in bf16 the gradients were 1.8 times as far from the formula as
// the rounding of a gradient alone, so 1.4 times. That rounding is the price of one
// product per gradient: with the operands in two 16-bit parts each there would be two.
//
// fp16 operands: dh u act'(g) passes 65504, or falls to subnormals, where the
// products behind it do not. A first pass finds the largest finite magnitude of both
// matrices (a maximum, so the order does not matter), and both are rounded as
// multiples of one power of two that takes it to [2^14, 2^15); the products' fp32 sums
// are multiplied back. One factor for both, because dx adds the two products, and for
// all rows and columns, because the products run along either. Scaling is exact, and
// elements down to 2^-28 of the largest keep fp16's relative precision. The pass adds
// 4 us to a training step of T = 333, F = 1416, K = 2048 (34.3 -> 38.1), 19 us at T =
// 4003, F = 2048 (cold).
#include "kp_ffn.cuh"

namespace kp {

namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 8;

// Eight columns of a row of dh, g and u, zeros past F.
struct Chunk {
    union {
        uint4 v;
        uint16_t h[8];
    } a;
    union {
        float4 v[2];
        float f[8];
    } b, c;
    __device__ void load(const uint16_t *dh, const float *g, const float *u, int f, int F, int vec) {
        if (vec) {
            a.v = __ldg(reinterpret_cast<const uint4 *>(dh + f));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                b.v[k] = __ldg(reinterpret_cast<const float4 *>(g + f) + k);
                c.v[k] = __ldg(reinterpret_cast<const float4 *>(u + f) + k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool in = f + k < F;
                a.h[k] = in ? dh[f + k] : 0;
                b.f[k] = in ? g[f + k] : 0.f;
                c.f[k] = in ? u[f + k] : 0.f;
            }
        }
    }
    // dG and dU of column k
    template <int kAct>
    __device__ void grads(int k, int dtype, float &dg, float &du) const {
        const float d = elem_widen(a.h[k], dtype);
        float av, dav;
        ffn_act_grad<kAct>(b.f[k], av, dav);
        du = d * av;
        dg = d * c.f[k] * dav;
    }
};

// The larger of two magnitudes' bits (ordered like magnitudes), infinity and NaN left out.
__device__ __forceinline__ uint32_t finite_max(uint32_t m, float v) {
    const uint32_t b = __float_as_uint(v) & 0x7FFFFFFFu;
    return b < 0x7F800000u ? max(m, b) : m;
}
// The largest of all threads' m, for thread 0.
__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t *sh) {
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x < 32) m = __reduce_max_sync(0xFFFFFFFFu, threadIdx.x < kThreads / 32 ? sh[threadIdx.x] : 0u);
    return m;
}

// Rows that hold anything.
__device__ __forceinline__ int64_t used_rows(const int32_t *rows, int T) {
    return rows ? min(max(__ldg(rows), 0), T) : T;
}

// Each block's largest finite |dG|, |dU| (bits), to top[block].
template <int kAct>
__global__ void __launch_bounds__(kThreads)
    gate_max_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ g,
                    const float *__restrict__ u, uint32_t *__restrict__ top, int T, int F, int dtype, int vec,
                    const int32_t *__restrict__ rows) {
    __shared__ uint32_t sh[kThreads / 32];
    const int chunks = (F + 7) >> 3;
    const int64_t total = used_rows(rows, T) * chunks;
    uint32_t m = 0;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / chunks;
        const int f = static_cast<int>(i - t * chunks) * 8;
        Chunk e;
        e.load(dh + t * lddh, g + t * F, u + t * F, f, F, vec);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float dg, du;
            e.grads<kAct>(k, dtype, dg, du);
            m = finite_max(finite_max(m, dg), du);
        }
    }
    m = block_max(m, sh);
    if (threadIdx.x == 0) top[blockIdx.x] = m;
}

// tops: blocks of the first pass, whose maxima are in top (0: no scaling). The factor
// that the products' sums are multiplied with goes to *back.
template <int kAct>
__global__ void __launch_bounds__(kThreads)
    gate_grad_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ g,
                     const float *__restrict__ u, uint16_t *__restrict__ dg, uint16_t *__restrict__ du,
                     int64_t ld, const uint32_t *__restrict__ top, int tops, float *__restrict__ back, int T, int F,
                     int dtype, int vec, const int32_t *__restrict__ rows) {
    pdl_trigger();   // a product launched programmatically behind this waits for it all the same
    float scale = 1.f;
    if (tops) {
        __shared__ uint32_t sh[kThreads / 32];
        __shared__ float sh_scale;
        uint32_t m = 0;
        for (int i = threadIdx.x; i < tops; i += kThreads) m = max(m, top[i]);
        m = block_max(m, sh);
        if (threadIdx.x == 0) {
            // the largest in [2^14, 2^15); both factors normal. All zero: nothing to scale.
            const int e = m ? min(14 + 127 - static_cast<int>(m >> 23), 126) : 0;
            sh_scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
            if (blockIdx.x == 0) *back = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        }
        __syncthreads();
        scale = sh_scale;
    }
    const int chunks = (F + 7) >> 3;
    const int64_t total = used_rows(rows, T) * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * kThreads) {
        const int64_t t = i / chunks;
        const int f = static_cast<int>(i - t * chunks) * 8;
        Chunk e;
        e.load(dh + t * lddh, g + t * F, u + t * F, f, F, vec);
        union {
            uint4 v;
            uint16_t h[8];
        } og, ou;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float a, b;
            e.grads<kAct>(k, dtype, a, b);
            og.h[k] = elem_round(a * scale, dtype);
            ou.h[k] = elem_round(b * scale, dtype);
        }
        // ld is a multiple of 8 and both buffers have its padding
        *reinterpret_cast<uint4 *>(dg + t * ld + f) = og.v;
        *reinterpret_cast<uint4 *>(du + t * ld + f) = ou.v;
    }
}

template <int kAct>
cudaError_t launch(const uint16_t *dh, int64_t lddh, const float *g, const float *u, uint16_t *dg, uint16_t *du,
                   int64_t ld, float *scaling, int T, int F, int dtype, int grid, int vec, const int32_t *rows, cudaStream_t s) {
    uint32_t *top = scaling ? reinterpret_cast<uint32_t *>(scaling) + 1 : nullptr;
    if (scaling) {
        gate_max_kernel<kAct><<<grid, kThreads, 0, s>>>(dh, lddh, g, u, top, T, F, dtype, vec, rows);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    gate_grad_kernel<kAct><<<grid, kThreads, 0, s>>>(dh, lddh, g, u, dg, du, ld, top, scaling ? grid : 0, scaling, T, F,
                                                     dtype, vec, rows);
    return cudaGetLastError();
}

}  // namespace

size_t ffn_gate_grad_scratch(int sms) { return (static_cast<size_t>(sms) * kBlocksPerSm + 1) * sizeof(float); }

cudaError_t ffn_gate_grad_launch(const void *dh, int64_t lddh, const float *g, const float *u, void *dg, void *du,
                                 int64_t ld, float *scaling, int T, int F, int act, int dtype, int sms,
                                 cudaStream_t s, const int32_t *rows) {
    const int64_t total = static_cast<int64_t>(T) * ((F + 7) / 8);
    const int64_t blocks = (total + kThreads - 1) / kThreads;
    const int64_t most = static_cast<int64_t>(sms) * kBlocksPerSm;
    const int grid = static_cast<int>(blocks < most ? blocks : most);
    const bool vec = F % 8 == 0 && lddh % 8 == 0 && (reinterpret_cast<uintptr_t>(dh) & 15) == 0;
    auto go = act == KP_ACT_SILU ? launch<KP_ACT_SILU> : act == KP_ACT_GELU ? launch<KP_ACT_GELU> : launch<KP_ACT_GELU_TANH>;
    return go(static_cast<const uint16_t *>(dh), lddh, g, u, static_cast<uint16_t *>(dg), static_cast<uint16_t *>(du), ld,
              scaling, T, F, dtype, grid, vec, rows, s);
}

}  // namespace kp
