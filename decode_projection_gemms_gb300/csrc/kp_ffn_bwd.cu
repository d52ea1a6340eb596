// Gradients of the gated block's two products, element by element:
//     dU = dh act(g),   dG = dh u act'(g).
// Three matrices read and two written, nothing reused: bound by HBM (T = 4003, F =
// 2048: 115 MB in 17 us). A thread takes eight columns. They are
// rounded to 16 bits because the tensor cores of the three products behind them
// read 16-bit operands; everything before that rounding is fp32, g and u included:
// with those saved in bf16 the gradients were 1.8 times as far from the formula as
// the rounding of a gradient alone, so 1.4 times.
#include "kp_ffn.cuh"

namespace kp {

namespace {

template <int kAct>
__global__ void __launch_bounds__(256)
    gate_grad_kernel(const uint16_t *__restrict__ dh, int64_t lddh, const float *__restrict__ g,
                     const float *__restrict__ u, uint16_t *__restrict__ dg, uint16_t *__restrict__ du,
                     int64_t ld, int T, int F, int dtype, int vec) {
    const int chunks = (F + 7) >> 3;
    const int64_t total = static_cast<int64_t>(T) * chunks;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(gridDim.x) * 256) {
        const int64_t t = i / chunks;
        const int f = static_cast<int>(i - t * chunks) * 8;
        union {
            uint4 v;
            uint16_t h[8];
        } a, og, ou;
        union {
            float4 v[2];
            float f[8];
        } b, c;
        if (vec) {
            a.v = __ldg(reinterpret_cast<const uint4 *>(dh + t * lddh + f));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                b.v[k] = __ldg(reinterpret_cast<const float4 *>(g + t * F + f) + k);
                c.v[k] = __ldg(reinterpret_cast<const float4 *>(u + t * F + f) + k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const bool in = f + k < F;
                a.h[k] = in ? dh[t * lddh + f + k] : 0;
                b.f[k] = in ? g[t * F + f + k] : 0.f;
                c.f[k] = in ? u[t * F + f + k] : 0.f;
            }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float d = elem_widen(a.h[k], dtype);
            float av, dav;
            ffn_act_grad<kAct>(b.f[k], av, dav);
            ou.h[k] = elem_round(d * av, dtype);
            og.h[k] = elem_round(d * c.f[k] * dav, dtype);
        }
        // ld is a multiple of 8 and both buffers have its padding
        *reinterpret_cast<uint4 *>(dg + t * ld + f) = og.v;
        *reinterpret_cast<uint4 *>(du + t * ld + f) = ou.v;
    }
}

}  // namespace

cudaError_t ffn_gate_grad_launch(const void *dh, int64_t lddh, const float *g, const float *u, void *dg, void *du,
                                 int64_t ld, int T, int F, int act, int dtype, int sms, cudaStream_t s) {
    const int64_t total = static_cast<int64_t>(T) * ((F + 7) / 8);
    const int64_t blocks = (total + 255) / 256;
    const int grid = static_cast<int>(blocks < sms * 8LL ? blocks : sms * 8LL);
    const bool vec = F % 8 == 0 && lddh % 8 == 0 && (reinterpret_cast<uintptr_t>(dh) & 15) == 0;
    using Fn = void (*)(const uint16_t *, int64_t, const float *, const float *, uint16_t *, uint16_t *, int64_t, int,
                        int, int, int);
    static const Fn kernels[] = {gate_grad_kernel<KP_ACT_SILU>, gate_grad_kernel<KP_ACT_GELU>,
                                 gate_grad_kernel<KP_ACT_GELU_TANH>};
    kernels[act]<<<grid, 256, 0, s>>>(static_cast<const uint16_t *>(dh), lddh, g, u, static_cast<uint16_t *>(dg),
                                      static_cast<uint16_t *>(du), ld, T, F, dtype, vec);
    return cudaGetLastError();
}

}  // namespace kp
