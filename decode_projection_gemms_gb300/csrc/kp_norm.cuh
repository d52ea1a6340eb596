// Layer norm and its gradients (kp_norm.cu).
#pragma once

#include "kp_ffn.cuh"

namespace kp {

constexpr int kNormMaxCols = 16384;

struct NormArgs {
    const void *x = nullptr, *w = nullptr, *b = nullptr;   // [T, K]; [K], b may be NULL
    const void *dy = nullptr;                              // backward: [T, K]
    void *y = nullptr;                                     // y; backward: dx
    float *mean = nullptr, *rstd = nullptr;                // [T], forward: may be NULL
    void *dw = nullptr, *dbias = nullptr;                  // backward: [K], dbias may be NULL
    float *part = nullptr;                                 // backward: workspace
    int64_t ldx = 0, ldy = 0, lddy = 0;
    int T = 0, K = 0, dtype = KP_BF16;
    bool center = true;
    float eps = 0.f;
};
size_t norm_backward_scratch(int T, int K, int sms);   // bytes of part
cudaError_t norm_launch(const NormArgs &a, cudaStream_t s);
cudaError_t norm_backward_launch(const NormArgs &a, const FfnDev &d, cudaStream_t s);

}  // namespace kp
