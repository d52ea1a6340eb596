// Shared parts of the mixture-of-experts operators: the router (kp_moe_route.cu), the
// rows' way to their experts and back (kp_moe_rows.cu) and the products grouped by
// expert (kp_moe_tile.cu), behind kp_moe_api.cu.
#pragma once

#include "kp_ffn.cuh"

namespace kp {

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeMaxTopK = 32;

// ---- router ---------------------------------------------------------------------
struct MoeRouteArgs {
    const void *logits = nullptr;
    int64_t ld = 0;
    const float *bias = nullptr;   // [E] or NULL
    int T = 0, E = 0, k = 0, score = 0, dtype = KP_BF16;
    int32_t *ids = nullptr;        // [T, k]
    float *weights = nullptr;      // [T, k]
    int32_t *offsets = nullptr;    // [E + 1]
    int32_t *order = nullptr;      // [T k]
    int32_t *position = nullptr;   // [T, k]
    void *work = nullptr;
};
size_t moe_route_scratch(int T, int E);   // bytes of work
cudaError_t moe_route_launch(const MoeRouteArgs &a, const FfnDev &d, cudaStream_t s);
cudaError_t moe_route_backward_launch(const float *dweights, const void *logits, int64_t ld, const int32_t *ids,
                                      const float *weights, void *dlogits, int64_t ldd, int T, int E, int k,
                                      int score, int dtype, const FfnDev &d, cudaStream_t s);

// ---- rows -------------------------------------------------------------------------
// rows[position[t, s]] = x[t]
cudaError_t moe_dispatch_launch(const void *x, int64_t ldx, const int32_t *position, void *rows, int64_t ldr, int T,
                                int k, int K, const FfnDev &d, cudaStream_t s);
// y[t] = round(sum_s weights[t, s] rows[position[t, s]]); weights NULL: ones
cudaError_t moe_combine_launch(const void *rows, int64_t ldr, const float *weights, const int32_t *position, void *y,
                               int64_t ldy, int T, int k, int K, int dtype, const FfnDev &d, cudaStream_t s);
cudaError_t moe_combine_backward_launch(const void *dy, int64_t lddy, const void *rows, int64_t ldr,
                                        const float *weights, const int32_t *position, void *drows, int64_t lddr,
                                        float *dweights, int T, int k, int K, int dtype, const FfnDev &d,
                                        cudaStream_t s);

// ---- grouped products ---------------------------------------------------------------
// The matrices of all experts: [E][rows][cols], row stride ld, expert stride se.
struct MoeMat {
    const void *p = nullptr;
    int64_t ld = 0, se = 0;
};
enum GroupedForm {
    GROUPED_PLAIN,     // y[r] = x[r] W_e^T
    GROUPED_GATED,     // h[r] = act(x[r] Wg_e^T) * (x[r] Wu_e^T); g, u
    GROUPED_BACKWARD   // dx[r] = d0[r] W0_e (+ d1[r] W1_e); dW0_e = d0^T x over the expert's rows (and dW1_e = d1^T x)
};
struct GroupedArgs {
    int form = GROUPED_PLAIN;
    int act = 0, dtype = KP_BF16;
    const int32_t *offsets = nullptr;
    int R = 0, E = 0, N = 0, K = 0;      // rows, experts, features, columns of x
    const void *x = nullptr;             // [R, K]
    int64_t ldx = 0;
    MoeMat w0, w1;                       // [E][N][K]
    const void *d0 = nullptr, *d1 = nullptr;   // backward: [R, N]; d1 may be NULL
    int64_t ldd = 0;
    void *y = nullptr;                   // y, h, dx
    int64_t ldy = 0;
    void *dw0 = nullptr, *dw1 = nullptr; // backward: [E][N][K], contiguous
    float *g = nullptr, *u = nullptr;    // gated: [R, N]
    const float *scale = nullptr;        // backward: device factor of every sum (NULL: 1)
    bool pdl = false;                    // launched behind a kernel that writes only d0, d1 and scale
    int *err = nullptr;
};
cudaError_t grouped_launch(const GroupedArgs &a, const FfnDev &d, cudaStream_t s);

}  // namespace kp
