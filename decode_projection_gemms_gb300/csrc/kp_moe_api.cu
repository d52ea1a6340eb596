// C entry points of the mixture-of-experts operators and of the layer norm in front of
// them (include/kdaproj.h): argument
// checks, workspace layout and the order of their launches. Nothing throws and nothing
// is kept between calls; the caller owns every buffer.
#include <cmath>

#include "kp_moe.cuh"
#include "kp_norm.cuh"

namespace kp {

static int cuda_failed(cudaError_t e, const char *what) {
    return set_error(KP_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}
static bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
static bool is16(int dtype) { return dtype == KP_BF16 || dtype == KP_FP16; }
static bool is_act(int act) { return act == KP_ACT_SILU || act == KP_ACT_GELU || act == KP_ACT_GELU_TANH; }
static size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// A matrix of 16-bit elements that a kernel reads or writes element by element.
static int check_rows(const char *fn, const char *name, const void *p, int64_t ld, int cols) {
    if (!p) return set_error(KP_EINVAL, "%s: %s is NULL", fn, name);
    if (misaligned(p, 2)) return set_error(KP_EALIGN, "%s: %s must be 2-byte aligned", fn, name);
    if (ld < cols) return set_error(KP_EINVAL, "%s: %s's row stride %lld is below its %d columns", fn, name,
                                    static_cast<long long>(ld), cols);
    return KP_OK;
}
// One that is read through a tensor map: 16-byte rows.
static int check_operand(const char *fn, const char *name, const void *p, int64_t ld, int cols) {
    const int rc = check_rows(fn, name, p, ld, cols);
    if (rc) return rc;
    if (misaligned(p, 16)) return set_error(KP_EALIGN, "%s: %s must be 16-byte aligned", fn, name);
    if (ld & 7) return set_error(KP_ESHAPE, "%s: %s's row stride %lld is not a multiple of 8", fn, name,
                                 static_cast<long long>(ld));
    return KP_OK;
}
// All experts' matrices [E][rows][cols].
static int check_experts(const char *fn, const char *name, const void *p, int64_t ld, int64_t se, int E, int rows,
                         int cols) {
    const int rc = check_operand(fn, name, p, ld, cols);
    if (rc) return rc;
    if (E > 1 && ((se & 7) || se < ld * (rows - 1) + cols))
        return set_error(KP_ESHAPE, "%s: %s's expert stride %lld is not a multiple of 8 or lets its matrices overlap", fn,
                         name, static_cast<long long>(se));
    return KP_OK;
}
static int check_ints(const char *fn, const char *name, const void *p) {
    if (!p) return set_error(KP_EINVAL, "%s: %s is NULL", fn, name);
    if (misaligned(p, 4)) return set_error(KP_EALIGN, "%s: %s must be 4-byte aligned", fn, name);
    return KP_OK;
}
static int check_workspace(const char *fn, const void *work, size_t have, size_t need) {
    if (have < need || (need && !work))
        return set_error(KP_EINVAL, "%s: the workspace has %zu bytes, %zu are needed (kp_moe_workspace)", fn,
                         work ? have : 0, need);
    if (need && misaligned(work, 256)) return set_error(KP_EALIGN, "%s: the workspace must be 256-byte aligned", fn);
    return KP_OK;
}
// Sizes that have the size of a block or a tile added to them in 32 bits.
static constexpr int kMost = 1 << 30;
static int check_pairs(const char *fn, int T, int k) {
    if (static_cast<int64_t>(T) * k > kMost)
        return set_error(KP_ESHAPE, "%s: %d tokens, top %d: at most 2^30 rows", fn, T, k);
    return KP_OK;
}
static int check_route(const char *fn, int T, int E, int k) {
    if (T < 0 || E < 1 || k < 1 || k > E)
        return set_error(KP_EINVAL, "%s: bad sizes: %d tokens, %d experts, top %d", fn, T, E, k);
    if (E > kMoeMaxExperts || k > kMoeMaxTopK)
        return set_error(KP_ESHAPE, "%s: %d experts, top %d: at most %d and %d", fn, E, k, kMoeMaxExperts, kMoeMaxTopK);
    return check_pairs(fn, T, k);
}
static int check_shuffle(const char *fn, int T, int k, int K, int dtype) {
    if (T < 0 || k < 1 || K < 1) return set_error(KP_EINVAL, "%s: bad sizes: %d tokens, top %d, %d columns", fn, T, k, K);
    if (!is16(dtype)) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (K > kMost) return set_error(KP_ESHAPE, "%s: %d columns: at most 2^30", fn, K);
    return check_pairs(fn, T, k);
}
static int check_norm(const char *fn, int T, int K, int dtype) {
    if (T < 0 || K < 1) return set_error(KP_EINVAL, "%s: bad sizes: %d rows, %d columns", fn, T, K);
    if (!is16(dtype) && dtype != KP_FP32) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (K > kNormMaxCols) return set_error(KP_ESHAPE, "%s: %d columns: at most %d", fn, K, kNormMaxCols);
    return KP_OK;
}
// A matrix of any of the three types, aligned to its elements.
static int check_matrix(const char *fn, const char *name, const void *p, int64_t ld, int cols, int dtype) {
    const int rc = check_rows(fn, name, p, ld, cols);
    if (rc || dtype != KP_FP32 || !misaligned(p, 4)) return rc;
    return set_error(KP_EALIGN, "%s: %s must be 4-byte aligned", fn, name);
}
static int check_grouped(const char *fn, int R, int E, int N, int K, int dtype) {
    if (R < 0 || E < 1 || N < 1 || K < 1)
        return set_error(KP_EINVAL, "%s: bad sizes: %d rows, %d experts, %d features, %d columns", fn, R, E, N, K);
    if (!is16(dtype)) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (E > kMoeMaxExperts) return set_error(KP_ESHAPE, "%s: %d experts: at most %d", fn, E, kMoeMaxExperts);
    if (K & 7) return set_error(KP_ESHAPE, "%s: K=%d is not a multiple of 8", fn, K);
    if (R > kMost || N > kMost || K > kMost)
        return set_error(KP_ESHAPE, "%s: %d rows, %d features, %d columns: at most 2^30", fn, R, N, K);
    return KP_OK;
}

// Gated backward: dG and dU [R][F rounded up to 8] in 16 bits, their scaling (fp16).
struct GatedBackwardWork {
    size_t du, scaling, bytes;
    int64_t ld;
};
static GatedBackwardWork gated_backward_work(int R, int F, int sms) {
    GatedBackwardWork w;
    w.ld = (static_cast<int64_t>(F) + 7) / 8 * 8;
    w.du = up256(static_cast<size_t>(R) * w.ld * 2);
    w.scaling = 2 * w.du;
    w.bytes = w.scaling + up256(ffn_gate_grad_scratch(sms));
    return w;
}

static cudaError_t zero(void *p, int E, int N, int K, cudaStream_t s) {
    return cudaMemsetAsync(p, 0, static_cast<size_t>(E) * N * K * 2, s);
}

}  // namespace kp

using namespace kp;

extern "C" {

int kp_moe_workspace(int op, int M, int N, int K, size_t *bytes) {
    const char *fn = "kp_moe_workspace";
    if (!bytes || M < 0 || N < 1 || K < 1)
        return set_error(KP_EINVAL, "%s: bad sizes: %d, %d, %d", fn, M, N, K);
    if (op != KP_MOE_ROUTE && op != KP_MOE_GATED_BACKWARD && op != KP_MOE_NORM_BACKWARD) return set_error(KP_EINVAL, "%s: unknown operator %d", fn, op);
    *bytes = 0;
    if (op == KP_MOE_ROUTE) {
        *bytes = moe_route_scratch(M, N);
        return KP_OK;
    }
    FfnDev d;
    const int rc = ffn_device(&d);
    if (rc) return rc;
    if (M) *bytes = op == KP_MOE_GATED_BACKWARD ? gated_backward_work(M, N, d.sms).bytes : norm_backward_scratch(M, K, d.sms);
    return KP_OK;
}

int kp_moe_route(const void *logits, int64_t ld, const float *bias, int T, int E, int k, int score, int dtype,
                 int32_t *ids, float *weights, int32_t *offsets, int32_t *order, int32_t *position, void *work,
                 size_t work_bytes, kp_stream_t stream) {
    const char *fn = "kp_moe_route";
    int rc = check_route(fn, T, E, k);
    if (rc) return rc;
    if (!is16(dtype) && dtype != KP_FP32) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (score != KP_SCORE_SOFTMAX && score != KP_SCORE_SIGMOID) return set_error(KP_EINVAL, "%s: unknown score %d", fn, score);
    if (bias && score != KP_SCORE_SIGMOID) return set_error(KP_EINVAL, "%s: a bias goes with the sigmoid score", fn);
    if (bias && misaligned(bias, 4)) return set_error(KP_EALIGN, "%s: bias must be 4-byte aligned", fn);
    if ((rc = check_ints(fn, "offsets", offsets))) return rc;
    FfnDev d;
    if (T == 0) {
        if ((rc = ffn_device(&d))) return rc;
        const cudaError_t e = cudaMemsetAsync(offsets, 0, (static_cast<size_t>(E) + 1) * sizeof(int32_t), stream);
        return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
    }
    if (!logits) return set_error(KP_EINVAL, "%s: logits is NULL", fn);
    if (misaligned(logits, dtype == KP_FP32 ? 4 : 2))
        return set_error(KP_EALIGN, "%s: logits must be aligned to its element size", fn);
    if (ld < E) return set_error(KP_EINVAL, "%s: logits' row stride %lld is below its %d experts", fn,
                                 static_cast<long long>(ld), E);
    if ((rc = check_ints(fn, "ids", ids)) || (rc = check_ints(fn, "weights", weights)) ||
        (rc = check_ints(fn, "order", order)) || (rc = check_ints(fn, "position", position)) ||
        (rc = check_workspace(fn, work, work_bytes, moe_route_scratch(T, E))) || (rc = ffn_device(&d)))
        return rc;
    MoeRouteArgs a;
    a.logits = logits;
    a.ld = ld;
    a.bias = bias;
    a.T = T;
    a.E = E;
    a.k = k;
    a.score = score;
    a.dtype = dtype;
    a.ids = ids;
    a.weights = weights;
    a.offsets = offsets;
    a.order = order;
    a.position = position;
    a.work = work;
    const cudaError_t e = moe_route_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_moe_route_backward(const float *dweights, const void *logits, int64_t ld, const int32_t *ids,
                          const float *weights, void *dlogits, int64_t ldd, int T, int E, int k, int score, int dtype,
                          kp_stream_t stream) {
    const char *fn = "kp_moe_route_backward";
    int rc = check_route(fn, T, E, k);
    if (rc) return rc;
    if (!is16(dtype) && dtype != KP_FP32) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (score != KP_SCORE_SOFTMAX && score != KP_SCORE_SIGMOID) return set_error(KP_EINVAL, "%s: unknown score %d", fn, score);
    if (T == 0) return KP_OK;
    const uintptr_t es = dtype == KP_FP32 ? 4 : 2;
    if (!logits || !dlogits) return set_error(KP_EINVAL, "%s: logits or dlogits is NULL", fn);
    if (misaligned(logits, es) || misaligned(dlogits, es))
        return set_error(KP_EALIGN, "%s: logits and dlogits must be aligned to their element size", fn);
    if (ld < E || ldd < E)
        return set_error(KP_EINVAL, "%s: a row stride (%lld, %lld) is below the %d experts", fn, static_cast<long long>(ld),
                         static_cast<long long>(ldd), E);
    FfnDev d;
    if ((rc = check_ints(fn, "dweights", dweights)) || (rc = check_ints(fn, "ids", ids)) ||
        (rc = check_ints(fn, "weights", weights)) || (rc = ffn_device(&d)))
        return rc;
    const cudaError_t e =
        moe_route_backward_launch(dweights, logits, ld, ids, weights, dlogits, ldd, T, E, k, score, dtype, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_moe_dispatch(const void *x, int64_t ldx, const int32_t *position, void *rows, int64_t ldr, int T, int k, int K,
                    int dtype, kp_stream_t stream) {
    const char *fn = "kp_moe_dispatch";
    int rc = check_shuffle(fn, T, k, K, dtype);
    if (rc || T == 0) return rc;
    FfnDev d;
    if ((rc = check_rows(fn, "x", x, ldx, K)) || (rc = check_rows(fn, "rows", rows, ldr, K)) ||
        (rc = check_ints(fn, "position", position)) || (rc = ffn_device(&d)))
        return rc;
    const cudaError_t e = moe_dispatch_launch(x, ldx, position, rows, ldr, T, k, K, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_moe_combine(const void *rows, int64_t ldr, const float *weights, const int32_t *position, void *y, int64_t ldy,
                   int T, int k, int K, int dtype, kp_stream_t stream) {
    const char *fn = "kp_moe_combine";
    int rc = check_shuffle(fn, T, k, K, dtype);
    if (rc || T == 0) return rc;
    FfnDev d;
    if ((rc = check_rows(fn, "rows", rows, ldr, K)) || (rc = check_rows(fn, "y", y, ldy, K)) ||
        (rc = check_ints(fn, "position", position)))
        return rc;
    if (weights && misaligned(weights, 4)) return set_error(KP_EALIGN, "%s: weights must be 4-byte aligned", fn);
    if ((rc = ffn_device(&d))) return rc;
    const cudaError_t e = moe_combine_launch(rows, ldr, weights, position, y, ldy, T, k, K, dtype, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_moe_combine_backward(const void *dy, int64_t lddy, const void *rows, int64_t ldr, const float *weights,
                            const int32_t *position, void *drows, int64_t lddr, float *dweights, int T, int k, int K,
                            int dtype, kp_stream_t stream) {
    const char *fn = "kp_moe_combine_backward";
    int rc = check_shuffle(fn, T, k, K, dtype);
    if (rc || T == 0) return rc;
    FfnDev d;
    if ((rc = check_rows(fn, "dy", dy, lddy, K)) || (rc = check_rows(fn, "rows", rows, ldr, K)) ||
        (rc = check_rows(fn, "drows", drows, lddr, K)) || (rc = check_ints(fn, "weights", weights)) ||
        (rc = check_ints(fn, "position", position)) || (rc = check_ints(fn, "dweights", dweights)) ||
        (rc = ffn_device(&d)))
        return rc;
    const cudaError_t e = moe_combine_backward_launch(dy, lddy, rows, ldr, weights, position, drows, lddr, dweights, T,
                                                      k, K, dtype, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_layer_norm(const void *x, int64_t ldx, const void *weight, const void *bias, void *y, int64_t ldy, float *mean,
                  float *rstd, int T, int K, float eps, int center, int dtype, kp_stream_t stream) {
    const char *fn = "kp_layer_norm";
    int rc = check_norm(fn, T, K, dtype);
    if (rc) return rc;
    if (!(eps >= 0.f) || !std::isfinite(eps)) return set_error(KP_EINVAL, "%s: eps must be finite and not negative", fn);
    if (T == 0) return KP_OK;
    if ((rc = check_matrix(fn, "x", x, ldx, K, dtype)) || (rc = check_matrix(fn, "y", y, ldy, K, dtype)) ||
        (rc = check_matrix(fn, "weight", weight, K, K, dtype)) ||
        (bias && (rc = check_matrix(fn, "bias", bias, K, K, dtype))) || (mean && (rc = check_ints(fn, "mean", mean))) ||
        (rstd && (rc = check_ints(fn, "rstd", rstd))))
        return rc;
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    NormArgs a;
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.b = bias;
    a.y = y;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.T = T;
    a.K = K;
    a.eps = eps;
    a.center = center != 0;
    a.dtype = dtype;
    const cudaError_t e = norm_launch(a, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_layer_norm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *weight,
                           const float *mean, const float *rstd, void *dx, int64_t lddx, void *dweight, void *dbias,
                           int T, int K, int dtype, void *work, size_t work_bytes, kp_stream_t stream) {
    const char *fn = "kp_layer_norm_backward";
    int rc = check_norm(fn, T, K, dtype);
    if (rc || (rc = check_matrix(fn, "dweight", dweight, K, K, dtype)) ||
        (dbias && (rc = check_matrix(fn, "dbias", dbias, K, K, dtype))))
        return rc;
    FfnDev d;
    const size_t row = static_cast<size_t>(K) * (dtype == KP_FP32 ? 4 : 2);
    if (T == 0) {   // no rows: the weights' gradients are zero
        if ((rc = ffn_device(&d))) return rc;
        cudaError_t e = cudaMemsetAsync(dweight, 0, row, stream);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, row, stream);
        return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
    }
    if ((rc = check_matrix(fn, "dy", dy, lddy, K, dtype)) || (rc = check_matrix(fn, "x", x, ldx, K, dtype)) ||
        (rc = check_matrix(fn, "weight", weight, K, K, dtype)) || (rc = check_matrix(fn, "dx", dx, lddx, K, dtype)) ||
        (mean && (rc = check_ints(fn, "mean", mean))) || (rc = check_ints(fn, "rstd", rstd)) || (rc = ffn_device(&d)) ||
        (rc = check_workspace(fn, work, work_bytes, norm_backward_scratch(T, K, d.sms))))
        return rc;
    NormArgs a;
    a.x = x;
    a.ldx = ldx;
    a.w = weight;
    a.dy = dy;
    a.lddy = lddy;
    a.y = dx;
    a.ldy = lddx;
    a.mean = const_cast<float *>(mean);
    a.rstd = const_cast<float *>(rstd);
    a.dw = dweight;
    a.dbias = dbias;
    a.part = static_cast<float *>(work);
    a.T = T;
    a.K = K;
    a.center = mean != nullptr;
    a.dtype = dtype;
    const cudaError_t e = norm_backward_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_grouped_gemm(const void *x, int64_t ldx, const void *W, int64_t ldw, int64_t sw, void *y, int64_t ldy,
                    const int32_t *offsets, int R, int E, int N, int K, int dtype, kp_stream_t stream) {
    const char *fn = "kp_grouped_gemm";
    int rc = check_grouped(fn, R, E, N, K, dtype);
    if (rc || R == 0) return rc;
    FfnDev d;
    if ((rc = check_operand(fn, "x", x, ldx, K)) || (rc = check_experts(fn, "W", W, ldw, sw, E, N, K)) ||
        (rc = check_rows(fn, "y", y, ldy, N)) || (rc = check_ints(fn, "offsets", offsets)) || (rc = ffn_device(&d)))
        return rc;
    GroupedArgs a;
    a.form = GROUPED_PLAIN;
    a.dtype = dtype;
    a.offsets = offsets;
    a.R = R;
    a.E = E;
    a.N = N;
    a.K = K;
    a.x = x;
    a.ldx = ldx;
    a.w0 = {W, ldw, sw};
    a.y = y;
    a.ldy = ldy;
    a.err = d.err;
    const cudaError_t e = grouped_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_grouped_gemm_backward(const void *dy, int64_t lddy, const void *x, int64_t ldx, const void *W, int64_t ldw,
                             int64_t sw, void *dx, int64_t lddx, void *dW, const int32_t *offsets, int R, int E, int N,
                             int K, int dtype, kp_stream_t stream) {
    const char *fn = "kp_grouped_gemm_backward";
    int rc = check_grouped(fn, R, E, N, K, dtype);
    if (rc) return rc;
    if (!dW) return set_error(KP_EINVAL, "%s: dW is NULL", fn);
    if (misaligned(dW, 16)) return set_error(KP_EALIGN, "%s: dW must be 16-byte aligned", fn);
    FfnDev d;
    if (R == 0) {   // no rows: the weights' gradients are zero
        if ((rc = ffn_device(&d))) return rc;
        const cudaError_t e = zero(dW, E, N, K, stream);
        return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
    }
    if ((rc = check_operand(fn, "dy", dy, lddy, N)) || (rc = check_operand(fn, "x", x, ldx, K)) ||
        (rc = check_experts(fn, "W", W, ldw, sw, E, N, K)) || (rc = check_rows(fn, "dx", dx, lddx, K)) ||
        (rc = check_ints(fn, "offsets", offsets)) || (rc = ffn_device(&d)))
        return rc;
    GroupedArgs a;
    a.form = GROUPED_BACKWARD;
    a.dtype = dtype;
    a.offsets = offsets;
    a.R = R;
    a.E = E;
    a.N = N;
    a.K = K;
    a.x = x;
    a.ldx = ldx;
    a.w0 = {W, ldw, sw};
    a.d0 = dy;
    a.ldd = lddy;
    a.y = dx;
    a.ldy = lddx;
    a.dw0 = dW;
    a.err = d.err;
    const cudaError_t e = grouped_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_grouped_gated_ffn(const void *x, int64_t ldx, const void *Wg, int64_t ldg, int64_t sg, const void *Wu,
                         int64_t ldu, int64_t su, void *h, int64_t ldh, float *g, float *u, const int32_t *offsets,
                         int R, int E, int F, int K, int act, int dtype, kp_stream_t stream) {
    const char *fn = "kp_grouped_gated_ffn";
    int rc = check_grouped(fn, R, E, F, K, dtype);
    if (rc) return rc;
    if (!is_act(act)) return set_error(KP_EINVAL, "%s: unknown activation %d", fn, act);
    if (R == 0) return KP_OK;
    if ((rc = check_operand(fn, "x", x, ldx, K)) || (rc = check_experts(fn, "Wg", Wg, ldg, sg, E, F, K)) ||
        (rc = check_experts(fn, "Wu", Wu, ldu, su, E, F, K)) || (rc = check_rows(fn, "h", h, ldh, F)) ||
        (rc = check_ints(fn, "offsets", offsets)))
        return rc;
    if ((g != nullptr) != (u != nullptr)) return set_error(KP_EINVAL, "%s: give both g and u, or neither", fn);
    if (g && (misaligned(g, 16) || misaligned(u, 16)))
        return set_error(KP_EALIGN, "%s: g and u must be 16-byte aligned", fn);
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    GroupedArgs a;
    a.form = GROUPED_GATED;
    a.act = act;
    a.dtype = dtype;
    a.offsets = offsets;
    a.R = R;
    a.E = E;
    a.N = F;
    a.K = K;
    a.x = x;
    a.ldx = ldx;
    a.w0 = {Wg, ldg, sg};
    a.w1 = {Wu, ldu, su};
    a.y = h;
    a.ldy = ldh;
    a.g = g;
    a.u = u;
    a.err = d.err;
    const cudaError_t e = grouped_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_grouped_gated_ffn_backward(const void *dh, int64_t lddh, const void *x, int64_t ldx, const void *Wg,
                                  int64_t ldg, int64_t sg, const void *Wu, int64_t ldu, int64_t su, const float *g,
                                  const float *u, void *dx, int64_t lddx, void *dWg, void *dWu,
                                  const int32_t *offsets, int R, int E, int F, int K, int act, int dtype, void *work,
                                  size_t work_bytes, kp_stream_t stream) {
    const char *fn = "kp_grouped_gated_ffn_backward";
    int rc = check_grouped(fn, R, E, F, K, dtype);
    if (rc) return rc;
    if (!is_act(act)) return set_error(KP_EINVAL, "%s: unknown activation %d", fn, act);
    if (!dWg || !dWu) return set_error(KP_EINVAL, "%s: dWg or dWu is NULL", fn);
    if (misaligned(dWg, 16) || misaligned(dWu, 16))
        return set_error(KP_EALIGN, "%s: dWg and dWu must be 16-byte aligned", fn);
    FfnDev d;
    cudaError_t e;
    if (R == 0) {   // no rows: the weights' gradients are zero
        if ((rc = ffn_device(&d))) return rc;
        e = zero(dWg, E, F, K, stream);
        if (e == cudaSuccess) e = zero(dWu, E, F, K, stream);
        return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
    }
    if ((rc = check_rows(fn, "dh", dh, lddh, F)) || (rc = check_operand(fn, "x", x, ldx, K)) ||
        (rc = check_experts(fn, "Wg", Wg, ldg, sg, E, F, K)) || (rc = check_experts(fn, "Wu", Wu, ldu, su, E, F, K)) ||
        (rc = check_rows(fn, "dx", dx, lddx, K)) || (rc = check_ints(fn, "offsets", offsets)))
        return rc;
    if (!g || !u) return set_error(KP_EINVAL, "%s: g or u is NULL", fn);
    if (misaligned(g, 16) || misaligned(u, 16)) return set_error(KP_EALIGN, "%s: g and u must be 16-byte aligned", fn);
    if ((rc = ffn_device(&d))) return rc;
    const GatedBackwardWork w = gated_backward_work(R, F, d.sms);
    if ((rc = check_workspace(fn, work, work_bytes, w.bytes))) return rc;
    uint8_t *base = static_cast<uint8_t *>(work);
    float *scaling = dtype == KP_FP16 ? reinterpret_cast<float *>(base + w.scaling) : nullptr;
    e = ffn_gate_grad_launch(dh, lddh, g, u, base, base + w.du, w.ld, scaling, R, F, act, dtype, d.sms, stream,
                             offsets + E);
    if (e != cudaSuccess) return cuda_failed(e, fn);
    GroupedArgs a;
    a.form = GROUPED_BACKWARD;
    a.dtype = dtype;
    a.offsets = offsets;
    a.R = R;
    a.E = E;
    a.N = F;
    a.K = K;
    a.x = x;
    a.ldx = ldx;
    a.w0 = {Wg, ldg, sg};
    a.w1 = {Wu, ldu, su};
    a.d0 = base;
    a.d1 = base + w.du;
    a.ldd = w.ld;
    a.y = dx;
    a.ldy = lddx;
    a.dw0 = dWg;
    a.dw1 = dWu;
    a.scale = scaling;
    a.pdl = true;
    a.err = d.err;
    e = grouped_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

}  // extern "C"
