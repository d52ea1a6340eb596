// C entry points of the feed-forward operators (include/kdaproj.h): argument
// checks, workspace layout and the order of their launches. Nothing throws and
// nothing is kept between calls; the caller owns every buffer.
#include <cuda.h>

#include <cstring>
#include <mutex>

#include "kp_ffn.cuh"

namespace kp {

// ---- tensor maps, shared-memory rule -------------------------------------------

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                             const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static std::mutex g_mu;
static EncodeFn g_encode = nullptr;

static cudaError_t encoder(EncodeFn *out) {
    std::lock_guard<std::mutex> lk(g_mu);
    if (!g_encode) {
        void *fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !fn) return cudaErrorNotSupported;
        g_encode = reinterpret_cast<EncodeFn>(fn);
    }
    *out = g_encode;
    return cudaSuccess;
}

cudaError_t ffn_tensor_map(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld,
                           int box_rows, int box_cols, int dtype, bool swizzle) {
    EncodeFn enc;
    cudaError_t e = encoder(&enc);
    if (e != cudaSuccess) return e;
    const cuuint64_t es = dtype == kMapU8 ? 1 : dtype == kMapF32 ? 4 : 2;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * es};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    const CUtensorMapDataType t = dtype == kMapU8    ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : dtype == kMapF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : dtype == KP_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUresult r = enc(map, t, 2, const_cast<void *>(ptr), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t ffn_tensor_map3(CUtensorMap *map, const void *ptr, int64_t n, int64_t rows, int64_t cols, int64_t ld,
                            int64_t step, int box_rows, int dtype) {
    EncodeFn enc;
    cudaError_t e = encoder(&enc);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(n)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(n > 1 ? step : ld * rows) * 2};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, dtype == KP_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                           const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t ffn_scale_map(CUtensorMap *map, const void *scales, int64_t tiles) {
    EncodeFn enc;
    cudaError_t e = encoder(&enc);
    if (e != cudaSuccess) return e;
    const cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(tiles)};   // 32-bit words
    const cuuint64_t strides[1] = {512};
    const cuuint32_t box[2] = {128, 2};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(scales), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t ffn_smem_for_tmem(int dev, uint32_t cols, size_t need, size_t *smem) {
    static std::mutex mu;
    static int known = -1, sm_smem = 0, reserved = 0;   // the last device asked about
    std::lock_guard<std::mutex> lk(mu);
    if (known != dev) {
        cudaError_t e = cudaDeviceGetAttribute(&sm_smem, cudaDevAttrMaxSharedMemoryPerMultiprocessor, dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&reserved, cudaDevAttrReservedSharedMemoryPerBlock, dev);
        if (e != cudaSuccess) return e;
        known = dev;
    }
    const long long least = (static_cast<long long>(sm_smem) * cols + 511) / 512 - reserved;
    *smem = least > static_cast<long long>(need) ? static_cast<size_t>(least) : need;
    return *smem > 227 * 1024 ? cudaErrorInvalidValue : cudaSuccess;
}

// ---- argument checks --------------------------------------------------------------

static int cuda_failed(cudaError_t e, const char *what) {
    return set_error(KP_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}
static bool misaligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
static bool is16(int dtype) { return dtype == KP_BF16 || dtype == KP_FP16; }
static bool is_act(int act) { return act == KP_ACT_SILU || act == KP_ACT_GELU || act == KP_ACT_GELU_TANH; }

// A 16-bit operand that is read through a tensor map: 16-byte rows.
static int check_operand(const char *fn, const char *name, const void *p, int64_t ld, int cols) {
    if (!p) return set_error(KP_EINVAL, "%s: %s is NULL", fn, name);
    if (misaligned(p, 16)) return set_error(KP_EALIGN, "%s: %s must be 16-byte aligned", fn, name);
    if (ld < cols) return set_error(KP_EINVAL, "%s: %s's row stride %lld is below its %d columns", fn, name,
                                    static_cast<long long>(ld), cols);
    if (ld & 7) return set_error(KP_ESHAPE, "%s: %s's row stride %lld is not a multiple of 8", fn, name,
                                 static_cast<long long>(ld));
    return KP_OK;
}
static int check_mx4(const char *fn, const char *name, const void *codes, const void *scales) {
    if (!codes || !scales) return set_error(KP_EINVAL, "%s: %s is NULL", fn, name);
    if (misaligned(codes, 16) || misaligned(scales, 16))
        return set_error(KP_EALIGN, "%s: %s's codes and scales must be 16-byte aligned", fn, name);
    return KP_OK;
}
// The 4-bit kernels count segments of 256 columns in 32 bits (that many hold
// half a terabyte of codes).
static int check_mx4_size(const char *fn, int64_t rows, int64_t cols) {
    if ((rows + 127) * ((cols + 255) / 256) >= (1ll << 32) || cols > (1 << 30))
        return set_error(KP_ESHAPE, "%s: %lld x %lld is too large", fn, static_cast<long long>(rows),
                         static_cast<long long>(cols));
    return KP_OK;
}
static int check_output(const char *fn, const char *name, const void *p, int64_t ld, int cols) {
    if (!p) return set_error(KP_EINVAL, "%s: %s is NULL", fn, name);
    if (misaligned(p, 2)) return set_error(KP_EALIGN, "%s: %s must be 2-byte aligned", fn, name);
    if (ld < cols) return set_error(KP_EINVAL, "%s: %s's row stride %lld is below its %d columns", fn, name,
                                    static_cast<long long>(ld), cols);
    return KP_OK;
}
static int check_workspace(const char *fn, const void *work, size_t have, size_t need) {
    if (have < need || (need && !work))
        return set_error(KP_EINVAL, "%s: the workspace has %zu bytes, %zu are needed (kp_ffn_workspace)", fn,
                         work ? have : 0, need);
    if (need && misaligned(work, 256)) return set_error(KP_EALIGN, "%s: the workspace must be 256-byte aligned", fn);
    return KP_OK;
}

// ---- workspaces -------------------------------------------------------------------

static size_t up256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

// Which kernel a forward product takes: see ffn_use_tile.
static size_t forward_scratch(bool mx4, bool gated, int M, int N, int K, int sms) {
    return ffn_use_tile(mx4, gated, M, N, K, sms) ? 0 : ffn_stream_scratch(mx4, gated, M, N, K, sms);
}

static cudaError_t forward_launch(const FfnArgs &a, const FfnDev &d, cudaStream_t s) {
    if (!ffn_use_tile(a.mx4, a.gated, a.M, a.N, a.K, d.sms)) return ffn_stream_launch(a, d, s);
    FfnTileArgs t;
    t.form = !a.mx4 ? TILE_GATED : a.gated ? TILE_MX4_GATED : TILE_MX4;
    t.act = a.act;
    t.dtype = a.dtype;
    t.A0 = a.x;
    t.B0 = a.Wa;
    t.B1 = a.Wb;
    t.lda = a.ldx;
    t.ldb0 = a.lda;
    t.ldb1 = a.ldb;
    t.qa = a.qx;
    t.qb0 = a.qa;
    t.qb1 = a.qb;
    t.y0 = a.y;
    t.ldy = a.ldy;
    t.g = a.g;
    t.u = a.u;
    t.M = a.M;
    t.N = a.N;
    t.K = a.K;
    t.pdl = a.pdl;
    t.err = a.err;
    return ffn_tile_launch(t, d, s);
}

// Whether a 4-bit product quantises x within its own launch.
static bool quantises_within(bool gated, int M, int N, int K, int sms) {
    return ffn_stream_quantises(M) && !ffn_use_tile(true, gated, M, N, K, sms);
}

// 4-bit products: x's codes, x's scales, split-K partial tiles; nothing where x is
// quantised within.
struct Mx4Work {
    size_t scales, part, bytes;
};
static Mx4Work mx4_work(bool gated, int M, int N, int K, int sms) {
    Mx4Work w = {};
    if (quantises_within(gated, M, N, K, sms)) return w;
    w.scales = up256(mx4_code_bytes(M, K));
    w.part = w.scales + up256(mx4_scale_bytes(M, K));
    w.bytes = w.part + forward_scratch(true, gated, M, N, K, sms);
    return w;
}

// Backward: dG and dU [T][F rounded up to 8] in 16 bits, their scaling (fp16), then
// dx's partial sums.
struct BwdWork {
    size_t du, scaling, part, bytes;
    int64_t ld;
};
static BwdWork bwd_work(int T, int F, int K, int sms) {
    BwdWork w;
    w.ld = (static_cast<int64_t>(F) + 7) / 8 * 8;
    w.du = up256(static_cast<size_t>(T) * w.ld * 2);
    w.scaling = 2 * w.du;
    w.part = w.scaling + up256(ffn_gate_grad_scratch(sms));
    w.bytes = w.part + ffn_backward_scratch(T, F, K, sms);
    return w;
}

static int bad_sizes(const char *fn, int M, int N, int K) {
    return set_error(KP_EINVAL, "%s: bad sizes: %d rows, %d features, %d columns", fn, M, N, K);
}

static int mx4_product(const char *fn, FfnArgs a, const void *x, int64_t ldx, const void *x_codes,
                       const void *x_scales, void *work, size_t work_bytes, cudaStream_t s) {
    if (a.M < 0 || a.N < 1 || a.K < 1) return bad_sizes(fn, a.M, a.N, a.K);
    if (!is16(a.dtype)) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, a.dtype);
    if (a.M == 0) return KP_OK;
    int rc = check_mx4_size(fn, a.M, a.K);
    if (rc) return rc;
    if ((x != nullptr) == (x_codes != nullptr))
        return set_error(KP_EINVAL, "%s: give x or its codes and scales, not both", fn);
    if (x) {
        if (misaligned(x, 2)) return set_error(KP_EALIGN, "%s: x must be 2-byte aligned", fn);
        if (ldx < a.K) return set_error(KP_EINVAL, "%s: x's row stride %lld is below its %d columns", fn,
                                        static_cast<long long>(ldx), a.K);
    } else if ((rc = check_mx4(fn, "x", x_codes, x_scales))) {
        return rc;
    }
    if ((rc = check_mx4(fn, a.gated ? "Wg" : "W", a.qa.codes, a.qa.scales))) return rc;
    if (a.gated && (rc = check_mx4(fn, "Wu", a.qb.codes, a.qb.scales))) return rc;
    if ((rc = check_output(fn, a.gated ? "h" : "y", a.y, a.ldy, a.N))) return rc;
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    const Mx4Work w = mx4_work(a.gated, a.M, a.N, a.K, d.sms);
    if ((rc = check_workspace(fn, work, work_bytes, w.bytes))) return rc;
    uint8_t *base = static_cast<uint8_t *>(work);
    a.mx4 = true;
    a.err = d.err;
    a.ws = reinterpret_cast<float *>(base + w.part);
    cudaError_t e;
    if (x && quantises_within(a.gated, a.M, a.N, a.K, d.sms)) {
        a.x = x;
        a.ldx = ldx;
    } else if (x) {
        // quantised on its way in; the product is launched behind it and
        // streams its weights meanwhile
        e = mx4_quantize_launch(x, ldx, a.M, a.K, a.dtype, base, base + w.scales, false, d.sms, s);
        if (e != cudaSuccess) return cuda_failed(e, fn);
        a.qx = {base, base + w.scales};
        a.pdl = true;
    } else {
        a.qx = {static_cast<const uint8_t *>(x_codes), static_cast<const uint8_t *>(x_scales)};
    }
    e = forward_launch(a, d, s);
    if (e != cudaSuccess) return cuda_failed(e, fn);
    return KP_OK;
}

}  // namespace kp

using namespace kp;

extern "C" {

int kp_mx4_bytes(int rows, int cols, size_t *code_bytes, size_t *scale_bytes) {
    if (rows < 0 || cols < 1 || !code_bytes || !scale_bytes)
        return set_error(KP_EINVAL, "kp_mx4_bytes: bad argument (%d rows, %d columns)", rows, cols);
    *code_bytes = mx4_code_bytes(rows, cols);
    *scale_bytes = mx4_scale_bytes(rows, cols);
    return KP_OK;
}

int kp_mx4_quantize(const void *x, int64_t ldx, int rows, int cols, int dtype, void *codes, void *scales,
                    kp_stream_t stream) {
    const char *fn = "kp_mx4_quantize";
    if (rows < 0 || cols < 1) return set_error(KP_EINVAL, "%s: bad sizes: %d rows, %d columns", fn, rows, cols);
    if (!is16(dtype) && dtype != KP_FP32) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (rows == 0) return KP_OK;
    if (!x) return set_error(KP_EINVAL, "%s: x is NULL", fn);
    if (misaligned(x, dtype == KP_FP32 ? 4 : 2))
        return set_error(KP_EALIGN, "%s: x must be aligned to its element size", fn);
    if (ldx < cols) return set_error(KP_EINVAL, "%s: x's row stride %lld is below its %d columns", fn,
                                     static_cast<long long>(ldx), cols);
    int rc = check_mx4_size(fn, rows, cols);
    if (rc || (rc = check_mx4(fn, "the output", codes, scales))) return rc;
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    cudaError_t e = mx4_quantize_launch(x, ldx, rows, cols, dtype, static_cast<uint8_t *>(codes),
                                        static_cast<uint8_t *>(scales), true, d.sms, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_mx4_dequantize(const void *codes, const void *scales, int rows, int cols, void *y, int64_t ldy, int dtype,
                      kp_stream_t stream) {
    const char *fn = "kp_mx4_dequantize";
    if (rows < 0 || cols < 1) return set_error(KP_EINVAL, "%s: bad sizes: %d rows, %d columns", fn, rows, cols);
    if (!is16(dtype) && dtype != KP_FP32) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (rows == 0) return KP_OK;
    int rc = check_mx4_size(fn, rows, cols);
    if (rc || (rc = check_mx4(fn, "the input", codes, scales))) return rc;
    if (!y) return set_error(KP_EINVAL, "%s: y is NULL", fn);
    if (misaligned(y, dtype == KP_FP32 ? 4 : 2))
        return set_error(KP_EALIGN, "%s: y must be aligned to its element size", fn);
    if (ldy < cols) return set_error(KP_EINVAL, "%s: y's row stride %lld is below its %d columns", fn,
                                     static_cast<long long>(ldy), cols);
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    cudaError_t e = mx4_dequantize_launch(static_cast<const uint8_t *>(codes), static_cast<const uint8_t *>(scales),
                                          rows, cols, y, ldy, dtype, d.sms, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_ffn_workspace(int op, int M, int N, int K, size_t *bytes) {
    if (!bytes || M < 0 || N < 1 || K < 1) return bad_sizes("kp_ffn_workspace", M, N, K);
    FfnDev d;
    int rc = ffn_device(&d);
    if (rc) return rc;
    *bytes = 0;
    switch (op) {
    case KP_FFN_MX4_GEMM:
    case KP_FFN_MX4_GATED:
        if (M) *bytes = mx4_work(op == KP_FFN_MX4_GATED, M, N, K, d.sms).bytes;
        return KP_OK;
    case KP_FFN_GATED:
        if (M) *bytes = forward_scratch(false, true, M, N, K, d.sms);
        return KP_OK;
    case KP_FFN_GATED_BACKWARD:
        if (M) *bytes = bwd_work(M, N, K, d.sms).bytes;
        return KP_OK;
    default: return set_error(KP_EINVAL, "kp_ffn_workspace: unknown operator %d", op);
    }
}

int kp_mx4_gemm(const void *x, int64_t ldx, const void *x_codes, const void *x_scales, const void *W_codes,
                const void *W_scales, void *y, int64_t ldy, int M, int N, int K, int dtype, void *work,
                size_t work_bytes, kp_stream_t stream) {
    FfnArgs a;
    a.dtype = dtype;
    a.qa = {static_cast<const uint8_t *>(W_codes), static_cast<const uint8_t *>(W_scales)};
    a.y = y;
    a.ldy = ldy;
    a.M = M;
    a.N = N;
    a.K = K;
    return mx4_product("kp_mx4_gemm", a, x, ldx, x_codes, x_scales, work, work_bytes, stream);
}

int kp_mx4_gated_ffn(const void *x, int64_t ldx, const void *x_codes, const void *x_scales, const void *Wg_codes,
                     const void *Wg_scales, const void *Wu_codes, const void *Wu_scales, void *h, int64_t ldh,
                     int T, int F, int K, int act, int dtype, void *work, size_t work_bytes, kp_stream_t stream) {
    if (!is_act(act)) return set_error(KP_EINVAL, "kp_mx4_gated_ffn: unknown activation %d", act);
    FfnArgs a;
    a.gated = true;
    a.act = act;
    a.dtype = dtype;
    a.qa = {static_cast<const uint8_t *>(Wg_codes), static_cast<const uint8_t *>(Wg_scales)};
    a.qb = {static_cast<const uint8_t *>(Wu_codes), static_cast<const uint8_t *>(Wu_scales)};
    a.y = h;
    a.ldy = ldh;
    a.M = T;
    a.N = F;
    a.K = K;
    return mx4_product("kp_mx4_gated_ffn", a, x, ldx, x_codes, x_scales, work, work_bytes, stream);
}

int kp_gated_ffn(const void *x, int64_t ldx, const void *Wg, int64_t ldg, const void *Wu, int64_t ldu, void *h,
                 int64_t ldh, float *g, float *u, int T, int F, int K, int act, int dtype, void *work,
                 size_t work_bytes, kp_stream_t stream) {
    const char *fn = "kp_gated_ffn";
    if (T < 0 || F < 1 || K < 1) return bad_sizes(fn, T, F, K);
    if (!is16(dtype)) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (!is_act(act)) return set_error(KP_EINVAL, "%s: unknown activation %d", fn, act);
    if (K & 7) return set_error(KP_ESHAPE, "%s: K=%d is not a multiple of 8", fn, K);
    if (T == 0) return KP_OK;
    int rc;
    if ((rc = check_operand(fn, "x", x, ldx, K)) || (rc = check_operand(fn, "Wg", Wg, ldg, K)) ||
        (rc = check_operand(fn, "Wu", Wu, ldu, K)) || (rc = check_output(fn, "h", h, ldh, F)))
        return rc;
    if ((g != nullptr) != (u != nullptr)) return set_error(KP_EINVAL, "%s: give both g and u, or neither", fn);
    if (g && (misaligned(g, 16) || misaligned(u, 16)))
        return set_error(KP_EALIGN, "%s: g and u must be 16-byte aligned", fn);
    FfnDev d;
    if ((rc = ffn_device(&d))) return rc;
    const size_t need = forward_scratch(false, true, T, F, K, d.sms);
    if ((rc = check_workspace(fn, work, work_bytes, need))) return rc;
    FfnArgs a;
    a.gated = true;
    a.act = act;
    a.dtype = dtype;
    a.x = x;
    a.ldx = ldx;
    a.Wa = Wg;
    a.lda = ldg;
    a.Wb = Wu;
    a.ldb = ldu;
    a.y = h;
    a.ldy = ldh;
    a.g = g;
    a.u = u;
    a.M = T;
    a.N = F;
    a.K = K;
    a.ws = static_cast<float *>(work);
    a.err = d.err;
    cudaError_t e = forward_launch(a, d, stream);
    return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
}

int kp_gated_ffn_backward(const void *dh, int64_t lddh, const void *x, int64_t ldx, const void *Wg, int64_t ldg,
                          const void *Wu, int64_t ldu, const float *g, const float *u, void *dx, void *dWg, void *dWu,
                          int T, int F, int K, int act, int dtype, void *work, size_t work_bytes,
                          kp_stream_t stream) {
    const char *fn = "kp_gated_ffn_backward";
    if (T < 0 || F < 1 || K < 1) return bad_sizes(fn, T, F, K);
    if (!is16(dtype)) return set_error(KP_EINVAL, "%s: unknown element type %d", fn, dtype);
    if (!is_act(act)) return set_error(KP_EINVAL, "%s: unknown activation %d", fn, act);
    if (K & 7) return set_error(KP_ESHAPE, "%s: K=%d is not a multiple of 8", fn, K);
    if (!dWg || !dWu) return set_error(KP_EINVAL, "%s: dWg or dWu is NULL", fn);
    if (misaligned(dWg, 16) || misaligned(dWu, 16))
        return set_error(KP_EALIGN, "%s: dWg and dWu must be 16-byte aligned", fn);
    int rc;
    FfnDev d;
    if (T == 0) {   // no tokens: the weights' gradients are zero
        if ((rc = ffn_device(&d))) return rc;
        cudaError_t e = cudaMemsetAsync(dWg, 0, static_cast<size_t>(F) * K * 2, stream);
        if (e == cudaSuccess) e = cudaMemsetAsync(dWu, 0, static_cast<size_t>(F) * K * 2, stream);
        return e == cudaSuccess ? KP_OK : cuda_failed(e, fn);
    }
    if ((rc = check_operand(fn, "x", x, ldx, K)) || (rc = check_operand(fn, "Wg", Wg, ldg, K)) ||
        (rc = check_operand(fn, "Wu", Wu, ldu, K)) || (rc = check_output(fn, "dh", dh, lddh, F)))
        return rc;
    if (!g || !u || !dx) return set_error(KP_EINVAL, "%s: g, u or dx is NULL", fn);
    if (misaligned(g, 16) || misaligned(u, 16) || misaligned(dx, 16))
        return set_error(KP_EALIGN, "%s: g, u and dx must be 16-byte aligned", fn);
    if ((rc = ffn_device(&d))) return rc;
    const BwdWork w = bwd_work(T, F, K, d.sms);
    if ((rc = check_workspace(fn, work, work_bytes, w.bytes))) return rc;
    uint8_t *base = static_cast<uint8_t *>(work);
    float *scaling = dtype == KP_FP16 ? reinterpret_cast<float *>(base + w.scaling) : nullptr;
    cudaError_t e = ffn_gate_grad_launch(dh, lddh, g, u, base, base + w.du, w.ld, scaling, T, F, act, dtype, d.sms,
                                         stream);
    if (e != cudaSuccess) return cuda_failed(e, fn);
    FfnTileArgs t;
    t.form = TILE_BACKWARD;
    t.dtype = dtype;
    t.A0 = base;
    t.A1 = base + w.du;
    t.lda = w.ld;
    t.B0 = Wg;
    t.B1 = Wu;
    t.ldb0 = ldg;
    t.ldb1 = ldu;
    t.X = x;
    t.ldx = ldx;
    t.y0 = dx;
    t.y1 = dWg;
    t.y2 = dWu;
    t.ldy = K;
    t.M = T;
    t.N = F;
    t.K = K;
    t.ws = reinterpret_cast<float *>(base + w.part);
    t.scale = scaling;
    t.err = d.err;
    if ((e = ffn_tile_launch(t, d, stream)) != cudaSuccess) return cuda_failed(e, fn);
    return KP_OK;
}

}  // extern "C"
