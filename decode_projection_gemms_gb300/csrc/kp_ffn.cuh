// Shared parts of the feed-forward operators: microscaled 4-bit quantisation
// (kp_mx4.cu), the weight-streaming kernel for few tokens (kp_ffn_stream.cu)
// and the tile kernel for many (kp_ffn_tile.cu), behind kp_ffn_api.cu.
//
// Microscaled 4-bit layout of a matrix [rows, cols] (cols the contraction):
//   codes   [rows][nb * 16] bytes, nb = ceil(cols / 32): two E2M1 codes a byte,
//           the lower column in the low nibble; columns past `cols` hold 0.
//   scales  one E8M0 byte per (row, 32-column block), in tiles of 128 rows x 4
//           blocks = 512 bytes, tile (rt, kt) at (rt * ceil(nb / 4) + kt) * 512,
//           byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 within it. This is
//           the order in which tcgen05.cp (32x128b, repeated for the four warps)
//           lays a tile into tensor memory where the block-scaled MMA reads it:
//           lane r % 32, column r / 32, byte b, so a tile is one 512-byte copy
//           in and one instruction on. Rows and blocks past the end hold 0.
#pragma once

#include "kp_internal.cuh"

namespace kp {

// Device properties of the current device and its error word (kp_api.cu).
struct FfnDev {
    int dev = 0;
    int sms = 0;
    int *err = nullptr;
};
int ffn_device(FfnDev *out);   // KP_OK, or a status with the message set (KP_EDEVICE included)

// Tensor map of a row-major matrix of 16-bit elements (KP_BF16, KP_FP16), of
// fp32 (kMapF32) or bytes (kMapU8), box_cols x box_rows, 128-byte swizzle or none, zero
// fill outside.
constexpr int kMapU8 = 16, kMapF32 = 17;
cudaError_t ffn_tensor_map(CUtensorMap *map, const void *ptr, int64_t rows, int64_t cols, int64_t ld,
                           int box_rows, int box_cols, int dtype, bool swizzle = true);
// The scale tiles of a microscaled matrix, 512 bytes each, boxes of two.
cudaError_t ffn_scale_map(CUtensorMap *map, const void *scales, int64_t tiles);
// Shared memory to request for a CTA that holds `cols` TMEM columns: at least
// cols/512 of the SM's, so CTAs that share an SM never need more than 512
// columns together and no allocation can wait for a CTA that waits for it.
cudaError_t ffn_smem_for_tmem(int dev, uint32_t cols, size_t need, size_t *smem);

// One operand in the microscaled layout.
struct Mx4Mat {
    const uint8_t *codes = nullptr;
    const uint8_t *scales = nullptr;
};
inline int64_t mx4_blocks(int64_t cols) { return (cols + 31) / 32; }
inline int64_t mx4_pitch(int64_t cols) { return mx4_blocks(cols) * 16; }
inline int64_t mx4_ktiles(int64_t cols) { return (mx4_blocks(cols) + 3) / 4; }
inline size_t mx4_code_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * mx4_pitch(cols); }
inline size_t mx4_scale_bytes(int64_t rows, int64_t cols) {
    return static_cast<size_t>((rows + 127) / 128) * mx4_ktiles(cols) * 512;
}
// pad: also write the scales of the rows that fill the last 128-row tile
// (operands that outlive the call); without it those bytes stay as they are,
// which only reaches products of rows that do not exist.
cudaError_t mx4_quantize_launch(const void *x, int64_t ldx, int rows, int cols, int dtype, uint8_t *codes,
                                uint8_t *scales, bool pad, int sms, cudaStream_t s);
cudaError_t mx4_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y,
                                  int64_t ldy, int dtype, int sms, cudaStream_t s);

// One forward product: y[M, N] = round(x W^T), or with Wb the gated block
// h[M, N] = round(act(x Wa^T) * (x Wb^T)), over 16-bit or microscaled operands.
struct FfnArgs {
    bool mx4 = false;
    bool gated = false;
    int act = 0;                 // enum kp_act
    int dtype = KP_BF16;         // x and W (16-bit), y, g, u
    const void *x = nullptr;     // 16 bits: [M, ldx] (microscaled products: then quantised within)
    int64_t ldx = 0;
    const void *Wa = nullptr, *Wb = nullptr;   // 16-bit: [N, lda / ldb]
    int64_t lda = 0, ldb = 0;
    Mx4Mat qx, qa, qb;           // microscaled operands
    void *y = nullptr;
    int64_t ldy = 0;
    float *g = nullptr, *u = nullptr;   // optional, 16-bit gated: both products' sums, [M, N]
    int M = 0, N = 0, K = 0;
    float *ws = nullptr;         // split-K partial tiles
    bool pdl = false;            // launched behind a kernel that writes only qx
    int *err = nullptr;
};
// Few tokens: weight streaming, split-K over a cluster (kp_ffn_stream.cu).
size_t ffn_stream_scratch(bool mx4, bool gated, int M, int N, int K, int sms);   // bytes
bool ffn_stream_quantises(int M);   // whether its 4-bit forms take x in 16 bits
float ffn_stream_us(bool mx4, bool gated, int M, int N, int K, int sms);   // estimate of its time
cudaError_t ffn_stream_launch(const FfnArgs &a, const FfnDev &d, cudaStream_t s);

// One launch of the tile kernel (kp_ffn_tile.cu), for many tokens and for the
// backward pass.
enum FfnTileForm {
    TILE_GATED,       // A = x, B = Wg and Wu side by side: h (and g, u)
    TILE_MX4_GATED,   // the same over microscaled operands
    TILE_MX4,         // A = x, B = W, microscaled: y
    TILE_BACKWARD     // dx = dG Wg + dU Wu, dWg = dG^T x and dWu = dU^T x
};
struct FfnTileArgs {
    int form = TILE_GATED;
    int act = 0, dtype = KP_BF16;
    const void *A0 = nullptr, *A1 = nullptr;     // x; backward: dG, dU [M, N]
    const void *B0 = nullptr, *B1 = nullptr;     // Wg, Wu
    const void *X = nullptr;                     // backward: x
    int64_t lda = 0, ldb0 = 0, ldb1 = 0, ldx = 0;
    Mx4Mat qa, qb0, qb1;
    void *y0 = nullptr, *y1 = nullptr, *y2 = nullptr;   // h or y; backward: dx, dWg, dWu (row stride K)
    int64_t ldy = 0;
    float *g = nullptr, *u = nullptr;
    int M = 0, N = 0, K = 0;     // tokens, features, columns of x
    float *ws = nullptr;         // backward: partial sums of dx
    const float *scale = nullptr;   // backward: device factor of every sum (none: 1)
    bool pdl = false;
    int *err = nullptr;
};
size_t ffn_backward_scratch(int T, int F, int K, int sms);   // bytes of ws (0: dx is not split)
cudaError_t ffn_tile_launch(const FfnTileArgs &a, const FfnDev &d, cudaStream_t s);

// Whether a forward product takes the tile kernel or the weight-streaming one.
bool ffn_use_tile(bool mx4, bool gated, int M, int N, int K, int sms);

// dG = dh u act'(g), dU = dh act(g): the gradients of both products, [T, F]
// with row stride ld (kp_ffn_bwd.cu). scaling (fp16; NULL: none): both come out as
// multiples of a power of two, whose reciprocal goes to scaling[0]; the rest of its
// ffn_gate_grad_scratch bytes is the kernels' own.
size_t ffn_gate_grad_scratch(int sms);
cudaError_t ffn_gate_grad_launch(const void *dh, int64_t lddh, const float *g, const float *u, void *dg, void *du,
                                 int64_t ld, float *scaling, int T, int F, int act, int dtype, int sms,
                                 cudaStream_t s);

}  // namespace kp

#if defined(__CUDACC__)

namespace kp {

// ---- activations ------------------------------------------------------------
// The normal distribution's integral up to g, and e = exp(-g^2 / 2). 1 + erf(g / sqrt 2)
// cancels for negative g (4 % off at -5, zero from -5.5 on); here the integral from |g|
// on is e times a polynomial in 1 / (1 + 0.3 |g|), which Mills' ratio is close to: a
// fit of least relative error over |g| <= 14, 2^-24 off and 2^-21 with fp32's roundings.
// erfcf gives the same values, but the epilogue of tiles with few K blocks waits for it
// (2000 x 4096 x 512: 27.8 us with erff, 40.3 with erfcf, 30.2 with this).
__device__ __forceinline__ float ffn_normal_cdf(float g, float &e) {
    const float t = __fdividef(1.f, fmaf(0.3f, fabsf(g), 1.f));
    float p = 0.0383782685f;
    p = fmaf(p, t, -0.169166028f);
    p = fmaf(p, t, 0.228659928f);
    p = fmaf(p, t, -0.0765063167f);
    p = fmaf(p, t, 0.142535433f);
    p = fmaf(p, t, 0.0946835577f);
    p = fmaf(p, t, 0.121920332f);
    p = fmaf(p, t, 0.119487688f);
    p = fmaf(p, t, 7.16883596e-06f);
    e = __expf(-0.5f * g * g);
    p *= e;
    return g < 0.f ? p : 1.f - p;
}
// act(g), in fp32.
template <int kAct>
__device__ __forceinline__ float ffn_act(float g) {
    if constexpr (kAct == KP_ACT_SILU) return __fdividef(g, 1.f + __expf(-g));
    if constexpr (kAct == KP_ACT_GELU) {
        float e;
        return g * ffn_normal_cdf(g, e);
    }
    // 0.5 (1 + tanh z) = 1 / (1 + exp(-2 z)), z = sqrt(2/pi) (g + 0.044715 g^3)
    const float z2 = 1.5957691216057308f * (g + 0.044715f * g * g * g);
    return __fdividef(g, 1.f + __expf(-z2));
}
// h = act(a) b. The choice is made once for all N, so only one activation's code
// runs through the instruction cache.
template <int N>
__device__ __forceinline__ void ffn_gate(const float (&a)[N], const float (&b)[N], int act, float (&h)[N]) {
    if (act == KP_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = ffn_act<KP_ACT_SILU>(a[i]) * b[i];
    } else if (act == KP_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = ffn_act<KP_ACT_GELU>(a[i]) * b[i];
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = ffn_act<KP_ACT_GELU_TANH>(a[i]) * b[i];
    }
}

// act(g) and act'(g), in fp32.
template <int kAct>
__device__ __forceinline__ void ffn_act_grad(float g, float &a, float &da) {
    a = ffn_act<kAct>(g);
    if constexpr (kAct == KP_ACT_SILU) {
        const float s = __fdividef(1.f, 1.f + __expf(-g));
        da = s * (1.f + g * (1.f - s));
    } else if constexpr (kAct == KP_ACT_GELU) {
        float e;
        const float cdf = ffn_normal_cdf(g, e);
        a = g * cdf;
        da = cdf + g * 0.39894228040143268f * e;
    } else {
        // a = g s(w), s the logistic function, w = 2 sqrt(2/pi) (g + 0.044715 g^3)
        const float w = 1.5957691216057308f * (g + 0.044715f * g * g * g);
        const float s = __fdividef(1.f, 1.f + __expf(-w));
        // from 20 on s (1 - s) is 0, and g^2 need not be finite
        const float c = fminf(fmaxf(g, -20.f), 20.f);
        da = s + c * s * (1.f - s) * 1.5957691216057308f * (1.f + 0.134145f * c * c);
    }
}

// ---- shared-memory matrix descriptors ----------------------------------------
// K-major, 128-byte swizzle: 8-row groups of 1024 bytes.
__device__ __forceinline__ uint64_t desc_kmajor(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}
// A 512-byte scale tile: no swizzle, 8-row (of 16 bytes) groups of 128 bytes.
__device__ __forceinline__ uint64_t desc_scales(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1) << 16) |
           (static_cast<uint64_t>(128 >> 4) << 32) | (static_cast<uint64_t>(1) << 46);
}

// ---- tcgen05 --------------------------------------------------------------------
// Scale tile from shared memory into four TMEM columns: lane i of each of the
// four 32-lane quarters gets 16-byte row i.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// D[tmem] (+)= (sA * A) (sB * B)^T over 64 E2M1 columns, one E8M0 scale per 32.
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t sa, uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
// 32 lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]),
          "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]),
          "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// kind::f16 instruction descriptor: D fp32, A and B bf16 or fp16, M x N tile;
// a_mn / b_mn: that operand is stored with M / N contiguous instead of K.
__host__ __device__ __forceinline__ uint32_t idesc_f16(int dtype, int M, int N, bool a_mn = false, bool b_mn = false) {
    const uint32_t ab = dtype == KP_FP16 ? 0u : (1u << 7) | (1u << 10);
    return (1u << 4) | ab | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// kind::mxf4 instruction descriptor: A and B E2M1 (1), E8M0 scales (bit 23).
// The scale bytes' position in their 32-bit column goes to bits 29 and 4.
__host__ __device__ __forceinline__ uint32_t idesc_mxf4(int M, int N) {
    return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_sf(uint32_t idesc, uint32_t byte) {
    return idesc | (byte << 29) | (byte << 4);
}

// One lane of a converged warp, the same one at every later call. Loops that issue
// MMAs or copies run with all 32 lanes and only their instructions are this
// lane's: operands then stay in the warp's uniform registers. In a branch taken by
// one lane each MMA is preceded by moves into them, which its queue does not hide
// (4-bit product 4096 x 4096 x 7168: 81 us against 58).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Wait (bounded by time only) for a barrier phase; used to drain copies.
__device__ __forceinline__ void ffn_drain_wait(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > 1000000000ull) break;
}

}  // namespace kp

#endif  // __CUDACC__
