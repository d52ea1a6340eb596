// Microscaled 4-bit floating point: quantisation and the values back.
//
// A block is 32 consecutive columns of a row. With m its largest magnitude,
//     scale = 2^max(-127, floor(log2 m) - 2)          (2 = the largest E2M1 exponent)
//     code  = E2M1 nearest to element / scale, ties to even, at most 6
// A block of zeros has scale 2^-127. The largest element lies in [4, 8) of its
// scale, so elements above 6 scales saturate to 6. A block that holds a NaN or
// an infinity gets the scale NaN (255): all of its values are NaN.
// Every step is exact or the one rounding: the scale comes from the exponent
// bits, and dividing by a power of two is a multiplication by its reciprocal.
//
// Both kernels only move bytes (4.25 bits an element on the 4-bit side). A lane
// takes 8 columns (16 bytes of a 16-bit type), four lanes a block, a warp 256
// columns of a row: reads of 512 contiguous bytes and writes of 128, and the
// block's maximum is two shuffles.
#include "kp_ffn.cuh"

namespace kp {

namespace {

constexpr int kQThreads = 256;

// fp32 bits of 2^-e for the scale byte e + 127 (0 .. 254): exact, also where
// the result is 2^127 (byte 0).
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// 2^(b - 127); b = 0 is a subnormal, 255 is NaN.
__device__ __forceinline__ float scale_value(uint32_t b) {
    return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FFFFFFFu : b << 23);
}

// Two E2M1 codes, `lo` in the low nibble (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
    uint16_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// 8 columns c .. c+7 of a row; `vec`: whole 16-byte words may be read.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int c, int cols, bool vec, float (&v)[8]) {
    if (vec && c + 8 <= cols) {
        if constexpr (sizeof(T) == 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + c));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(row + c) + 1);
            v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
            v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
            constexpr int D = sizeof(T) == 2 && __is_same(T, __half) ? KP_FP16 : KP_BF16;
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(row + c));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = elem_lo<D>(w[i]), v[2 * i + 1] = elem_hi<D>(w[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? static_cast<float>(row[c + i]) : 0.f;
    }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads)
    mx4_quantize_kernel(const T *__restrict__ x, int64_t ldx, int rows, int cols, int vec,
                        uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int rows_pad) {
    pdl_trigger();   // the product behind this kernel may start on its weights
    const int lane = threadIdx.x & 31;
    const int segs = (cols + 255) >> 8;
    const int nb = (cols + 31) >> 5;
    const int kt_n = (nb + 3) >> 2;
    const int64_t pitch = static_cast<int64_t>(nb) * 16;
    const int64_t units = static_cast<int64_t>(rows_pad) * segs;
    const int64_t nw = static_cast<int64_t>(gridDim.x) * (kQThreads / 32);
    for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5); w < units; w += nw) {
        const int r = static_cast<int>(w / segs);
        const int seg = static_cast<int>(w - static_cast<int64_t>(r) * segs);
        const int c = seg * 256 + lane * 8;
        float v[8];
        if (r < rows) {
            load8(x + r * ldx, c, cols, vec != 0, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.f;
        }
        // The largest magnitude as a bit pattern: it orders like the magnitude,
        // with infinity and NaN on top.
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        const uint32_t ex = m >> 23;                     // 0: zero or subnormal, 255: infinity or NaN
        const uint32_t b = ex == 255 ? 255u : ex > 2 ? ex - 2 : 0u;
        const float inv = inv_scale(b == 255 ? 127u : b);
        if (r < rows && c < nb * 32) {
            uint32_t q = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) q |= e2m1x2(v[2 * i] * inv, v[2 * i + 1] * inv) << (8 * i);
            *reinterpret_cast<uint32_t *>(codes + r * pitch + (c >> 1)) = q;
        }
        // four blocks' scales of a tile are one 32-bit word: lane 0 has tile
        // 2 seg's, lane 16 tile 2 seg + 1's
        uint32_t word = b;
#pragma unroll
        for (int i = 1; i < 4; ++i) word |= __shfl_down_sync(0xFFFFFFFFu, b, 4 * i) << (8 * i);
        const int kt = seg * 2 + (lane >> 4);
        if ((lane & 15) == 0 && kt < kt_n)
            *reinterpret_cast<uint32_t *>(scales + (static_cast<int64_t>(r >> 7) * kt_n + kt) * 512 +
                                          (r & 31) * 16 + ((r & 127) >> 5) * 4) = word;
    }
}

template <typename T>
__global__ void __launch_bounds__(kQThreads)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int rows,
                          int cols, T *__restrict__ y, int64_t ldy, int vec) {
    const int chunks = (cols + 7) >> 3;
    const int nb = (cols + 31) >> 5;
    const int kt_n = (nb + 3) >> 2;
    const int64_t pitch = static_cast<int64_t>(nb) * 16;
    const int64_t total = static_cast<int64_t>(rows) * chunks;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kQThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; i < total; i += step) {
        const int r = static_cast<int>(i / chunks);
        const int c = static_cast<int>(i - static_cast<int64_t>(r) * chunks) * 8;
        const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(codes + r * pitch + (c >> 1)));
        const int b = c >> 5;
        const float s = scale_value(__ldg(scales + (static_cast<int64_t>(r >> 7) * kt_n + (b >> 2)) * 512 +
                                          (r & 31) * 16 + ((r & 127) >> 5) * 4 + (b & 3)));
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            // magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: with exponent field e and
            // mantissa bit t, t/2 for e = 0 and (1 + t/2) 2^(e-1) above
            const uint32_t n = (q >> (4 * k)) & 15u;
            const uint32_t e = (n >> 1) & 3u, t = n & 1u;
            const float mag = e ? __uint_as_float((126u + e) << 23 | t << 22) : 0.5f * static_cast<float>(t);
            v[k] = ((n & 8u) ? -mag : mag) * s;
        }
        T *dst = y + r * ldy + c;
        if (vec && c + 8 <= cols) {
            if constexpr (sizeof(T) == 4) {
                reinterpret_cast<float4 *>(dst)[0] = make_float4(v[0], v[1], v[2], v[3]);
                reinterpret_cast<float4 *>(dst)[1] = make_float4(v[4], v[5], v[6], v[7]);
            } else {
                constexpr int D = __is_same(T, __half) ? KP_FP16 : KP_BF16;
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    o[k] = elem_round<D>(v[2 * k]) | static_cast<uint32_t>(elem_round<D>(v[2 * k + 1])) << 16;
                *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        } else {
            for (int k = 0; k < 8 && c + k < cols; ++k) dst[k] = static_cast<T>(v[k]);
        }
    }
}

bool rows_vectorise(const void *p, int64_t ld, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0;
}

int grid_for(int64_t warps, int sms) {
    const int64_t blocks = (warps + kQThreads / 32 - 1) / (kQThreads / 32);
    const int64_t most = static_cast<int64_t>(sms) * 8;
    return static_cast<int>(blocks < most ? blocks : most);
}

}  // namespace

cudaError_t mx4_quantize_launch(const void *x, int64_t ldx, int rows, int cols, int dtype, uint8_t *codes,
                                uint8_t *scales, bool pad, int sms, cudaStream_t s) {
    const int rows_pad = pad ? (rows + 127) / 128 * 128 : rows;
    const int64_t units = static_cast<int64_t>(rows_pad) * ((cols + 255) / 256);
    const int grid = grid_for(units, sms);
    const int vec = rows_vectorise(x, ldx, dtype == KP_FP32 ? 4 : 2);
    if (dtype == KP_FP32)
        mx4_quantize_kernel<<<grid, kQThreads, 0, s>>>(static_cast<const float *>(x), ldx, rows, cols, vec, codes,
                                                       scales, rows_pad);
    else if (dtype == KP_FP16)
        mx4_quantize_kernel<<<grid, kQThreads, 0, s>>>(static_cast<const __half *>(x), ldx, rows, cols, vec, codes,
                                                       scales, rows_pad);
    else
        mx4_quantize_kernel<<<grid, kQThreads, 0, s>>>(static_cast<const __nv_bfloat16 *>(x), ldx, rows, cols, vec,
                                                       codes, scales, rows_pad);
    return cudaGetLastError();
}

cudaError_t mx4_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y,
                                  int64_t ldy, int dtype, int sms, cudaStream_t s) {
    const int64_t units = static_cast<int64_t>(rows) * ((cols + 7) / 8);
    const int grid = grid_for((units + 31) / 32, sms);
    const int vec = rows_vectorise(y, ldy, dtype == KP_FP32 ? 4 : 2);
    if (dtype == KP_FP32)
        mx4_dequantize_kernel<<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, static_cast<float *>(y), ldy, vec);
    else if (dtype == KP_FP16)
        mx4_dequantize_kernel<<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, static_cast<__half *>(y), ldy, vec);
    else
        mx4_dequantize_kernel<<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, static_cast<__nv_bfloat16 *>(y),
                                                         ldy, vec);
    return cudaGetLastError();
}

}  // namespace kp
