// Device parts of microscaled 4-bit quantisation, shared by the quantising kernel
// and by the product that quantises a few tokens on their way in. The rule and its
// exactness are described in kp_mx4.cu.
#pragma once

#include "kp_ffn.cuh"

namespace kp {

// fp32 bits of 2^-e for the scale byte e + 127 (0 .. 254): exact, also where
// the result is 2^127 (byte 0).
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }
// Eight E2M1 codes, the first in the low nibble (round to nearest even,
// saturating).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight columns of a row as they lie in memory: four words of a 16-bit type,
// eight of fp32. amax gives the bits, as fp32, of the largest magnitude: bit
// patterns order like magnitudes, with infinity and NaN on top.
template <typename T>
struct Eight {
    static constexpr int D = __is_same(T, __half) ? KP_FP16 : KP_BF16;
    uint32_t w[4];
    __device__ void load_full(const T *p) {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    }
    __device__ void load(const T *row, int c, int cols) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t lo = c + 2 * i < cols ? h[c + 2 * i] : 0, hi = c + 2 * i + 1 < cols ? h[c + 2 * i + 1] : 0;
            w[i] = lo | hi << 16;
        }
    }
    __device__ uint32_t amax() const {   // of the four lanes of a block
        uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu),
                              __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        return __float_as_uint(elem_lo<D>(max(m & 0xFFFFu, m >> 16)));
    }
    __device__ void scaled(float inv, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = elem_lo<D>(w[i]) * inv, v[2 * i + 1] = elem_hi<D>(w[i]) * inv;
    }
};
template <>
struct Eight<float> {
    float f[8];
    __device__ void load_full(const float *p) {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(p));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
        f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
    }
    static constexpr int kWindow = 48;
    __device__ void load_shifted(const float *p) {
        const uint32_t d = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<uintptr_t>(p) - d);
        const float4 a = __ldg(q), b = __ldg(q + 1), e = __ldg(q + 2);
        float t[11] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, e.x, e.y, e.z};
        if (d & 8)
#pragma unroll
            for (int i = 0; i < 9; ++i) t[i] = t[i + 2];
        if (d & 4)
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] = t[i + 1];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = t[i];
    }
    __device__ void load(const float *row, int c, int cols) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? row[c + i] : 0.f;
    }
    __device__ uint32_t amax() const {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        return max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    }
    __device__ void scaled(float inv, float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i] * inv;
    }
};

// Scale byte of a block whose largest magnitude has these fp32 bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
    const uint32_t ex = amax >> 23;   // 0: zero or subnormal, 255: infinity or NaN
    return ex == 255 ? 255u : ex > 2 ? ex - 2 : 0u;
}

// Eight columns of a block that four neighbouring lanes hold: their codes, and in b
// the block's scale byte (the same in the four lanes).
template <typename T>
__device__ __forceinline__ uint32_t quantize8(const Eight<T> &e, uint32_t &b) {
    b = scale_byte(e.amax());
    float v[8];
    e.scaled(inv_scale(b == 255 ? 127u : b), v);
    return e2m1x8(v);
}

}  // namespace kp
