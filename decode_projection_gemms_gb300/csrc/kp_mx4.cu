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
// The kernels only move bytes (4.25 bits an element on the 4-bit side), so what
// counts is that every warp has several wide loads in flight, that reads and writes
// are contiguous, and that few instructions go to an element: 16-bit rows have a
// whole block in each lane (four 16-byte loads, no exchange, the scale once per 32
// elements; 4096 x 7168 bf16: 14.7 us with 8 columns a lane, 13.0 with 32; 4096 x 7167 22.7 and 15.1), fp32 rows
// 8 columns, four lanes a block. Rows that do not start on 16 bytes still move in
// aligned 16-byte words: a lane reads the words that hold its columns and shifts,
// and on the way back it takes the columns of one aligned word, whose codes may
// straddle two blocks.
#include "kp_mx4.cuh"

namespace kp {

namespace {

constexpr int kQThreads = 256;
constexpr int kQBlocks = 6;   // resident blocks per SM of the 16-bit kernel: its grid is one round

// A 32-column block of a 16-bit row as it lies in memory.
template <typename T>
struct Block16 {
    static constexpr int D = __is_same(T, __half) ? KP_FP16 : KP_BF16;
    uint32_t w[16];
    __device__ void load_full(const T *p) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p) + i);
            w[4 * i] = a.x, w[4 * i + 1] = a.y, w[4 * i + 2] = a.z, w[4 * i + 3] = a.w;
        }
    }
    // From an address aligned to the element only, through the five aligned words
    // around it: kWindow bytes from the last 16-byte boundary.
    static constexpr int kWindow = 80;
    __device__ void load_shifted(const T *p) {
        const uint32_t d = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) & 15u);
        const uint4 *q = reinterpret_cast<const uint4 *>(reinterpret_cast<uintptr_t>(p) - d);
        uint32_t t[20];
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            const uint4 a = __ldg(q + i);
            t[4 * i] = a.x, t[4 * i + 1] = a.y, t[4 * i + 2] = a.z, t[4 * i + 3] = a.w;
        }
        if (d & 8)
#pragma unroll
            for (int i = 0; i < 18; ++i) t[i] = t[i + 2];
        if (d & 4)
#pragma unroll
            for (int i = 0; i < 17; ++i) t[i] = t[i + 1];
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = __funnelshift_r(t[i], t[i + 1], (d & 2) * 8);
    }
    __device__ void load(const T *row, int c, int cols) {
        const uint16_t *h = reinterpret_cast<const uint16_t *>(row);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t lo = c + 2 * i < cols ? h[c + 2 * i] : 0, hi = c + 2 * i + 1 < cols ? h[c + 2 * i + 1] : 0;
            w[i] = lo | hi << 16;
        }
    }
    __device__ uint32_t amax() const {   // fp32 bits of the largest magnitude
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return __float_as_uint(elem_lo<D>(max(m & 0xFFFFu, m >> 16)));
    }
};

// Units of work: (row, 32 blocks), a block a lane. Their count fits 32 bits: the
// entry points refuse matrices of 2^32 segments of 256 columns and more.
template <typename T>
__global__ void __launch_bounds__(kQThreads, kQBlocks)
    mx4_quantize16_kernel(const T *__restrict__ x, int64_t ldx, int rows, int cols, uint8_t *__restrict__ codes,
                          uint8_t *__restrict__ scales, int rows_pad) {
    pdl_trigger();   // the product behind this kernel may start on its weights
    const int lane = threadIdx.x & 31;
    const int nb = (cols + 31) >> 5;
    const int kt_n = (nb + 3) >> 2;
    const uint32_t groups = (static_cast<uint32_t>(kt_n) + 7) >> 3;
    const uint32_t units = static_cast<uint32_t>(rows_pad) * groups;
    const uint32_t nw = gridDim.x * (kQThreads / 32);
    // the matrix's first and last byte, which no aligned word may leave
    const uintptr_t lo = reinterpret_cast<uintptr_t>(x);
    const uintptr_t hi = reinterpret_cast<uintptr_t>(x + static_cast<int64_t>(rows - 1) * ldx + cols);
    for (uint32_t u = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); u < units; u += nw) {
        const int r = static_cast<int>(u / groups);
        const int blk = static_cast<int>(u - static_cast<uint32_t>(r) * groups) * 32 + lane;
        const int c = blk * 32;
        const int have = r < rows ? cols : 0;   // rows that fill the last scale tile: zeros
        const T *row = x + r * ldx;
        const uintptr_t at = reinterpret_cast<uintptr_t>(row + c), word = at & ~static_cast<uintptr_t>(15);
        Block16<T> e;
        if (c + 32 <= have && at == word)
            e.load_full(row + c);
        else if (c + 32 <= have && word >= lo && word + Block16<T>::kWindow <= hi)
            e.load_shifted(row + c);
        else
            e.load(row, c, have);
        const uint32_t b = scale_byte(e.amax());
        const float inv = inv_scale(b == 255 ? 127u : b);
        uint32_t q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[2 * k] = elem_lo<Block16<T>::D>(e.w[4 * i + k]) * inv;
                v[2 * k + 1] = elem_hi<Block16<T>::D>(e.w[4 * i + k]) * inv;
            }
            q[i] = e2m1x8(v);
        }
        if (r < rows && blk < nb)
            *reinterpret_cast<uint4 *>(codes + (static_cast<int64_t>(r) * nb + blk) * 16) = make_uint4(q[0], q[1], q[2], q[3]);
        if ((blk >> 2) < kt_n)   // zero for blocks that fill the tile
            scales[(static_cast<int64_t>(r >> 7) * kt_n + (blk >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (blk & 3)] =
                static_cast<uint8_t>(b);
    }
}

// fp32: units of (row, U segments of 256 columns); large matrices take four
// segments at a time, small ones, where latency counts, one.
template <int U>
__global__ void __launch_bounds__(kQThreads)
    mx4_quantize32_kernel(const float *__restrict__ x, int64_t ldx, int rows, int cols, int vec,
                        uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, int rows_pad) {
    pdl_trigger();   // the product behind this kernel may start on its weights
    const int lane = threadIdx.x & 31;
    const uint32_t groups = (static_cast<uint32_t>(cols) + 256 * U - 1) / (256 * U);
    const int nb = (cols + 31) >> 5;
    const int kt_n = (nb + 3) >> 2;
    const uint32_t units = static_cast<uint32_t>(rows_pad) * groups;
    const uint32_t nw = gridDim.x * (kQThreads / 32);
    for (uint32_t w = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); w < units; w += nw) {
        const int r = static_cast<int>(w / groups);
        const int first = static_cast<int>(w - static_cast<uint32_t>(r) * groups) * 256 * U;
        const int c0 = first + lane * 8;
        const float *row = x + r * ldx;
        uint32_t *crow = reinterpret_cast<uint32_t *>(codes + static_cast<int64_t>(r) * nb * 16);
        uint8_t *srow = scales + static_cast<int64_t>(r >> 7) * kt_n * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
        Eight<float> e[U];
        if (r < rows && vec && first + 256 * U <= cols) {
#pragma unroll
            for (int s = 0; s < U; ++s) e[s].load_full(row + c0 + 256 * s);
        } else {
            const int have = r < rows ? cols : 0;   // rows that fill the last scale tile: zeros
            // the matrix's first and last byte, which no aligned word may leave
            const uintptr_t lo = reinterpret_cast<uintptr_t>(x);
            const uintptr_t hi = reinterpret_cast<uintptr_t>(x + static_cast<int64_t>(rows - 1) * ldx + cols);
#pragma unroll
            for (int s = 0; s < U; ++s) {
                const int c = c0 + 256 * s;
                const uintptr_t at = reinterpret_cast<uintptr_t>(row + c), word = at & ~static_cast<uintptr_t>(15);
                if (c + 8 <= have && at == word)
                    e[s].load_full(row + c);
                else if (c + 8 <= have && word >= lo && word + Eight<float>::kWindow <= hi)
                    e[s].load_shifted(row + c);
                else
                    e[s].load(row, c, have);
            }
        }
#pragma unroll
        for (int s = 0; s < U; ++s) {
            const int c = c0 + 256 * s;
            uint32_t b;
            const uint32_t q = quantize8(e[s], b);
            if (r < rows && c < nb * 32) crow[c >> 3] = q;
            // one lane of a block writes its scale, zero for blocks that fill the tile
            if ((lane & 3) == 0 && (c >> 7) < kt_n) srow[static_cast<int64_t>(c >> 7) * 512 + ((c >> 5) & 3)] = static_cast<uint8_t>(b);
        }
    }
}

// Four codes (the low 16 bits of q), unscaled, as four bf16 in two words. The
// magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 are 0000, 3F00, 3F80, 3FC0, 4000, 4040,
// 4080, 40C0 in bf16: their high and low bytes are looked up four at a time with a
// byte permutation.
__device__ __forceinline__ void decode4(uint32_t q, uint32_t &first, uint32_t &second) {
    const uint32_t m = q & 0x7777u;
    uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, m);
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, m);
    // a selector with its top bit set repeats the byte's sign bit: FF where the
    // code is negative, 80 elsewhere
    uint32_t sign;
    asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(q));
    hi |= (sign & 0x01010101u) << 7;
    first = __byte_perm(lo, hi, 0x5140);
    second = __byte_perm(lo, hi, 0x7362);
}
// bf16 bits of the scale 2^(b - 127): a subnormal for b = 0, NaN for b = 255.
__device__ __forceinline__ uint32_t scale_bits(uint32_t b) { return max(b << 7, 0x40u) + ((b + 1) >> 8); }
// A bf16 pair times two scales: exact, since a code has two significant bits.
__device__ __forceinline__ uint32_t mul2(uint32_t v, uint32_t s) {
    union {
        uint32_t u;
        __nv_bfloat162 h;
    } a, b;
    a.u = v;
    b.u = s;
    a.h = __hmul2_rn(a.h, b.h);
    return a.u;
}

// bf16 values to the output type: one, or 16 bytes of them in stores of kPiece bytes.
template <typename T>
__device__ __forceinline__ void store_one(T *dst, uint32_t bf16) {
    if constexpr (sizeof(T) == 4)
        *dst = bf16lo(bf16);
    else
        *reinterpret_cast<uint16_t *>(dst) =
            __is_same(T, __half) ? elem_round<KP_FP16>(bf16lo(bf16)) : static_cast<uint16_t>(bf16);
}
template <typename T, int kPiece>
__device__ __forceinline__ void store_word(T *dst, const uint32_t (&h)[4]) {
    uint32_t o[4];
    if constexpr (sizeof(T) == 4) {
        o[0] = h[0] << 16, o[1] = h[0] & 0xFFFF0000u, o[2] = h[1] << 16, o[3] = h[1] & 0xFFFF0000u;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            o[k] = __is_same(T, __half) ? elem_round<KP_FP16>(bf16lo(h[k])) |
                                              static_cast<uint32_t>(elem_round<KP_FP16>(bf16hi(h[k]))) << 16
                                        : h[k];
    }
    if constexpr (kPiece == 16) {
        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    } else if constexpr (kPiece == 8) {
        reinterpret_cast<uint2 *>(dst)[0] = make_uint2(o[0], o[1]);
        reinterpret_cast<uint2 *>(dst)[1] = make_uint2(o[2], o[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) reinterpret_cast<uint32_t *>(dst)[k] = o[k];
    }
}

// A warp takes 1024 columns of a row, a lane the V columns of 16 bytes of every 32 V,
// in stores of kPiece bytes: as wide as the rows' starts allow (8191 x 7156 in bf16,
// rows of 14312 bytes: 28 us in two stores a lane, 32 with 8 bytes a lane, 42 with the
// shifts below; 4096 x 7166 in four stores 16 us, with shifts 19). kShift, for 16-bit
// rows that start on 2 bytes: the columns before a row's first 16-byte boundary (h of
// them) are stored one by one, and the V columns of a store start inside a code word and
// may straddle two blocks (4096 x 7167: 19 us, with eight 2-byte stores a lane 87).
constexpr int kDqSpan = 1024;
template <typename T, int kPiece, bool kShift>
__global__ void __launch_bounds__(kQThreads)
    mx4_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int rows,
                          int cols, T *__restrict__ y, int64_t ldy) {
    constexpr int V = 16 / sizeof(T);
    constexpr int kSteps = kDqSpan / (32 * V);
    const int lane = threadIdx.x & 31;
    const int nb = (cols + 31) >> 5;
    const int kt_n = (nb + 3) >> 2;
    const uint32_t groups = (static_cast<uint32_t>(cols) + kDqSpan - 1) / kDqSpan;
    const uint32_t units = static_cast<uint32_t>(rows) * groups;
    const uint32_t nw = gridDim.x * (kQThreads / 32);
    for (uint32_t w = blockIdx.x * (kQThreads / 32) + (threadIdx.x >> 5); w < units; w += nw) {
        const int r = static_cast<int>(w / groups);
        const int first = static_cast<int>(w - static_cast<uint32_t>(r) * groups) * kDqSpan;
        const uint32_t *crow = reinterpret_cast<const uint32_t *>(codes + static_cast<int64_t>(r) * nb * 16);
        const uint8_t *srow = scales + static_cast<int64_t>(r >> 7) * kt_n * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4;
        auto scale_at = [&](int c) { return static_cast<uint32_t>(__ldg(srow + static_cast<int64_t>(c >> 7) * 512 + ((c >> 5) & 3))); };
        T *row = y + r * ldy;
        int h = 0;
        if constexpr (kShift) {
            h = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / static_cast<int>(sizeof(T));
            if (first == 0 && lane < h && lane < cols) {
                uint32_t a, b;
                decode4(__ldg(crow + (lane >> 3)) >> (4 * (lane & 7)), a, b);
                store_one(row + lane, mul2(a, scale_bits(scale_at(lane))));
            }
        }
        const int c0 = first + h + lane * V;
        uint32_t q[kSteps], s0[kSteps], s1[kSteps];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = c0 + s * 32 * V;
            q[s] = s0[s] = s1[s] = 0;
            if (c < cols) {   // a row's codes fill whole blocks, so the word is there
                if constexpr (kShift) {
                    const int i = c >> 3;
                    q[s] = __funnelshift_r(__ldg(crow + i), i + 1 < nb * 4 ? __ldg(crow + i + 1) : 0u, 4 * (c & 7));
                    s0[s] = scale_at(c);
                    s1[s] = scale_at(min(c + V, cols) - 1);
                } else {
                    q[s] = V == 8 ? __ldg(crow + (c >> 3)) : __ldg(crow + (c >> 3)) >> (4 * (c & 7));
                    s0[s] = scale_at(c);
                }
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            const int c = c0 + s * 32 * V;
            uint32_t v[4] = {0, 0, 0, 0};
            decode4(q[s], v[0], v[1]);
            if constexpr (V == 8) decode4(q[s] >> 16, v[2], v[3]);
            const uint32_t a = scale_bits(s0[s]);
            if constexpr (kShift) {
                const uint32_t b = scale_bits(s1[s]);
                const int left = 32 - (c & 31);   // columns up to the next block
#pragma unroll
                for (int k = 0; k < V / 2; ++k)
                    v[k] = mul2(v[k], (2 * k < left ? a : b) | (2 * k + 1 < left ? a : b) << 16);
            } else {
#pragma unroll
                for (int k = 0; k < V / 2; ++k) v[k] = mul2(v[k], a | a << 16);
            }
            if (c + V <= cols) {
                store_word<T, kPiece>(row + c, v);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    if (c + k < cols) store_one(row + c + k, k & 1 ? v[k / 2] >> 16 : v[k / 2]);
            }
        }
    }
}

bool rows_vectorise(const void *p, int64_t ld, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * es) % 16 == 0;
}

int grid_for(int64_t warps, int sms, int per_sm) {
    const int64_t blocks = (warps + kQThreads / 32 - 1) / (kQThreads / 32);
    const int64_t most = static_cast<int64_t>(sms) * per_sm;
    return static_cast<int>(blocks < most ? blocks : most);
}

template <typename T>
void quantize16(const void *x, int64_t ldx, int rows, int cols, uint8_t *codes, uint8_t *scales, int rows_pad, int sms,
                cudaStream_t s) {
    const int64_t units = static_cast<int64_t>(rows_pad) * ((cols + 1023) / 1024);
    mx4_quantize16_kernel<T><<<grid_for(units, sms, kQBlocks), kQThreads, 0, s>>>(static_cast<const T *>(x), ldx, rows, cols,
                                                                                  codes, scales, rows_pad);
}

void quantize32(const void *x, int64_t ldx, int rows, int cols, uint8_t *codes, uint8_t *scales, int rows_pad, int sms,
                cudaStream_t s) {
    const int vec = rows_vectorise(x, ldx, 4);
    const float *p = static_cast<const float *>(x);
    const int64_t segs = static_cast<int64_t>(rows_pad) * ((cols + 255) / 256);
    if (segs >= static_cast<int64_t>(sms) * 8 * (kQThreads / 32) * 4)   // four segments for every warp
        mx4_quantize32_kernel<4><<<grid_for(static_cast<int64_t>(rows_pad) * ((cols + 1023) / 1024), sms, 8), kQThreads, 0, s>>>(
            p, ldx, rows, cols, vec, codes, scales, rows_pad);
    else
        mx4_quantize32_kernel<1><<<grid_for(segs, sms, 8), kQThreads, 0, s>>>(p, ldx, rows, cols, vec, codes, scales,
                                                                              rows_pad);
}

template <typename T>
void dequantize_go(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y, int64_t ldy, int sms,
                   cudaStream_t s) {
    T *p = static_cast<T *>(y);
    const int grid = grid_for(static_cast<int64_t>(rows) * ((cols + kDqSpan - 1) / kDqSpan), sms, 8);
    const uintptr_t starts = reinterpret_cast<uintptr_t>(y) | static_cast<uintptr_t>(ldy * sizeof(T));
    if (starts % 16 == 0)
        mx4_dequantize_kernel<T, 16, false><<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, p, ldy);
    else if (starts % 8 == 0)
        mx4_dequantize_kernel<T, 8, false><<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, p, ldy);
    else if (sizeof(T) == 4 || starts % 4 == 0)
        mx4_dequantize_kernel<T, 4, false><<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, p, ldy);
    else if constexpr (sizeof(T) == 2)
        mx4_dequantize_kernel<T, 16, true><<<grid, kQThreads, 0, s>>>(codes, scales, rows, cols, p, ldy);
}

}  // namespace

cudaError_t mx4_quantize_launch(const void *x, int64_t ldx, int rows, int cols, int dtype, uint8_t *codes,
                                uint8_t *scales, bool pad, int sms, cudaStream_t s) {
    const int rows_pad = pad ? (rows + 127) / 128 * 128 : rows;
    if (dtype == KP_FP32)
        quantize32(x, ldx, rows, cols, codes, scales, rows_pad, sms, s);
    else if (dtype == KP_FP16)
        quantize16<__half>(x, ldx, rows, cols, codes, scales, rows_pad, sms, s);
    else
        quantize16<__nv_bfloat16>(x, ldx, rows, cols, codes, scales, rows_pad, sms, s);
    return cudaGetLastError();
}

cudaError_t mx4_dequantize_launch(const uint8_t *codes, const uint8_t *scales, int rows, int cols, void *y,
                                  int64_t ldy, int dtype, int sms, cudaStream_t s) {
    if (dtype == KP_FP32)
        dequantize_go<float>(codes, scales, rows, cols, y, ldy, sms, s);
    else if (dtype == KP_FP16)
        dequantize_go<__half>(codes, scales, rows, cols, y, ldy, sms, s);
    else
        dequantize_go<__nv_bfloat16>(codes, scales, rows, cols, y, ldy, sms, s);
    return cudaGetLastError();
}

}  // namespace kp
