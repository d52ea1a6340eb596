// Products grouped by expert.
#include "kp_moe.cuh"

namespace kp {

namespace {

constexpr int kT = 64, kKb = 16;

struct GroupedParams {
    GroupedArgs a;
    int tiles_m;
};

// out[n][m] = sum_k A[m, k] B[n, k] for one 64 x 64 tile; n the rows (WGRAD: features).
template <int kForm>
__global__ void __launch_bounds__(256) grouped_kernel(const GroupedParams p) {
    const GroupedArgs &a = p.a;
    __shared__ float sa[2][kKb][kT + 1], sb[2][kKb][kT + 1];
    const uint16_t *x = static_cast<const uint16_t *>(a.x);
    const int e = blockIdx.z;
    int first, count;
    expert_rows(a.offsets, e, a.R, first, count);
    const int tm = blockIdx.x * kT;
    const int cols = kForm == GROUPED_DGRAD || kForm == GROUPED_WGRAD ? a.K : a.N;
    const int rows = kForm == GROUPED_WGRAD ? a.N : count;
    const int depth = kForm == GROUPED_WGRAD ? count : kForm == GROUPED_DGRAD ? a.N : a.K;
    const bool two = kForm == GROUPED_GATED || a.d1;
    const float scale = a.scale ? __ldg(a.scale) : 1.f;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int tn = blockIdx.y * kT; tn < rows; tn += gridDim.y * kT) {
        float acc[2][4][4] = {};
        for (int q = 0; q < (two ? 2 : 1); ++q) {
            const MoeMat &w = q ? a.w1 : a.w0;
            const uint16_t *W = static_cast<const uint16_t *>(w.p) + e * w.se;
            const uint16_t *d = static_cast<const uint16_t *>(q ? a.d1 : a.d0);
            for (int k0 = 0; k0 < depth; k0 += kKb) {
                for (int i = threadIdx.x; i < kT * kKb; i += 256) {
                    const int m = kForm == GROUPED_PLAIN || kForm == GROUPED_GATED ? i / kKb : i % kT;
                    const int k = kForm == GROUPED_PLAIN || kForm == GROUPED_GATED ? i % kKb : i / kT;
                    float va = 0.f, vb = 0.f;
                    if (k0 + k < depth && tm + m < cols) {
                        const uint16_t *s = kForm == GROUPED_WGRAD   ? x + static_cast<int64_t>(first + k0 + k) * a.ldx + tm + m
                                            : kForm == GROUPED_DGRAD ? W + static_cast<int64_t>(k0 + k) * w.ld + tm + m
                                                                     : W + static_cast<int64_t>(tm + m) * w.ld + k0 + k;
                        va = elem_widen(*s, a.dtype);
                    }
                    if (k0 + k < depth && tn + m < rows) {
                        const uint16_t *s = kForm == GROUPED_WGRAD   ? d + static_cast<int64_t>(first + k0 + k) * a.ldd + tn + m
                                            : kForm == GROUPED_DGRAD ? d + static_cast<int64_t>(first + tn + m) * a.ldd + k0 + k
                                                                     : x + static_cast<int64_t>(first + tn + m) * a.ldx + k0 + k;
                        vb = elem_widen(*s, a.dtype);
                    }
                    sa[0][k][m] = va;
                    sb[0][k][m] = vb;
                }
                __syncthreads();
                float(&c)[4][4] = acc[kForm == GROUPED_DGRAD ? 0 : q];
#pragma unroll
                for (int k = 0; k < kKb; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sb[0][k][ty * 4 + i], sa[0][k][tx + 16 * j], c[i][j]);
                __syncthreads();
            }
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) {
                const int n = tn + ty * 4 + i, m = tm + tx + 16 * j;
                if (n >= rows || m >= cols) continue;
                if (kForm == GROUPED_WGRAD) {
                    const int64_t at = (static_cast<int64_t>(e) * a.N + n) * a.K + m;
                    static_cast<uint16_t *>(a.y0)[at] = elem_round(acc[0][i][j] * scale, a.dtype);
                    if (two) static_cast<uint16_t *>(a.y1)[at] = elem_round(acc[1][i][j] * scale, a.dtype);
                } else {
                    float v = acc[0][i][j] * scale;
                    if (kForm == GROUPED_GATED) {
                        const float ga[1] = {acc[0][i][j]}, ub[1] = {acc[1][i][j]};
                        float h[1];
                        ffn_gate(ga, ub, a.act, h);
                        v = h[0];
                        if (a.g) {
                            a.g[static_cast<int64_t>(first + n) * a.N + m] = ga[0];
                            a.u[static_cast<int64_t>(first + n) * a.N + m] = ub[0];
                        }
                    }
                    static_cast<uint16_t *>(a.y0)[(first + n) * a.ldy + m] = elem_round(v, a.dtype);
                }
            }
    }
}

}  // namespace

cudaError_t grouped_launch(const GroupedArgs &a, const FfnDev &d, cudaStream_t s) {
    GroupedParams p;
    p.a = a;
    const bool wgrad = a.form == GROUPED_WGRAD;
    const int cols = wgrad || a.form == GROUPED_DGRAD ? a.K : a.N;
    const int rows = wgrad ? a.N : a.R;
    const dim3 grid((cols + kT - 1) / kT, rows < 64 * kT ? (rows + kT - 1) / kT : 64, a.E);
    switch (a.form) {
    case GROUPED_PLAIN: grouped_kernel<GROUPED_PLAIN><<<grid, 256, 0, s>>>(p); break;
    case GROUPED_GATED: grouped_kernel<GROUPED_GATED><<<grid, 256, 0, s>>>(p); break;
    case GROUPED_DGRAD: grouped_kernel<GROUPED_DGRAD><<<grid, 256, 0, s>>>(p); break;
    default: grouped_kernel<GROUPED_WGRAD><<<grid, 256, 0, s>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace kp
