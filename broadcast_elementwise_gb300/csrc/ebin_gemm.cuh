// Matrix products with bias, activation and residual in the epilogue.
#pragma once

#include <type_traits>

#include "ebin_act.cuh"

namespace ebin {

struct GemmEpilogue {
    const void *bias;       // [n], or null
    const void *residual;   // [m][n], or null
    void *y;
    void *z;                // receives the pre-activation, or null
    int64_t ld_residual, ldy, ldz;
    int32_t bias_f32;
    int32_t act;
};

struct GemmShape {
    int64_t m, n, k;
};

// ------------------------------------------------------------------ the simple kernel
//
// One output element per accumulator, operands through shared memory element
// by element: any transposes, strides and alignment.

struct GemmAnyArgs {
    const void *a, *b;
    int64_t a_m, a_k, b_k, b_n;   // element strides
    GemmShape s;
    GemmEpilogue e;
};

template <class T, int ACT>
__device__ __forceinline__ void gemm_store(const GemmEpilogue &e, int64_t m, int64_t n, float z) {
    if (e.bias)
        z += e.bias_f32 ? static_cast<const float *>(e.bias)[n]
                        : to_f(static_cast<const T *>(e.bias)[n]);
    if (e.z) static_cast<T *>(e.z)[m * e.ldz + n] = from_f<T>(z);
    float y = act_value<ACT>(z);
    if (e.residual) y += to_f(static_cast<const T *>(e.residual)[m * e.ld_residual + n]);
    static_cast<T *>(e.y)[m * e.ldy + n] = from_f<T>(y);
}

template <class T, int ACT>
__global__ void __launch_bounds__(256) k_gemm_any(const GemmAnyArgs g) {
    __shared__ float s_a[16][64 + 1], s_b[16][64 + 1];
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    layer_pdl_launch();
    layer_pdl_wait();
    const T *a = static_cast<const T *>(g.a), *b = static_cast<const T *>(g.b);
    for (int64_t k0 = 0; k0 < g.s.k; k0 += 16) {
        for (int i = threadIdx.x; i < 16 * 64; i += 256) {
            // neighbouring threads along the dense direction of each operand
            const int ka = g.a_k == 1 ? i & 15 : i >> 6, ma = g.a_k == 1 ? i >> 4 : i & 63;
            const int kb = g.b_k == 1 ? i & 15 : i >> 6, nb = g.b_k == 1 ? i >> 4 : i & 63;
            s_a[ka][ma] = m0 + ma < g.s.m && k0 + ka < g.s.k
                ? to_f(a[(m0 + ma) * g.a_m + (k0 + ka) * g.a_k]) : 0.0f;
            s_b[kb][nb] = n0 + nb < g.s.n && k0 + kb < g.s.k
                ? to_f(b[(k0 + kb) * g.b_k + (n0 + nb) * g.b_n]) : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(s_a[k][ty + 16 * i], s_b[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < g.s.m && n < g.s.n) gemm_store<T, ACT>(g.e, m, n, acc[i][j]);
        }
}

}  // namespace ebin
