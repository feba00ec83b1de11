// Kernels on the heads of q and k: rotary positions, and the RMS norm of each
// head with the rotation in the same pass, forward and gradient.
//
// Every kernel reads each input element once and writes each output element
// once; the floor is that traffic.  Arithmetic is binary32 throughout, with
// one rounding to the element type at the store.
#pragma once

#include "ebin_layer.h"

namespace ebin {

constexpr int kHeadsThreads = 256;
constexpr int kHeadsMaxDim = 1024;

enum HeadsMode : int { HEADS_ROTATE = 0, HEADS_NORM = 1, HEADS_NORM_GRAD = 2 };

struct HeadsTensor {
    const void *p;
    int64_t sb, st, sh;   // element strides: batch, token, head
};

struct HeadsArgs {
    HeadsTensor x[2];     // forward inputs of q and k (without a norm: what is rotated)
    HeadsTensor dy[2];    // incoming gradients (HEADS_NORM_GRAD)
    HeadsTensor y[2];     // outputs
    const void *w[2];     // norm weights, or null for 1
    const float *cos, *sin;   // [table, half]
    const void *pos;
    int64_t ps_b, ps_t;   // position strides
    int64_t table;
    int64_t tokens, rows; // tokens of a sequence; batch * tokens
    int32_t heads[2];
    int32_t dim, half;    // head_dim, rotary_dim / 2
    int32_t pos_size;     // 0 (the token's index), 4 or 8
    int32_t w_f32;        // weights are binary32
    float eps;
    float sign;           // -1: the transposed rotation
    uint32_t *status;
    float *partial[2];    // HEADS_NORM_GRAD: [CTAs of the tensor][dim] weight-gradient sums
};

__device__ __forceinline__ int64_t heads_offset(const HeadsTensor &t, int64_t b, int64_t s,
                                                int64_t h) {
    return b * t.sb + s * t.st + h * t.sh;
}

// The table row of token s of sequence b; -1 when it lies outside the table.
__device__ __forceinline__ int64_t heads_position(const HeadsArgs &a, int64_t b, int64_t s) {
    if (a.half == 0) return 0;
    int64_t p = s;
    if (a.pos_size == 4)
        p = static_cast<const int32_t *>(a.pos)[b * a.ps_b + s * a.ps_t];
    else if (a.pos_size == 8)
        p = static_cast<const int64_t *>(a.pos)[b * a.ps_b + s * a.ps_t];
    return (p >= 0 && p < a.table) ? p : -1;
}

template <class T>
__device__ __forceinline__ float heads_weight(const HeadsArgs &a, int which, int j) {
    if (!a.w[which]) return 1.0f;
    return a.w_f32 ? static_cast<const float *>(a.w[which])[j]
                   : to_f(static_cast<const T *>(a.w[which])[j]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// One warp per (token, head) row, element by element: any head_dim, any
// strides, any alignment.  A lane owns whole pairs (and single elements past
// rotary_dim), so an output may be its own input.  grid.y picks q or k; a CTA
// of the gradient keeps its warps' weight-gradient sums in shared memory.
template <class T, int MODE>
__global__ void __launch_bounds__(kHeadsThreads) k_heads_any(const HeadsArgs a, int interleaved) {
    extern __shared__ float s_dw[];   // HEADS_NORM_GRAD: [warps][dim]
    const int which = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int kWarps = kHeadsThreads / 32;
    const int D = a.dim, half = a.half, slots = D - half;   // a pair or a single element each
    const int heads = a.heads[which];
    layer_pdl_launch();
    if constexpr (MODE == HEADS_NORM_GRAD)
        for (int j = threadIdx.x; j < kWarps * D; j += kHeadsThreads) s_dw[j] = 0.0f;
    layer_pdl_wait();
    if constexpr (MODE == HEADS_NORM_GRAD) __syncthreads();
    bool bad = false;
    const int64_t total = a.rows * heads;
    for (int64_t row = (int64_t)blockIdx.x * kWarps + warp; row < total;
         row += (int64_t)gridDim.x * kWarps) {
        const int64_t bs = row / heads, h = row - bs * heads;
        const int64_t b = bs / a.tokens, s = bs - b * a.tokens;
        const T *x = static_cast<const T *>(a.x[which].p) + heads_offset(a.x[which], b, s, h);
        T *y = static_cast<T *>(const_cast<void *>(a.y[which].p)) +
               heads_offset(a.y[which], b, s, h);
        const T *dy = nullptr;
        if constexpr (MODE == HEADS_NORM_GRAD)
            dy = static_cast<const T *>(a.dy[which].p) + heads_offset(a.dy[which], b, s, h);
        const int64_t p = heads_position(a, b, s);
        if (p < 0) {
            bad = true;
            for (int j = lane; j < D; j += 32) y[j] = from_f<T>(0.0f);
            continue;
        }
        const float *cs = a.cos + p * half, *sn = a.sin + p * half;
        // a slot's elements: i0 and, in a rotated pair, i1
        auto first = [&](int k) { return k >= half ? k + half : (interleaved ? 2 * k : k); };
        auto second = [&](int k) { return interleaved ? 2 * k + 1 : k + half; };
        float ss = 0.0f, dot = 0.0f;
        if constexpr (MODE != HEADS_ROTATE) {
            for (int k = lane; k < slots; k += 32) {
                const int i0 = first(k);
                const float x0 = to_f(x[i0]);
                ss = fmaf(x0, x0, ss);
                float x1 = 0.0f;
                if (k < half) {
                    x1 = to_f(x[second(k)]);
                    ss = fmaf(x1, x1, ss);
                }
                if constexpr (MODE == HEADS_NORM_GRAD) {
                    float g0 = to_f(dy[i0]);
                    if (k < half) {
                        const int i1 = second(k);
                        const float d1 = to_f(dy[i1]), c = cs[k], n = sn[k];
                        const float g1 = d1 * c - g0 * n;
                        g0 = g0 * c + d1 * n;
                        dot = fmaf(g1 * heads_weight<T>(a, which, i1), x1, dot);
                    }
                    dot = fmaf(g0 * heads_weight<T>(a, which, i0), x0, dot);
                }
            }
            ss = warp_sum(ss);
            if constexpr (MODE == HEADS_NORM_GRAD) dot = warp_sum(dot);
        }
        const float rstd = MODE == HEADS_ROTATE ? 1.0f : rsqrtf(ss / (float)D + a.eps);
        const float mean = dot * rstd / (float)D;
        for (int k = lane; k < slots; k += 32) {
            const int i0 = first(k), i1 = k < half ? second(k) : -1;
            float x0 = to_f(x[i0]) * rstd, x1 = i1 >= 0 ? to_f(x[i1]) * rstd : 0.0f;
            const float c = i1 >= 0 ? cs[k] : 1.0f, n = i1 >= 0 ? sn[k] * a.sign : 0.0f;
            if constexpr (MODE == HEADS_NORM_GRAD) {
                float g0 = to_f(dy[i0]);
                const float w0 = heads_weight<T>(a, which, i0);
                if (i1 >= 0) {
                    const float d1 = to_f(dy[i1]), w1 = heads_weight<T>(a, which, i1);
                    const float g1 = d1 * c + g0 * n;      // n carries the transpose's sign
                    g0 = g0 * c - d1 * n;
                    s_dw[warp * D + i1] += g1 * x1;
                    y[i1] = from_f<T>(rstd * (g1 * w1 - x1 * mean));
                }
                s_dw[warp * D + i0] += g0 * x0;
                y[i0] = from_f<T>(rstd * (g0 * w0 - x0 * mean));
            } else {
                if constexpr (MODE == HEADS_NORM) {
                    x0 *= heads_weight<T>(a, which, i0);
                    if (i1 >= 0) x1 *= heads_weight<T>(a, which, i1);
                }
                if (i1 >= 0) {
                    y[i0] = from_f<T>(x0 * c - x1 * n);
                    y[i1] = from_f<T>(x1 * c + x0 * n);
                } else {
                    y[i0] = from_f<T>(x0);
                }
            }
        }
    }
    if (bad && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
    if constexpr (MODE == HEADS_NORM_GRAD) {
        __syncthreads();
        for (int j = threadIdx.x; j < D; j += kHeadsThreads) {
            float v = 0.0f;
            for (int w = 0; w < kWarps; ++w) v += s_dw[w * D + j];
            a.partial[which][(int64_t)blockIdx.x * D + j] = v;
        }
    }
}

// The last step of the weight gradients: dw[j] = the sum of partial[.][j] over
// the CTAs, in an order fixed by their number.  grid (columns / 32, 2).
struct HeadsDwArgs {
    const float *partial[2];
    int64_t count[2];
    float *dw[2];
    int32_t dim;
};

__global__ void __launch_bounds__(1024) k_heads_dw(const HeadsDwArgs a);

}  // namespace ebin
