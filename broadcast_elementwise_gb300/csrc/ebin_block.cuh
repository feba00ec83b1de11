// Kernels of the norms around a block: norm of the block's output, gate, dropout,
// scaled addition to the residual stream, norm of the stream and its modulation,
// forward and gradient.  Bound by memory: forward x and y in, h and z out; a gradient dz,
// dh, h and y in, dx and dy out, and the parameters' sums.  Three sets of kernels:
// units of a CTA (ebin_block_unit.cuh), where nearly all rows go; a row a team
// (ebin_block_rows.cuh); and those of any width, below.
#pragma once

#include "ebin_philox.cuh"

namespace ebin {

// The rows of a group in `parts` parts of `rows`.
struct BlockUnits {
    int64_t parts = 1, rows = 0;
};

// The kernels of CTAs' units: chunks of 256 columns that a lane owns, threads and warps.
constexpr int kUnitVpt = 4, kUnitThreads = 512, kUnitWarps = kUnitThreads / 32;
constexpr int64_t kUnitColumns = 8192;   // the widest rows that they take
// A gradient's chunks: what it keeps of a column fits 128 registers (with a layer norm
// and none after the block three sums: [16388,1152] bf16 66 us, 80 with three chunks a lane).
template <bool FULL, bool POST> constexpr int kUnitGradVpt = FULL && POST ? 1 : 2;

struct BlockArgs {
    // forward: x, y -> h, z; gradient: dz, dh, h, y -> dx, dy
    const void *x, *y, *dz, *dh;   // x: the gradient's h
    void *h, *z;                   // the gradient's dx, dy
    int64_t ld_x, ld_y, ld_dz, ld_dh, ld_h, ld_z;
    const void *gate, *w_post, *b_post, *w_pre, *b_pre, *scale, *shift;
    int64_t ld_gate, ld_scale, ld_shift;
    int64_t gate_rows, mod_rows;   // rows that share a row of them, at least 1
    int64_t rows, n;
    float stream_scale, branch_scale;
    float eps_post, eps_pre;
    int32_t post, pre;             // ebin_norm
    int32_t w_f32, mod_f32;
    DropArgs drop;
    BlockUnits cta, team;          // units of a CTA, of a team
    int64_t groups, group_rows;
    float *partial;                // [units][4][pad]: sums of dz hh, dz, e yh, e; or null
    int64_t pad;                   // n in whole vectors of four
    int32_t need;                  // which of the four, by bit
};

enum BlockSum : int { SUM_DZ_HH = 0, SUM_DZ = 1, SUM_E_YH = 2, SUM_E = 3 };

// Whether a gradient's units take the full kernel: a layer norm, or a shift's or a bias's
// gradient.
inline bool unit_grad_full(int post, int pre, int need) {
    return post == EBIN_NORM_LAYER || pre == EBIN_NORM_LAYER || need >> SUM_DZ & 1 ||
           need >> SUM_E & 1;
}

struct BlockSumsArgs {
    float *partial;                // [groups * parts][4][pad]
    int64_t parts, groups, n, pad;
    int64_t tiles;                 // of 32 columns
    const void *gate, *w_post, *b_post, *w_pre, *b_pre, *scale;
    int64_t ld_gate, ld_scale;
    int32_t gate_grouped, mod_grouped;
    int32_t w_f32, mod_f32, dtype;
    int32_t need;
    int32_t second;                // a second launch joins the groups
    float *dgate, *dw_post, *db_post, *dw_pre, *db_pre, *dscale, *dshift;
};

// Element j of a parameter row; `none` where there is none.
template <class T>
__device__ __forceinline__ float block_param(const void *p, int64_t j, int f32, float none) {
    if (!p) return none;
    return f32 ? static_cast<const float *>(p)[j] : to_f(static_cast<const T *>(p)[j]);
}

template <class T>
__device__ __forceinline__ const void *block_row(const void *p, int64_t index, int f32) {
    if (!p) return nullptr;
    return f32 ? static_cast<const void *>(static_cast<const float *>(p) + index)
               : static_cast<const void *>(static_cast<const T *>(p) + index);
}

// ------------------------------------------------------------------ any width

constexpr int kBlockAnyThreads = 1024;

// The sum over the CTA of each v; every thread gets it.
template <int K> __device__ __forceinline__ void cta_sums(float (&v)[K], float *s) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    __syncthreads();   // the last sums have been read
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) s[(threadIdx.x >> 5) * K + k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = 0.0f;
        for (int w = 0; w < kBlockAnyThreads / 32; ++w) v[k] += s[w * K + k];
    }
}

// (mean, 1 / deviation) of value(0 .. n - 1): the mean first, then the squares
// about it (a RMS norm: about 0).
template <class F>
__device__ __forceinline__ float2 row_moments(const F &value, int64_t n, int norm, float eps,
                                              float *s) {
    if (norm == EBIN_NORM_NONE) return make_float2(0.0f, 1.0f);
    float v[1] = {0.0f}, mean = 0.0f;
    if (norm == EBIN_NORM_LAYER) {
        for (int64_t j = threadIdx.x; j < n; j += kBlockAnyThreads) v[0] += value(j);
        cta_sums(v, s);
        mean = v[0] / (float)n;
        v[0] = 0.0f;
    }
    for (int64_t j = threadIdx.x; j < n; j += kBlockAnyThreads) {
        const float d = value(j) - mean;
        v[0] = fmaf(d, d, v[0]);
    }
    cta_sums(v, s);
    return make_float2(mean, rsqrtf(v[0] / (float)n + eps));
}

__device__ __forceinline__ bool block_kept(const BlockArgs &a, int64_t row, int64_t j,
                                           uint2 offset) {
    if (!a.drop.least) return true;
    const uint4 w = drop_words(a.drop, (uint32_t)(j >> 2), (uint32_t)row, offset);
    const uint32_t word = (j & 2) ? ((j & 1) ? w.w : w.z) : ((j & 1) ? w.y : w.x);
    return word >= a.drop.least;
}
__device__ __forceinline__ float block_keep(const BlockArgs &a, float v, int64_t row, int64_t j,
                                            uint2 offset) {
    if (!a.drop.least) return v;
    return block_kept(a, row, j, offset) ? v * a.drop.scale : 0.0f;
}

// A CTA walks rows, a thread every 1024th column of each, with one pass over the
// row for each sum (from the L1 and L2 after the first): any width, any stride, any
// alignment, for rows of more than 32768 columns ([1000,40000] bf16 310 us, a sixth of
// the copy's rate; with 256 threads 1.2 times that).  A thread reads and writes the same columns in every
// pass, so an output may be an input.
template <class T, class S>
__global__ void __launch_bounds__(kBlockAnyThreads) k_block_any(const BlockArgs a) {
    __shared__ float s[kBlockAnyThreads / 32];
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const S *x = static_cast<const S *>(a.x) + row * a.ld_x;
        const T *y = static_cast<const T *>(a.y) + (a.y ? row * a.ld_y : 0);
        const void *gate = block_row<T>(a.gate, row / a.gate_rows * a.ld_gate, a.mod_f32);
        const void *scale = block_row<T>(a.scale, row / a.mod_rows * a.ld_scale, a.mod_f32);
        const void *shift = block_row<T>(a.shift, row / a.mod_rows * a.ld_shift, a.mod_f32);
        const float2 my = row_moments([&](int64_t j) { return to_f(y[j]); }, a.n, a.post,
                                      a.eps_post, s);
        auto stream = [&](int64_t j) {
            const float t = a.stream_scale * to_f(x[j]);
            if (!a.y) return t;
            float v = (to_f(y[j]) - my.x) * my.y;
            v = fmaf(v, block_param<T>(a.w_post, j, a.w_f32, 1.0f),
                     block_param<T>(a.b_post, j, a.w_f32, 0.0f));
            v = block_keep(a, v, row, j, offset);
            return fmaf(a.branch_scale * block_param<T>(gate, j, a.mod_f32, 1.0f), v, t);
        };
        const float2 mh = row_moments(stream, a.n, a.pre, a.eps_pre, s);
        for (int64_t j = threadIdx.x; j < a.n; j += kBlockAnyThreads) {
            const float h = stream(j);
            float z = (h - mh.x) * mh.y;
            z = fmaf(z, block_param<T>(a.w_pre, j, a.w_f32, 1.0f),
                     block_param<T>(a.b_pre, j, a.w_f32, 0.0f));
            z = fmaf(z, 1.0f + block_param<T>(scale, j, a.mod_f32, 0.0f),
                     block_param<T>(shift, j, a.mod_f32, 0.0f));
            if (a.h) static_cast<S *>(a.h)[row * a.ld_h + j] = from_f<S>(h);
            if (a.z) static_cast<T *>(a.z)[row * a.ld_z + j] = from_f<T>(z);
        }
    }
}

// The gradient, for rows of more than 16384 columns: a CTA takes a unit, rows of one group;
// its column sums stay in its part of the workspace, each column its thread's own, read
// and written for every row ([1000,20000] bf16 0.55 ms, with 256 threads and
// all four kinds 2.1).
template <class T, class S>
__global__ void __launch_bounds__(kBlockAnyThreads) k_block_any_grad(const BlockArgs a) {
    __shared__ float s[2 * (kBlockAnyThreads / 32)];
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    const int64_t group = blockIdx.x / a.team.parts, part = blockIdx.x - group * a.team.parts;
    const int64_t r0 = group * a.group_rows + part * a.team.rows;
    const int64_t r1 = min(r0 + a.team.rows, (group + 1) * a.group_rows);
    float *const sums = a.partial ? a.partial + (int64_t)blockIdx.x * 4 * a.pad : nullptr;
    if (sums)
        for (int64_t j = threadIdx.x; j < a.n; j += kBlockAnyThreads)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (a.need >> k & 1) sums[k * a.pad + j] = 0.0f;
    const float inv = 1.0f / (float)a.n;
    for (int64_t row = r0; row < r1; ++row) {
        const S *h = static_cast<const S *>(a.x) + (a.x ? row * a.ld_x : 0);
        const T *y = static_cast<const T *>(a.y) + (a.y ? row * a.ld_y : 0);
        const T *dz = static_cast<const T *>(a.dz) + (a.dz ? row * a.ld_dz : 0);
        const S *dh = static_cast<const S *>(a.dh) + (a.dh ? row * a.ld_dh : 0);
        const void *gate = block_row<T>(a.gate, row / a.gate_rows * a.ld_gate, a.mod_f32);
        const void *scale = block_row<T>(a.scale, row / a.mod_rows * a.ld_scale, a.mod_f32);
        const float2 mh = row_moments([&](int64_t j) { return to_f(h[j]); }, a.n, a.pre,
                                      a.eps_pre, s);
        auto normed = [&](int64_t j) { return (to_f(h[j]) - mh.x) * mh.y; };
        auto into = [&](int64_t j) {    // m
            return to_f(dz[j]) * (1.0f + block_param<T>(scale, j, a.mod_f32, 0.0f)) *
                   block_param<T>(a.w_pre, j, a.w_f32, 1.0f);
        };
        float c[2] = {0.0f, 0.0f};   // sums of m and of m hh
        if (a.pre != EBIN_NORM_NONE) {
            for (int64_t j = threadIdx.x; j < a.n; j += kBlockAnyThreads) {
                const float m = into(j);
                c[0] += m;
                c[1] = fmaf(m, normed(j), c[1]);
            }
            cta_sums(c, s);
            c[0] = a.pre == EBIN_NORM_LAYER ? c[0] * inv : 0.0f;
            c[1] *= inv;
        }
        auto total = [&](int64_t j) {   // D
            const float d = a.dh ? to_f(dh[j]) : 0.0f;
            if (a.pre == EBIN_NORM_NONE) return d;
            return fmaf(mh.y, into(j) - c[0] - normed(j) * c[1], d);
        };
        auto branch = [&](int64_t j, float d) {   // e
            return block_keep(a, a.branch_scale * d, row, j, offset);
        };
        const float2 my = row_moments([&](int64_t j) { return to_f(y[j]); }, a.n, a.post,
                                      a.eps_post, s);
        auto weigh = [&](int64_t j) {
            return block_param<T>(gate, j, a.mod_f32, 1.0f) *
                   block_param<T>(a.w_post, j, a.w_f32, 1.0f);
        };
        float b[2] = {0.0f, 0.0f};   // sums of u and of u yh
        if (a.post != EBIN_NORM_NONE) {
            for (int64_t j = threadIdx.x; j < a.n; j += kBlockAnyThreads) {
                const float u = branch(j, total(j)) * weigh(j);
                b[0] += u;
                b[1] = fmaf(u, (to_f(y[j]) - my.x) * my.y, b[1]);
            }
            cta_sums(b, s);
            b[0] = a.post == EBIN_NORM_LAYER ? b[0] * inv : 0.0f;
            b[1] *= inv;
        }
        for (int64_t j = threadIdx.x; j < a.n; j += kBlockAnyThreads) {
            const float d = total(j), e = branch(j, d);
            const float yh = a.y ? (to_f(y[j]) - my.x) * my.y : 0.0f;
            if (sums) {
                if (a.dz) {
                    const float g = to_f(dz[j]);
                    if (a.need >> SUM_DZ_HH & 1) sums[SUM_DZ_HH * a.pad + j] += g * normed(j);
                    if (a.need >> SUM_DZ & 1) sums[SUM_DZ * a.pad + j] += g;
                }
                // what is dropped adds nothing, whatever y is there
                if (a.need >> SUM_E_YH & 1 && block_kept(a, row, j, offset))
                    sums[SUM_E_YH * a.pad + j] += e * yh;
                if (a.need >> SUM_E & 1) sums[SUM_E * a.pad + j] += e;
            }
            float u = e * weigh(j);
            if (a.post != EBIN_NORM_NONE) u = my.y * (u - b[0] - yh * b[1]);
            if (a.h) static_cast<S *>(a.h)[row * a.ld_h + j] = from_f<S>(a.stream_scale * d);
            if (a.z) static_cast<T *>(a.z)[row * a.ld_z + j] = from_f<T>(u);
        }
    }
}

// The row kernels of a pair of types (0: float32, 1: float16, 2: bfloat16; 3, 4: these
// two beside a float32 stream; ebin_block_rows.cu).  parts: the units of a group that
// they took, 0 where they do not take rows of this width.
#define EBIN_DECLARE_ROWS(dt)                                                                \
    cudaError_t launch_block_rows_##dt(const BlockArgs &, bool vec, int64_t *parts,           \
                                       cudaStream_t);                                        \
    cudaError_t launch_block_rows_grad_##dt(const BlockArgs &, bool vec, int64_t *parts,      \
                                            cudaStream_t);
EBIN_DECLARE_ROWS(0)
EBIN_DECLARE_ROWS(1)
EBIN_DECLARE_ROWS(2)
EBIN_DECLARE_ROWS(3)
EBIN_DECLARE_ROWS(4)
#undef EBIN_DECLARE_ROWS

}  // namespace ebin
