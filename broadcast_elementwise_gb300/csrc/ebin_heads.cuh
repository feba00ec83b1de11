// Kernels on the heads of q and k: rotary positions, and the RMS norm of each
// head with the rotation in the same pass, forward and gradient.
//
// Every kernel reads each input element once and writes each output element
// once; the floor is that traffic.  Arithmetic is binary32 throughout, with
// one rounding to the element type at the store.
#pragma once

#include <type_traits>

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

// ------------------------------------------------------------------ 16-byte vectors
//
// The path of heads whose rows are whole 16-byte vectors on 16-byte
// boundaries.  A group of L lanes (a power of two) takes a token; a lane owns
// one unit of its heads, two vectors whose elements form V = 16 / sizeof(T)
// pairs (a[i], b[i]):
//   half layout          vectors at u V and half + u V for u < half / V, then
//                        two neighbouring vectors of what passes through
//   interleaved layout   vectors at 2 u V and (2 u + 1) V: pairs of neighbours
// so a rotation needs no exchange between lanes, and a norm one tree over L.
// Cosines, sines and weights stay in registers over the heads of one item.

struct HeadsVecArgs {
    int32_t log_lanes;
    int32_t units;          // lanes of a group with work
    int32_t rot_units;      // half layout: units that rotate
    int32_t table_vec;      // table rows may be read 16 bytes at a time
    int32_t groups[2];      // items of a token: groups of HPT heads of q, then of k
    int32_t wide;           // item indices pass 32 bits
    int32_t ctas[2];        // the gradient's CTAs for q and for k
};

template <class T, int V> struct HeadsVec {
    uint4 w;
    __device__ __forceinline__ float at(int i) const {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float((&w.x)[i]);
        } else {
            const uint32_t x = (&w.x)[i / 2];
            if constexpr (std::is_same<T, __nv_bfloat16>::value)
                return __uint_as_float(i % 2 ? (x & 0xFFFF0000u) : (x << 16));
            else
                return __half2float(__ushort_as_half((unsigned short)(i % 2 ? x >> 16 : x)));
        }
    }
};

template <class T> __device__ __forceinline__ uint32_t heads_pack2(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __half2 p = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
}

template <class T> __device__ __forceinline__ uint4 heads_load(const T *p) {
    uint4 r;
    // not .nc: an output may be its own input
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

template <class T, int V>
__device__ __forceinline__ void heads_store(T *p, const float *v) {
    uint4 r;
    if constexpr (sizeof(T) == 4)
        r = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                       __float_as_uint(v[3]));
    else
        r = make_uint4(heads_pack2<T>(v[0], v[1]), heads_pack2<T>(v[2], v[3]),
                       heads_pack2<T>(v[V - 4], v[V - 3]), heads_pack2<T>(v[V - 2], v[V - 1]));
    *reinterpret_cast<uint4 *>(p) = r;
}

// Where a lane's unit lies, and how its pairs read.
template <class T, bool IL> struct HeadsUnit {
    static constexpr int V = 16 / sizeof(T);
    int off0, off1;    // element offsets of the two vectors
    bool on, second;   // the lane has work; its second vector exists
    int pairs;         // leading pairs that rotate
    int pair0;         // the first pair's index in the table row

    __device__ __forceinline__ void place(const HeadsArgs &a, const HeadsVecArgs &v, int lane) {
        on = lane < v.units;
        if constexpr (IL) {
            off0 = 2 * lane * V;
            off1 = off0 + V;
            pair0 = lane * V;
            pairs = min(max(a.half - pair0, 0), V);
        } else {
            const bool rot = lane < v.rot_units;
            off0 = rot ? lane * V : 2 * a.half + 2 * (lane - v.rot_units) * V;
            off1 = rot ? a.half + off0 : off0 + V;
            pair0 = lane * V;
            pairs = rot ? V : 0;
        }
        second = on && off1 < a.dim;
    }
    __device__ __forceinline__ void load(const T *p, uint4 &x0, uint4 &x1) const {
        x0 = x1 = make_uint4(0, 0, 0, 0);
        if (on) x0 = heads_load(p + off0);
        if (second) x1 = heads_load(p + off1);
    }
    __device__ __forceinline__ static void open(const uint4 &x0, const uint4 &x1, float *a,
                                                float *b) {
        const HeadsVec<T, V> v0{x0}, v1{x1};
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (IL) {
                a[i] = i < V / 2 ? v0.at(2 * i) : v1.at(2 * i - V);
                b[i] = i < V / 2 ? v0.at(2 * i + 1) : v1.at(2 * i + 1 - V);
            } else {
                a[i] = v0.at(i);
                b[i] = v1.at(i);
            }
        }
    }
    __device__ __forceinline__ void store(T *p, const float *a, const float *b) const {
        float v0[V], v1[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if constexpr (IL) {
                v0[i] = i % 2 ? b[i / 2] : a[i / 2];
                v1[i] = i % 2 ? b[(i + V) / 2] : a[(i + V) / 2];
            } else {
                v0[i] = a[i];
                v1[i] = b[i];
            }
        }
        if (on) heads_store<T, V>(p + off0, v0);
        if (second) heads_store<T, V>(p + off1, v1);
    }
    __device__ __forceinline__ void angles(const HeadsArgs &a, const HeadsVecArgs &v, int64_t p,
                                           float *c, float *s) const {
        const float *cr = a.cos + p * a.half + pair0, *sr = a.sin + p * a.half + pair0;
        if (on && pairs == V && v.table_vec) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(cr + i));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(sr + i));
                c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
                s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const bool r = on && i < pairs;
                c[i] = r ? __ldg(cr + i) : 1.0f;
                s[i] = r ? __ldg(sr + i) : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] *= a.sign;
    }
    __device__ __forceinline__ void weights(const HeadsArgs &a, int which, float *wa,
                                            float *wb) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j0 = IL ? off0 + 2 * i : off0 + i, j1 = IL ? j0 + 1 : off1 + i;
            wa[i] = on && j0 < a.dim ? heads_weight<T>(a, which, j0) : 0.0f;
            wb[i] = on && j1 < a.dim ? heads_weight<T>(a, which, j1) : 0.0f;
        }
    }
    // a pair that does not rotate is left alone: an infinity times a zero sine is no number
    __device__ __forceinline__ void turn(float *a, float *b, const float *c,
                                         const float *s) const {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float x = a[i] * c[i] - b[i] * s[i], y = b[i] * c[i] + a[i] * s[i];
            const bool r = i < pairs;
            a[i] = r ? x : a[i];
            b[i] = r ? y : b[i];
        }
    }
};

__device__ __forceinline__ float group_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Quotient and remainder of an item index by a count (32-bit when it fits).
__device__ __forceinline__ void heads_split(int64_t i, int64_t n, int wide, int64_t &q,
                                            int64_t &r) {
    if (wide) {
        q = i / n;
        r = i - q * n;
    } else {
        const uint32_t qi = (uint32_t)i / (uint32_t)n;
        q = qi;
        r = (uint32_t)i - qi * (uint32_t)n;
    }
}

// Rotation, and norm with rotation.  An item is a token and HPT heads of q or
// of k; all its loads are issued before the first is used.
template <class T, bool IL, int MODE, int HPT>
__global__ void __launch_bounds__(kHeadsThreads)
k_heads_vec(const HeadsArgs a, const HeadsVecArgs v) {
    constexpr int V = 16 / sizeof(T);
    const int lanes = 1 << v.log_lanes, lane = threadIdx.x & (lanes - 1);
    layer_pdl_launch();
    const int64_t item = ((int64_t)blockIdx.x * kHeadsThreads + threadIdx.x) >> v.log_lanes;
    int64_t bs, g, b, s;
    heads_split(item, v.groups[0] + v.groups[1], v.wide, bs, g);
    const bool live = bs < a.rows;
    if (!live) bs = 0;            // the group still takes part in the warp's exchanges
    heads_split(bs, a.tokens, v.wide, b, s);
    const int which = g >= v.groups[0];
    const int h0 = (int)(which ? g - v.groups[0] : g) * HPT;
    const int count = live ? min(HPT, a.heads[which] - h0) : 0;
    HeadsUnit<T, IL> u;
    u.place(a, v, lane);
    const HeadsTensor tx = which ? a.x[1] : a.x[0], ty = which ? a.y[1] : a.y[0];
    const T *x = static_cast<const T *>(tx.p) + heads_offset(tx, b, s, h0);
    T *y = static_cast<T *>(const_cast<void *>(ty.p)) + heads_offset(ty, b, s, h0);
    layer_pdl_wait();
    uint4 x0[HPT], x1[HPT];
#pragma unroll
    for (int h = 0; h < HPT; ++h)
        if (h < count) u.load(x + h * tx.sh, x0[h], x1[h]);
        else x0[h] = x1[h] = make_uint4(0, 0, 0, 0);
    const int64_t p = heads_position(a, b, s);
    float c[V], sn[V], wa[V], wb[V];
    u.angles(a, v, p < 0 ? 0 : p, c, sn);
    if constexpr (MODE == HEADS_NORM) u.weights(a, which, wa, wb);
    if (p < 0 && live && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
#pragma unroll
    for (int h = 0; h < HPT; ++h) {
        float va[V], vb[V];
        u.open(x0[h], x1[h], va, vb);
        if constexpr (MODE == HEADS_NORM) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < V; ++i) ss = fmaf(va[i], va[i], fmaf(vb[i], vb[i], ss));
            const float rstd = rsqrtf(group_sum(ss, lanes) / (float)a.dim + a.eps);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                va[i] *= rstd * wa[i];
                vb[i] *= rstd * wb[i];
            }
        }
        u.turn(va, vb, c, sn);
        if (p < 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) va[i] = vb[i] = 0.0f;
        }
        if (h < count) u.store(y + h * ty.sh, va, vb);
    }
}

// The gradient of norm and rotation.  CTAs take items of q or of k only, in
// steps of their number, so a thread's weight-gradient sums stay in registers
// to the end; the CTA's sums then join in shared memory and go to its row of
// the workspace.
template <class T, bool IL>
__global__ void __launch_bounds__(kHeadsThreads)
k_heads_vec_grad(const HeadsArgs a, const HeadsVecArgs v) {
    constexpr int V = 16 / sizeof(T);
    extern __shared__ float s_dw[];   // [groups of the CTA][dim]
    const int lanes = 1 << v.log_lanes, lane = threadIdx.x & (lanes - 1);
    const int which = (int)blockIdx.x >= v.ctas[0];
    const int cta = (int)blockIdx.x - (which ? v.ctas[0] : 0);
    const int heads = a.heads[which];
    const HeadsTensor tx = which ? a.x[1] : a.x[0], tg = which ? a.dy[1] : a.dy[0],
                      ty = which ? a.y[1] : a.y[0];
    const int64_t total = a.rows * heads;
    const int per = kHeadsThreads >> v.log_lanes, group = threadIdx.x >> v.log_lanes;
    HeadsUnit<T, IL> u;
    u.place(a, v, lane);
    layer_pdl_launch();
    layer_pdl_wait();
    float wa[V], wb[V], da[V], db[V];
    u.weights(a, which, wa, wb);
#pragma unroll
    for (int i = 0; i < V; ++i) da[i] = db[i] = 0.0f;
    bool bad = false;
    // every lane of a warp makes the same number of steps: the exchanges are warp-wide
    const int64_t step = (int64_t)v.ctas[which] * per;
    for (int64_t base = (int64_t)cta * per; base < total; base += step) {
        const int64_t row = base + group;
        const bool live = row < total;
        int64_t bs, h, b, s;
        heads_split(live ? row : 0, heads, v.wide, bs, h);
        heads_split(bs, a.tokens, v.wide, b, s);
        uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, g0 = x0, g1 = x0;
        if (live) {
            u.load(static_cast<const T *>(tx.p) + heads_offset(tx, b, s, h), x0, x1);
            u.load(static_cast<const T *>(tg.p) + heads_offset(tg, b, s, h), g0, g1);
        }
        const int64_t p = heads_position(a, b, s);
        float c[V], sn[V], xa[V], xb[V], ga[V], gb[V];
        u.angles(a, v, p < 0 ? 0 : p, c, sn);
        u.open(x0, x1, xa, xb);
        u.open(g0, g1, ga, gb);
        u.turn(ga, gb, c, sn);
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            ss = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], ss));
            dot = fmaf(ga[i] * wa[i], xa[i], fmaf(gb[i] * wb[i], xb[i], dot));
        }
        ss = group_sum(ss, lanes);
        dot = group_sum(dot, lanes);
        const float rstd = rsqrtf(ss / (float)a.dim + a.eps);
        const float mean = dot * rstd / (float)a.dim;
        const bool use = live && p >= 0;
        bad |= live && p < 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            xa[i] *= rstd;
            xb[i] *= rstd;
            if (use) {
                da[i] = fmaf(ga[i], xa[i], da[i]);
                db[i] = fmaf(gb[i], xb[i], db[i]);
            }
            ga[i] = use ? rstd * (ga[i] * wa[i] - xa[i] * mean) : 0.0f;
            gb[i] = use ? rstd * (gb[i] * wb[i] - xb[i] * mean) : 0.0f;
        }
        if (live)
            u.store(static_cast<T *>(const_cast<void *>(ty.p)) + heads_offset(ty, b, s, h), ga,
                    gb);
    }
    if (bad && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int j0 = IL ? u.off0 + 2 * i : u.off0 + i, j1 = IL ? j0 + 1 : u.off1 + i;
        if (u.on && j0 < a.dim) s_dw[group * a.dim + j0] = da[i];
        if (u.on && j1 < a.dim) s_dw[group * a.dim + j1] = db[i];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.dim; j += kHeadsThreads) {
        float t = 0.0f;
        for (int r = 0; r < per; ++r) t += s_dw[r * a.dim + j];
        a.partial[which][(int64_t)cta * a.dim + j] = t;
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
