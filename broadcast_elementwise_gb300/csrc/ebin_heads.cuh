// Kernels on the heads of q and k: rotary positions, and the RMS norm of each
// head with the rotation in the same pass, forward and gradient.
//
// Bound by memory: every kernel but k_heads_any reads each input element once
// and writes each output element once, and the floor is that traffic.  Measured
// on GB300, bf16, q and k of 32 and 8 heads of 128, over sets of inputs that
// together pass the L2 (copy: 6694 GB/s):
//   rotation            [1,16384] tokens   52.5 us   6550 GB/s   k_heads_vec
//   norm and rotation   [2,4096] tokens    29.4 us   5780 GB/s   k_heads_ring
//   its gradient        [2,4096] tokens    46.1 us   5500 GB/s   k_heads_vec_grad
// With 62 of the 128 rotated (HEADS_ODD), [2,4096] tokens: 47.6, 70.0 and 82.0 us.
// Arithmetic is binary32 throughout, with one rounding to the element type at
// the store.
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
// rotary_dim), so an output may be its own input; a norm reads its row twice,
// the second time from the L1.  grid.y picks q or k; a CTA of the gradient keeps
// its warps' weight-gradient sums in shared memory.  The path of what has no
// vectors, one element a lane and access: an eighth of the copy's rate for heads of
// 128 off 16 bytes (rotation of [2,4096,40,128] bf16 195 us, norm 219, its gradient
// 271), a twentieth for heads of 33, where a row of 66 bytes takes a warp (143 us).
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
//   half layout whose half is no whole number of vectors   vectors at 2 u V and
//   (2 u + 1) V; the other element of each pair comes through shared memory
// Cosines, sines and weights stay in registers over the heads of one item.
enum HeadsKind : int { HEADS_HALF = 0, HEADS_PAIRS = 1, HEADS_ODD = 2 };

struct HeadsNear {          // a tensor whose token and head strides fit 32 bits
    const void *p;
    int64_t sb;
    int32_t st, sh;
};

struct HeadsVecArgs {
    HeadsNear x[2], dy[2], y[2];
    FastDiv per_token;     // items of a token: groups of HPT heads of q, then of k
    FastDiv tokens;        // tokens of a sequence
    FastDiv heads[2];      // the gradient's items of a token: kRingHeads heads of q, of k
    uint32_t q_items;       // of per_token
    uint32_t items;         // of the launch
    int32_t log_lanes;
    int32_t units;          // lanes of a group with work
    int32_t rot_units;      // half layout: units that rotate
    int32_t table_vec;      // table rows may be read 16 bytes at a time
    int32_t weight_vec;     // and the weights
    int32_t ctas[2];        // the gradient's CTAs for q and for k
};

__device__ __forceinline__ int64_t heads_near(const HeadsNear &t, uint32_t b, uint32_t s,
                                              uint32_t h) {
    return (int64_t)b * t.sb + (int64_t)(int32_t)s * t.st + (int64_t)(int32_t)h * t.sh;
}

template <class T> __device__ __forceinline__ uint4 heads_load(const T *p) {
    uint4 r;
    // not .nc: an output may be its own input
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// Where a lane's unit lies and how its pairs read: pairs 2i and 2i + 1 are
// (a[i].x, b[i].x) and (a[i].y, b[i].y), ready for the packed binary32 pipe.
template <class T, int KIND> struct HeadsUnit {
    static constexpr bool IL = KIND == HEADS_PAIRS, ODD = KIND == HEADS_ODD;
    static constexpr int V = 16 / sizeof(T), N = V / 2;
    int off0, off1;    // element offsets of the two vectors
    bool on, second;   // the lane has work; its second vector exists
    int pairs;         // leading pairs that rotate
    int pair0;         // the first pair's index in the table row

    __device__ __forceinline__ void place(const HeadsArgs &a, const HeadsVecArgs &v, int lane) {
        on = lane < v.units;
        if constexpr (ODD) {
            off0 = 2 * lane * V;
            off1 = off0 + V;
            pair0 = 0;
            pairs = min(max(2 * a.half - off0, 0), 2 * V);   // leading elements that rotate
        } else if constexpr (IL) {
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
        if (!on) pairs = 0;
        second = on && off1 < a.dim;
    }
    // every lane loads from inside the row: one without work (or without a
    // second vector) repeats the row's first vector, and masks what it sums
    __device__ __forceinline__ void load(const T *p, uint4 &x0, uint4 &x1) const {
        x0 = heads_load(p + (on ? off0 : 0));
        x1 = heads_load(p + (second ? off1 : 0));
    }
    __device__ __forceinline__ static void open(const uint4 &x0, const uint4 &x1, float2 *a,
                                                float2 *b) {
        if constexpr (sizeof(T) == 4) {
            float2 e[4];
            e[0] = make_float2(__uint_as_float(x0.x), __uint_as_float(x0.y));
            e[1] = make_float2(__uint_as_float(x0.z), __uint_as_float(x0.w));
            e[2] = make_float2(__uint_as_float(x1.x), __uint_as_float(x1.y));
            e[3] = make_float2(__uint_as_float(x1.z), __uint_as_float(x1.w));
            split(e, a, b);
        } else {
            float2 e[8];
            e[0] = open2<T>(x0.x);
            e[1] = open2<T>(x0.y);
            e[2] = open2<T>(x0.z);
            e[3] = open2<T>(x0.w);
            e[4] = open2<T>(x1.x);
            e[5] = open2<T>(x1.y);
            e[6] = open2<T>(x1.z);
            e[7] = open2<T>(x1.w);
            split(e, a, b);
        }
    }
    // e: the unit's elements two by two, in memory order
    __device__ __forceinline__ static void split(const float2 *e, float2 *a, float2 *b) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (IL) {
                a[i] = make_float2(e[2 * i].x, e[2 * i + 1].x);
                b[i] = make_float2(e[2 * i].y, e[2 * i + 1].y);
            } else {
                a[i] = e[i];
                b[i] = e[N + i];
            }
        }
    }
    __device__ __forceinline__ void store(T *p, const float2 *a, const float2 *b) const {
        float2 e[V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (IL) {
                e[2 * i] = make_float2(a[i].x, b[i].x);
                e[2 * i + 1] = make_float2(a[i].y, b[i].y);
            } else {
                e[i] = a[i];
                e[N + i] = b[i];
            }
        }
        uint4 r0, r1;
        if constexpr (sizeof(T) == 4) {
            r0 = make_uint4(__float_as_uint(e[0].x), __float_as_uint(e[0].y),
                            __float_as_uint(e[1].x), __float_as_uint(e[1].y));
            r1 = make_uint4(__float_as_uint(e[2].x), __float_as_uint(e[2].y),
                            __float_as_uint(e[3].x), __float_as_uint(e[3].y));
        } else {
            r0 = make_uint4(pack2<T>(e[0]), pack2<T>(e[1]), pack2<T>(e[2]),
                            pack2<T>(e[3]));
            r1 = make_uint4(pack2<T>(e[V - 4]), pack2<T>(e[V - 3]),
                            pack2<T>(e[V - 2]), pack2<T>(e[V - 1]));
        }
        if (on) *reinterpret_cast<uint4 *>(p + off0) = r0;
        if (second) *reinterpret_cast<uint4 *>(p + off1) = r1;
    }
    // ODD: element k of the unit (0 .. 2 V - 1) turns with element other(k) of
    // the row: y = x c + x_other s, s = -sin for the row's first half and sin for
    // its second, times `sign`
    __device__ __forceinline__ int other(int half, int k) const {
        const int j = off0 + k;
        return j < half ? j + half : j - half;
    }
    __device__ __forceinline__ void factors(const HeadsArgs &a, int64_t p, float sign, float2 *ca,
                                            float2 *cb, float2 *sa, float2 *sb) const {
        const float *cr = a.cos + p * a.half, *sr = a.sin + p * a.half;
        auto one = [&](int k, float &c, float &s) {
            c = 1.0f;
            s = 0.0f;
            if (k < pairs) {
                const int j = off0 + k;
                const bool first = j < a.half;
                const int at = first ? j : j - a.half;
                c = __ldg(cr + at);
                s = __ldg(sr + at) * (first ? -sign : sign);
            }
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            one(2 * i, ca[i].x, sa[i].x);
            one(2 * i + 1, ca[i].y, sa[i].y);
            one(V + 2 * i, cb[i].x, sb[i].x);
            one(V + 2 * i + 1, cb[i].y, sb[i].y);
        }
    }
    // the weights that the other elements carry, into s
    __device__ __forceinline__ void weigh_others(const HeadsArgs &a, int which, float2 *sa,
                                                 float2 *sb) const {
        auto one = [&](int k, float &s) {
            if (k < pairs) s *= heads_weight<T>(a, which, other(a.half, k));
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            one(2 * i, sa[i].x);
            one(2 * i + 1, sa[i].y);
            one(V + 2 * i, sb[i].x);
            one(V + 2 * i + 1, sb[i].y);
        }
    }
    // a pair's factors: y_a = x_a ca + x_b nb, y_b = x_b cb + x_a sa: cos, sin and
    // -sin, with a norm times the weights of the elements they meet
    // (ODD: y_a = x_a ca + other sa, y_b = x_b cb + other nb)
    template <bool NORM>
    __device__ __forceinline__ void folded(const HeadsArgs &a, const HeadsVecArgs &v, int which,
                                           int64_t p, float2 *ca, float2 *cb, float2 *sa,
                                           float2 *nb) const {
        if constexpr (ODD) factors(a, p, a.sign, ca, cb, sa, nb);
        else angles(a, v, p, ca, sa, nb);
        if constexpr (NORM) {
            float2 wa[N], wb[N];
            weights(a, v, which, wa, wb);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                cb[i] = __fmul2_rn(ODD ? cb[i] : ca[i], wb[i]);
                ca[i] = __fmul2_rn(ca[i], wa[i]);
                if constexpr (!ODD) {
                    sa[i] = __fmul2_rn(sa[i], wa[i]);
                    nb[i] = __fmul2_rn(nb[i], wb[i]);
                }
            }
            if constexpr (ODD) weigh_others(a, which, sa, nb);
        } else if constexpr (!ODD) {
#pragma unroll
            for (int i = 0; i < N; ++i) cb[i] = ca[i];
        }
    }
    __device__ __forceinline__ void share(T *row, const uint4 &x0, const uint4 &x1) const {
        if (on) *reinterpret_cast<uint4 *>(row + off0) = x0;
        if (second) *reinterpret_cast<uint4 *>(row + off1) = x1;
    }
    // row: the unpacked row's other elements, as shared; scale: what a, b were scaled by
    __device__ __forceinline__ void turn_odd(const T *row, int half, float scale, float2 *a,
                                             float2 *b, const float2 *ca, const float2 *cb,
                                             const float2 *sa, const float2 *sb) const {
        auto one = [&](int k, float x, float c, float s) {
            x *= c;
            return k < pairs ? fmaf(to_f(row[other(half, k)]) * scale, s, x) : x;
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i].x = one(2 * i, a[i].x, ca[i].x, sa[i].x);
            a[i].y = one(2 * i + 1, a[i].y, ca[i].y, sa[i].y);
            b[i].x = one(V + 2 * i, b[i].x, cb[i].x, sb[i].x);
            b[i].y = one(V + 2 * i + 1, b[i].y, cb[i].y, sb[i].y);
        }
    }
    // the unit's cosines and sines (pairs past `pairs`: 1 and 0)
    __device__ __forceinline__ void table(const HeadsArgs &a, const HeadsVecArgs &v, int64_t p,
                                          float2 *c, float2 *s) const {
        const float *cr = a.cos + p * a.half + pair0, *sr = a.sin + p * a.half + pair0;
        if (pairs == V && v.table_vec) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(cr + 2 * i));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(sr + 2 * i));
                c[i] = make_float2(x.x, x.y);
                c[i + 1] = make_float2(x.z, x.w);
                s[i] = make_float2(y.x, y.y);
                s[i + 1] = make_float2(y.z, y.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                c[i].x = 2 * i < pairs ? __ldg(cr + 2 * i) : 1.0f;
                s[i].x = 2 * i < pairs ? __ldg(sr + 2 * i) : 0.0f;
                c[i].y = 2 * i + 1 < pairs ? __ldg(cr + 2 * i + 1) : 1.0f;
                s[i].y = 2 * i + 1 < pairs ? __ldg(sr + 2 * i + 1) : 0.0f;
            }
        }
    }
    // c = cos, s = sin with the direction's sign, n = -s
    __device__ __forceinline__ void angles(const HeadsArgs &a, const HeadsVecArgs &v, int64_t p,
                                           float2 *c, float2 *s, float2 *n) const {
        table(a, v, p, c, s);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            n[i] = __fmul2_rn(s[i], both(-a.sign));
            s[i] = __fmul2_rn(s[i], both(a.sign));
        }
    }
    __device__ __forceinline__ void weights(const HeadsArgs &a, const HeadsVecArgs &v, int which,
                                            float2 *wa, float2 *wb) const {
        const void *w = which ? a.w[1] : a.w[0];
        if (w && v.weight_vec && !a.w_f32) {
            uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0;
            if (on) x0 = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + off0));
            if (second)
                x1 = __ldg(reinterpret_cast<const uint4 *>(static_cast<const T *>(w) + off1));
            open(x0, x1, wa, wb);
            return;
        }
        float2 e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int j = (i < N ? off0 : off1 - V) + 2 * i;
            const bool has = i < N ? on : second;
            e[i].x = has ? heads_weight<T>(a, which, j) : 0.0f;
            e[i].y = has ? heads_weight<T>(a, which, j + 1) : 0.0f;
        }
        split(e, wa, wb);
    }
    // a pair that does not rotate takes its factors ca, cb alone: an infinity
    // times a zero sine would be no number
    __device__ __forceinline__ void turn(float2 *a, float2 *b, const float2 *ca, const float2 *sa,
                                         const float2 *nb, const float2 *cb) const {
        if (pairs == V) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 x = a[i];
                a[i] = __ffma2_rn(x, ca[i], __fmul2_rn(b[i], nb[i]));
                b[i] = __ffma2_rn(x, sa[i], __fmul2_rn(b[i], cb[i]));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 x = a[i], y = b[i];
                a[i] = __fmul2_rn(x, ca[i]);
                b[i] = __fmul2_rn(y, cb[i]);
                if (2 * i < pairs) {
                    a[i].x = fmaf(y.x, nb[i].x, a[i].x);
                    b[i].x = fmaf(x.x, sa[i].x, b[i].x);
                }
                if (2 * i + 1 < pairs) {
                    a[i].y = fmaf(y.y, nb[i].y, a[i].y);
                    b[i].y = fmaf(x.y, sa[i].y, b[i].y);
                }
            }
        }
    }
    // the transposed rotation (a gradient's): y_a = a cos + b sin, y_b = b cos - a sin
    __device__ __forceinline__ void turn_back(float2 *a, float2 *b, const float2 *c,
                                              const float2 *s) const {
        if (pairs == V) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 x = a[i];
                a[i] = __ffma2_rn(x, c[i], __fmul2_rn(b[i], s[i]));
                b[i] = __ffma2_rn(b[i], c[i], neg2(__fmul2_rn(x, s[i])));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float2 x = a[i], y = b[i];
                if (2 * i < pairs) {
                    a[i].x = fmaf(x.x, c[i].x, y.x * s[i].x);
                    b[i].x = fmaf(y.x, c[i].x, -(x.x * s[i].x));
                }
                if (2 * i + 1 < pairs) {
                    a[i].y = fmaf(x.y, c[i].y, y.y * s[i].y);
                    b[i].y = fmaf(y.y, c[i].y, -(x.y * s[i].y));
                }
            }
        }
    }
    // the sum over the lane's elements of x^2 (0 where it has none)
    __device__ __forceinline__ float squares(const float2 *a, const float2 *b) const {
        float2 x = both(0.0f), y = both(0.0f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (!IL || i < N / 2) {
                x = __ffma2_rn(a[i], a[i], x);
                if (IL) x = __ffma2_rn(b[i], b[i], x);
            }
            if (!IL || i >= N / 2) {
                if (IL) y = __ffma2_rn(a[i], a[i], y);
                y = __ffma2_rn(b[i], b[i], y);
            }
        }
        return (on ? x.x + x.y : 0.0f) + (second ? y.x + y.y : 0.0f);
    }
};

// Keeps the compiler from holding a vector's unpacked form across this point.
__device__ __forceinline__ void keep_packed(uint4 &x) {
    asm volatile("" : "+r"(x.x), "+r"(x.y), "+r"(x.z), "+r"(x.w));
}

// Rotation, and norm with rotation.  An item is a token and HPT heads of q or
// of k; all its loads are issued before the first is used.  Four heads an item
// and three CTAs an SM (80 registers): rotation of [1,16384,40,128] bf16 52.9 us;
// two heads 61.6, four at two CTAs 58.8; one head where rows are few.
template <class T, int KIND, int MODE, int HPT>
__global__ void __launch_bounds__(kHeadsThreads, sizeof(T) == 4 ? 1 : KIND == HEADS_ODD ? 2 : 3)
k_heads_vec(const HeadsArgs a, const HeadsVecArgs v) {
    using Unit = HeadsUnit<T, KIND>;
    constexpr int N = Unit::N;
    const int lanes = 1 << v.log_lanes, lane = threadIdx.x & (lanes - 1);
    layer_pdl_launch();
    uint32_t item = (blockIdx.x * kHeadsThreads + threadIdx.x) >> v.log_lanes;
    const bool live = item < v.items;
    if (!live) item = 0;          // the group still takes part in the warp's exchanges
    uint32_t bs, g, b, s;
    v.per_token.split(item, bs, g);
    v.tokens.split(bs, b, s);
    const bool which = g >= v.q_items;
    const int h0 = (int)(which ? g - v.q_items : g) * HPT;
    const int count = min(HPT, (which ? a.heads[1] : a.heads[0]) - h0);
    Unit u;
    u.place(a, v, lane);
    const T *const x = static_cast<const T *>(which ? v.x[1].p : v.x[0].p) +
                       heads_near(which ? v.x[1] : v.x[0], b, s, h0);
    const int xsh = which ? v.x[1].sh : v.x[0].sh;
    layer_pdl_wait();
    const int64_t p = heads_position(a, b, s);
    uint4 x0[HPT], x1[HPT];
#pragma unroll
    for (int h = 0; h < HPT; ++h) u.load(x + (h < count ? (int64_t)h * xsh : 0), x0[h], x1[h]);
    extern __shared__ uint4 s_rows[];   // HEADS_ODD: the groups' rows, [groups][HPT][dim]
    T *const rows = reinterpret_cast<T *>(s_rows) +
                    (int64_t)(threadIdx.x >> v.log_lanes) * HPT * a.dim;
    if constexpr (Unit::ODD) {
#pragma unroll
        for (int h = 0; h < HPT; ++h) u.share(rows + h * a.dim, x0[h], x1[h]);
        __syncwarp();
    }
    float rstd[HPT];
    if constexpr (MODE == HEADS_NORM) {
        // the heads' sums cross the lanes together, so that their shuffles overlap
#pragma unroll
        for (int h = 0; h < HPT; ++h) {
            float2 va[N], vb[N];
            Unit::open(x0[h], x1[h], va, vb);
            rstd[h] = u.squares(va, vb);
            keep_packed(x0[h]);
            keep_packed(x1[h]);
        }
        for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int h = 0; h < HPT; ++h) rstd[h] += __shfl_xor_sync(0xFFFFFFFFu, rstd[h], o);
        const float inv = 1.0f / (float)a.dim;
#pragma unroll
        for (int h = 0; h < HPT; ++h) rstd[h] = rsqrtf(fmaf(rstd[h], inv, a.eps));
    }
    float2 ca[N], cb[N], sa[N], nb[N];
    u.template folded<MODE == HEADS_NORM>(a, v, which, p < 0 ? 0 : p, ca, cb, sa, nb);
    if (p < 0 && live && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
    T *const y = static_cast<T *>(const_cast<void *>(which ? v.y[1].p : v.y[0].p)) +
                 heads_near(which ? v.y[1] : v.y[0], b, s, h0);
    const int ysh = which ? v.y[1].sh : v.y[0].sh;
#pragma unroll
    for (int h = 0; h < HPT; ++h) {
        float2 va[N], vb[N];
        Unit::open(x0[h], x1[h], va, vb);
        if constexpr (MODE == HEADS_NORM) {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                va[i] = __fmul2_rn(va[i], both(rstd[h]));
                vb[i] = __fmul2_rn(vb[i], both(rstd[h]));
            }
        }
        if constexpr (Unit::ODD)
            u.turn_odd(rows + h * a.dim, a.half, MODE == HEADS_NORM ? rstd[h] : 1.0f, va, vb, ca,
                       cb, sa, nb);
        else
            u.turn(va, vb, ca, sa, nb, cb);
        if (p < 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) va[i] = vb[i] = both(0.0f);
        }
        if (live && h < count) u.store(y + (int64_t)h * ysh, va, vb);
    }
}

// Rows through a ring in shared memory.  A group of lanes walks items (a token
// and kRingHeads heads of q or of k) in steps of the launch's groups; their
// rows are fetched kAhead before they are worked on, by asynchronous copies.
// Each thread copies what it will read itself, so that nothing but its own
// copies is waited for.  What is fetched runs at most one item ahead, so one
// set of the next item's facts is enough.
constexpr int kRingHeads = 4;

__device__ __forceinline__ void heads_copy(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// GRAD: rows of x and of dy, of one tensor; else rows of x, of q then of k.
template <class T, int KIND, bool GRAD> struct HeadsRing {
    using Unit = HeadsUnit<T, KIND>;
    static constexpr int kAhead = GRAD ? 3 : 4, kSlots = kAhead + 1;
    static constexpr int kVectors = GRAD ? 4 : 2;             // of a thread and row
    static constexpr int kBytes = kSlots * kVectors * kHeadsThreads * 16;
    static_assert(kAhead <= kRingHeads, "at most one item ahead");

    uint4 *mine;                // this thread's place in the ring's first vector
    uint32_t item, step, total; // the group's item being fetched; items of the walk
    uint32_t end;               // past the last item that any group of the CTA fetches as this one does
    FastDiv parts;              // items of a token
    const T *x, *dy;            // the row being fetched
    int xsh, gsh;
    int row, fill, slot;        // row of the item; ring slots to fill and to read
    // of the item whose fetching began last
    T *y;
    int64_t position;
    int count, ysh;
    bool k;                     // of k

    __device__ __forceinline__ void start(const HeadsArgs &a, const HeadsVecArgs &v, int one) {
        uint32_t bs, h, b, s;
        const bool live = item < total;   // an item past the end has no rows
        parts.split(live ? item : 0, bs, h);
        v.tokens.split(bs, b, s);
        k = one >= 0 ? one == 1 : h >= v.q_items;
        if (one < 0 && k) h -= v.q_items;
        h *= kRingHeads;
        position = heads_position(a, b, s);
        x = static_cast<const T *>(k ? v.x[1].p : v.x[0].p) +
            heads_near(k ? v.x[1] : v.x[0], b, s, h);
        xsh = k ? v.x[1].sh : v.x[0].sh;
        if constexpr (GRAD) {
            dy = static_cast<const T *>(k ? v.dy[1].p : v.dy[0].p) +
                 heads_near(k ? v.dy[1] : v.dy[0], b, s, h);
            gsh = k ? v.dy[1].sh : v.dy[0].sh;
        }
        y = static_cast<T *>(const_cast<void *>(k ? v.y[1].p : v.y[0].p)) +
            heads_near(k ? v.y[1] : v.y[0], b, s, h);
        ysh = k ? v.y[1].sh : v.y[0].sh;
        count = live ? min(kRingHeads, (k ? a.heads[1] : a.heads[0]) - (int)h) : 0;
    }
    // one: 0 or 1, the walk's tensor, or -1, both
    __device__ __forceinline__ void fetch(const HeadsArgs &a, const HeadsVecArgs &v, const Unit &u,
                                          int one) {
        if (item < end) {
            if (row == 0) start(a, v, one);
            if (row < count) {
                const uint32_t to = (uint32_t)__cvta_generic_to_shared(
                    mine + fill * (kVectors * kHeadsThreads));
                if (u.on) {
                    heads_copy(to, x + u.off0);
                    if constexpr (GRAD) heads_copy(to + 2 * kHeadsThreads * 16, dy + u.off0);
                }
                if (u.second) {
                    heads_copy(to + kHeadsThreads * 16, x + u.off1);
                    if constexpr (GRAD) heads_copy(to + 3 * kHeadsThreads * 16, dy + u.off1);
                }
                x += xsh;
                if constexpr (GRAD) dy += gsh;
            }
            if (++row == kRingHeads) {
                row = 0;
                item += step;
            }
            fill = fill + 1 == kSlots ? 0 : fill + 1;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    // lanes without work, or without a second vector, read zeros
    __device__ __forceinline__ void clear(const Unit &u) {
        for (int i = 0; i < kSlots * kVectors; ++i)
            if (!(i & 1 ? u.second : u.on)) mine[i * kHeadsThreads] = make_uint4(0, 0, 0, 0);
    }
    // the next row's vectors, once they have arrived
    __device__ __forceinline__ const uint4 *take() {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        const uint4 *const p = mine + slot * (kVectors * kHeadsThreads);
        slot = slot + 1 == kSlots ? 0 : slot + 1;
        return p;
    }
};

// Norm and rotation of many rows: the ring's rows, a token's angles and weights
// in registers over its item.  Three CTAs an SM (80 registers): [2,4096,40,128] bf16
// 29.0 us, two 32.2; a CTA an item, without the ring, 32.3.
template <class T, int KIND>
__global__ void __launch_bounds__(kHeadsThreads, KIND == HEADS_ODD ? 2 : 3)
k_heads_ring(const HeadsArgs a, const HeadsVecArgs v) {
    using Ring = HeadsRing<T, KIND, false>;
    using Unit = HeadsUnit<T, KIND>;
    constexpr int N = Unit::N;
    extern __shared__ uint4 s_ring[];   // the ring, after it (HEADS_ODD) the groups' rows
    const int lanes = 1 << v.log_lanes, lane = threadIdx.x & (lanes - 1);
    const int per = kHeadsThreads >> v.log_lanes, group = threadIdx.x >> v.log_lanes;
    layer_pdl_launch();
    Unit u;
    u.place(a, v, lane);
    Ring r{};
    r.mine = s_ring + threadIdx.x;
    r.item = blockIdx.x * per + group;
    r.step = gridDim.x * per;
    r.total = v.items;
    r.end = v.items + group;
    r.parts = v.per_token;
    T *const shared_row = reinterpret_cast<T *>(s_ring + Ring::kBytes / 16) + group * a.dim;
    r.clear(u);
    layer_pdl_wait();
#pragma unroll 1
    for (int i = 0; i < Ring::kAhead; ++i) r.fetch(a, v, u, -1);
    const float inv = 1.0f / (float)a.dim;
    // every lane of a warp makes the same number of steps: the exchanges are warp-wide
    for (uint32_t base = blockIdx.x * per; base < r.total; base += r.step) {
        const int64_t p = r.position;
        const int count = r.count;
        T *y = r.y;
        const int ysh = r.ysh;
        if (count > 0 && p < 0 && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
        float2 ca[N], cb[N], sa[N], nb[N];
        u.template folded<true>(a, v, r.k, p < 0 ? 0 : p, ca, cb, sa, nb);
        const bool out = __any_sync(0xFFFFFFFFu, p < 0);   // rare
#pragma unroll 1
        for (int h = 0; h < kRingHeads; ++h) {
            const uint4 *const in = r.take();
            const uint4 x0 = in[0], x1 = in[kHeadsThreads];
            r.fetch(a, v, u, -1);
            float2 va[N], vb[N];
            Unit::open(x0, x1, va, vb);
            if constexpr (Unit::ODD) {
                __syncwarp();   // the row before has been read
                u.share(shared_row, x0, x1);
                __syncwarp();
            }
            float ss = u.squares(va, vb);
            for (int o = lanes >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
            const float rstd = rsqrtf(fmaf(ss, inv, a.eps));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                va[i] = __fmul2_rn(va[i], both(rstd));
                vb[i] = __fmul2_rn(vb[i], both(rstd));
            }
            if constexpr (Unit::ODD) u.turn_odd(shared_row, a.half, rstd, va, vb, ca, cb, sa, nb);
            else u.turn(va, vb, ca, sa, nb, cb);
            if (out) {
                if (p < 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i) va[i] = vb[i] = both(0.0f);
                }
            }
            if (h < count) u.store(y, va, vb);
            y += ysh;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// The gradient of norm and rotation.  CTAs take items of q or of k only, so a
// thread's weight-gradient sums stay in registers to the end; the CTA's sums
// then join in shared memory and go to its row of the workspace.  118 registers,
// two CTAs an SM, 98 KB of rows on their way to them: [2,4096,40,128] bf16 46.3 us;
// with one row ahead in registers instead 60.1.
template <class T, int KIND>
__global__ void __launch_bounds__(kHeadsThreads, 2)
k_heads_vec_grad(const HeadsArgs a, const HeadsVecArgs v) {
    using Ring = HeadsRing<T, KIND, true>;
    using Unit = HeadsUnit<T, KIND>;
    constexpr int N = Unit::N;
    // the ring, after it the weights [lanes][2 V] and (HEADS_ODD) the groups' rows; at
    // the end the sums [groups of the CTA][dim]
    extern __shared__ uint4 s_ring[];
    float *const s_dw = reinterpret_cast<float *>(s_ring);
    const int lanes = 1 << v.log_lanes, lane = threadIdx.x & (lanes - 1);
    const int which = (int)blockIdx.x >= v.ctas[0];
    const uint32_t cta = blockIdx.x - (which ? v.ctas[0] : 0);
    const int per = kHeadsThreads >> v.log_lanes, group = threadIdx.x >> v.log_lanes;
    layer_pdl_launch();
    Unit u;
    u.place(a, v, lane);
    Ring r{};
    r.mine = s_ring + threadIdx.x;
    r.parts = which ? v.heads[1] : v.heads[0];
    r.total = (uint32_t)a.rows * r.parts.n;
    r.item = cta * per + group;
    r.step = (which ? v.ctas[1] : v.ctas[0]) * per;
    r.end = r.total + group;
    // a lane's weights in shared memory, in the order that it uses them: sixteen
    // registers less
    float4 *const s_w = reinterpret_cast<float4 *>(s_ring + Ring::kBytes / 16) + lane;
    T *const shared_row = reinterpret_cast<T *>(s_dw + Ring::kBytes / 4 +
                                                (2 * Unit::V << v.log_lanes)) + group * a.dim;
    r.clear(u);
    layer_pdl_wait();
#pragma unroll 1
    for (int i = 0; i < Ring::kAhead; ++i) r.fetch(a, v, u, which);
    if (threadIdx.x < lanes) {
        float2 wa[N], wb[N];
        u.weights(a, v, which, wa, wb);
#pragma unroll
        for (int i = 0; i < N; ++i)
            s_w[i * lanes] = make_float4(wa[i].x, wa[i].y, wb[i].x, wb[i].y);
    }
    __syncthreads();
    float2 da[N], db[N];
#pragma unroll
    for (int i = 0; i < N; ++i) da[i] = db[i] = both(0.0f);
    bool bad = false;
    const float inv = 1.0f / (float)a.dim;
    // every lane of a warp makes the same number of steps: the exchanges are warp-wide
    for (uint32_t base = cta * per; base < r.total; base += r.step) {
        const int64_t p = r.position;
        const int count = r.count;
        T *y = r.y;
        const int ysh = r.ysh;
        bad |= count > 0 && p < 0;
        float2 c[N], sn[N], cb[N], sb[N];
        if constexpr (Unit::ODD) u.factors(a, p < 0 ? 0 : p, -1.0f, c, cb, sn, sb);
        else u.table(a, v, p < 0 ? 0 : p, c, sn);
        const bool out = __any_sync(0xFFFFFFFFu, p < 0);   // rare
#pragma unroll 1
        for (int h = 0; h < kRingHeads; ++h) {
            const uint4 *const in = r.take();
            float2 xa[N], xb[N], ga[N], gb[N];
            {
                const uint4 g0 = in[2 * kHeadsThreads], g1 = in[3 * kHeadsThreads];
                Unit::open(g0, g1, ga, gb);
                Unit::open(in[0], in[kHeadsThreads], xa, xb);
                if constexpr (Unit::ODD) {
                    __syncwarp();   // the row before has been read
                    u.share(shared_row, g0, g1);
                    __syncwarp();
                }
            }
            r.fetch(a, v, u, which);
            if constexpr (Unit::ODD) u.turn_odd(shared_row, a.half, 1.0f, ga, gb, c, cb, sn, sb);
            else u.turn_back(ga, gb, c, sn);
            float ss = u.squares(xa, xb);
            // sum of g w x, the absent elements' weights being 0
            float2 dot = both(0.0f);
            float2 wa[N], wb[N];   // g w
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float4 w = s_w[i * lanes];
                wa[i] = __fmul2_rn(ga[i], make_float2(w.x, w.y));
                wb[i] = __fmul2_rn(gb[i], make_float2(w.z, w.w));
                dot = __ffma2_rn(wa[i], xa[i], __ffma2_rn(wb[i], xb[i], dot));
            }
            float gx = dot.x + dot.y;
            for (int o = lanes >> 1; o > 0; o >>= 1) {
                ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
                gx += __shfl_xor_sync(0xFFFFFFFFu, gx, o);
            }
            const float rstd = rsqrtf(fmaf(ss, inv, a.eps));
            const float2 mean = both(-gx * rstd * inv), r2 = both(rstd);
            const bool live = h < count, use = live && p >= 0;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                xa[i] = __fmul2_rn(xa[i], r2);
                xb[i] = __fmul2_rn(xb[i], r2);
                if (use) {
                    da[i] = __ffma2_rn(ga[i], xa[i], da[i]);
                    db[i] = __ffma2_rn(gb[i], xb[i], db[i]);
                }
                ga[i] = __fmul2_rn(__ffma2_rn(xa[i], mean, wa[i]), r2);
                gb[i] = __fmul2_rn(__ffma2_rn(xb[i], mean, wb[i]), r2);
            }
            if (out) {
                if (p < 0) {
#pragma unroll
                    for (int i = 0; i < N; ++i) ga[i] = gb[i] = both(0.0f);
                }
            }
            if (live) u.store(y, ga, gb);
            y += ysh;
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad && lane == 0) atomicOr(a.status, EBIN_DEVICE_POSITION_RANGE);
    __syncthreads();   // the ring and the weights have been read
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // pairs 2i and 2i + 1 of the unit
        constexpr bool IL = Unit::IL;
        const int j = IL ? (i < N / 2 ? u.off0 : u.off1 - Unit::V) + 4 * i : u.off0 + 2 * i;
        const int k = IL ? j + 1 : u.off1 + 2 * i, next = IL ? 2 : 1;
        const bool first = IL ? (i < N / 2 ? u.on : u.second) : u.on;
        const bool other = IL ? first : u.second;
        if (first) {
            s_dw[group * a.dim + j] = da[i].x;
            s_dw[group * a.dim + j + next] = da[i].y;
        }
        if (other) {
            s_dw[group * a.dim + k] = db[i].x;
            s_dw[group * a.dim + k + next] = db[i].y;
        }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.dim; j += kHeadsThreads) {
        float t = 0.0f;
        for (int r = 0; r < per; ++r) t += s_dw[r * a.dim + j];
        a.partial[which][(int64_t)cta * a.dim + j] = t;
    }
}

}  // namespace ebin
