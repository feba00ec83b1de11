// The norms around a block on rows of up to 32768 elements (a gradient's: 16384): a
// team of warps takes a row, each lane eight columns of every chunk of 256 that its
// warp owns, and a row's data is read from memory once.
#pragma once

#include "ebin_block.cuh"

namespace ebin {

constexpr int kChunk = 256;         // columns of a warp's share
constexpr int kRowsMaxWarps = 32;

struct RowsGeom {
    int32_t warps;     // of a team
    int32_t teams;     // of a CTA: 1, or one for each warp
    int32_t slots;     // rows in shared memory: the one worked on and those on their way
    FastDiv gate, mod; // rows that share a row of gate, of scale and shift
    // a gradient's: where h, dz, dh and y lie among a thread's vectors, and how many these are
    int32_t at[4], vectors;
    int64_t units;
};

// Which columns a lane owns, and how it reaches them.  With vectors: eight
// neighbours (16-bit rows), or two fours 128 columns apart (a 32-bit type takes
// part: 16 bytes a lane and access either way); else eight columns 32 apart.
template <class T, class S, bool VEC> struct RowsLane {
    static constexpr bool WIDE = sizeof(S) == 4;
    int lane, base, n;   // base: the chunk's first column

    // first column of quad q (vectors)
    __device__ __forceinline__ int quad(int q) const {
        return base + (WIDE ? q * 128 + lane * 4 : lane * 8 + q * 4);
    }
    // column of element e
    __device__ __forceinline__ int col(int e) const {
        return VEC ? quad(e >> 2) + (e & 3) : base + e * 32 + lane;
    }
    __device__ __forceinline__ bool live(int e) const { return col(e) < n; }

    template <class E>
    __device__ __forceinline__ static void open4(const E *p, float2 *v) {
        if constexpr (sizeof(E) == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(p);
            v[0] = make_float2(x.x, x.y);
            v[1] = make_float2(x.z, x.w);
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(p);
            v[0] = open2<E>(x.x);
            v[1] = open2<E>(x.y);
        }
    }
    // the lane's columns of a row in global memory; 0 past the row's end
    template <class E> __device__ __forceinline__ void load(const E *p, float2 *v) const {
        if constexpr (VEC) {
            if constexpr (!WIDE && sizeof(E) == 2) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (quad(0) < n) x = *reinterpret_cast<const uint4 *>(p + quad(0));
                v[0] = open2<E>(x.x);
                v[1] = open2<E>(x.y);
                v[2] = open2<E>(x.z);
                v[3] = open2<E>(x.w);
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    v[2 * q] = v[2 * q + 1] = make_float2(0.0f, 0.0f);
                    if (quad(q) < n) open4(p + quad(q), v + 2 * q);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k].x = live(2 * k) ? to_f(p[col(2 * k)]) : 0.0f;
                v[k].y = live(2 * k + 1) ? to_f(p[col(2 * k + 1)]) : 0.0f;
            }
        }
    }
    template <class E> __device__ __forceinline__ void store(E *p, const float2 *v) const {
        if constexpr (VEC) {
            if constexpr (!WIDE && sizeof(E) == 2) {
                if (quad(0) < n)
                    *reinterpret_cast<uint4 *>(p + quad(0)) =
                        make_uint4(pack2<E>(v[0]), pack2<E>(v[1]), pack2<E>(v[2]), pack2<E>(v[3]));
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (quad(q) >= n) continue;
                    if constexpr (sizeof(E) == 4)
                        *reinterpret_cast<float4 *>(p + quad(q)) =
                            make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
                    else
                        *reinterpret_cast<uint2 *>(p + quad(q)) =
                            make_uint2(pack2<E>(v[2 * q]), pack2<E>(v[2 * q + 1]));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (live(2 * k)) p[col(2 * k)] = from_f<E>(v[k].x);
                if (live(2 * k + 1)) p[col(2 * k + 1)] = from_f<E>(v[k].y);
            }
        }
    }
    // a row of parameters in type T or binary32
    __device__ __forceinline__ void params(const void *p, int f32, float2 *v) const {
        if (f32) load(static_cast<const float *>(p), v);
        else load(static_cast<const T *>(p), v);
    }
    // keep bits of the lane's columns of a row, element e in bit e
    __device__ __forceinline__ uint32_t kept(const DropArgs &d, uint32_t row, uint2 offset) const {
        auto bits = [&](uint32_t quad) {
            const uint4 w = drop_words(d, quad, row, offset);
            return (uint32_t)(w.x >= d.least) | (uint32_t)(w.y >= d.least) << 1 |
                   (uint32_t)(w.z >= d.least) << 2 | (uint32_t)(w.w >= d.least) << 3;
        };
        if constexpr (VEC) {
            return bits((uint32_t)quad(0) >> 2) | bits((uint32_t)quad(1) >> 2) << 4;
        } else {
            // a lane draws two of the chunk's 64 quads; element e's lies with lane
            // (8 e + lane / 4) % 32, in its first for e < 4
            const uint32_t mine = bits((uint32_t)(base >> 2) + lane) |
                                  bits((uint32_t)(base >> 2) + 32 + lane) << 4;
            uint32_t r = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t theirs =
                    __shfl_sync(0xFFFFFFFFu, mine, (8 * e + (lane >> 2)) & 31);
                r |= (theirs >> ((e & 4) + (lane & 3)) & 1) << e;
            }
            return r;
        }
    }
};

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// What is kept times the scale; exactly 0 for what is dropped.
__device__ __forceinline__ void keep8(float2 *v, uint32_t bits, float scale) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        v[k].x = bits >> (2 * k) & 1 ? v[k].x * scale : 0.0f;
        v[k].y = bits >> (2 * k + 1) & 1 ? v[k].y * scale : 0.0f;
    }
}

// A team's exchange of partial sums through shared memory, [2][warps] of K floats:
// consecutive exchanges take the halves in turn, so that one barrier each is enough.
struct Team {
    int lane, warp, warps;
    float *s;           // 2 * kRowsMaxWarps * 8 floats
    int half;
    int count;          // live columns of the warp that this lane stands for in joins
    float inv_mine;     // 1 / live columns of this warp (0: none)
    float inv_n;

    template <int VPT> __device__ __forceinline__ void start(int n) {
        auto columns = [&](int w) {
            int c = 0;
            for (int i = 0; i < VPT; ++i) c += min(max(n - (i * warps + w) * kChunk, 0), kChunk);
            return c;
        };
        count = lane < warps ? columns(lane) : 0;
        const int mine = columns(warp);
        inv_mine = mine ? 1.0f / (float)mine : 0.0f;
        inv_n = 1.0f / (float)n;
        half = 0;
    }
    // v: a warp's values, the same in each lane; after it lane w has warp w's (0 past the last)
    template <int K> __device__ __forceinline__ void gather(float (&v)[K]) {
        if (warps == 1) {
            if (lane)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] = 0.0f;
            return;
        }
        float *const at = s + half * kRowsMaxWarps * 8;
        half ^= 1;
        if (lane == 0)
#pragma unroll
            for (int k = 0; k < K; ++k) at[k * kRowsMaxWarps + warp] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = lane < warps ? at[k * kRowsMaxWarps + lane] : 0.0f;
    }
};

template <int K> __device__ __forceinline__ void warp_sums(float (&v)[K]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
}

__device__ __forceinline__ float sum8(const float2 *v) {
    const float2 a = __fadd2_rn(v[0], v[1]), b = __fadd2_rn(v[2], v[3]);
    const float2 c = __fadd2_rn(a, b);
    return c.x + c.y;
}

// Sum of squares about `mean` of the live ones of eight.
template <class L>
__device__ __forceinline__ float squares8(const L &l, const float2 *v, float mean) {
    float2 t = two(0.0f);
    if (mean == 0.0f) {   // columns past the row's end hold 0
#pragma unroll
        for (int k = 0; k < 4; ++k) t = __ffma2_rn(v[k], v[k], t);
        return t.x + t.y;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float2 d = __fadd2_rn(v[k], two(-mean));
        if (!l.live(2 * k)) d.x = 0.0f;
        if (!l.live(2 * k + 1)) d.y = 0.0f;
        t = __ffma2_rn(d, d, t);
    }
    return t.x + t.y;
}

// Joined moments: each warp's squares lie about its own mean, and move to the
// row's (the pairwise rule of Chan, Golub and LeVeque): one exchange, and no loss
// for rows far from 0.  v[0]: the warp's sum, v[1]: its squares; lane w's warp's.
__device__ __forceinline__ float2 join_moments(const Team &t, float sum, float squares, int norm,
                                               float eps) {
    float mean = 0.0f;
    if (norm == EBIN_NORM_LAYER) {
        float m[1] = {sum};
        warp_sums(m);
        mean = m[0] * t.inv_n;
        if (t.count) {
            const float d = sum / (float)t.count - mean;
            squares = fmaf(d * d, (float)t.count, squares);
        }
    }
    float q[1] = {squares};
    warp_sums(q);
    return make_float2(mean, rsqrtf(fmaf(q[0], t.inv_n, eps)));
}

template <class L, int VPT>
__device__ __forceinline__ float2 row_moments(Team &t, const L (&l)[VPT], const float2 (&v)[VPT][4],
                                              int norm, float eps) {
    float s[1] = {0.0f}, mean = 0.0f;
    if (norm == EBIN_NORM_LAYER) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) s[0] += sum8(v[i]);
        warp_sums(s);
        mean = s[0] * t.inv_mine;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i) q[0] += squares8(l[i], v[i], mean);
    warp_sums(q);
    float both[2] = {s[0], q[0]};
    t.gather(both);
    return join_moments(t, both[0], both[1], norm, eps);
}

// Asynchronous copies of a lane's columns: COUNT rows of a step, types by SIZE.
__device__ __forceinline__ void rows_copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void rows_copy8(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `left` of the newest groups are under way
__device__ __forceinline__ void rows_wait(int left) {
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// A thread's part of a row of one tensor in shared memory: what it copied itself,
// 16-byte vectors `stride` apart.
template <class L, class E> struct RowsPart {
    // vectors of a chunk: 1 (eight 16-bit columns) or 2
    static constexpr int N = sizeof(E) == 4 ? 2 : 1;
    __device__ __forceinline__ static void fetch(const L &l, uint4 *at, int stride, const E *row) {
        const uint32_t to = (uint32_t)__cvta_generic_to_shared(at);
        if constexpr (!L::WIDE) {
            if (l.quad(0) < l.n) rows_copy16(to, row + l.quad(0));
        } else {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (l.quad(q) >= l.n) continue;
                if constexpr (sizeof(E) == 4) rows_copy16(to + q * stride * 16, row + l.quad(q));
                else rows_copy8(to + q * 8, row + l.quad(q));
            }
        }
    }
    __device__ __forceinline__ static void open(const L &l, const uint4 *at, int stride,
                                                float2 *v) {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint4 x = at[q * stride];
                const bool in = l.quad(q) < l.n;
                v[2 * q] = in ? make_float2(__uint_as_float(x.x), __uint_as_float(x.y)) : two(0.0f);
                v[2 * q + 1] = in ? make_float2(__uint_as_float(x.z), __uint_as_float(x.w))
                                  : two(0.0f);
            }
        } else {
            uint4 x = at[0];
            if (l.quad(0) >= l.n) x.x = x.y = 0;
            if (l.quad(1) >= l.n) x.z = x.w = 0;
            v[0] = open2<E>(x.x);
            v[1] = open2<E>(x.y);
            v[2] = open2<E>(x.z);
            v[3] = open2<E>(x.w);
        }
    }
};

template <class T, class S, int VPT, bool VEC>
__global__ void __launch_bounds__(VPT == 2 ? 512 : 1024, VPT == 2 ? 2 : 1)
k_block_rows(const BlockArgs a, const RowsGeom g) {
    using Lane = RowsLane<T, S, VEC>;
    using PartS = RowsPart<Lane, S>;
    using PartT = RowsPart<Lane, T>;
    __shared__ float s_sums[2 * kRowsMaxWarps * 8];
    extern __shared__ uint4 s_rows[];   // [slots][vectors of a thread][threads]
    constexpr int kVectors = VPT * (PartS::N + PartT::N);
    Team t;
    t.lane = threadIdx.x & 31;
    t.warps = g.warps;
    t.warp = g.teams > 1 ? 0 : threadIdx.x >> 5;
    t.s = s_sums;
    t.start<VPT>((int)a.n);
    Lane l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) l[i] = Lane{t.lane, (i * g.warps + t.warp) * kChunk, (int)a.n};
    const int64_t first = g.teams > 1 ? (int64_t)blockIdx.x * g.teams + (threadIdx.x >> 5)
                                      : blockIdx.x;
    const int64_t step = (int64_t)gridDim.x * g.teams;
    const int threads = blockDim.x;
    uint4 *const mine = s_rows + threadIdx.x;
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    const int ahead = g.slots - 1;
    int fill = 0, slot = 0;
    int64_t next = first;   // the row to fetch
    auto fetch = [&]() {
        if constexpr (VEC) {
            if (next < a.rows) {
                uint4 *const at = mine + fill * kVectors * threads;
                const S *const x = static_cast<const S *>(a.x) + next * a.ld_x;
                const T *const y = static_cast<const T *>(a.y) + (a.y ? next * a.ld_y : 0);
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    PartS::fetch(l[i], at + i * PartS::N * threads, threads, x);
                    if (a.y)
                        PartT::fetch(l[i], at + (VPT * PartS::N + i * PartT::N) * threads, threads,
                                     y);
                }
                next += step;
            }
            fill = fill + 1 == g.slots ? 0 : fill + 1;
            rows_commit();
        }
    };
    if constexpr (VEC)
        for (int i = 0; i < ahead; ++i) fetch();
    for (int64_t row = first; row < a.rows; row += step) {
        fetch();
        if constexpr (VEC) rows_wait(ahead);
        const uint4 *const at = mine + slot * kVectors * threads;
        slot = slot + 1 == g.slots ? 0 : slot + 1;
        uint32_t group, rest;
        g.gate.split((uint32_t)row, group, rest);
        const void *const gate = block_row<T>(a.gate, group * a.ld_gate, a.mod_f32);
        g.mod.split((uint32_t)row, group, rest);
        float2 v[VPT][4];
        float2 my = make_float2(0.0f, 1.0f);
        if (a.y) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if constexpr (VEC)
                    PartT::open(l[i], at + (VPT * PartS::N + i * PartT::N) * threads, threads,
                                v[i]);
                else
                    l[i].load(static_cast<const T *>(a.y) + row * a.ld_y, v[i]);
            }
            if (a.post != EBIN_NORM_NONE) my = row_moments(t, l, v, a.post, a.eps_post);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float2 x[4], p[4];
            if constexpr (VEC) PartS::open(l[i], at + i * PartS::N * threads, threads, x);
            else l[i].load(static_cast<const S *>(a.x) + row * a.ld_x, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], two(a.stream_scale));
            if (a.y) {
                if (a.post != EBIN_NORM_NONE) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        v[i][k] = __fmul2_rn(__fadd2_rn(v[i][k], two(-my.x)), two(my.y));
                    if (a.w_post) {
                        l[i].params(a.w_post, a.w_f32, p);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[i][k] = __fmul2_rn(v[i][k], p[k]);
                    }
                    if (a.b_post) {
                        l[i].params(a.b_post, a.w_f32, p);
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[i][k] = __fadd2_rn(v[i][k], p[k]);
                    }
                }
                if (a.drop.least)
                    keep8(v[i], l[i].kept(a.drop, (uint32_t)row, offset), a.drop.scale);
                if (a.gate) {
                    l[i].params(gate, a.mod_f32, p);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][k] = __fmul2_rn(v[i][k], p[k]);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    x[k] = __ffma2_rn(v[i][k], two(a.branch_scale), x[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = x[k];
            if (a.h) l[i].store(static_cast<S *>(a.h) + row * a.ld_h, v[i]);
            // a layer's bias, or a mean taken off, leaves something past the row's end
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (!l[i].live(2 * k)) v[i][k].x = 0.0f;
                if (!l[i].live(2 * k + 1)) v[i][k].y = 0.0f;
            }
        }
        if (!a.z) continue;
        const float2 mh = row_moments(t, l, v, a.pre, a.eps_pre);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float2 p[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                v[i][k] = __fmul2_rn(__fadd2_rn(v[i][k], two(-mh.x)), two(mh.y));
            if (a.w_pre) {
                l[i].params(a.w_pre, a.w_f32, p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __fmul2_rn(v[i][k], p[k]);
            }
            if (a.b_pre) {
                l[i].params(a.b_pre, a.w_f32, p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __fadd2_rn(v[i][k], p[k]);
            }
            if (a.scale) {
                l[i].params(block_row<T>(a.scale, group * a.ld_scale, a.mod_f32), a.mod_f32, p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __ffma2_rn(v[i][k], p[k], v[i][k]);
            }
            if (a.shift) {
                l[i].params(block_row<T>(a.shift, group * a.ld_shift, a.mod_f32), a.mod_f32, p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __fadd2_rn(v[i][k], p[k]);
            }
            l[i].store(static_cast<T *>(a.z) + row * a.ld_z, v[i]);
        }
    }
    if constexpr (VEC) rows_wait(0);
}

// The gradient.  A team takes a unit, consecutive rows of one group, and keeps its
// columns' sums for the parameters in registers to the unit's end (ALL: the four of
// BlockSum, else those without a bias).  A row costs two exchanges: the moments of
// h and y with the products of m and h, then, with a post norm, those of u.
// GLOBAL: the sums of wide rows, which registers do not hold, are kept in the
// unit's part of the workspace.
template <class T, class S, int VPT, bool VEC, bool ALL, bool GLOBAL>
__global__ void __launch_bounds__(512, 1) k_block_rows_grad(const BlockArgs a, const RowsGeom g) {
    using Lane = RowsLane<T, S, VEC>;
    using PartS = RowsPart<Lane, S>;
    using PartT = RowsPart<Lane, T>;
    constexpr int kKinds = ALL ? 4 : 2;   // without ALL: SUM_DZ_HH, SUM_E_YH
    __shared__ float s_sums[2 * kRowsMaxWarps * 8];
    extern __shared__ uint4 s_rows[];
    Team t;
    t.lane = threadIdx.x & 31;
    t.warps = g.warps;
    t.warp = g.teams > 1 ? 0 : threadIdx.x >> 5;
    t.s = s_sums;
    t.start<VPT>((int)a.n);
    Lane l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) l[i] = Lane{t.lane, (i * g.warps + t.warp) * kChunk, (int)a.n};
    const int64_t unit = g.teams > 1 ? (int64_t)blockIdx.x * g.teams + (threadIdx.x >> 5)
                                     : blockIdx.x;
    if (unit >= g.units) return;   // a whole team, and one without barriers
    const int64_t group = unit / a.parts, part = unit - group * a.parts;
    const int64_t r0 = group * a.group_rows + part * a.unit_rows;
    const int64_t r1 = min(r0 + a.unit_rows, (group + 1) * a.group_rows);
    const int threads = blockDim.x;
    uint4 *const mine = s_rows + threadIdx.x;
    const bool pre = a.pre != EBIN_NORM_NONE, post = a.post != EBIN_NORM_NONE;
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    uint32_t index, rest;
    g.gate.split((uint32_t)r0, index, rest);
    const void *const gate = block_row<T>(a.gate, index * a.ld_gate, a.mod_f32);
    g.mod.split((uint32_t)r0, index, rest);
    const void *const scale = block_row<T>(a.scale, index * a.ld_scale, a.mod_f32);
    float *const partial = a.partial ? a.partial + unit * 4 * a.n : nullptr;
    float2 acc[GLOBAL ? 1 : kKinds][VPT][4];
    if constexpr (!GLOBAL) {
#pragma unroll
        for (int k = 0; k < kKinds; ++k)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[k][i][j] = two(0.0f);
    }
    // kind's place among those kept
    auto place = [](int kind) { return ALL ? kind : kind >> 1; };
    bool begun = false;
    // sums of x y (y null: x) of chunk i
    auto add = [&](int kind, int i, const float2 *x, const float2 *y) {
        if constexpr (GLOBAL) {
            if (!partial) return;
            float2 s[4];
            float *const to = partial + kind * a.n;
            if (begun) l[i].load(to, s);
            else s[0] = s[1] = s[2] = s[3] = two(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = y ? __ffma2_rn(x[j], y[j], s[j]) : __fadd2_rn(s[j], x[j]);
            l[i].store(to, s);
        } else {
            float2 *const s = acc[place(kind)][i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = y ? __ffma2_rn(x[j], y[j], s[j]) : __fadd2_rn(s[j], x[j]);
        }
    };
    const int ahead = g.slots - 1;
    int fill = 0, slot = 0;
    int64_t next = r0;
    auto fetch = [&]() {
        if constexpr (VEC) {
            if (next < r1) {
                uint4 *const at = mine + fill * g.vectors * threads;
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    auto of = [&](int k, int vectors) {
                        return at + (g.at[k] + i * vectors) * threads;
                    };
                    if (a.x)
                        PartS::fetch(l[i], of(0, PartS::N), threads,
                                     static_cast<const S *>(a.x) + next * a.ld_x);
                    if (a.dz)
                        PartT::fetch(l[i], of(1, PartT::N), threads,
                                     static_cast<const T *>(a.dz) + next * a.ld_dz);
                    if (a.dh)
                        PartS::fetch(l[i], of(2, PartS::N), threads,
                                     static_cast<const S *>(a.dh) + next * a.ld_dh);
                    if (a.y)
                        PartT::fetch(l[i], of(3, PartT::N), threads,
                                     static_cast<const T *>(a.y) + next * a.ld_y);
                }
                ++next;
            }
            fill = fill + 1 == g.slots ? 0 : fill + 1;
            rows_commit();
        }
    };
    if constexpr (VEC)
        for (int i = 0; i < ahead; ++i) fetch();
    for (int64_t row = r0; row < r1; ++row) {
        fetch();
        if constexpr (VEC) rows_wait(ahead);
        const uint4 *const at = mine + slot * g.vectors * threads;
        slot = slot + 1 == g.slots ? 0 : slot + 1;
        auto open_h = [&](int i, float2 *v) {
            if constexpr (VEC)
                PartS::open(l[i], at + (g.at[0] + i * PartS::N) * threads, threads, v);
            else l[i].load(static_cast<const S *>(a.x) + row * a.ld_x, v);
        };
        auto open_dz = [&](int i, float2 *v) {
            if constexpr (VEC)
                PartT::open(l[i], at + (g.at[1] + i * PartT::N) * threads, threads, v);
            else l[i].load(static_cast<const T *>(a.dz) + row * a.ld_dz, v);
        };
        auto open_dh = [&](int i, float2 *v) {
            if constexpr (VEC)
                PartS::open(l[i], at + (g.at[2] + i * PartS::N) * threads, threads, v);
            else l[i].load(static_cast<const S *>(a.dh) + row * a.ld_dh, v);
        };
        auto open_y = [&](int i, float2 *v) {
            if constexpr (VEC)
                PartT::open(l[i], at + (g.at[3] + i * PartT::N) * threads, threads, v);
            else l[i].load(static_cast<const T *>(a.y) + row * a.ld_y, v);
        };
        // this warp's sums of h, of its squares about their mean, of m and of m with h
        // less that mean, and the sums and squares of y
        float w[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        float2 v[VPT][4];   // m, then D
        if (pre) {
            float mean = 0.0f;
            if (a.pre == EBIN_NORM_LAYER) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float2 h[4];
                    open_h(i, h);
                    s[0] += sum8(h);
                }
                warp_sums(s);
                w[0] = s[0];
                mean = s[0] * t.inv_mine;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float2 h[4], p[4];
                open_dz(i, v[i]);
                if (scale) {
                    l[i].params(scale, a.mod_f32, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = __ffma2_rn(v[i][j], p[j], v[i][j]);
                }
                if (a.w_pre) {
                    l[i].params(a.w_pre, a.w_f32, p);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], p[j]);
                }
                open_h(i, h);
                w[1] += squares8(l[i], h, mean);
                w[2] += sum8(v[i]);
                float2 c = two(0.0f);   // m is 0 past the row's end
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    c = __ffma2_rn(v[i][j], __fadd2_rn(h[j], two(-mean)), c);
                w[3] += c.x + c.y;
            }
        }
        if (post) {
            float mean = 0.0f;
            float2 y[VPT][4];
#pragma unroll
            for (int i = 0; i < VPT; ++i) open_y(i, y[i]);
            if (a.post == EBIN_NORM_LAYER) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) s[0] += sum8(y[i]);
                warp_sums(s);
                w[4] = s[0];
                mean = s[0] * t.inv_mine;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) w[5] += squares8(l[i], y[i], mean);
        }
        float2 mh = make_float2(0.0f, 1.0f), my = mh;
        float c0 = 0.0f, c1 = 0.0f;   // means of m and of m hh
        if (pre || post) {
            {
                float q[4] = {w[1], w[2], w[3], w[5]};
                warp_sums(q);
                w[1] = q[0];
                w[2] = q[1];
                w[3] = q[2];
                w[5] = q[3];
            }
            t.gather(w);
            if (pre) {
                mh = join_moments(t, w[0], w[1], a.pre, a.eps_pre);
                // the products about the row's mean
                const bool layer = a.pre == EBIN_NORM_LAYER;
                if (layer && t.count) w[3] = fmaf(w[2], w[0] / (float)t.count - mh.x, w[3]);
                float c[2] = {w[2], w[3]};
                warp_sums(c);
                c0 = layer ? c[0] * t.inv_n : 0.0f;
                c1 = c[1] * mh.y * t.inv_n;
            }
            if (post) my = join_moments(t, w[4], w[5], a.post, a.eps_post);
        }
        float2 u[VPT][4];
        float b[2] = {0.0f, 0.0f};   // sums of u and of u yh
        // yh of chunk i, 0 past the row's end
        auto normed_y = [&](int i, float2 *yh) {
            open_y(i, yh);
            if (!post) return;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                yh[j] = __fmul2_rn(__fadd2_rn(yh[j], two(-my.x)), two(my.y));
                if (!l[i].live(2 * j)) yh[j].x = 0.0f;
                if (!l[i].live(2 * j + 1)) yh[j].y = 0.0f;
            }
        };
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float2 d[4];
            if (a.dh) open_dh(i, d);
            else d[0] = d[1] = d[2] = d[3] = two(0.0f);
            if (pre) {
                float2 h[4], dz[4];
                open_h(i, h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    h[j] = __fmul2_rn(__fadd2_rn(h[j], two(-mh.x)), two(mh.y));
                    const float2 m = __ffma2_rn(h[j], two(-c1), __fadd2_rn(v[i][j], two(-c0)));
                    d[j] = __ffma2_rn(m, two(mh.y), d[j]);
                }
                open_dz(i, dz);
                add(SUM_DZ_HH, i, dz, h);
                if constexpr (ALL) add(SUM_DZ, i, dz, nullptr);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[i][j] = d[j];
                if (!l[i].live(2 * j)) v[i][j].x = 0.0f;
                if (!l[i].live(2 * j + 1)) v[i][j].y = 0.0f;
            }
            // e, then u
#pragma unroll
            for (int j = 0; j < 4; ++j) u[i][j] = __fmul2_rn(v[i][j], two(a.branch_scale));
            if (a.drop.least)
                keep8(u[i], l[i].kept(a.drop, (uint32_t)row, offset), a.drop.scale);
            float2 yh[4];
            if (a.y) {
                normed_y(i, yh);
                add(SUM_E_YH, i, u[i], yh);
            }
            if constexpr (ALL) add(SUM_E, i, u[i], nullptr);
            float2 p[4];
            if (gate) {
                l[i].params(gate, a.mod_f32, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[i][j] = __fmul2_rn(u[i][j], p[j]);
            }
            if (a.w_post) {
                l[i].params(a.w_post, a.w_f32, p);
#pragma unroll
                for (int j = 0; j < 4; ++j) u[i][j] = __fmul2_rn(u[i][j], p[j]);
            }
            if (post) {
                float2 c = two(0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) c = __ffma2_rn(u[i][j], yh[j], c);
                b[0] += sum8(u[i]);
                b[1] += c.x + c.y;
            }
        }
        begun = true;
        if (post) {
            warp_sums(b);
            t.gather(b);
            warp_sums(b);
            b[0] = a.post == EBIN_NORM_LAYER ? b[0] * t.inv_n : 0.0f;
            b[1] *= t.inv_n;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (post && a.z) {
                float2 yh[4];
                normed_y(i, yh);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    u[i][j] = __fmul2_rn(
                        __ffma2_rn(yh[j], two(-b[1]), __fadd2_rn(u[i][j], two(-b[0]))), two(my.y));
            }
            if (a.z) l[i].store(static_cast<T *>(a.z) + row * a.ld_z, u[i]);
            if (a.h) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], two(a.stream_scale));
                l[i].store(static_cast<S *>(a.h) + row * a.ld_h, v[i]);
            }
        }
    }
    if constexpr (VEC) rows_wait(0);
    if constexpr (!GLOBAL) {
        if (!partial) return;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (!ALL && (k == SUM_DZ || k == SUM_E)) continue;
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                l[i].store(partial + k * a.n, acc[place(k)][i]);
        }
    }
}

}  // namespace ebin
