// The norms around a block, a row a team of warps: each lane owns eight columns of every
// chunk of 256 that its warp owns, and a row's data is read from memory once.  The
// path of what the kernels of CTAs' units (ebin_block_unit.cuh) leave.  Forward: few rows,
// small groups, rows whose factors leave no room for them in shared memory, rows of 8193
// to 32768 columns, and off the vectors 32-bit streams and rows of at most 2048 columns.  Of
// gradients: small groups, those without a norm before the next block, rows of 8193 to
// 16384 columns, and, with a norm after the block and a layer norm or the gradient of a
// shift or a bias, of 4097 and more ([4096,8192] bf16 with layer norms on both sides 176 us).
#pragma once

#include "ebin_block.cuh"

namespace ebin {

constexpr int kChunk = 256;         // columns of a warp's share
constexpr int kRowsMaxWarps = 32;

struct RowsGeom {
    int32_t warps;     // of a team
    int32_t joins;     // the power of two that holds them
    int32_t teams;     // of a CTA: 1, or one for each warp
    int32_t slots;     // rows in shared memory: the one worked on and those on their way
    FastDiv gate, mod; // rows that share a row of gate, of scale and shift
    // a gradient's: where h, dz, dh and y lie among a thread's vectors (-1: read where they
    // lie in memory), how many these are, and the vectors of its factors (-1: all 1)
    int32_t at[4], vectors;
    int32_t factor[2], factors;
    int64_t units;
    // of a CTA that takes a unit: which of its columns' factors there are, by bit, and
    // the 16-byte vectors of one
    int32_t tables, table;
    int32_t slot_bytes;   // of its teams' rows
};

__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }

// Four q of eight columns by a quad's words: exactly 0 for what is dropped, in each row.
template <class... V>
__device__ __forceinline__ void drop_four(uint4 w, uint32_t least, int q, V *...rows) {
    auto one = [&](float2 *v) {
        v[2 * q].x = w.x >= least ? v[2 * q].x : 0.0f;
        v[2 * q].y = w.y >= least ? v[2 * q].y : 0.0f;
        v[2 * q + 1].x = w.z >= least ? v[2 * q + 1].x : 0.0f;
        v[2 * q + 1].y = w.w >= least ? v[2 * q + 1].y : 0.0f;
    };
    (one(rows), ...);
}

// Which columns a lane owns, and how it reaches them.  With vectors: eight
// neighbours (16-bit rows), or two fours 128 columns apart (a 32-bit type takes
// part: 16 bytes a lane and access either way); else eight columns 32 apart.
template <class T, class S, bool VEC> struct RowsLane {
    static constexpr bool WIDE = sizeof(S) == 4;
    int lane, base, n;   // base: the chunk's first column
    bool on0, on1;       // whether the fours lie within the row (vectors)
    int at0, at1;        // where they are read: what lies past the end reads column 0

    __device__ __forceinline__ void place(int lane_, int base_, int n_) {
        lane = lane_;
        base = base_;
        n = n_;
        on0 = quad(0) < n;
        on1 = WIDE ? quad(1) < n : on0;
        at0 = on0 ? quad(0) : 0;
        at1 = WIDE ? (on1 ? quad(1) : 0) : at0 + 4;
    }
    // no column of the chunk lies in the row (the same for a whole warp)
    __device__ __forceinline__ bool none() const { return base >= n; }
    // first column of four q (vectors)
    __device__ __forceinline__ int quad(int q) const {
        return base + (WIDE ? q * 128 + lane * 4 : lane * 8 + q * 4);
    }
    __device__ __forceinline__ bool on(int q) const { return q ? on1 : on0; }
    // column of element e
    __device__ __forceinline__ int col(int e) const {
        return VEC ? quad(e >> 2) + (e & 3) : base + e * 32 + lane;
    }
    __device__ __forceinline__ bool live(int e) const {
        return VEC ? on(e >> 2) : col(e) < n;
    }
    // the sum of eight (v: two by two) over the columns within the row
    __device__ __forceinline__ float within(const float2 *v) const {
        if constexpr (VEC && !WIDE) {
            const float2 a = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
            return on0 ? a.x + a.y : 0.0f;
        } else if constexpr (VEC) {
            const float2 a = __fadd2_rn(v[0], v[1]), b = __fadd2_rn(v[2], v[3]);
            return (on0 ? a.x + a.y : 0.0f) + (on1 ? b.x + b.y : 0.0f);
        } else {
            float s = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                s += (live(2 * k) ? v[k].x : 0.0f) + (live(2 * k + 1) ? v[k].y : 0.0f);
            return s;
        }
    }

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
    // the lane's columns of a row in global memory; past the row's end anything (vectors) or 0
    template <class E> __device__ __forceinline__ void load(const E *p, float2 *v) const {
        if constexpr (VEC) {
            if constexpr (!WIDE && sizeof(E) == 2) {
                const uint4 x = *reinterpret_cast<const uint4 *>(p + at0);
                v[0] = open2<E>(x.x);
                v[1] = open2<E>(x.y);
                v[2] = open2<E>(x.z);
                v[3] = open2<E>(x.w);
            } else {
                open4(p + at0, v);
                open4(p + at1, v + 2);
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
                if (on0)
                    *reinterpret_cast<uint4 *>(p + quad(0)) =
                        make_uint4(pack2<E>(v[0]), pack2<E>(v[1]), pack2<E>(v[2]), pack2<E>(v[3]));
            } else {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (!on(q)) continue;
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

    // keep bits of the lane's columns of a row, element e in bit e (columns 32 apart): a lane
    // draws two of the chunk's 64 quads; element e's lies with lane (8 e + lane / 4) % 32, in
    // its first for e < 4
    __device__ __forceinline__ uint32_t kept(const DropArgs &d, uint32_t row, uint2 offset) const {
        auto bits = [&](uint32_t quad) {
            const uint4 w = drop_words(d, quad, row, offset);
            return (uint32_t)(w.x >= d.least) | (uint32_t)(w.y >= d.least) << 1 |
                   (uint32_t)(w.z >= d.least) << 2 | (uint32_t)(w.w >= d.least) << 3;
        };
        const uint32_t mine = bits((uint32_t)(base >> 2) + lane) |
                              bits((uint32_t)(base >> 2) + 32 + lane) << 4;
        uint32_t r = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t theirs = __shfl_sync(0xFFFFFFFFu, mine, (8 * e + (lane >> 2)) & 31);
            r |= (theirs >> ((e & 4) + (lane & 3)) & 1) << e;
        }
        return r;
    }
    // exactly 0 for what is dropped, in each of the rows
    template <class... V>
    __device__ __forceinline__ void drop(const DropArgs &d, uint32_t row, uint2 offset,
                                         V *...rows) const {
        if constexpr (VEC) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                drop_four(drop_words(d, (uint32_t)quad(q) >> 2, row, offset), d.least, q, rows...);
        } else {
            const uint32_t bits = kept(d, row, offset);
            (drop_bits(bits, rows), ...);
        }
    }
    __device__ __forceinline__ static void drop_bits(uint32_t bits, float2 *v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            v[k].x = bits >> (2 * k) & 1 ? v[k].x : 0.0f;
            v[k].y = bits >> (2 * k + 1) & 1 ? v[k].y : 0.0f;
        }
    }
};

// A team's exchange of partial sums through shared memory, [2][8][warps]: consecutive
// exchanges take the halves in turn, so that one barrier each is enough.
// The CTA is the team, or its teams are single warps.
struct Team {
    int lane, warp, warps, joins;
    float *s;           // 2 * 8 * kRowsMaxWarps floats
    int half;
    float count;        // live columns of the warp that this lane stands for in joins
    float inv_count;    // and 1 / that (0: none)
    float inv_mine;     // 1 / live columns of this warp (0: none)
    float inv_n;

    template <int VPT> __device__ __forceinline__ void start(const RowsGeom &g, int n, float *sums) {
        lane = threadIdx.x & 31;
        const int team = (threadIdx.x >> 5) / g.warps;
        warp = (threadIdx.x >> 5) - team * g.warps;
        sums += team * g.warps;   // a team's columns of the sums
        warps = g.warps;
        joins = g.joins;
        s = sums;
        half = 0;
        auto columns = [&](int w) {
            int c = 0;
            for (int i = 0; i < VPT; ++i) c += min(max(n - (i * warps + w) * kChunk, 0), kChunk);
            return c;
        };
        const int from = lane & (joins - 1);
        count = from < warps ? (float)columns(from) : 0.0f;
        inv_count = count > 0.0f ? 1.0f / count : 0.0f;
        const int mine = columns(warp);
        inv_mine = mine ? 1.0f / (float)mine : 0.0f;
        inv_n = 1.0f / (float)n;
    }
    // v: a warp's values, the same in each lane; after it lane w has warp w % joins' (0 past
    // the last)
    template <int K> __device__ __forceinline__ void gather(float (&v)[K]) {
        if (warps == 1) return;
        float *const at = s + half * 8 * kRowsMaxWarps;
        half ^= 1;
        float mine = v[0];      // lane k stores value k
#pragma unroll
        for (int k = 1; k < K; ++k) mine = lane == k ? v[k] : mine;
        if (lane < K) at[lane * kRowsMaxWarps + warp] = mine;
        __syncthreads();
        const int from = lane & (joins - 1);
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = from < warps ? at[k * kRowsMaxWarps + from] : 0.0f;
    }
    // the sums over the warps of what gather gave
    template <int K> __device__ __forceinline__ void join(float (&v)[K]) const {
        for (int o = joins >> 1; o > 0; o >>= 1)
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
    }
    // (mean, 1 / deviation) from the warps' sums and squares: each warp's squares lie
    // about its own mean, and move to the row's (the pairwise rule of Chan, Golub and
    // LeVeque): one exchange, and no loss for rows far from 0
    __device__ __forceinline__ float2 moments(float sum, float squares, bool layer,
                                              float eps) const {
        float mean = 0.0f;
        if (layer) {
            float m[1] = {sum};
            join(m);
            mean = m[0] * inv_n;
            const float d = fmaf(sum, inv_count, -mean);
            squares = fmaf(d * d, count, squares);
        }
        float q[1] = {squares};
        join(q);
        return make_float2(mean, rsqrtf(fmaf(q[0], inv_n, eps)));
    }
};

template <int K> __device__ __forceinline__ void warp_sums(float (&v)[K]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
}

// The lane's sum of squares about `mean` (not read without LAYER: about 0).
template <bool LAYER, class L>
__device__ __forceinline__ float squares8(const L &l, const float2 *v, float mean) {
    float2 t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 d = LAYER ? __fadd2_rn(v[k], two(-mean)) : v[k];
        t[k] = __fmul2_rn(d, d);
    }
    return l.within(t);
}

// LAYER: either norm may be a layer norm; else neither is.
template <bool LAYER, class L, int VPT>
__device__ __forceinline__ float2 row_moments(Team &t, const L (&l)[VPT], const float2 (&v)[VPT][4],
                                              int norm, float eps) {
    const bool layer = LAYER && norm == EBIN_NORM_LAYER;
    float s[1] = {0.0f}, mean = 0.0f;
    if (layer) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (!i || !l[i].none()) s[0] += l[i].within(v[i]);
        warp_sums(s);
        mean = s[0] * t.inv_mine;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        if (!i || !l[i].none()) q[0] += squares8<LAYER>(l[i], v[i], mean);
    warp_sums(q);
    if constexpr (LAYER) {
        float both[2] = {s[0], q[0]};
        t.gather(both);
        return t.moments(both[0], both[1], layer, eps);
    } else {
        t.gather(q);
        return t.moments(0.0f, q[0], false, eps);
    }
}

// Asynchronous copies of a lane's columns.
__device__ __forceinline__ void rows_copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void rows_copy8(uint32_t to, const void *from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}
// One element of SIZE bytes, at once.
template <int SIZE> __device__ __forceinline__ void rows_move(uint32_t to, const char *from) {
    if constexpr (SIZE == 4)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(*reinterpret_cast<const uint32_t *>(from)) : "memory");
    else
        asm volatile("st.shared.b16 [%0], %1;" ::"r"(to), "h"(*reinterpret_cast<const uint16_t *>(from)) : "memory");
}
__device__ __forceinline__ void rows_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most `left` of the newest groups are under way
__device__ __forceinline__ void rows_wait(int left) {
    if (left == 0) asm volatile("cp.async.wait_group 0;" ::: "memory");
    else if (left == 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
    else asm volatile("cp.async.wait_group 2;" ::: "memory");
}

// A thread's part of a row of one tensor in shared memory: what it copied itself,
// 16-byte vectors `stride` apart.  What it holds past the row's end is anything:
// sums leave it out (within), and nothing is stored there.
template <class L, class E> struct RowsPart {
    // vectors of a chunk: 1 (eight 16-bit columns) or 2
    static constexpr int N = sizeof(E) == 4 ? 2 : 1;
    __device__ __forceinline__ static void fetch(const L &l, uint32_t to, int stride,
                                                 const E *row) {
        if constexpr (!L::WIDE) {
            rows_copy16(to, row + l.at0);
        } else if constexpr (sizeof(E) == 4) {
            rows_copy16(to, row + l.at0);
            rows_copy16(to + stride * 16, row + l.at1);
        } else {
            rows_copy8(to, row + l.at0);
            rows_copy8(to + 8, row + l.at1);
        }
    }
    __device__ __forceinline__ static void open(const uint4 *at, int stride, float2 *v) {
        if constexpr (sizeof(E) == 4) {
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint4 x = at[q * stride];
                v[2 * q] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
                v[2 * q + 1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
            }
        } else {
            const uint4 x = at[0];
            v[0] = open2<E>(x.x);
            v[1] = open2<E>(x.y);
            v[2] = open2<E>(x.z);
            v[3] = open2<E>(x.w);
        }
    }
};

__device__ __forceinline__ void mul8(float2 *v, const float2 *p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fmul2_rn(v[k], p[k]);
}
__device__ __forceinline__ void add8(float2 *v, const float2 *p) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __fadd2_rn(v[k], p[k]);
}
// (v - m.x) m.y
template <bool LAYER> __device__ __forceinline__ void norm8(float2 *v, float2 m) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (LAYER) v[k] = __fadd2_rn(v[k], two(-m.x));
        v[k] = __fmul2_rn(v[k], two(m.y));
    }
}

// A team, a row after another.  One chunk a lane to 8192 columns, so that a row spreads over
// many warps ([16,4096] bf16 2.3 us in a graph); four past it ([2048,16384] 86 us).
template <class T, class S, int VPT, bool VEC, bool LAYER>
__global__ void __launch_bounds__(1024, 1)
k_block_rows(const BlockArgs a, const RowsGeom g) {
    using Lane = RowsLane<T, S, VEC>;
    using PartS = RowsPart<Lane, S>;
    using PartT = RowsPart<Lane, T>;
    __shared__ float s_sums[2 * 8 * kRowsMaxWarps];
    extern __shared__ uint4 s_rows[];   // [slots][vectors of a thread][threads]
    constexpr int kX = VPT * PartS::N, kVectors = kX + VPT * PartT::N;
    Team t;
    t.start<VPT>(g, (int)a.n, s_sums);
    Lane l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        l[i].place(t.lane, (i * g.warps + t.warp) * kChunk, (int)a.n);
    const int first = g.teams > 1 ? (int)blockIdx.x * g.teams + (threadIdx.x >> 5)
                                  : (int)blockIdx.x;
    const int step = (int)gridDim.x * g.teams, rows = (int)a.rows;
    const int threads = blockDim.x;
    uint4 *const mine = s_rows + threadIdx.x;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine);
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    const float branch = a.branch_scale * (a.drop.least ? a.drop.scale : 1.0f);
    const int ahead = g.slots - 1;
    int fill = 0, slot = 0, next = first;
    auto fetch = [&]() {
        if constexpr (VEC) {
            if (next < rows) {
                const uint32_t at = to + fill * kVectors * threads * 16;
                const S *const x = static_cast<const S *>(a.x) + next * a.ld_x;
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (!i || !l[i].none())
                        PartS::fetch(l[i], at + i * PartS::N * threads * 16, threads, x);
                if (a.y) {
                    const T *const y = static_cast<const T *>(a.y) + next * a.ld_y;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (!i || !l[i].none())
                            PartT::fetch(l[i], at + (kX + i * PartT::N) * threads * 16, threads, y);
                }
                next += step;
            }
            fill = fill + 1 == g.slots ? 0 : fill + 1;
            rows_commit();
        }
    };
    if constexpr (VEC)
        for (int i = 0; i < ahead; ++i) fetch();
    for (int row = first; row < rows; row += step) {
        fetch();
        if constexpr (VEC) rows_wait(ahead);
        const uint4 *const at = mine + slot * kVectors * threads;
        slot = slot + 1 == g.slots ? 0 : slot + 1;
        float2 v[VPT][4];
        float2 my = make_float2(0.0f, 1.0f);
        const void *gate = nullptr;
        if (a.y) {
            if (a.gate) {
                uint32_t group, rest;
                g.gate.split((uint32_t)row, group, rest);
                gate = block_row<T>(a.gate, group * a.ld_gate, a.mod_f32);
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
            if (i && l[i].none()) continue;
                if constexpr (VEC) PartT::open(at + (kX + i * PartT::N) * threads, threads, v[i]);
                else l[i].load(static_cast<const T *>(a.y) + row * a.ld_y, v[i]);
            }
            if (a.post != EBIN_NORM_NONE) my = row_moments<LAYER>(t, l, v, a.post, a.eps_post);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i && l[i].none()) continue;
            float2 x[4], p[4];
            if constexpr (VEC) PartS::open(at + i * PartS::N * threads, threads, x);
            else l[i].load(static_cast<const S *>(a.x) + row * a.ld_x, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], two(a.stream_scale));
            if (a.y) {
                if (a.post != EBIN_NORM_NONE) {
                    norm8<LAYER>(v[i], my);
                    if (a.w_post) {
                        l[i].params(a.w_post, a.w_f32, p);
                        mul8(v[i], p);
                    }
                    if (a.b_post) {
                        l[i].params(a.b_post, a.w_f32, p);
                        add8(v[i], p);
                    }
                }
                if (a.drop.least) l[i].drop(a.drop, (uint32_t)row, offset, v[i]);
                if (gate) {
                    l[i].params(gate, a.mod_f32, p);
                    mul8(v[i], p);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = __ffma2_rn(v[i][k], two(branch), x[k]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = x[k];
            if (a.h) l[i].store(static_cast<S *>(a.h) + row * a.ld_h, v[i]);
        }
        if (!a.z) continue;
        const float2 mh = row_moments<LAYER>(t, l, v, a.pre, a.eps_pre);
        const void *scale = nullptr, *shift = nullptr;
        if (a.scale || a.shift) {
            uint32_t group, rest;
            g.mod.split((uint32_t)row, group, rest);
            scale = block_row<T>(a.scale, group * a.ld_scale, a.mod_f32);
            shift = block_row<T>(a.shift, group * a.ld_shift, a.mod_f32);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (i && l[i].none()) continue;
            float2 p[4];
            norm8<LAYER>(v[i], mh);
            if (a.w_pre) {
                l[i].params(a.w_pre, a.w_f32, p);
                mul8(v[i], p);
            }
            if (a.b_pre) {
                l[i].params(a.b_pre, a.w_f32, p);
                add8(v[i], p);
            }
            if (scale) {
                l[i].params(scale, a.mod_f32, p);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = __ffma2_rn(v[i][k], p[k], v[i][k]);
            }
            if (shift) {
                l[i].params(shift, a.mod_f32, p);
                add8(v[i], p);
            }
            l[i].store(static_cast<T *>(a.z) + row * a.ld_z, v[i]);
        }
    }
    if constexpr (VEC) rows_wait(0);
}

// The gradient.  A team takes a unit, consecutive rows of one group, and keeps its
// columns' sums for the parameters in registers to the unit's end.  A row costs two
// exchanges: the moments of h and y with the products of m and h, then, with a post
// norm, those of u.  A column's factors (1 + scale) w_pre and branch_scale gate w_post
// / (1 - p) lie in shared memory, each thread's its own.
// GLOBAL: the sums of wide rows, which registers do not hold, are kept in the
// unit's part of the workspace, those that are wanted ([2048,16384] bf16 with norms on both
// sides 196 us, all four kinds 253; a layer norm with dropout 181 and 209).
template <class T, class S, int VPT, bool VEC, bool GLOBAL>
__global__ void __launch_bounds__(512, 1) k_block_rows_grad(const BlockArgs a, const RowsGeom g) {
    using Lane = RowsLane<T, S, VEC>;
    using PartS = RowsPart<Lane, S>;
    using PartT = RowsPart<Lane, T>;
    __shared__ float s_sums[2 * 8 * kRowsMaxWarps];
    extern __shared__ uint4 s_rows[];   // the rows' slots, then the factors
    Team t;
    t.start<VPT>(g, (int)a.n, s_sums);
    Lane l[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
        l[i].place(t.lane, (i * g.warps + t.warp) * kChunk, (int)a.n);
    const int64_t unit = g.teams > 1 ? (int64_t)blockIdx.x * g.teams + (threadIdx.x >> 5)
                                     : blockIdx.x;
    if (unit >= g.units) return;   // a whole team, and one without barriers
    const int64_t group = unit / a.team.parts, part = unit - group * a.team.parts;
    const int r0 = (int)(group * a.group_rows + part * a.team.rows);
    const int r1 = (int)min(r0 + a.team.rows, (group + 1) * a.group_rows);
    const int threads = blockDim.x;
    uint4 *const mine = s_rows + threadIdx.x;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine);
    const bool pre = a.pre != EBIN_NORM_NONE, post = a.post != EBIN_NORM_NONE;
    const bool layer_h = a.pre == EBIN_NORM_LAYER;
    const bool layer_y = a.post == EBIN_NORM_LAYER;
    const float branch = a.branch_scale * (a.drop.least ? a.drop.scale : 1.0f);
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    const int ahead = g.slots - 1;
    int fill = 0, slot = 0, next = r0;
    // whether an input's rows go through shared memory (of 8192 columns all that are there)
    auto held = [&](int k, const void *p) { return GLOBAL ? g.at[k] >= 0 : p != nullptr; };
    auto fetch = [&]() {
        if constexpr (VEC) {
            if (next < r1) {
                const uint32_t at = to + fill * g.vectors * threads * 16;
                const uint32_t s_step = PartS::N * threads * 16, t_step = PartT::N * threads * 16;
                if (held(0, a.x)) {
                    const S *const p = static_cast<const S *>(a.x) + next * a.ld_x;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        PartS::fetch(l[i], at + g.at[0] * threads * 16 + i * s_step, threads, p);
                }
                if (held(1, a.dz)) {
                    const T *const p = static_cast<const T *>(a.dz) + next * a.ld_dz;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        PartT::fetch(l[i], at + g.at[1] * threads * 16 + i * t_step, threads, p);
                }
                if (held(2, a.dh)) {
                    const S *const p = static_cast<const S *>(a.dh) + next * a.ld_dh;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        PartS::fetch(l[i], at + g.at[2] * threads * 16 + i * s_step, threads, p);
                }
                if (held(3, a.y)) {
                    const T *const p = static_cast<const T *>(a.y) + next * a.ld_y;
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        PartT::fetch(l[i], at + g.at[3] * threads * 16 + i * t_step, threads, p);
                }
                ++next;
            }
            fill = fill + 1 == g.slots ? 0 : fill + 1;
            rows_commit();
        }
    };
    if constexpr (VEC)
        for (int i = 0; i < ahead; ++i) fetch();
    // the factors: two vectors a chunk
    float4 *const factors = reinterpret_cast<float4 *>(mine + g.slots * g.vectors * threads);
    {
        uint32_t index, rest;
        g.gate.split((uint32_t)r0, index, rest);
        const void *const gate = block_row<T>(a.gate, index * a.ld_gate, a.mod_f32);
        g.mod.split((uint32_t)r0, index, rest);
        const void *const scale = block_row<T>(a.scale, index * a.ld_scale, a.mod_f32);
#pragma unroll 1
        for (int f = 0; f < 2; ++f) {
            const int place = f ? g.factor[1] : g.factor[0];
            if (place < 0) continue;
            const void *const w = f ? a.w_post : a.w_pre, *const m = f ? gate : scale;
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float2 p[4], q[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) q[k] = two(f ? branch : 1.0f);
                if (m) {
                    l[i].params(m, a.mod_f32, p);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        q[k] = f ? __fmul2_rn(q[k], p[k]) : __fadd2_rn(q[k], p[k]);
                }
                if (w) {
                    l[i].params(w, a.w_f32, p);
                    mul8(q, p);
                }
                float4 *const at = factors + (place + 2 * i) * threads;
                at[0] = make_float4(q[0].x, q[0].y, q[1].x, q[1].y);
                at[threads] = make_float4(q[2].x, q[2].y, q[3].x, q[3].y);
            }
        }
    }
    auto times = [&](int f, int i, float2 *v) {
        if (g.factor[f] < 0) return;
        const float4 *const at = factors + (g.factor[f] + 2 * i) * threads;
        const float4 x = at[0], y = at[threads];
        v[0] = __fmul2_rn(v[0], make_float2(x.x, x.y));
        v[1] = __fmul2_rn(v[1], make_float2(x.z, x.w));
        v[2] = __fmul2_rn(v[2], make_float2(y.x, y.y));
        v[3] = __fmul2_rn(v[3], make_float2(y.z, y.w));
    };
    float *const partial = a.partial ? a.partial + unit * 4 * a.pad : nullptr;
    float2 acc[GLOBAL ? 1 : 4][VPT][4];
    if constexpr (!GLOBAL) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[k][i][j] = two(0.0f);
    }
    bool begun = false;
    // sums of x y (y null: x) of chunk i
    auto add = [&](int kind, int i, const float2 *x, const float2 *y) {
        if constexpr (GLOBAL) {
            if (!partial || !(a.need >> kind & 1)) return;
            float2 s[4];
            float *const at = partial + kind * a.pad;
            if (begun) l[i].load(at, s);
            else s[0] = s[1] = s[2] = s[3] = two(0.0f);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = y ? __ffma2_rn(x[j], y[j], s[j]) : __fadd2_rn(s[j], x[j]);
            l[i].store(at, s);
        } else {
            float2 *const s = acc[kind][i];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[j] = y ? __ffma2_rn(x[j], y[j], s[j]) : __fadd2_rn(s[j], x[j]);
        }
    };
    for (int row = r0; row < r1; ++row) {
        fetch();
        if constexpr (VEC) rows_wait(ahead);
        const uint4 *const at = mine + slot * g.vectors * threads;
        slot = slot + 1 == g.slots ? 0 : slot + 1;
        auto open_h = [&](int i, float2 *v) {
            if (VEC && held(0, a.x))
                PartS::open(at + (g.at[0] + i * PartS::N) * threads, threads, v);
            else l[i].load(static_cast<const S *>(a.x) + row * a.ld_x, v);
        };
        auto open_dz = [&](int i, float2 *v) {
            if (VEC && held(1, a.dz))
                PartT::open(at + (g.at[1] + i * PartT::N) * threads, threads, v);
            else l[i].load(static_cast<const T *>(a.dz) + row * a.ld_dz, v);
        };
        auto open_dh = [&](int i, float2 *v) {
            if (VEC && held(2, a.dh))
                PartS::open(at + (g.at[2] + i * PartS::N) * threads, threads, v);
            else l[i].load(static_cast<const S *>(a.dh) + row * a.ld_dh, v);
        };
        auto open_y = [&](int i, float2 *v) {
            if (VEC && held(3, a.y))
                PartT::open(at + (g.at[3] + i * PartT::N) * threads, threads, v);
            else l[i].load(static_cast<const T *>(a.y) + row * a.ld_y, v);
        };
        // this warp's sums of the squares of h about their mean, of m with h less that
        // mean, of the squares of y, of m, of h and of y
        float w[6] = {};
        float2 v[VPT][4];   // m, then D
        if (pre) {
            float mean = 0.0f;
            if (layer_h) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float2 h[4];
                    open_h(i, h);
                    s[0] += l[i].within(h);
                }
                warp_sums(s);
                w[4] = s[0];
                mean = s[0] * t.inv_mine;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float2 h[4], c[4];
                open_dz(i, v[i]);
                times(0, i, v[i]);
                open_h(i, h);
                w[3] += l[i].within(v[i]);
#pragma unroll
                for (int j = 0; j < 4; ++j) h[j] = __fadd2_rn(h[j], two(-mean));
                w[0] += squares8<false>(l[i], h, 0.0f);
#pragma unroll
                for (int j = 0; j < 4; ++j) c[j] = __fmul2_rn(v[i][j], h[j]);
                w[1] += l[i].within(c);
            }
        }
        if (post) {
            float mean = 0.0f;
            if (layer_y) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < VPT; ++i) {
                    float2 y[4];
                    open_y(i, y);
                    s[0] += l[i].within(y);
                }
                warp_sums(s);
                w[5] = s[0];
                mean = s[0] * t.inv_mine;
            }
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                float2 y[4];
                open_y(i, y);
                w[2] += squares8<true>(l[i], y, mean);
            }
        }
        float2 mh = make_float2(0.0f, 1.0f), my = mh;
        float c0 = 0.0f, c1 = 0.0f;   // means of m and of m hh
        if (pre || post) {
            float q[4] = {w[0], w[1], w[2], w[3]};
            warp_sums(q);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = q[k];
            t.gather(w);
            if (pre) {
                mh = t.moments(w[4], w[0], layer_h, a.eps_pre);
                // the products about the row's mean
                float c[2] = {w[3], w[1]};
                if (layer_h) c[1] = fmaf(w[3], fmaf(w[4], t.inv_count, -mh.x), c[1]);
                t.join(c);
                c0 = layer_h ? c[0] * t.inv_n : 0.0f;
                c1 = c[1] * mh.y * t.inv_n;
            }
            if (post) my = t.moments(w[5], w[2], layer_y, a.eps_post);
        }
        float2 u[VPT][4];
        float b[2] = {0.0f, 0.0f};   // sums of u yh and of u
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float2 d[4], yh[4];
            if (a.dh) open_dh(i, d);
            else d[0] = d[1] = d[2] = d[3] = two(0.0f);
            if (pre) {
                float2 h[4], dz[4];
                open_h(i, h);
                norm8<true>(h, mh);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 m = __fadd2_rn(v[i][j], two(-c0));
                    d[j] = __ffma2_rn(__ffma2_rn(h[j], two(-c1), m), two(mh.y), d[j]);
                }
                open_dz(i, dz);
                add(SUM_DZ_HH, i, dz, h);
                add(SUM_DZ, i, dz, nullptr);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][j] = u[i][j] = d[j];
            if (a.y) {
                open_y(i, yh);
                if (post) norm8<true>(yh, my);
            } else {
                yh[0] = yh[1] = yh[2] = yh[3] = two(0.0f);
            }
            // e / branch, then u; what is dropped adds nothing, whatever y is there
            if (a.drop.least) l[i].drop(a.drop, (uint32_t)row, offset, u[i], yh);
            if (a.y) add(SUM_E_YH, i, u[i], yh);
            add(SUM_E, i, u[i], nullptr);
            times(1, i, u[i]);
            if (post) {
                b[1] += l[i].within(u[i]);
                mul8(yh, u[i]);
                b[0] += l[i].within(yh);
            }
        }
        begun = true;
        if (post) {
            warp_sums(b);
            t.gather(b);
            t.join(b);
            b[0] *= t.inv_n;
            b[1] = layer_y ? b[1] * t.inv_n : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (a.z) {
                if (post) {
                    float2 yh[4];
                    open_y(i, yh);
                    norm8<true>(yh, my);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        u[i][j] = __fadd2_rn(u[i][j], two(-b[1]));
                        u[i][j] = __fmul2_rn(__ffma2_rn(yh[j], two(-b[0]), u[i][j]), two(my.y));
                    }
                }
                l[i].store(static_cast<T *>(a.z) + row * a.ld_z, u[i]);
            }
            if (a.h) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[i][j] = __fmul2_rn(v[i][j], two(a.stream_scale));
                l[i].store(static_cast<S *>(a.h) + row * a.ld_h, v[i]);
            }
        }
    }
    if constexpr (VEC) rows_wait(0);
    if (!partial) return;
    // the sums of e carry its factor from here on
#pragma unroll
    for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float2 s[4];
            if constexpr (GLOBAL) {
                if (k == SUM_DZ_HH || k == SUM_DZ || !(a.need >> k & 1)) continue;
                l[i].load(partial + k * a.pad, s);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = acc[k][i][j];
            }
            if (k == SUM_E_YH || k == SUM_E) {
#pragma unroll
                for (int j = 0; j < 4; ++j) s[j] = __fmul2_rn(s[j], two(branch));
            }
            l[i].store(partial + k * a.pad, s);
        }
    }
}

}  // namespace ebin
