// The norms around a block on many rows of at most 8192 columns: one CTA an SM takes a unit,
// consecutive rows of one group, and its teams walk them in turn.  (A gradient whose sums take
// a chunk a lane, kUnitGradVpt: at most 4096.)  What a column's
// elements are multiplied by and added to lies in shared memory in binary32, formed
// once from the parameters: two 16-byte loads in place of one and eight conversions,
// which a row of weights in the L1 costs for each use ([8192,4096] bf16 with both
// norms' weights: 60 us so, 48 without the weights).
//
// 512 threads of 128 registers an SM, each row through shared memory by asynchronous copies, up
// to three rows a team there.  bf16, against a copy's 6683 GB/s:
//   [8192,4096] norms on both sides   forward 49.0 us 5480 GB/s, gradient 69.1 us 5830
//   [16380,1536] f32 stream, gate, scale, shift   forward 52.2 us 5790 GB/s
//   [16388,1152] the same with dropout, gradient 66.6 us 3400 GB/s
//   [8192,4096] layer norms on both sides   forward 59.7 us 4490 GB/s, gradient 144 us 2800
// RMS norms and plain modulation are bound by memory, with the issue of instructions close behind.
// The modulated gradient is not: 43 million warp instructions are 35 of its 67 us, the rest a
// row's chain of two exchanges and three passes, with 15 warps an SM to cover it (a capture:
// issue 55 %, memory 36 %, stalls at barriers 1.25, of fixed latency 1.38 and on shared memory
// 1.02 an issue).
//
// RAGGED: rows that do not start and end on vectors.  A row's copies begin on the
// vector that holds its first element; a lane takes its columns from two neighbouring
// vectors and shifts them into place, and an output's vectors are made of two
// neighbouring lanes' words.  Shifts and the ends of stores about double the instructions:
// [8191,4097] bf16 122 us and 237, element by element 198 and 803.  Of a tensor's first and last
// rows the vectors that pass its ends are copied by elements: nothing outside is read
// ([8185,4096], rows 4097 apart, bf16 100 us and 155, whole vectors everywhere 96 and 148).
#pragma once

#include "ebin_block_copy.h"
#include "ebin_block_rows.cuh"

namespace ebin {

// A table of a factor for the lane's columns: the fours of chunk i, [2][32] vectors.
template <class L> struct UnitTable {
    const float4 *at;   // this lane's first
    int warps;
    __device__ __forceinline__ void read(int i, float2 *p) const {
        const float4 x = at[i * warps * 64], y = at[i * warps * 64 + 32];
        p[0] = make_float2(x.x, x.y);
        p[1] = make_float2(x.z, x.w);
        p[2] = make_float2(y.x, y.y);
        p[3] = make_float2(y.z, y.w);
    }
    __device__ __forceinline__ void times(int i, float2 *v) const {
        float2 p[4];
        read(i, p);
        mul8(v, p);
    }
};

// value(col, q, p): a table's four values at col; written by the whole CTA.
template <class L, class F>
__device__ __forceinline__ void unit_fill(float4 *table, int vectors, int n, const F &value) {
    for (int j = threadIdx.x; j < vectors; j += blockDim.x) {
        const int lane = j & 31, q = j >> 5 & 1, base = (j >> 6) * kChunk;
        const int col = base + (L::WIDE ? q * 128 + lane * 4 : lane * 8 + q * 4);
        float4 v = col < n ? value(col) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (L::RAGGED) {   // 0 past the row's end
            if (col + 1 >= n) v.y = 0.0f;
            if (col + 2 >= n) v.z = 0.0f;
            if (col + 3 >= n) v.w = 0.0f;
        }
        table[j] = v;
    }
}

// Four of a row of n parameters in type T or binary32; `none` where there is no row.
template <class T, bool RAGGED>
__device__ __forceinline__ float4 params4(const void *p, int col, int n, int f32, float none) {
    if (!p) return make_float4(none, none, none, none);
    if constexpr (RAGGED) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = col + e < n ? block_param<T>(p, col + e, f32, none) : 0.0f;
        return make_float4(v[0], v[1], v[2], v[3]);
    }
    if (f32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(p) + col);
    if constexpr (sizeof(T) == 2) {
        const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const T *>(p) + col);
        const float2 a = open2<T>(x.x), b = open2<T>(x.y);
        return make_float4(a.x, a.y, b.x, b.y);
    } else {
        return *reinterpret_cast<const float4 *>(static_cast<const T *>(p) + col);
    }
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
    return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}
__device__ __forceinline__ float4 four(float v) { return make_float4(v, v, v, v); }

enum UnitTables : int {
    TABLE_Y = 1,       // branch_scale / (1 - p) gate w_post
    TABLE_Y_ADD = 2,   // branch_scale / (1 - p) gate b_post
    TABLE_H = 4,       // (1 + scale) w_pre
    TABLE_H_ADD = 8    // (1 + scale) b_pre + shift
};

// x: two vectors of W words; y: the W words that begin s bytes into them (s < 4 W, the same
// for a whole warp, whole halves of words).
template <int W, bool HALVES>
__device__ __forceinline__ void shift_words(uint32_t (&x)[2 * W], uint32_t (&y)[W], int s) {
    if (W == 4 && s & 8)
#pragma unroll
        for (int k = 0; k < 2 * W - 2; ++k) x[k] = x[k + 2];
    if (s & 4)
#pragma unroll
        for (int k = 0; k <= W; ++k) x[k] = x[k + 1 < 2 * W ? k + 1 : k];
#pragma unroll
    for (int k = 0; k < W; ++k) y[k] = HALVES ? __funnelshift_r(x[k], x[k + 1], (s & 2) * 8) : x[k];
}

// A lane's columns as RowsLane's with vectors, for all its chunks: those of chunk i
// begin `stride` columns after those of chunk i - 1.  A chunk of a lane is one piece of
// eight columns, or (WIDE) two of four, 128 columns apart.
template <class T, class S, bool RAG> struct UnitLane {
    static constexpr bool WIDE = sizeof(S) == 4, RAGGED = RAG;
    static constexpr int P = WIDE ? 2 : 1, C = 8 / P;   // pieces, columns of one
    int first, stride, n;   // the first column of chunk 0
    int chunk;              // and the chunk's own
    int lane, warp, warps;  // among the CTA's

    __device__ __forceinline__ void place(int lane_, int team_warp, int team_warps, int teams,
                                          int n_) {
        lane = lane_;
        warp = threadIdx.x >> 5;
        warps = team_warps * teams;
        chunk = team_warp * kChunk;
        first = chunk + lane * C;
        stride = team_warps * kChunk;
        n = n_;
    }
    // no column of chunk i lies in the row (the same for a whole warp; never of chunk 0)
    __device__ __forceinline__ bool none(int i) const { return i && chunk + i * stride >= n; }
    // the row ends in chunk i, or with it (the same for a whole warp)
    __device__ __forceinline__ bool ends(int i) const { return chunk + (i * stride + kChunk) > n; }
    // column of four q
    __device__ __forceinline__ int col(int i, int q) const {
        return first + i * stride + (WIDE ? q * 128 : q * 4);
    }
    // four q lies in the row (rows on vectors)
    __device__ __forceinline__ bool on(int i, int q) const {
        return first + i * stride + (WIDE ? q * 128 : 0) < n;
    }

    // ---- a row in shared memory
    //
    // On vectors: a thread's own, [vectors][512].  RAGGED: the chunk as it lies in memory,
    // from the vector with its first column on, and one vector more: [chunks][warps].
    template <class E> __host__ __device__ static constexpr int bytes() { return C * (int)sizeof(E); }   // of a piece
    template <class E> __host__ __device__ static constexpr int buffer() { return kChunk * (int)sizeof(E) + 16; }
    template <class E> __host__ __device__ static constexpr int vectors() { return sizeof(E) == 4 ? 2 : 1; }
    template <class E> __device__ __forceinline__ int lane_base() const {
        return RAG ? warp * buffer<E>() + lane * bytes<E>() : (int)threadIdx.x * 16;
    }
    template <class E> __device__ __forceinline__ int chunk_step() const {
        return RAG ? warps * buffer<E>() : vectors<E>() * kUnitThreads * 16;
    }
    template <class E> __host__ __device__ static constexpr int piece_step() {
        return RAG ? 128 * (int)sizeof(E) : sizeof(E) == 4 ? kUnitThreads * 16 : 8;
    }
    // how far an address lies past a piece's boundary
    template <class E> __device__ __forceinline__ static int past(const E *p) {
        return RAG ? (int)((uintptr_t)p & (bytes<E>() - 1)) : 0;
    }
    template <class E> __device__ __forceinline__ static void copy(uint32_t to, const char *from) {
        if constexpr (bytes<E>() == 16) rows_copy16(to, from);
        else rows_copy8(to, from);
    }
    // each(to, from) for the vectors of chunk i; to: this lane's place in shared memory; row: at
    // this lane's first column
    template <class E, class F>
    __device__ __forceinline__ void vectors_of(int i, uint32_t to, const E *row,
                                               const F &each) const {
        row += i * stride;
        to += i * chunk_step<E>();
        const int s = past(row);
        const char *const p = reinterpret_cast<const char *>(row) - s;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const int at = (first + i * stride + q * 128) * (int)sizeof(E) - s;
            const int count = row_vectors(at, bytes<E>(), n * (int)sizeof(E),
                                          RAG && q == P - 1 && lane == 31);
            if (count > 0) each(to + q * piece_step<E>(), p + q * 128 * (int)sizeof(E));
            if (RAG && q == P - 1 && count > 1)
                each(to + q * piece_step<E>() + bytes<E>(),
                     p + q * 128 * (int)sizeof(E) + bytes<E>());
        }
    }
    template <class E>
    __device__ __forceinline__ void fetch(int i, uint32_t to, const E *row) const {
        vectors_of(i, to, row, [](uint32_t there, const char *from) { copy<E>(there, from); });
    }
    // the same of a row whose vectors may leave the tensor, [begin, end)
    template <class E>
    __device__ __forceinline__ void fetch_within(int i, uint32_t to, const E *row, const E *begin,
                                                 const E *end) const {
        vectors_of(i, to, row, [&](uint32_t there, const char *from) {
            copy_within((uintptr_t)from, bytes<E>(), (int)sizeof(E), (uintptr_t)begin,
                        (uintptr_t)end, [&] { copy<E>(there, from); },
                        [&](int b) { rows_move<sizeof(E)>(there + b, from + b); });
        });
    }
    // Columns past the row's end are never copied to: zero, once, for good (on vectors).
    template <class E> __device__ __forceinline__ void clear(int i, char *at) const {
        if constexpr (RAG) return;
        at += i * chunk_step<E>();
#pragma unroll
        for (int q = 0; q < P; ++q) {
            if (on(i, q)) continue;
            uint2 *const p = reinterpret_cast<uint2 *>(at + q * piece_step<E>());
            p[0] = make_uint2(0, 0);
            if (bytes<E>() == 16) p[1] = make_uint2(0, 0);
        }
    }
    // A chunk of the lane, packed, 0 past the row's end where it was cleared (or RAGGED).
    template <class E> struct Words {
        uint32_t w[2 * sizeof(E)];
        __device__ __forceinline__ void zero() {
#pragma unroll
            for (int k = 0; k < (int)(2 * sizeof(E)); ++k) w[k] = 0;
        }
        __device__ __forceinline__ float2 pair(int j) const {
            if constexpr (sizeof(E) == 4)
                return make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
            else
                return open2<E>(w[j]);
        }
        // pair j: 0 where its bits of a chunk's are
        __device__ __forceinline__ void mask(int j, uint32_t bits) {
            if constexpr (sizeof(E) == 4) {
                if (!(bits >> (2 * j) & 1)) w[2 * j] = 0;
                if (!(bits >> (2 * j + 1) & 1)) w[2 * j + 1] = 0;
            } else {
                w[j] &= (bits >> (2 * j) & 1 ? 0xFFFFu : 0u) |
                        (bits >> (2 * j + 1) & 1 ? 0xFFFF0000u : 0u);
            }
        }
    };
    // s: past() of the row in memory
    template <class E>
    __device__ __forceinline__ void read(Words<E> &r, int i, const char *at, int s) const {
        constexpr int W = bytes<E>() / 4;
        at += i * chunk_step<E>();
#pragma unroll
        for (int q = 0; q < P; ++q) {
            const char *const p = at + q * piece_step<E>();
            uint32_t x[2 * W];
#pragma unroll
            for (int k = 0; k < (RAG ? 2 : 1); ++k) {
                if constexpr (W == 4) {
                    const uint4 v = reinterpret_cast<const uint4 *>(p)[k];
                    x[4 * k] = v.x;
                    x[4 * k + 1] = v.y;
                    x[4 * k + 2] = v.z;
                    x[4 * k + 3] = v.w;
                } else {
                    const uint2 v = reinterpret_cast<const uint2 *>(p)[k];
                    x[2 * k] = v.x;
                    x[2 * k + 1] = v.y;
                }
            }
            uint32_t y[W];
            if constexpr (RAG) {
                shift_words<W, sizeof(E) == 2>(x, y, s);
                if (ends(i)) {
                    const int left = n - (first + i * stride + q * 128);   // columns from the piece on
                    constexpr int each = 4 / (int)sizeof(E);
#pragma unroll
                    for (int k = 0; k < W; ++k) {
                        if (left < each * k + 1) y[k] = 0;
                        else if (each == 2 && left < each * k + 2) y[k] &= 0xFFFF;
                    }
                }
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) y[k] = x[k];
            }
#pragma unroll
            for (int k = 0; k < W; ++k) r.w[q * W + k] = y[k];
        }
    }
    template <class E>
    __device__ __forceinline__ void open(int i, const char *at, int s, float2 *v) const {
        Words<E> w;
        read<E>(w, i, at, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w.pair(j);
    }
    // pair j of chunk i, 0 past the row's end
    __device__ __forceinline__ float2 live(int i, int j, float2 v) const {
        if constexpr (RAG) {
            if (ends(i)) {
                const int left = n - (col(i, j >> 1) + 2 * (j & 1));
                v = make_float2(left > 0 ? v.x : 0.0f, left > 1 ? v.y : 0.0f);
            }
            return v;
        } else {
            return on(i, j >> 1) ? v : two(0.0f);
        }
    }

    // ---- an output
    template <class E> __device__ __forceinline__ void store(int i, E *row, const float2 *v) const {
        row += i * stride;
#pragma unroll
        for (int q = 0; q < P; ++q) {
            constexpr int W = bytes<E>() / 4;
            uint32_t own[W];
#pragma unroll
            for (int k = 0; k < W; ++k) {
                if constexpr (sizeof(E) == 4)
                    own[k] = __float_as_uint(k & 1 ? v[q * W / 2 + k / 2].y : v[q * W / 2 + k / 2].x);
                else
                    own[k] = pack2<E>(v[q * W + k]);
            }
            E *p = row + q * 128;
            if constexpr (!RAG) {
                if (on(i, q)) vector<W>(p, own);
            } else {
                const int at = first + i * stride + q * 128, s = past(p), se = s / (int)sizeof(E);
                // the vector at p - s: the neighbour's last s bytes, then this lane's first
                uint32_t x[2 * W], y[W];
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    x[k] = __shfl_up_sync(0xFFFFFFFFu, own[k], 1);
                    x[W + k] = own[k];
                }
                const bool mine = s == 0 ? at + C <= n : lane > 0 && at - se + C <= n;
                const bool next = s == 0 ? mine : lane < 31 && at + 2 * C - se <= n;
                if (s) {
                    shift_words<W, sizeof(E) == 2>(x, y, bytes<E>() - s);
                } else {
#pragma unroll
                    for (int k = 0; k < W; ++k) y[k] = own[k];
                }
                if (mine) vector<W>(reinterpret_cast<char *>(p) - s, y);
                // columns in no whole vector of the warp's
                if (!mine || !next) {
#pragma unroll
                    for (int e = 0; e < C; ++e)
                        if (at + e < n && !(e < C - se ? mine : next)) {
                            const float2 w = v[q * C / 2 + e / 2];
                            p[e] = from_f<E>(e & 1 ? w.y : w.x);
                        }
                }
            }
        }
    }
    template <int W> __device__ __forceinline__ static void vector(void *p, const uint32_t (&w)[W]) {
        if constexpr (W == 4) *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
    // binary32 sums of chunk i's columns, into a row of them that ends on a vector
    __device__ __forceinline__ void store_sums(int i, float *row, const float2 *v) const {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            if (col(i, q) < n)
                *reinterpret_cast<float4 *>(row + col(i, q)) =
                    make_float4(v[2 * q].x, v[2 * q].y, v[2 * q + 1].x, v[2 * q + 1].y);
    }

    // ---- what is kept: element e of chunk i in bit e
    __device__ __forceinline__ uint32_t kept(int i, const DropArgs &d, uint32_t row,
                                             uint2 offset) const {
        uint32_t r = 0;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint4 w = drop_words(d, (uint32_t)col(i, q) >> 2, row, offset);
            r |= ((uint32_t)(w.x >= d.least) | (uint32_t)(w.y >= d.least) << 1 |
                  (uint32_t)(w.z >= d.least) << 2 | (uint32_t)(w.w >= d.least) << 3) << (4 * q);
        }
        return r;
    }
    template <class... V>
    __device__ __forceinline__ void drop(int i, const DropArgs &d, uint32_t row, uint2 offset,
                                         V *...rows) const {
#pragma unroll
        for (int q = 0; q < 2; ++q)
            drop_four(drop_words(d, (uint32_t)col(i, q) >> 2, row, offset), d.least, q, rows...);
    }
};

// sums of eight, and of their squares
__device__ __forceinline__ float sum8(const float2 *v) {
    const float2 a = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    return a.x + a.y;
}
__device__ __forceinline__ float squares(const float2 *v) {
    float2 x = __fmul2_rn(v[0], v[0]);
#pragma unroll
    for (int j = 1; j < 4; ++j) x = __ffma2_rn(v[j], v[j], x);
    return x.x + x.y;
}

// Four values' sums over a warp: lanes 8 k .. 8 k + 7 get that of v[k].  Six
// exchanges: each halves what a lane still carries.
__device__ __forceinline__ float warp_sums4(const float (&v)[4], int lane) {
    const bool up = lane & 16;
    float a = up ? v[2] : v[0], b = up ? v[3] : v[1];
    a += __shfl_xor_sync(0xFFFFFFFFu, up ? v[0] : v[2], 16);
    b += __shfl_xor_sync(0xFFFFFFFFu, up ? v[1] : v[3], 16);
    const bool odd = lane & 8;
    float r = odd ? b : a;
    r += __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    return r;
}

__device__ __forceinline__ float eighth_sums(float r) {   // over lanes 8 k .. 8 k + 7
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) r += __shfl_xor_sync(0xFFFFFFFFu, r, o);
    return r;
}

// A team of at most 16 warps, one of a CTA's: its exchanges go through [2][12][warps] floats
// in turn, with a barrier each (1 .. 8; 0 is the CTA's, and teams of one warp have none).
// In a join lane l stands for warps l % 8 and l % 8 + 8.
struct UnitTeam {
    int lane, warp, warps, id, half;
    float *s;
    float inv_n;

    __device__ __forceinline__ void start(const RowsGeom &g, int n, float *sums) {
        lane = threadIdx.x & 31;
        warps = g.warps;
        id = (threadIdx.x >> 5) / warps;
        warp = (threadIdx.x >> 5) - id * warps;
        s = sums + id * 24 * warps;
        half = 0;
        inv_n = 1.0f / (float)n;
    }
    __device__ __forceinline__ float *turn() {
        half = half ? 0 : 12 * warps;
        return s + half;
    }
    __device__ __forceinline__ void meet() const {
        asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(warps * 32) : "memory");
    }
    // over the warps, of row k of what they left; the same in lanes 8 j .. 8 j + 7
    __device__ __forceinline__ float join(const float *at, int k) const {
        at += k * warps;
        const int w = lane & 7;
        float r = w < warps ? at[w] : 0.0f;
        if (warps > 8) r += w + 8 < warps ? at[w + 8] : 0.0f;
        return eighth_sums(r);
    }
    // the team's sum of v
    __device__ __forceinline__ float sum(float v) {
        float one[1] = {v};
        warp_sums(one);
        if (warps == 1) return one[0];
        float *const at = turn();
        if (lane == 0) at[warp] = one[0];
        meet();
        return join(at, 0);
    }
    // the team's sums of each v
    template <int K> __device__ __forceinline__ void sums(float (&v)[K]) {
        constexpr int G = (K + 3) / 4;
        float r[G];
#pragma unroll
        for (int g = 0; g < G; ++g) {
            float four[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) four[k] = 4 * g + k < K ? v[4 * g + k] : 0.0f;
            r[g] = warp_sums4(four, lane);
        }
        if (warps > 1) {
            float *const at = turn();
#pragma unroll
            for (int g = 0; g < G; ++g)
                if ((lane & 7) == 0) at[(4 * g + (lane >> 3)) * warps + warp] = r[g];
            meet();
#pragma unroll
            for (int g = 0; g < G; ++g) r[g] = join(at, 4 * g + (lane >> 3));
        }
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = __shfl_sync(0xFFFFFFFFu, r[k / 4], 8 * (k % 4));
    }
};

// (mean, 1 / deviation) of a row in registers, 0 past its end: the mean first, then the
// squares about it (a RMS norm: about 0).
template <bool LAYER, class L, int VPT>
__device__ __forceinline__ float2 unit_moments(UnitTeam &t, const L &l, const float2 (&v)[VPT][4],
                                               int norm, float eps) {
    float mean = 0.0f, q = 0.0f;
    const bool layer = LAYER && norm == EBIN_NORM_LAYER;
    if (layer) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (!l.none(i)) s += sum8(v[i]);
        mean = t.sum(s) * t.inv_n;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if (l.none(i)) continue;
        if (layer) {
            float2 d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = l.live(i, k, __fadd2_rn(v[i][k], two(-mean)));
            q += squares(d);
        } else {
            q += squares(v[i]);
        }
    }
    return make_float2(mean, rsqrtf(fmaf(t.sum(q), t.inv_n, eps)));
}

// The copies of a row whose vectors may leave the tensor, [begin, end): rare, and a call, so that
// it takes no registers from the rows between.
template <int VPT, class L, class E>
__device__ __noinline__ void unit_fetch_within(const L l, uint32_t to, const E *row,
                                               const E *begin, const E *end) {
#pragma unroll 1
    for (int i = 0; i < VPT; ++i)
        if (!l.none(i)) l.fetch_within(i, to, row, begin, end);
}

// A tensor's rows on their way to shared memory: the next row, and its step.
template <class E> struct UnitFrom {
    const E *row;
    int64_t step;
    template <class L>
    __device__ __forceinline__ UnitFrom(const L &l, const void *p, int64_t ld, int first, int rows)
        : row(static_cast<const E *>(p) + (p ? first * ld + l.first : 0)), step(p ? rows * ld : 0) {}
    template <int VPT, class L> __device__ __forceinline__ void fetch(const L &l, uint32_t to) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
            if (!l.none(i)) l.fetch(i, to, row);
        row += step;
    }
    // of a row whose vectors may leave the tensor, `rows` rows from p on
    template <int VPT, class L>
    __device__ __forceinline__ void fetch_within(const L &l, uint32_t to, const void *p, int64_t ld,
                                                 int64_t rows) {
        const E *const begin = static_cast<const E *>(p);
        unit_fetch_within<VPT>(l, to, row, begin, begin + ((rows - 1) * ld + l.n));
        row += step;
    }
};

template <class T, class S, bool LAYER, bool RAG>
__global__ void __launch_bounds__(kUnitThreads, 1)
k_block_unit(const BlockArgs a, const RowsGeom g) {
    using Lane = UnitLane<T, S, RAG>;
    constexpr int VPT = kUnitVpt;
    __shared__ float s_sums[24 * kUnitWarps];
    extern __shared__ uint4 s_rows[];   // the tables, then the slots: x, then y
    UnitTeam t;
    t.start(g, (int)a.n, s_sums);
    Lane l;
    l.place(t.lane, t.warp, g.warps, g.teams, (int)a.n);
    const int64_t unit = blockIdx.x, group = unit / a.cta.parts, part = unit - group * a.cta.parts;
    const int r0 = (int)(group * a.group_rows + part * a.cta.rows);
    const int r1 = (int)min(r0 + a.cta.rows, (group + 1) * a.group_rows);
    const int step = g.teams;
    const bool post = a.post != EBIN_NORM_NONE;
    const float branch = a.branch_scale * (a.drop.least ? a.drop.scale : 1.0f);
    float4 *table = reinterpret_cast<float4 *>(s_rows);
    UnitTable<Lane> by[4];   // of bit k
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        by[k] = UnitTable<Lane>{table + t.warp * 64 + t.lane, g.warps};
        if (g.tables >> k & 1) table += g.table;
    }
    char *const mine = reinterpret_cast<char *>(table);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine);
    const int ahead = g.slots - 1, last = ahead * g.slot_bytes;
    const int x_at = l.template lane_base<S>();
    const int y_at = VPT * l.template chunk_step<S>() + l.template lane_base<T>();
    for (int k = 0; k <= last; k += g.slot_bytes)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            l.template clear<S>(i, mine + k + x_at);
            if (a.y) l.template clear<T>(i, mine + k + y_at);
        }
    int fill = 0, slot = 0, next = r0 + t.id;
    UnitFrom<S> from_x(l, a.x, a.ld_x, next, step);
    UnitFrom<T> from_y(l, a.y, a.ld_y, next, step);
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    auto fetch = [&]() {
        if (next < r1) {
            if (RAG) __syncwarp();   // the slot has been read
            if (RAG && __builtin_expect(row_at_edge(next, (int)a.rows), 0)) {
                from_x.template fetch_within<VPT>(l, to + fill + x_at, a.x, a.ld_x, a.rows);
                if (a.y) from_y.template fetch_within<VPT>(l, to + fill + y_at, a.y, a.ld_y, a.rows);
            } else {
                from_x.template fetch<VPT>(l, to + fill + x_at);
                if (a.y) from_y.template fetch<VPT>(l, to + fill + y_at);
            }
            next += step;
        }
        fill = fill == last ? 0 : fill + g.slot_bytes;
        rows_commit();
    };
    for (int i = 0; i < ahead; ++i) fetch();
    {
        uint32_t index, rest;
        g.gate.split((uint32_t)r0, index, rest);
        const void *const gate = block_row<T>(a.gate, index * a.ld_gate, a.mod_f32);
        g.mod.split((uint32_t)r0, index, rest);
        const void *const scale = block_row<T>(a.scale, index * a.ld_scale, a.mod_f32);
        const void *const shift = block_row<T>(a.shift, index * a.ld_shift, a.mod_f32);
        float4 *at = reinterpret_cast<float4 *>(s_rows);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
            if (!(g.tables >> k & 1)) continue;
            const bool y = k < 2, more = k & 1;
            unit_fill<Lane>(at, g.table, (int)a.n, [&](int col) {
                const float4 m = y ? mul4(four(branch), params4<T, RAG>(gate, col, l.n, a.mod_f32, 1.0f))
                                   : add4(four(1.0f), params4<T, RAG>(scale, col, l.n, a.mod_f32, 0.0f));
                const void *const w = y ? (more ? a.b_post : a.w_post) : (more ? a.b_pre : a.w_pre);
                float4 r = mul4(m, params4<T, RAG>(w, col, l.n, a.w_f32, more ? 0.0f : 1.0f));
                if (k == 3) r = add4(r, params4<T, RAG>(shift, col, l.n, a.mod_f32, 0.0f));
                return r;
            });
            at += g.table;
        }
    }
    __syncthreads();
    S *h = static_cast<S *>(a.h) + (a.h ? (r0 + t.id) * a.ld_h + l.first : 0);
    T *z = static_cast<T *>(a.z) + (a.z ? (r0 + t.id) * a.ld_z + l.first : 0);
    const int64_t step_h = step * a.ld_h, step_z = step * a.ld_z;
    for (int row = r0 + t.id; row < r1; row += step, h += step_h, z += step_z) {
        fetch();
        rows_wait(ahead);
        if (RAG) __syncwarp();   // a lane reads what its neighbour copied
        const char *const at = mine + slot;
        slot = slot == last ? 0 : slot + g.slot_bytes;
        const int s_x = Lane::past(static_cast<const S *>(a.x) + row * a.ld_x + l.first);
        const int s_y = Lane::past(static_cast<const T *>(a.y) + (a.y ? row * a.ld_y + l.first : 0));
        float2 v[VPT][4];
        float2 my = make_float2(0.0f, 1.0f);
        if (a.y) {
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (l.none(i)) continue;
                l.template open<T>(i, at + y_at, s_y, v[i]);
            }
            if (post) my = unit_moments<LAYER>(t, l, v, a.post, a.eps_post);
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (l.none(i)) continue;
            float2 x[4];
            l.template open<S>(i, at + x_at, s_x, x);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = __fmul2_rn(x[k], two(a.stream_scale));
            if (a.y) {
                if (post) norm8<LAYER>(v[i], my);
                if (!(g.tables & TABLE_Y_ADD)) {
                    if (a.drop.least) l.drop(i, a.drop, (uint32_t)row, offset, v[i]);
                    if (g.tables & TABLE_Y) {
                        float2 p[4];
                        by[0].read(i, p);
#pragma unroll
                        for (int k = 0; k < 4; ++k) x[k] = __ffma2_rn(v[i][k], p[k], x[k]);
                    } else {
                        add8(x, v[i]);
                    }
                } else {   // with a bias the mask comes after the factor
                    float2 p[4], q[4];
                    by[0].read(i, q);
                    by[1].read(i, p);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][k] = __ffma2_rn(v[i][k], q[k], p[k]);
                    if (a.drop.least) l.drop(i, a.drop, (uint32_t)row, offset, v[i]);
                    add8(x, v[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i][k] = x[k];
            if (a.h) l.store(i, h, v[i]);
            // the tables end with the row, and so does v, but for a mean taken off y
            if (LAYER)
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i][k] = l.live(i, k, v[i][k]);
        }
        if (!a.z) continue;
        const float2 mh = unit_moments<LAYER>(t, l, v, a.pre, a.eps_pre);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (l.none(i)) continue;
            norm8<LAYER>(v[i], mh);
            if (g.tables & TABLE_H) by[2].times(i, v[i]);
            if (g.tables & TABLE_H_ADD) {
                float2 p[4];
                by[3].read(i, p);
                add8(v[i], p);
            }
            l.store(i, z, v[i]);
        }
    }
    rows_wait(0);
}

__device__ __forceinline__ float2 mask2(float2 v, uint32_t bits, int j) {
    return make_float2(bits >> (2 * j) & 1 ? v.x : 0.0f, bits >> (2 * j + 1) & 1 ? v.y : 0.0f);
}

// The gradient of such units, with a pre norm; its sums in registers as
// k_block_rows_grad's, the teams' joined in shared memory at the end, one after another.
// A row takes one exchange (FULL, with a layer norm: one more before it, of the means).
// What dy needs of D before D is known comes from D's parts: with t = (factor of y) (y
// - mean) the mean of u yh is that of t D, and
//     sum t D = sum t dh + r (sum t m - c0 sum t - r c1 sum t (h - mean)),
// c0 and c1 the means of m and of m hh; so nothing of a row is kept in registers from
// the sums' pass to the outputs'.  Both factors have tables.
template <class T, class S, bool FULL, bool POST, bool RAG>
__global__ void __launch_bounds__(kUnitThreads, 1)
k_block_unit_grad(const BlockArgs a, const RowsGeom g) {
    using Lane = UnitLane<T, S, RAG>;
    using WordsS = typename Lane::template Words<S>;
    using WordsT = typename Lane::template Words<T>;
    constexpr int VPT = kUnitGradVpt<FULL, POST>;
    // the sums kept: SUM_E is a post norm's bias' alone
    constexpr int kKinds = !FULL ? 2 : POST ? 4 : 3;
    __shared__ float s_sums[24 * kUnitWarps];
    extern __shared__ uint4 s_rows[];   // the tables, then the rows; at the end the sums
    UnitTeam t;
    t.start(g, (int)a.n, s_sums);
    Lane l;
    l.place(t.lane, t.warp, g.warps, g.teams, (int)a.n);
    const int64_t unit = blockIdx.x, group = unit / a.cta.parts, part = unit - group * a.cta.parts;
    const int r0 = (int)(group * a.group_rows + part * a.cta.rows);
    const int r1 = (int)min(r0 + a.cta.rows, (group + 1) * a.group_rows);
    const int step = g.teams;
    const bool layer_h = FULL && a.pre == EBIN_NORM_LAYER;
    const bool layer_y = FULL && POST && a.post == EBIN_NORM_LAYER;
    const float branch = a.branch_scale * (a.drop.least ? a.drop.scale : 1.0f);
    float4 *const tables = reinterpret_cast<float4 *>(s_rows);
    const float4 *const by_y = tables + t.warp * 64 + t.lane, *const by_h = by_y + g.table;
    const int table_step = g.warps * 64;
    char *const mine = reinterpret_cast<char *>(s_rows + 2 * g.table);
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(mine);
    const int ahead = g.slots - 1, last = ahead * g.slot_bytes;
    // h, dz, dh and y of a row lie behind one another
    const int s_bytes = VPT * l.template chunk_step<S>(), t_bytes = VPT * l.template chunk_step<T>();
    const int h_at = l.template lane_base<S>(), dh_at = s_bytes + t_bytes + h_at;
    const int dz_at = s_bytes + l.template lane_base<T>(), y_at = dz_at + t_bytes + s_bytes;
    for (int k = 0; k <= last; k += g.slot_bytes)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            l.template clear<S>(i, mine + k + h_at);
            l.template clear<T>(i, mine + k + dz_at);
            l.template clear<S>(i, mine + k + dh_at);
            if (a.y) l.template clear<T>(i, mine + k + y_at);
        }
    int fill = 0, slot = 0, next = r0 + t.id;
    UnitFrom<S> from_h(l, a.x, a.ld_x, next, step), from_dh(l, a.dh, a.ld_dh, next, step);
    UnitFrom<T> from_dz(l, a.dz, a.ld_dz, next, step), from_y(l, a.y, a.ld_y, next, step);
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    auto fetch = [&]() {
        if (next < r1) {
            if (RAG) __syncwarp();   // the slot has been read
            if (RAG && __builtin_expect(row_at_edge(next, (int)a.rows), 0)) {
                from_h.template fetch_within<VPT>(l, to + fill + h_at, a.x, a.ld_x, a.rows);
                from_dz.template fetch_within<VPT>(l, to + fill + dz_at, a.dz, a.ld_dz, a.rows);
                if (a.dh)
                    from_dh.template fetch_within<VPT>(l, to + fill + dh_at, a.dh, a.ld_dh, a.rows);
                if (a.y) from_y.template fetch_within<VPT>(l, to + fill + y_at, a.y, a.ld_y, a.rows);
            } else {
                from_h.template fetch<VPT>(l, to + fill + h_at);
                from_dz.template fetch<VPT>(l, to + fill + dz_at);
                if (a.dh) from_dh.template fetch<VPT>(l, to + fill + dh_at);
                if (a.y) from_y.template fetch<VPT>(l, to + fill + y_at);
            }
            next += step;
        }
        fill = fill == last ? 0 : fill + g.slot_bytes;
        rows_commit();
    };
    for (int i = 0; i < ahead; ++i) fetch();
    {
        uint32_t index, rest;
        g.gate.split((uint32_t)r0, index, rest);
        const void *const gate = block_row<T>(a.gate, index * a.ld_gate, a.mod_f32);
        g.mod.split((uint32_t)r0, index, rest);
        const void *const scale = block_row<T>(a.scale, index * a.ld_scale, a.mod_f32);
        unit_fill<Lane>(tables, g.table, (int)a.n, [&](int col) {
            return mul4(mul4(four(branch), params4<T, RAG>(gate, col, l.n, a.mod_f32, 1.0f)),
                        params4<T, RAG>(a.w_post, col, l.n, a.w_f32, 1.0f));
        });
        unit_fill<Lane>(tables + g.table, g.table, (int)a.n, [&](int col) {
            return mul4(add4(four(1.0f), params4<T, RAG>(scale, col, l.n, a.mod_f32, 0.0f)),
                        params4<T, RAG>(a.w_pre, col, l.n, a.w_f32, 1.0f));
        });
    }
    __syncthreads();
    float2 acc[kKinds][VPT][4];
#pragma unroll
    for (int k = 0; k < kKinds; ++k)
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[k][i][j] = two(0.0f);
    constexpr int kEYh = FULL ? (int)SUM_E_YH : 1;
    T *dy = static_cast<T *>(a.z) + (a.z ? (r0 + t.id) * a.ld_z + l.first : 0);
    S *dx = static_cast<S *>(a.h) + (a.h ? (r0 + t.id) * a.ld_h + l.first : 0);
    const int64_t step_y = step * a.ld_z, step_x = step * a.ld_h;
    auto factor = [&](const float4 *table, int i, float2 *p) {
        const float4 x = table[i * table_step], y = table[i * table_step + 32];
        p[0] = make_float2(x.x, x.y);
        p[1] = make_float2(x.z, x.w);
        p[2] = make_float2(y.x, y.y);
        p[3] = make_float2(y.z, y.w);
    };
    for (int row = r0 + t.id; row < r1; row += step, dy += step_y, dx += step_x) {
        fetch();
        // what both passes keep, drawn while the row is on its way
        uint32_t bits[VPT];
        if (POST && a.drop.least)
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (!l.none(i)) bits[i] = l.kept(i, a.drop, (uint32_t)row, offset);
        rows_wait(ahead);
        if (RAG) __syncwarp();   // a lane reads what its neighbour copied
        const char *const at = mine + slot;
        slot = slot == last ? 0 : slot + g.slot_bytes;
        const int s_h = Lane::past(static_cast<const S *>(a.x) + row * a.ld_x + l.first);
        const int s_dz = Lane::past(static_cast<const T *>(a.dz) + row * a.ld_dz + l.first);
        const int s_dh =
            Lane::past(static_cast<const S *>(a.dh) + (a.dh ? row * a.ld_dh + l.first : 0));
        const int s_y = Lane::past(static_cast<const T *>(a.y) + (a.y ? row * a.ld_y + l.first : 0));
        auto read_h = [&](int i, WordsS &w) { l.template read<S>(w, i, at + h_at, s_h); };
        auto read_dz = [&](int i, WordsT &w) { l.template read<T>(w, i, at + dz_at, s_dz); };
        auto read_dh = [&](int i, WordsS &w) {
            if (a.dh) l.template read<S>(w, i, at + dh_at, s_dh);
            else w.zero();
        };
        auto read_y = [&](int i, WordsT &w) { l.template read<T>(w, i, at + y_at, s_y); };
        float2 mh = make_float2(0.0f, 1.0f), my = mh;
        float c0 = 0.0f, c1 = 0.0f, b0 = 0.0f, b1 = 0.0f;
        if (FULL && (layer_h || layer_y)) {
            float2 s[3] = {two(0.0f), two(0.0f), two(0.0f)};   // of h, y and m: 0 past the row
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (l.none(i)) continue;
                WordsS h;
                WordsT z, y;
                float2 k[4];
                read_h(i, h);
                read_dz(i, z);
                if (POST) read_y(i, y);
                factor(by_h, i, k);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[0] = __fadd2_rn(s[0], h.pair(j));
                    if (POST) s[1] = __fadd2_rn(s[1], y.pair(j));
                    s[2] = __ffma2_rn(z.pair(j), k[j], s[2]);
                }
            }
            float q[3];
#pragma unroll
            for (int k = 0; k < 3; ++k) q[k] = s[k].x + s[k].y;
            t.sums(q);
            if (layer_h) {
                mh.x = q[0] * t.inv_n;
                c0 = q[2] * t.inv_n;
            }
            if (layer_y) my.x = q[1] * t.inv_n;
        }
        {
            // sums of h h, m h, y y, t dh, t m, t h, then (FULL) of t, f dh, f m, f h and f, the
            // factor; h and y less their means
            constexpr int K = !POST ? 2 : FULL ? 11 : 6;
            float2 q[K];
#pragma unroll
            for (int k = 0; k < K; ++k) q[k] = two(0.0f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (l.none(i)) continue;
                WordsS h, d;
                WordsT z, y;
                float2 k[4], f[4];
                read_h(i, h);
                read_dz(i, z);
                factor(by_h, i, k);
                if constexpr (POST) {
                    read_y(i, y);
                    read_dh(i, d);
                    factor(by_y, i, f);
                    if (a.drop.least)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            f[j] = mask2(f[j], bits[i], j);
                            d.mask(j, bits[i]);   // 0 times it may be NaN
                        }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 m = __fmul2_rn(z.pair(j), k[j]);
                    float2 x = h.pair(j);
                    if constexpr (FULL) x = l.live(i, j, __fadd2_rn(x, two(-mh.x)));
                    q[0] = __ffma2_rn(x, x, q[0]);
                    q[1] = __ffma2_rn(m, x, q[1]);
                    if constexpr (POST) {
                        float2 yy = y.pair(j);
                        const float2 dh = d.pair(j);
                        if constexpr (FULL) yy = l.live(i, j, __fadd2_rn(yy, two(-my.x)));
                        q[2] = __ffma2_rn(yy, yy, q[2]);
                        const float2 tt = __fmul2_rn(yy, f[j]);
                        q[3] = __ffma2_rn(tt, dh, q[3]);
                        q[4] = __ffma2_rn(tt, m, q[4]);
                        q[5] = __ffma2_rn(tt, x, q[5]);
                        if constexpr (FULL) {
                            q[6] = __fadd2_rn(q[6], tt);
                            q[7] = __ffma2_rn(f[j], dh, q[7]);
                            q[8] = __ffma2_rn(f[j], m, q[8]);
                            q[9] = __ffma2_rn(f[j], x, q[9]);
                            q[10] = __fadd2_rn(q[10], f[j]);
                        }
                    }
                }
            }
            float w[K];
#pragma unroll
            for (int k = 0; k < K; ++k) w[k] = q[k].x + q[k].y;
            t.sums(w);
            mh.y = rsqrtf(fmaf(w[0], t.inv_n, a.eps_pre));
            c1 = w[1] * mh.y * t.inv_n;
            if constexpr (POST) {
                my.y = rsqrtf(fmaf(w[2], t.inv_n, a.eps_post));
                const float back = mh.y * c1;
                float d = fmaf(-back, w[5], w[4]);
                if constexpr (FULL) d = fmaf(-c0, w[6], d);
                b0 = fmaf(mh.y, d, w[3]) * my.y * t.inv_n;
                if (FULL && layer_y) {
                    d = fmaf(-c0, w[FULL ? 10 : 0], fmaf(-back, w[FULL ? 9 : 0], w[FULL ? 8 : 0]));
                    b1 = fmaf(mh.y, d, w[FULL ? 7 : 0]) * t.inv_n;
                }
            }
        }
        const float2 rh = two(mh.y), ry = two(my.y), down = two(-c1), off = two(-b0);
        const float2 rb = two(-b1 * my.y);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (l.none(i)) continue;
            float2 v[4];   // D, then e, then u and dy
            {
                WordsS h, d;
                WordsT z;
                float2 k[4];
                read_h(i, h);
                read_dz(i, z);
                read_dh(i, d);
                factor(by_h, i, k);
                float2 out[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 x = h.pair(j);
                    if constexpr (FULL) x = __fadd2_rn(x, two(-mh.x));
                    x = __fmul2_rn(x, rh);
                    const float2 dz = z.pair(j);
                    acc[0][i][j] = __ffma2_rn(dz, x, acc[0][i][j]);
                    float2 m;
                    if constexpr (FULL) {
                        acc[1][i][j] = __fadd2_rn(acc[1][i][j], dz);
                        m = __ffma2_rn(dz, k[j], two(-c0));
                    } else {
                        m = __fmul2_rn(dz, k[j]);
                    }
                    v[j] = __ffma2_rn(__ffma2_rn(x, down, m), rh, d.pair(j));
                    out[j] = __fmul2_rn(v[j], two(a.stream_scale));
                }
                if (a.h) l.store(i, dx, out);
            }
            if (a.drop.least) {
                if constexpr (!POST) bits[i] = l.kept(i, a.drop, (uint32_t)row, offset);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = mask2(v[j], bits[i], j);
            }
            if constexpr (FULL && POST) add8(acc[kKinds - 1][i], v);
            float2 f[4];
            factor(by_y, i, f);
            if (POST || a.y) {
                WordsT y;
                read_y(i, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float2 x = y.pair(j);
                    // What is dropped adds nothing to the gate's, whatever y is there.  Its bits
                    // hold fewer registers than y over Philox's rounds (66.6 us, and 70.7).
                    if (!POST && a.drop.least) x = mask2(x, bits[i], j);
                    if constexpr (POST) {
                        if constexpr (FULL) x = __fadd2_rn(x, two(-my.x));
                        x = __fmul2_rn(x, ry);
                    }
                    acc[kEYh][i][j] = __ffma2_rn(v[j], x, acc[kEYh][i][j]);
                    v[j] = __fmul2_rn(v[j], f[j]);
                    if constexpr (POST) {
                        v[j] = __ffma2_rn(x, off, v[j]);
                        v[j] = FULL ? __ffma2_rn(v[j], ry, rb) : __fmul2_rn(v[j], ry);
                    }
                }
            } else {
                mul8(v, f);
            }
            if (a.z) l.store(i, dy, v);
        }
    }
    rows_wait(0);
    if (!a.partial) return;
    float2 *const sums = reinterpret_cast<float2 *>(s_rows) + t.warp * 32 + t.lane;
    const int team_threads = g.warps * 32;
    for (int team = 0; team < g.teams; ++team) {
        __syncthreads();   // the rows have been read; the team before has added
        if (t.id != team) continue;
        float *const partial = a.partial + unit * 4 * a.pad;
#pragma unroll
        for (int k = 0; k < kKinds; ++k)
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (l.none(i)) continue;
                float2 *const at = sums + (k * VPT + i) * 4 * team_threads;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (team > 0) acc[k][i][j] = __fadd2_rn(at[j * team_threads], acc[k][i][j]);
                    if (team + 1 < g.teams) at[j * team_threads] = acc[k][i][j];
                }
                if (team + 1 < g.teams) continue;
                const int kind = FULL ? k : 2 * k;
                if (kind == SUM_E_YH || kind == SUM_E) {   // they carry their factor from here on
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[k][i][j] = __fmul2_rn(acc[k][i][j], two(branch));
                }
                l.store_sums(i, partial + kind * a.pad, acc[k][i]);
            }
    }
}

}  // namespace ebin
