// The product on the tensor cores: operand tiles by tensor copies (TMA) into
// swizzled shared memory, tcgen05.mma into accumulators in tensor memory, the
// epilogue from there.
//
// Mathematics: D = P Q^T over k, P's rows the lanes of the accumulator (128 a
// CTA), Q's rows its columns (BN).  A product runs either way round: P = A
// and Q = B, or, for few rows of A, P = B and Q = A, so that the long operand
// fills the 128 lanes.  Either operand may be dense along k or across it: the
// shared-memory descriptors say which, nothing is transposed.
//
// Warps of a CTA: 0 issues the copies, 1 the matrix instructions, 2 holds the
// tensor memory, 4.. run the epilogue.  Barriers between them: `full` and
// `empty` per stage of operands, `tfull` and `tempty` per accumulator.  Every
// wait has a limit.  One that runs out, in any warp, is told to every CTA of the
// cluster; they meet, the leader waits (each wait again with the limit) for the
// products and the copies that are still on their way, both CTAs' on a pair, and
// only then is shared memory reused or left and the tensor memory given back.
// EBIN_DEVICE_WAIT_LIMIT is raised and the output is not valid.
//
// What bounds it.  Large products: the matrix instructions (a pair's 256 x 256 x
// 64 step takes 512 clocks at best) and the power they draw, so that times go by
// the clock that the limit leaves (1.5 to 1.7 GHz in a long run): [4096,4096] x
// [4096,8192] bf16 154 us, with bias and GELU 160 to 168, 1640 to 1720 TFLOP/s; 8192^3
// 547 to 630 us.  Few rows: reading B, [4,4096] x [4096,4096] 9.8 us from memory: 5.0
// us of reading at the copy's rate, the rest launch, set-up, the cluster's meetings
// and the join (7.2 us with B in the L2).  In between, a CTA's copies (190 bytes a
// ns) and the 4 to 6 us of an unoverlapped first tile and last epilogue.
#pragma once

#include <type_traits>

#include <cuda.h>

#include "ebin_gemm.cuh"
#include "ebin_gemm_drain.h"

namespace ebin {

constexpr int kTcBK = 64;                    // k per stage: one 128-byte swizzle row
constexpr int kTcRows = 128;                 // accumulator lanes of a CTA
constexpr int kTcSmem = 227 * 1024;

struct TcArgs {
    GemmEpilogue e;
    int64_t m, n;
    int32_t kblocks;            // k in steps of kTcBK
    int32_t p_tiles, q_tiles;   // tiles of P's rows (kTcRows * CTAs) and of Q's (BN)
    int32_t p_mn, q_mn;         // the operand is dense across k
    int32_t q_box;              // Q's rows a copy brings when it is dense along k
    int32_t stage, stages;      // bytes of a stage of operands, and how many
    int32_t vec;                // y, z, residual and bias take accesses of 16 bytes (1) or 32 (2)
    long long limit;            // clocks of a wait
    uint32_t *status;
};

__device__ __forceinline__ uint32_t tc_smem(const void *p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void tc_bar_init(uint32_t bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void tc_bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
// take bytes that will not come off a barrier's count
__device__ __forceinline__ void tc_bar_count_off(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
// arrive at a barrier of this cluster, by its cluster address
__device__ __forceinline__ void tc_bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool tc_bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return ok != 0;
}
// Wait for the phase of the given parity; false when the limit ran out.
__device__ __forceinline__ bool tc_bar_wait(uint32_t bar, uint32_t parity, long long limit) {
    for (int i = 0; i < 32; ++i)
        if (tc_bar_try(bar, parity)) return true;
    const long long t0 = clock64();
    while (clock64() - t0 < limit)
        if (tc_bar_try(bar, parity)) return true;
    return false;
}
// a CTA of this cluster's view of a shared-memory address of this CTA's layout
__device__ __forceinline__ uint32_t tc_map(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t tc_cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t tc_cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void tc_put_word(uint32_t cluster_addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ void tc_cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool tc_elect() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one));
    return one != 0;
}

template <int CTAS>
__device__ __forceinline__ void tc_copy(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global"
                     ".mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(map), "r"(bar), "r"(x), "r"(y)
                     : "memory");
    else
        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
                     "[%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
                     "l"(map), "r"(bar), "r"(x), "r"(y)
                     : "memory");
}

template <int CTAS> __device__ __forceinline__ void tc_alloc(uint32_t dst, int columns) {
    if constexpr (CTAS == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}
template <int CTAS> __device__ __forceinline__ void tc_free(uint32_t addr, int columns) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr),
                     "r"(columns));
}

// Shared-memory operand descriptor: 128-byte swizzle; rows of 128 bytes, eight
// of them 1024 bytes on (k-dense operands), or, for operands dense across k,
// blocks of 64 k by 64 rows 8192 bytes on.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, bool mn) {
    const uint64_t lead = mn ? 8192 >> 4 : 1, stride = 1024 >> 4;
    return (uint64_t)((addr >> 4) & 0x3FFF) | (lead << 16) | (stride << 32) | (1ull << 46) |
           (2ull << 61);
}

template <int CTAS>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t add) {
    if constexpr (CTAS == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(add)
                     : "memory");
    else
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                     "l"(a), "l"(b), "r"(idesc), "r"(add)
                     : "memory");
}

// Arrive at `bar` (of both CTAs of a pair) when the products issued so far are done.
template <int CTAS> __device__ __forceinline__ void tc_commit(uint32_t bar) {
    if constexpr (CTAS == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                     ".multicast::cluster.b64 [%0], %1;" ::"r"(bar),
                     "h"((uint16_t)3)
                     : "memory");
    else
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
                     "[%0];" ::"r"(bar)
                     : "memory");
}

__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

// Accumulator columns of a warp's 32 lanes: thread = lane.  The load and its
// wait are one statement: the registers hold nothing before the wait.
__device__ __forceinline__ void tc_load16(uint32_t addr, float *v) {
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tc_load32(uint32_t addr, float *v) {
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
                 "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]),
                   "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
                   "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
                   "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
                   "=r"(r[30]), "=r"(r[31])
                 : "r"(addr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

template <class T> __device__ __forceinline__ uint32_t tc_pack(float lo, float hi) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __half2 p = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
}
template <class T> __device__ __forceinline__ void tc_unpack8(const uint4 &w, float *v) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}
template <class T> __device__ __forceinline__ uint4 tc_pack8(const float *v) {
    return make_uint4(tc_pack<T>(v[0], v[1]), tc_pack<T>(v[2], v[3]), tc_pack<T>(v[4], v[5]),
                      tc_pack<T>(v[6], v[7]));
}

template <int ACT, int N> __device__ __forceinline__ void tc_act_all(float *v) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = act_value<ACT>(v[i]);
}
template <int N> __device__ __forceinline__ void tc_act(int act, float *v) {
    switch (act) {
    case EBIN_ACT_RELU: tc_act_all<EBIN_ACT_RELU, N>(v); break;
    case EBIN_ACT_GELU: tc_act_all<EBIN_ACT_GELU, N>(v); break;
    case EBIN_ACT_GELU_TANH: tc_act_all<EBIN_ACT_GELU_TANH, N>(v); break;
    case EBIN_ACT_SILU: tc_act_all<EBIN_ACT_SILU, N>(v); break;
    }
}

template <class T>
__device__ __forceinline__ float tc_bias(const GemmEpilogue &e, int64_t n) {
    if (!e.bias) return 0.0f;
    return e.bias_f32 ? static_cast<const float *>(e.bias)[n]
                      : to_f(static_cast<const T *>(e.bias)[n]);
}

// `most` (or N) neighbouring rows m of column n, where neighbouring lanes hold
// neighbouring n.
template <class T, int N>
__device__ __forceinline__ void tc_store_down(const GemmEpilogue &e, int64_t m, int64_t n,
                                              float *v, int most, float bias) {
    float r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += bias;
    if (e.residual) {
        const T *p = static_cast<const T *>(e.residual) + m * e.ld_residual + n;
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = i < most ? to_f(p[i * e.ld_residual]) : 0.0f;
    }
    if (e.z) {
        T *p = static_cast<T *>(e.z) + m * e.ldz + n;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < most) p[i * e.ldz] = from_f<T>(v[i]);
    }
    tc_act<N>(e.act, v);
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += r[i];
    }
    T *p = static_cast<T *>(e.y) + m * e.ldy + n;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < most) p[i * e.ldy] = from_f<T>(v[i]);
}

// 32 bytes: in one access (a whole sector a lane) or in two.
template <bool WIDE> __device__ __forceinline__ void tc_put32(void *p, const uint4 &a, const uint4 &b) {
    if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x),
                     "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = a;
        static_cast<uint4 *>(p)[1] = b;
    }
}
template <bool WIDE> __device__ __forceinline__ void tc_get32(const void *p, uint4 &a, uint4 &b) {
    if constexpr (WIDE) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z),
                       "=r"(b.w)
                     : "l"(p)
                     : "memory");
    } else {
        a = static_cast<const uint4 *>(p)[0];
        b = static_cast<const uint4 *>(p)[1];
    }
}

// 16 neighbouring columns n of row m, all inside the output, vectors aligned.
template <class T, bool WIDE>
__device__ __forceinline__ void tc_store16(const GemmEpilogue &e, int64_t m, int64_t n, float *v) {
    uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
    if (e.residual)
        tc_get32<WIDE>(static_cast<const T *>(e.residual) + m * e.ld_residual + n, r0, r1);
    if (e.bias) {
        if (e.bias_f32) {
            const float4 *b = reinterpret_cast<const float4 *>(static_cast<const float *>(e.bias) + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldg(b + i);
                v[4 * i] += f.x;
                v[4 * i + 1] += f.y;
                v[4 * i + 2] += f.z;
                v[4 * i + 3] += f.w;
            }
        } else {
            const uint4 *b = reinterpret_cast<const uint4 *>(static_cast<const T *>(e.bias) + n);
            float f[16];
            tc_unpack8<T>(__ldg(b), f);
            tc_unpack8<T>(__ldg(b + 1), f + 8);
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += f[i];
        }
    }
    if (e.z)
        tc_put32<WIDE>(static_cast<T *>(e.z) + m * e.ldz + n, tc_pack8<T>(v), tc_pack8<T>(v + 8));
    tc_act<16>(e.act, v);
    if (e.residual) {
        float f[16];
        tc_unpack8<T>(r0, f);
        tc_unpack8<T>(r1, f + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] += f[i];
    }
    tc_put32<WIDE>(static_cast<T *>(e.y) + m * e.ldy + n, tc_pack8<T>(v), tc_pack8<T>(v + 8));
}

// What a kernel's shared memory holds, in bytes.  The stages fill what is left:
// a weight that streams from memory wants all the copies in flight that fit
// (one CTA an SM with eight stages against two with four: [64,8192] x
// [8192,8192] bf16 31.5 -> 28.5 us).
template <int CTAS, int BN, bool SPLIT> struct TcLayout {
    static constexpr int kP = kTcRows * 128;
    static constexpr int kQRows = (BN / CTAS + 63) / 64 * 64;       // dense across k: blocks of 64
    static constexpr int kEpilogueWarps = SPLIT ? 4 : 8;
    static constexpr int kScratch = SPLIT ? 0 : kEpilogueWarps * 32 * 33 * 4;   // 32 x 32 transposes
    static constexpr int kBarriers = 512;
    static constexpr int kRoom = kTcSmem - 1024 - kScratch - kBarriers;
    static constexpr int kAccumulators = SPLIT ? 1 : 2;
    static constexpr int kAccStep = BN <= 32 ? 32 : BN <= 64 ? 64 : BN <= 128 ? 128 : 256;
    static constexpr int kColumns = kAccumulators * kAccStep;
    static constexpr int kBytes = kTcSmem;
    static constexpr int kThreads = 128 + 32 * kEpilogueWarps;
    static constexpr int kMostStages = 12;
    static_assert(8 * (2 * kMostStages + 5) + 24 <= kBarriers, "room for the barriers and words");
    // bytes of a stage: P's rows, and Q's (rows or blocks), on 1024-byte boundaries
    static int stage(bool q_mn) { return kP + (q_mn ? kQRows : (BN / CTAS + 7) / 8 * 8) * 128; }
    static int stages(bool q_mn) {
        const int n = kRoom / stage(q_mn);
        return n > kMostStages ? kMostStages : n;
    }
};

// One tile after another (SPLIT = false): clusters of CTAS CTAs take tiles in
// steps of their number; a pair's accumulator is 256 lanes over two CTAs, the
// leader issues the products for both, each brings its own half of Q.
// SPLIT: the CTAs of a cluster share one tile's k and join their sums in each
// other's shared memory, in rank order; P = B, Q = A.
template <class T, int CTAS, int BN, bool SPLIT>
__global__ void __launch_bounds__(TcLayout<CTAS, BN, SPLIT>::kThreads, 1)
k_gemm_tc(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
          const TcArgs a) {
    using L = TcLayout<CTAS, BN, SPLIT>;
    static_assert(!SPLIT || CTAS == 1, "a split tile is a single CTA's");
    extern __shared__ uint8_t s_raw[];
    const uint32_t base = (tc_smem(s_raw) + 1023) & ~1023u;
    uint8_t *const s_base = s_raw + (base - tc_smem(s_raw));
    const uint32_t scratch = base + a.stages * a.stage;
    const uint32_t bars = scratch + L::kScratch;
    auto full = [&](int i) { return bars + 8 * i; };
    auto empty = [&](int i) { return bars + 8 * (L::kMostStages + i); };
    auto tfull = [&](int i) { return bars + 8 * (2 * L::kMostStages + i); };
    auto tempty = [&](int i) { return bars + 8 * (2 * L::kMostStages + 2 + i); };
    const uint32_t drain = bars + 8 * (2 * L::kMostStages + 4);
    const uint32_t s_tmem = drain + 8;
    const uint32_t s_failed = drain + 12;   // a wait of this cluster ran out
    const uint32_t s_issued = drain + 16;   // the leader's: steps issued by it, by its peer
    auto word = [&](uint32_t at) {
        return *reinterpret_cast<volatile uint32_t *>(s_base + (at - base));
    };
    // uniform in the warp, so that what follows from it can stay in uniform registers
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = tc_cluster_rank(), ranks = tc_cluster_size();
    const bool leader = CTAS == 1 || rank == 0;

    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            tc_bar_init(full(i), 1);
            tc_bar_init(empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc_bar_init(tfull(i), 1);
            tc_bar_init(tempty(i), CTAS * L::kEpilogueWarps);
        }
        tc_bar_init(drain, 1);
        *reinterpret_cast<volatile uint32_t *>(s_base + (s_failed - base)) = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 2) tc_alloc<CTAS>(s_tmem, L::kColumns);
    layer_pdl_launch();
    tc_fence_before();
    __syncthreads();
    tc_cluster_sync();
    tc_fence_after();
    const uint32_t tmem = word(s_tmem);
    layer_pdl_wait();

    // the work of this cluster (and, split, this CTA's part of k)
    const int tiles = a.p_tiles * a.q_tiles;
    const int cluster = blockIdx.x / ranks, clusters = gridDim.x / ranks;
    const int kb0 = SPLIT ? (int)((long long)a.kblocks * rank / ranks) : 0;
    const int kb1 = SPLIT ? (int)((long long)a.kblocks * (rank + 1) / ranks) : a.kblocks;
    const uint32_t q_bytes = (a.q_mn ? L::kQRows : a.q_box) * 128;   // Q's, of a step
    auto place = [&](int t, int &p, int &q) {
        // groups of eight tiles of P walk along Q: the tiles in flight form a block
        constexpr int G = 8;
        const int group = t / (G * a.q_tiles), in = t - group * G * a.q_tiles;
        const int size = min(G, a.p_tiles - group * G);
        p = group * G + in % size;
        q = in / size;
    };
    bool ok = true;

    if (warp == 0) {
        // the whole warp walks the loop (its values stay uniform), one lane issues
        const bool one = tc_elect();
        int s = 0, issued = 0;
        uint32_t phase = 1;
        for (int t = cluster; t < tiles && ok; t += clusters) {
            int p, q;
            place(t, p, q);
            const int pr = (p * CTAS + (CTAS == 2 ? (int)rank : 0)) * kTcRows;
            const int qr = q * BN + (CTAS == 2 ? (int)rank * (BN / 2) : 0);
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                if (!tc_bar_wait(empty(s), phase, a.limit)) {
                    ok = false;
                    break;
                }
                if (one) {
                    const uint32_t sp = base + s * a.stage, sq = sp + L::kP;
                    const uint32_t bar = CTAS == 2 ? tc_map(full(s), 0) : full(s);
                    if (leader) tc_bar_expect(full(s), CTAS * (L::kP + q_bytes));
                    if (a.p_mn) {
                        tc_copy<CTAS>(sp, &p_map, pr, kb * kTcBK, bar);
                        tc_copy<CTAS>(sp + 8192, &p_map, pr + 64, kb * kTcBK, bar);
                    } else {
                        tc_copy<CTAS>(sp, &p_map, kb * kTcBK, pr, bar);
                    }
                    if (a.q_mn) {
#pragma unroll
                        for (int i = 0; i < L::kQRows / 64; ++i)
                            tc_copy<CTAS>(sq + 8192 * i, &q_map, qr + 64 * i, kb * kTcBK, bar);
                    } else {
                        tc_copy<CTAS>(sq, &q_map, kb * kTcBK, qr, bar);
                    }
                }
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
        }
        if (one) tc_put_word(tc_map(s_issued + (leader ? 0 : 4), leader ? rank : 0), (uint32_t)issued);
    } else if (warp == 1 && leader) {
        // f32 accumulators; operands f16 or bf16, their major directions; N / 8, M / 16
        constexpr uint32_t type = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
        const uint32_t idesc = (1u << 4) | (type << 7) | (type << 10) | ((uint32_t)a.p_mn << 15) |
                               ((uint32_t)a.q_mn << 16) | ((uint32_t)(BN / 8) << 17) |
                               ((uint32_t)(CTAS * kTcRows / 16) << 24);
        const uint32_t p_step = a.p_mn ? 2048 >> 4 : 32 >> 4, q_step = a.q_mn ? 2048 >> 4 : 32 >> 4;
        const uint64_t p_desc = tc_desc(base, a.p_mn), q_desc = tc_desc(base + L::kP, a.q_mn);
        const bool one = tc_elect();
        int s = 0, n = 0;
        uint32_t phase = 0;
        for (int t = cluster; t < tiles && ok; t += clusters, ++n) {
            const int acc = n & 1;
            if (!tc_bar_wait(tempty(acc), (n >> 1 & 1) ^ 1, a.limit)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t d = tmem + acc * L::kAccStep;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!tc_bar_wait(full(s), phase, a.limit)) {
                    ok = false;
                    break;
                }
                if (one) {
                    // addresses stay below 2^18: no carry leaves the descriptor's field
                    uint64_t pd = p_desc + (uint32_t)(s * (a.stage >> 4));
                    uint64_t qd = q_desc + (uint32_t)(s * (a.stage >> 4));
#pragma unroll
                    for (int k = 0; k < kTcBK / 16; ++k) {
                        tc_mma<CTAS>(d, pd, qd, idesc, kb > kb0 || k > 0);
                        pd += p_step;
                        qd += q_step;
                    }
                    tc_commit<CTAS>(empty(s));
                }
                if (++s == a.stages) {
                    s = 0;
                    phase ^= 1;
                }
            }
            if (ok && one) tc_commit<CTAS>(tfull(acc));
        }
    } else if (warp >= 4 && !SPLIT) {
        // a warp reads its own quarter of the lanes; two warps share a quarter's columns
        const int quarter = warp & 3, side = (warp - 4) >> 2;
        float *const s_t = reinterpret_cast<float *>(s_base + (scratch - base)) +
                           (warp - 4) * 32 * 33;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        int n = 0;
        for (int t = cluster; t < tiles && ok; t += clusters, ++n) {
            int p, q;
            place(t, p, q);
            const int acc = n & 1;
            ok = tc_bar_wait(tfull(acc), n >> 1 & 1, a.limit);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            tc_fence_after();
            const int64_t row0 = (int64_t)(p * CTAS + (CTAS == 2 ? (int)rank : 0)) * kTcRows +
                                 quarter * 32;
            const int64_t col0 = (int64_t)q * BN;
            const bool live = row0 < a.m;
            if (a.vec && col0 + BN <= a.n) {
#pragma unroll 1
                for (int c = 16 * side; c < BN && live; c += 32) {
                    float v[16];
                    tc_load16(lanes + acc * L::kAccStep + c, v);
                    if (kb1 == kb0) {   // no k: nothing was summed
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                    }
                    if (row0 + lane < a.m) {
                        if (a.vec == 2) tc_store16<T, true>(a.e, row0 + lane, col0 + c, v);
                        else tc_store16<T, false>(a.e, row0 + lane, col0 + c, v);
                    }
                }
            } else {
                // off alignment or at the edge: through shared memory, so that
                // neighbouring lanes store neighbouring columns
#pragma unroll 1
                for (int c = 32 * side; c < BN && live && col0 + c < a.n; c += 64) {
                    float v[32];
                    tc_load32(lanes + acc * L::kAccStep + c, v);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s_t[lane * 33 + i] = kb1 == kb0 ? 0.0f : v[i];
                    __syncwarp();
                    const int64_t col = col0 + c + lane;
                    if (col < a.n) {
                        const float bias = tc_bias<T>(a.e, col);
                        const int rows = (int)min((int64_t)32, a.m - row0);
#pragma unroll 1
                        for (int r = 0; r < rows; r += 4) {
                            float w[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) w[i] = s_t[(r + i) * 33 + lane];
                            tc_store_down<T, 4>(a.e, row0 + r, col, w, rows - r, bias);
                        }
                    }
                    __syncwarp();
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tc_bar_arrive(CTAS == 2 ? tc_map(tempty(acc), 0) : tc_map(tempty(acc), rank));
        }
    }

    // every role is over, and said so if it failed, before the cluster next meets
    auto tell = [&] {
        if (!ok)
            for (uint32_t r = 0; r < ranks; ++r) tc_put_word(tc_map(s_failed, r), 1);
    };
    if constexpr (SPLIT) {
        // P is B: lanes are n, columns are m
        int p, q;
        place(cluster, p, q);
        const int64_t row0 = (int64_t)p * kTcRows, col0 = (int64_t)q * BN;
        const int most = (int)min((int64_t)BN, a.m - col0);
        const int quarter = warp & 3;
        const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
        if (warp >= 4) {
            ok = tc_bar_wait(tfull(0), 0, a.limit);
            ok = __all_sync(0xFFFFFFFFu, ok);
            tc_fence_after();
        }
        if (ranks == 1) {
            const int64_t n = row0 + quarter * 32 + lane;
            if (warp >= 4) {
                const float bias = n < a.n ? tc_bias<T>(a.e, n) : 0.0f;
#pragma unroll 1
                for (int c = 0; c < most; c += 16) {
                    float v[16];
                    tc_load16(lanes + c, v);
                    if (!ok || kb1 == kb0) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) v[i] = 0.0f;
                    }
                    if (n < a.n) tc_store_down<T, 16>(a.e, col0 + c, n, v, most - c, bias);
                }
            }
        } else {
            // A rank joins `width` neighbouring columns.  Once every CTA's products are
            // done, the stages are free: each sends its sums to the ranks that join
            // them, [from][width / 4][128 lanes][4] there, a warp's vectors side by side
            // ([256,4096] x [4096,4096] on tiles of 128 columns, operands in the L2, 13.4
            // us; column by column 18.7).
            tell();
            __syncwarp();
            __syncthreads();
            tc_cluster_sync();
            if (!word(s_failed)) {   // the same in every CTA of the cluster
                const uint32_t width = BN / ranks, shift = __popc(width - 1);   // powers of two
                const uint32_t four = width < 4 ? width : 4;                    // columns of a vector
                if (warp >= 4) {
                    const uint32_t at = quarter * 32 + lane;
#pragma unroll 1
                    for (int c = 0; c < most; c += 16) {
                        float v[16];
                        tc_load16(lanes + c, v);
                        auto place_of = [&](int i) {
                            const uint32_t within = (uint32_t)(c + i) & (width - 1);
                            return tc_map(base + 4 * (rank * width * kTcRows + within * kTcRows +
                                                      at * four), (uint32_t)(c + i) >> shift);
                        };
                        if (four == 4) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::
                                                 "r"(place_of(i)), "f"(v[i]), "f"(v[i + 1]),
                                             "f"(v[i + 2]), "f"(v[i + 3])
                                             : "memory");
                        } else {
#pragma unroll
                            for (int i = 0; i < 16; i += 2)
                                asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::
                                                 "r"(place_of(i)), "f"(v[i]), "f"(v[i + 1])
                                             : "memory");
                        }
                    }
                    tc_fence_before();
                }
                __syncwarp();
                __syncthreads();
                tc_cluster_sync();
                const int row = threadIdx.x & 127;
                const int64_t n = row0 + row;
                const int first = (int)(rank * width), last = min(first + (int)width, most);
                if (n < a.n) {
                    const float bias = tc_bias<T>(a.e, n);
                    const float *const in = reinterpret_cast<const float *>(s_base) + row * four;
                    // two threads a row, a vector of columns at a time
                    for (int c = first + (threadIdx.x >> 7) * (int)four; c < last;
                         c += (L::kThreads >> 7) * (int)four) {
                        float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        for (uint32_t r = 0; r < ranks; ++r) {
                            const float *const from = in + (r * width + (c - first)) * kTcRows;
                            if (four == 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(from);
                                z[0] += f.x;
                                z[1] += f.y;
                                z[2] += f.z;
                                z[3] += f.w;
                            } else {
                                const float2 f = *reinterpret_cast<const float2 *>(from);
                                z[0] += f.x;
                                z[1] += f.y;
                            }
                        }
                        tc_store_down<T, 4>(a.e, col0 + c, n, z, min((int)four, last - c), bias);
                    }
                }
            }
        }
    }

    tell();
    tc_fence_before();
    __syncwarp();
    __syncthreads();
    tc_cluster_sync();
    tc_fence_after();
    if (word(s_failed)) {   // wind down: what is on its way first
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, EBIN_DEVICE_WAIT_LIMIT);
        if (warp == 0 && leader) {
            const int own = (int)word(s_issued), peer = CTAS == 2 ? (int)word(s_issued + 4) : own;
            const int end = tc_drain_end(own, peer);
            for (int j = tc_drain_first(own, peer, a.stages); j < end; ++j) {
                const uint32_t bar = full(j % a.stages);
                const TcDrain todo = tc_drain_step(j, own, peer);
                if (lane == 0 && todo == TC_DRAIN_EXPECT) tc_bar_expect(bar, L::kP + q_bytes);
                if (lane == 0 && todo == TC_DRAIN_COUNT_OFF) tc_bar_count_off(bar, L::kP + q_bytes);
                if (!__all_sync(0xFFFFFFFFu, tc_bar_wait(bar, j / a.stages & 1, a.limit))) break;
            }
        }
        if (warp == 1) {
            if (leader && tc_elect()) tc_commit<CTAS>(drain);
            __syncwarp();
            tc_bar_wait(drain, 0, a.limit);
        }
        __syncwarp();
        __syncthreads();
        tc_cluster_sync();
        tc_fence_after();
    }
    if (warp == 2) tc_free<CTAS>(tmem, L::kColumns);
}

}  // namespace ebin
