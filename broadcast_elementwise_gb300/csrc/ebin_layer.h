// Shared by the translation units of the layer operators (heads, matrix
// products, epilogue gradients).  Not part of the public C ABI.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "ebin.h"
#include "ebin_plan.h"

namespace ebin {

// The current stream's status word and device facts (ebin_host.cpp).
uint32_t *stream_status_word(cudaStream_t s);
int current_sm_count();

inline bool ranges_overlap(const void *p, int64_t pb, const void *q, int64_t qb) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return pb > 0 && qb > 0 && a < b + (uintptr_t)qb && b < a + (uintptr_t)pb;
}

// Whether two matrices of `rows` rows share a byte: rows of xb bytes that start ldx bytes
// apart from x on, of yb bytes ldy apart from y on.  Columns of one wider buffer, side by side,
// share none.
inline bool rows_share(const void *x, int64_t xb, int64_t ldx, const void *y, int64_t yb,
                       int64_t ldy, int64_t rows) {
    if (xb <= 0 || yb <= 0 || rows <= 0 ||
        !ranges_overlap(x, (rows - 1) * ldx + xb, y, (rows - 1) * ldy + yb))
        return false;
    if (ldx != ldy) return true;
    // where y's rows begin behind those of x
    const int64_t at = ((int64_t)((uintptr_t)y - (uintptr_t)x) % ldx + ldx) % ldx;
    return at < xb || at + yb > ldx;
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// a * b < EBIN_MAX_ELEMENTS for a, b >= 0, without overflow.
inline bool product_fits(int64_t a, int64_t b, int64_t *out) {
    if (a != 0 && b > (EBIN_MAX_ELEMENTS - 1) / a) return false;
    *out = a * b;
    return true;
}

// Division of 32-bit indices by a launch's constant n: with 2^(l-1) < n <= 2^l
// and m = floor(2^32 (2^l - n) / n) + 1, x / n = (hi(x m) + x) >> l exactly,
// the sum taken in 33 bits (Granlund and Montgomery's multiplier).
struct FastDiv {
    uint32_t n, mul, shift;
#ifdef __CUDACC__
    __device__ __forceinline__ void split(uint32_t x, uint32_t &q, uint32_t &r) const {
        q = (uint32_t)(((uint64_t)__umulhi(x, mul) + x) >> shift);
        r = x - q * n;
    }
#endif
};

inline FastDiv fast_div(uint32_t n) {
    uint32_t l = 0;
    while (((uint64_t)1 << l) < n) ++l;
    const uint64_t m = (((uint64_t)1 << 32) * (((uint64_t)1 << l) - n)) / n + 1;
    return FastDiv{n, (uint32_t)m, l};
}

// Let KERNEL take `bytes` of dynamic shared memory on the current device (asked
// of the runtime once per kernel and device).
template <auto KERNEL> cudaError_t allow_smem(size_t bytes) {
    static std::atomic<bool> done[128];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool slot = dev >= 0 && dev < 128;
    if (slot && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && slot) done[dev].store(true, std::memory_order_relaxed);
    return e;
}

// Launch with programmatic dependent launch (the kernel calls
// griddepcontrol.wait before its first global access) and count it.
template <class... KParams, class... Args>
cudaError_t launch_layer(void (*kernel)(KParams...), dim3 grid, int block, size_t smem,
                         cudaStream_t stream, int cluster, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    cfg.attrs = attr;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// sum[w][j] = the sum over rows of partial[w], [count[w]][dim], for `tensors`
// (1 or 2) tensors, in a fixed order (ebin_layer.cu).
cudaError_t launch_sum_rows(const float *const partial[2], const int64_t count[2],
                            float *const sum[2], int64_t dim, int tensors, cudaStream_t s);

#ifdef __CUDACC__
__device__ __forceinline__ void layer_pdl_launch() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void layer_pdl_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}

// Two elements of a 16-bit word as a binary32 pair, and back.
template <class T> __device__ __forceinline__ float2 open2(uint32_t w) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value)
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

template <class T> __device__ __forceinline__ uint32_t pack2(float2 v) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 p = __float22bfloat162_rn(v);
        return *reinterpret_cast<const uint32_t *>(&p);
    } else {
        const __half2 p = __float22half2_rn(v);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
}
#endif

}  // namespace ebin
