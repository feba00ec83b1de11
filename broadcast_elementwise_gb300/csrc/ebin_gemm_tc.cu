// The tensor-core product kernels of one element type (-DEBIN_DT: 1 float16,
// 2 bfloat16): pairs of CTAs on tiles of 256 rows, and split tiles.
#include "ebin_gemm_tc.cuh"

namespace ebin {

#if EBIN_DT == 1
using GemmT = __half;
#define EBIN_GEMM_NAME launch_tc_f16
#else
using GemmT = __nv_bfloat16;
#define EBIN_GEMM_NAME launch_tc_bf16
#endif

template <int CTAS, int BN, bool SPLIT>
static cudaError_t run(const CUtensorMap &p, const CUtensorMap &q, const TcArgs &a, int grid,
                       int cluster, cudaStream_t s) {
    using L = TcLayout<CTAS, BN, SPLIT>;
    static_assert(L::kBytes <= kTcSmem, "shared memory of a CTA");
    static const cudaError_t opted = cudaFuncSetAttribute(
        k_gemm_tc<GemmT, CTAS, BN, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
    if (opted != cudaSuccess) return opted;
    return launch_layer(k_gemm_tc<GemmT, CTAS, BN, SPLIT>, dim3((unsigned)grid), L::kThreads,
                        L::kBytes, s, cluster, p, q, a);
}

// bn: the accumulator columns of a tile; grid CTAs in clusters.
cudaError_t EBIN_GEMM_NAME(const CUtensorMap &p, const CUtensorMap &q, const TcArgs &a, int bn,
                           int grid, int cluster, cudaStream_t s) {
    if (bn == 256) return run<2, 256, false>(p, q, a, grid, cluster, s);
    if (bn == 224) return run<2, 224, false>(p, q, a, grid, cluster, s);
    if (bn == 192) return run<2, 192, false>(p, q, a, grid, cluster, s);
    if (bn == 160) return run<2, 160, false>(p, q, a, grid, cluster, s);
    if (bn == 16) return run<1, 16, true>(p, q, a, grid, cluster, s);
    if (bn == 32) return run<1, 32, true>(p, q, a, grid, cluster, s);
    if (bn == 64) return run<1, 64, true>(p, q, a, grid, cluster, s);
    if (bn == 128) return run<1, 128, true>(p, q, a, grid, cluster, s);
    return cudaErrorInvalidValue;
}

}  // namespace ebin
