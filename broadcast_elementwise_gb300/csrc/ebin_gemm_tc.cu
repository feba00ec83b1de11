// The tensor-core product kernels of one element type (-DEBIN_DT: 1 float16,
// 2 bfloat16): pairs of CTAs on tiles of 256 rows, and split tiles.
#include "ebin_gemm_tc.cuh"

namespace ebin {

#if EBIN_DT == 1
using GemmT = __half;
#define EBIN_GEMM_NAME launch_tc_f16
#define EBIN_GEMM_CLUSTERS tc_clusters_f16
#else
using GemmT = __nv_bfloat16;
#define EBIN_GEMM_NAME launch_tc_bf16
#define EBIN_GEMM_CLUSTERS tc_clusters_bf16
#endif

template <int CTAS, int BN, bool SPLIT> static cudaError_t opt_in() {
    using L = TcLayout<CTAS, BN, SPLIT>;
    return allow_smem<k_gemm_tc<GemmT, CTAS, BN, SPLIT>>(L::kBytes);
}

template <int CTAS, int BN, bool SPLIT>
static cudaError_t run(const CUtensorMap &p, const CUtensorMap &q, TcArgs a, int grid,
                       int cluster, cudaStream_t s) {
    using L = TcLayout<CTAS, BN, SPLIT>;
    const cudaError_t opted = opt_in<CTAS, BN, SPLIT>();
    if (opted != cudaSuccess) return opted;
    a.stage = L::stage(a.q_mn);
    a.stages = L::stages(a.q_mn);
    return launch_layer(k_gemm_tc<GemmT, CTAS, BN, SPLIT>, dim3((unsigned)grid), L::kThreads,
                        L::kBytes, s, cluster, p, q, a);
}

template <int BN, int CLUSTER> static int clusters() {
    using L = TcLayout<1, BN, true>;
    static const int held = [] {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(CLUSTER);
        cfg.blockDim = dim3(L::kThreads);
        cfg.dynamicSmemBytes = L::kBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = CLUSTER;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (opt_in<1, BN, true>() != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k_gemm_tc<GemmT, 1, BN, true>, &cfg) !=
                cudaSuccess) {
            cudaGetLastError();
            n = 0;
        }
        return n;
    }();
    return held;
}
template <int BN> static int clusters_of(int cluster) {
    return cluster == 2 ? clusters<BN, 2>() : cluster == 4 ? clusters<BN, 4>() : clusters<BN, 8>();
}

int EBIN_GEMM_CLUSTERS(int bn, int cluster) {
    return bn == 16 ? clusters_of<16>(cluster) : bn == 32 ? clusters_of<32>(cluster)
         : bn == 64 ? clusters_of<64>(cluster) : clusters_of<128>(cluster);
}

// bn: the accumulator columns of a tile (on a pair of CTAs, or split); grid CTAs
// in clusters.
cudaError_t EBIN_GEMM_NAME(const CUtensorMap &p, const CUtensorMap &q, const TcArgs &a, int bn,
                           bool pair, int grid, int cluster, cudaStream_t s) {
    if (bn == 256) return run<2, 256, false>(p, q, a, grid, cluster, s);
    if (bn == 224) return run<2, 224, false>(p, q, a, grid, cluster, s);
    if (bn == 192) return run<2, 192, false>(p, q, a, grid, cluster, s);
    if (bn == 160) return run<2, 160, false>(p, q, a, grid, cluster, s);
    if (bn == 128 && pair) return run<2, 128, false>(p, q, a, grid, cluster, s);
    if (bn == 96) return run<2, 96, false>(p, q, a, grid, cluster, s);
    if (bn == 64 && pair) return run<2, 64, false>(p, q, a, grid, cluster, s);
    if (bn == 16) return run<1, 16, true>(p, q, a, grid, cluster, s);
    if (bn == 32) return run<1, 32, true>(p, q, a, grid, cluster, s);
    if (bn == 64) return run<1, 64, true>(p, q, a, grid, cluster, s);
    if (bn == 128) return run<1, 128, true>(p, q, a, grid, cluster, s);
    return cudaErrorInvalidValue;
}

}  // namespace ebin
