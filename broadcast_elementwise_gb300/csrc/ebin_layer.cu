// The last step of sums that CTAs began: weight gradients and bias gradients.
#include "ebin_layer.h"

namespace ebin {

struct SumRowsArgs {
    const float *partial[2];   // [count][dim]
    int64_t count[2];
    float *sum[2];             // [dim], or null
    int64_t dim;
};

// sum[j] = the sum of partial[.][j], in an order fixed by the count: 32 threads
// take every 32nd row, then join in order.  grid (columns / 32, tensors).
__global__ void __launch_bounds__(1024) k_sum_rows(const SumRowsArgs a) {
    __shared__ float s[32][33];
    const float *partial = blockIdx.y ? a.partial[1] : a.partial[0];
    float *sum = blockIdx.y ? a.sum[1] : a.sum[0];
    const int64_t count = blockIdx.y ? a.count[1] : a.count[0];
    const int64_t j = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const bool live = j < a.dim && sum;
    layer_pdl_launch();
    layer_pdl_wait();
    float v = 0.0f;
    if (live) {
#pragma unroll 8
        for (int64_t c = threadIdx.y; c < count; c += 32) v += partial[c * a.dim + j];
    }
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && live) {
        float t = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) t += s[r][threadIdx.x];
        sum[j] = t;
    }
}

cudaError_t launch_sum_rows(const float *const partial[2], const int64_t count[2],
                            float *const sum[2], int64_t dim, int tensors, cudaStream_t s) {
    SumRowsArgs a{};
    for (int w = 0; w < tensors; ++w) {
        a.partial[w] = partial[w];
        a.count[w] = count[w];
        a.sum[w] = sum[w];
    }
    a.dim = dim;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)div_up(dim, 32), (unsigned)tensors);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launch();
    return cudaLaunchKernelEx(&cfg, k_sum_rows, a);
}

}  // namespace ebin
