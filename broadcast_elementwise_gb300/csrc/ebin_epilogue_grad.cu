// The gradient of a product's epilogue: dz = dy act'(z), and dbias = the sum
// over rows of dy act'(z), in one pass over dy and z.
//
// Bound by that traffic (two inputs and one output, each once): [8192,8192] bf16
// with SiLU takes 63.1 us, 6380 GB/s of the 6694 measured by a copy.  A thread
// owns one vector of columns and walks the rows of its CTA's part with the
// column sums in registers; the CTA's warps join in shared memory in a fixed
// order, the parts in a second, small launch.  16-bit data takes its slopes two
// at a time in the fast forms of ebin_act.cuh ([4096,4096]: SiLU 34.3 us in
// scalar form with full exp and quotient, 18.5 so; GELU with erff 43.5, 19.1).
#include <new>

#include "ebin_act.cuh"

namespace ebin {

constexpr int kEgWarps = 8, kEgThreads = 32 * kEgWarps;

struct EgArgs {
    const void *dy, *z;
    void *dz;
    int64_t ld_dy, ld_z, ld_dz;
    int64_t m, n;
    int64_t rows;        // rows of a CTA's part
    float *partial;      // [parts][n], or null
};

template <class T, int V> struct alignas(sizeof(T) * V) EgVec {
    T v[V];
};

// dz of one vector, and its sums.
template <class T, int V, int ACT>
__device__ __forceinline__ EgVec<T, V> eg_vector(const EgVec<T, V> &g, const EgVec<T, V> &z,
                                                 float *sum) {
    EgVec<T, V> out;
    if constexpr (sizeof(T) == 2 && V == 8) {
        uint32_t gw[4], zw[4], ow[4];
        memcpy(gw, &g, 16);
        if constexpr (ACT != EBIN_ACT_NONE) memcpy(zw, &z, 16);
        float2 *const s2 = reinterpret_cast<float2 *>(sum);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 d = open2<T>(gw[i]);
            if constexpr (ACT != EBIN_ACT_NONE) d = __fmul2_rn(d, act_slope2<ACT>(open2<T>(act_near2<T>(zw[i]))));
            s2[i] = __fadd2_rn(s2[i], d);
            ow[i] = pack2<T>(d);
        }
        memcpy(&out, ow, 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float d = to_f(g.v[i]);
            if constexpr (ACT != EBIN_ACT_NONE) {
                const float x = to_f(act_near(z.v[i]));
                if constexpr (sizeof(T) == 2) d *= act_slope2<ACT>(act_pair(x)).x;
                else d *= act_slope_full<ACT>(x);
            }
            sum[i] += d;
            out.v[i] = from_f<T>(d);
        }
    }
    return out;
}

// Rows in flight per thread, at four CTAs an SM (dz and dbias of [4096,4096] bf16
// with SiLU: two rows 18.6 us, one 21.0, four at two CTAs an SM 20.2).
constexpr int kEgRows = 2;

template <class T, int V, int ACT>
__global__ void __launch_bounds__(kEgThreads, 4) k_epilogue_grad(const EgArgs a) {
    __shared__ float s_sum[kEgWarps][32 * V + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = ((int64_t)blockIdx.x * 32 + lane) * V;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows, r1 = min(a.m, r0 + a.rows);
    const T *dy = static_cast<const T *>(a.dy) + (r0 + warp) * a.ld_dy + col;
    const T *z = static_cast<const T *>(a.z) + (r0 + warp) * a.ld_z + col;
    T *dz = static_cast<T *>(a.dz) + (r0 + warp) * a.ld_dz + col;
    layer_pdl_launch();
    layer_pdl_wait();
    alignas(8) float sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) sum[i] = 0.0f;
    if (col < a.n) {
        for (int64_t r = r0 + warp; r < r1; r += kEgWarps * kEgRows) {
            EgVec<T, V> g[kEgRows], x[kEgRows];
#pragma unroll
            for (int k = 0; k < kEgRows; ++k) {
                // a row past the end repeats the first of its step
                const int64_t down = r + k * kEgWarps < r1 ? k * kEgWarps : 0;
                g[k] = *reinterpret_cast<const EgVec<T, V> *>(dy + down * a.ld_dy);
                if constexpr (ACT != EBIN_ACT_NONE)
                    x[k] = *reinterpret_cast<const EgVec<T, V> *>(z + down * a.ld_z);
            }
#pragma unroll
            for (int k = 0; k < kEgRows; ++k)
                if (r + k * kEgWarps < r1)
                    *reinterpret_cast<EgVec<T, V> *>(dz + k * kEgWarps * a.ld_dz) =
                        eg_vector<T, V, ACT>(g[k], x[k], sum);
            dy += kEgWarps * kEgRows * a.ld_dy;
            z += kEgWarps * kEgRows * a.ld_z;
            dz += kEgWarps * kEgRows * a.ld_dz;
        }
    }
    if (!a.partial) return;
#pragma unroll
    for (int i = 0; i < V; ++i) s_sum[warp][lane * V + i] = sum[i];
    __syncthreads();
    for (int j = threadIdx.x; j < 32 * V; j += kEgThreads) {
        const int64_t c = (int64_t)blockIdx.x * 32 * V + j;
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < kEgWarps; ++w) t += s_sum[w][j];
        if (c < a.n) a.partial[(int64_t)blockIdx.y * a.n + c] = t;
    }
}

}  // namespace ebin

struct ebin_epilogue_grad_plan_s {
    ebin_epilogue_grad_attrs at;
    int64_t ld_dy, ld_z, ld_dz;
    int64_t isz;
    int64_t parts[2] = {};      // CTAs down the rows, for vectors of 16 bytes and of one element
    size_t workspace = 0;
};

using namespace ebin;

namespace {

int64_t matrix_span(int64_t rows, int64_t cols, int64_t ld) {
    return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0;
}

template <class T, int V>
cudaError_t launch_eg(const EgArgs &a, int act, int64_t parts, cudaStream_t s) {
    const dim3 grid((unsigned)div_up(a.n, 32 * V), (unsigned)parts);
    switch (act) {
    case EBIN_ACT_RELU:
        return launch_layer(k_epilogue_grad<T, V, EBIN_ACT_RELU>, grid, kEgThreads, 0, s, 1, a);
    case EBIN_ACT_GELU:
        return launch_layer(k_epilogue_grad<T, V, EBIN_ACT_GELU>, grid, kEgThreads, 0, s, 1, a);
    case EBIN_ACT_GELU_TANH:
        return launch_layer(k_epilogue_grad<T, V, EBIN_ACT_GELU_TANH>, grid, kEgThreads, 0, s, 1,
                            a);
    case EBIN_ACT_SILU:
        return launch_layer(k_epilogue_grad<T, V, EBIN_ACT_SILU>, grid, kEgThreads, 0, s, 1, a);
    default:
        return launch_layer(k_epilogue_grad<T, V, EBIN_ACT_NONE>, grid, kEgThreads, 0, s, 1, a);
    }
}

template <class T>
cudaError_t launch_eg_type(const EgArgs &a, int act, bool vec, int64_t parts, cudaStream_t s) {
    return vec ? launch_eg<T, 16 / sizeof(T)>(a, act, parts, s) : launch_eg<T, 1>(a, act, parts, s);
}

// Parts down the rows: about one wave of CTAs (four to each of 152 SMs), at
// least one step of every warp each.
int64_t eg_parts(int64_t m, int64_t n, int64_t V) {
    const int64_t strips = std::max<int64_t>(1, div_up(n, 32 * V));
    const int64_t want = std::max<int64_t>(1, div_up(4 * 152, strips));
    return std::max<int64_t>(1, std::min<int64_t>({want, div_up(m, kEgWarps * kEgRows), 1024}));
}

}  // namespace

extern "C" ebin_status ebin_epilogue_grad_plan_create(const ebin_epilogue_grad_attrs *attrs,
                                                      ebin_epilogue_grad_plan_t *out) {
    if (!attrs || !out) return EBIN_ERR_INVALID_ARG;
    *out = nullptr;
    const ebin_epilogue_grad_attrs &a = *attrs;
    if (a.dtype != EBIN_FLOAT16 && a.dtype != EBIN_BFLOAT16 && a.dtype != EBIN_FLOAT32)
        return EBIN_ERR_UNSUPPORTED_TYPE;
    if (a.activation < EBIN_ACT_NONE || a.activation > EBIN_ACT_SILU ||
        (a.has_bias != 0 && a.has_bias != 1))
        return EBIN_ERR_INVALID_ATTR;
    const int64_t most = int64_t(1) << 30;
    if (a.m < 0 || a.n < 0 || a.m > most || a.n > most) return EBIN_ERR_INVALID_ARG;
    const int64_t ld[3] = {a.ld_dy ? a.ld_dy : a.n, a.ld_z ? a.ld_z : a.n,
                           a.ld_dz ? a.ld_dz : a.n};
    for (int64_t v : ld) {
        int64_t span;
        if (v < a.n || !product_fits(std::max<int64_t>(a.m, 1), v, &span))
            return EBIN_ERR_INVALID_ARG;
    }
    auto *p = new (std::nothrow) ebin_epilogue_grad_plan_s;
    if (!p) return EBIN_ERR_INVALID_ARG;
    p->at = a;
    p->ld_dy = ld[0];
    p->ld_z = ld[1];
    p->ld_dz = ld[2];
    p->isz = (int64_t)ebin_dtype_size(a.dtype);
    if (a.m > 0 && a.n > 0) {
        p->parts[0] = eg_parts(a.m, a.n, 16 / p->isz);
        p->parts[1] = eg_parts(a.m, a.n, 1);
        if (a.has_bias)
            p->workspace = sizeof(float) * (size_t)(std::max(p->parts[0], p->parts[1]) * a.n);
    }
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_epilogue_grad_plan_workspace(ebin_epilogue_grad_plan_t plan,
                                                         size_t *bytes) {
    if (!plan || !bytes) return EBIN_ERR_INVALID_ARG;
    *bytes = plan->workspace;
    return EBIN_OK;
}

extern "C" void ebin_epilogue_grad_plan_release(ebin_epilogue_grad_plan_t plan) { delete plan; }

extern "C" ebin_status ebin_epilogue_grad_execute(ebin_epilogue_grad_plan_t plan, const void *dy,
                                                  const void *z, void *dz, float *dbias,
                                                  void *workspace, size_t workspace_bytes,
                                                  void *stream) {
    if (!plan) return EBIN_ERR_INVALID_ARG;
    const ebin_epilogue_grad_plan_s &p = *plan;
    const ebin_epilogue_grad_attrs &at = p.at;
    if (at.n == 0) return EBIN_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (at.has_bias && !dbias) return EBIN_ERR_INVALID_ARG;
    if (at.m == 0) {
        if (at.has_bias && cudaMemsetAsync(dbias, 0, sizeof(float) * at.n, s) != cudaSuccess)
            return EBIN_ERR_CUDA;
        return EBIN_OK;
    }
    const bool has_z = at.activation != EBIN_ACT_NONE;
    if (!has_z) z = nullptr;
    if (!dy || !dz || (has_z && !z)) return EBIN_ERR_INVALID_ARG;
    if (((uintptr_t)dy | (uintptr_t)z | (uintptr_t)dz) % (uintptr_t)p.isz)
        return EBIN_ERR_INVALID_ARG;
    if (at.has_bias && (!workspace || workspace_bytes < p.workspace ||
                        (uintptr_t)workspace % 16 != 0 || (uintptr_t)dbias % 4 != 0))
        return EBIN_ERR_INVALID_ARG;
    const int64_t dy_b = matrix_span(at.m, at.n, p.ld_dy) * p.isz;
    const int64_t z_b = has_z ? matrix_span(at.m, at.n, p.ld_z) * p.isz : 0;
    const int64_t dz_b = matrix_span(at.m, at.n, p.ld_dz) * p.isz;
    if (ranges_overlap(dy, dy_b, dz, dz_b) && !(dy == dz && p.ld_dy == p.ld_dz))
        return EBIN_ERR_ALIAS;
    if (ranges_overlap(z, z_b, dz, dz_b) && !(z == dz && p.ld_z == p.ld_dz))
        return EBIN_ERR_ALIAS;
    if (at.has_bias) {
        const int64_t b = sizeof(float) * at.n, w = (int64_t)p.workspace;
        const void *others[3] = {dy, z, dz};
        const int64_t sizes[3] = {dy_b, z_b, dz_b};
        for (int i = 0; i < 3; ++i)
            if (ranges_overlap(dbias, b, others[i], sizes[i]) ||
                ranges_overlap(workspace, w, others[i], sizes[i]))
                return EBIN_ERR_ALIAS;
        if (ranges_overlap(dbias, b, workspace, w)) return EBIN_ERR_ALIAS;
    }
    const int64_t V = 16 / p.isz;
    const bool vec = at.n % V == 0 && p.ld_dy % V == 0 && p.ld_dz % V == 0 &&
                     (!has_z || p.ld_z % V == 0) &&
                     ((uintptr_t)dy | (uintptr_t)z | (uintptr_t)dz) % 16 == 0;
    EgArgs a{};
    a.dy = dy;
    a.z = z;
    a.dz = dz;
    a.ld_dy = p.ld_dy;
    a.ld_z = p.ld_z;
    a.ld_dz = p.ld_dz;
    a.m = at.m;
    a.n = at.n;
    const int64_t parts = p.parts[vec ? 0 : 1];
    a.rows = div_up(at.m, parts);
    a.partial = at.has_bias ? static_cast<float *>(workspace) : nullptr;
    cudaError_t e;
    if (at.dtype == EBIN_FLOAT32) e = launch_eg_type<float>(a, at.activation, vec, parts, s);
    else if (at.dtype == EBIN_FLOAT16) e = launch_eg_type<__half>(a, at.activation, vec, parts, s);
    else e = launch_eg_type<__nv_bfloat16>(a, at.activation, vec, parts, s);
    if (e != cudaSuccess) return EBIN_ERR_CUDA;
    if (!at.has_bias) return EBIN_OK;
    const float *part[2] = {a.partial, nullptr};
    const int64_t count[2] = {parts, 0};
    float *sum[2] = {dbias, nullptr};
    return launch_sum_rows(part, count, sum, at.n, 1, s) == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}
