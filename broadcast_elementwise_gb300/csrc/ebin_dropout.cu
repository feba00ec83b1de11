// Dropout: y = residual + keep(x + bias) / (1 - p), and its gradient with the
// bias's, in one pass; the mask comes from ebin_philox.cuh and is never stored.
//
// Time goes by elements, not by bytes: the ten rounds take 20 wide products and 20 exclusive
// ors for four elements, and a warp has one row on its way and none while it draws (a capture
// of the first below: issue 55 %, 8.7 warps waiting for memory an issue).  bf16, against the
// bytes at a copy's 6683 GB/s:
//   [16384,8192] with bias and residual 136 us (120), alone 123 (80), gradient 112 (80)
//   [8192,4096] with bias and residual 39 us (30), alone 36 (20), gradient 31, with the bias's 34 (20)
// [8192,4096] f32 alone 47 us (40); [4095,1543] f16, off the vectors, 12.7 (3.8).
#include <new>

#include "ebin_philox.cuh"

namespace ebin {

constexpr int kDropWarps = 8, kDropThreads = 32 * kDropWarps;

struct DropoutArgs {
    const void *x, *residual, *bias;
    void *y;
    int64_t ld_x, ld_r, ld_y;
    int64_t m, n;
    int64_t rows;        // rows of a CTA's part
    int32_t bias_f32;
    DropArgs drop;
    float *partial;      // a gradient's sums over a part's rows, [parts][n], or null
};

template <class T, int V> struct alignas(sizeof(T) * V) DropVec {
    T v[V];
};

// A lane owns V neighbouring columns, a whole number of quads; warps walk the rows
// of the CTA's part.  VEC: one access of V elements; else element by element, up to
// the row's end.  Many warps cover the rounds better than many rows a thread: forward five
// CTAs an SM (four 139 us, six 138, eight 180), one row a step (two 142, three 155); a
// gradient's sums leave room for four (33 us at [8192,4096], 45 with two rows).
template <class T, int V, bool VEC, bool GRAD>
__global__ void __launch_bounds__(kDropThreads, GRAD ? 4 : 5) k_dropout(const DropoutArgs a) {
    __shared__ float s_sum[GRAD ? kDropWarps : 1][32 * V + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col = ((int64_t)blockIdx.x * 32 + lane) * V;
    const int64_t r0 = (int64_t)blockIdx.y * a.rows, r1 = min(a.m, r0 + a.rows);
    layer_pdl_launch();
    layer_pdl_wait();
    const uint2 offset = drop_offset(a.drop);
    const int live = (int)min((int64_t)V, a.n - col);   // columns of the lane, maybe none
    float bias[V], sum[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        bias[i] = sum[i] = 0.0f;
        if (!GRAD && a.bias && i < live)
            bias[i] = a.bias_f32 ? static_cast<const float *>(a.bias)[col + i]
                                 : to_f(static_cast<const T *>(a.bias)[col + i]);
    }
    if (live > 0) {
        for (int64_t r = r0 + warp; r < r1; r += kDropWarps) {
            const T *x = static_cast<const T *>(a.x) + r * a.ld_x + col;
            const T *res = static_cast<const T *>(a.residual) + r * a.ld_r + col;
            T *y = static_cast<T *>(a.y) + r * a.ld_y + col;
            DropVec<T, V> in, add, out;
            if constexpr (VEC) {
                in = *reinterpret_cast<const DropVec<T, V> *>(x);
                if (!GRAD && a.residual) add = *reinterpret_cast<const DropVec<T, V> *>(res);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    in.v[i] = i < live ? x[i] : from_f<T>(0.0f);
                    if (!GRAD && a.residual) add.v[i] = i < live ? res[i] : from_f<T>(0.0f);
                }
            }
            float v[V];
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = to_f(in.v[i]) + bias[i];
            if (a.drop.least) {
#pragma unroll
                for (int i = 0; i < V; i += 4)
                    drop_quad(a.drop, (uint32_t)((col + i) >> 2), (uint32_t)r, offset, v + i);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (GRAD) sum[i] += v[i];
                else if (a.residual) v[i] += to_f(add.v[i]);
                out.v[i] = from_f<T>(v[i]);
            }
            if constexpr (VEC) {
                *reinterpret_cast<DropVec<T, V> *>(y) = out;
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < live) y[i] = out.v[i];
            }
        }
    }
    if constexpr (GRAD) {
        if (!a.partial) return;
#pragma unroll
        for (int i = 0; i < V; ++i) s_sum[warp][lane * V + i] = sum[i];
        __syncthreads();
        for (int j = threadIdx.x; j < 32 * V; j += kDropThreads) {
            const int64_t c = (int64_t)blockIdx.x * 32 * V + j;
            float t = 0.0f;
#pragma unroll
            for (int w = 0; w < kDropWarps; ++w) t += s_sum[w][j];
            if (c < a.n) a.partial[(int64_t)blockIdx.y * a.n + c] = t;
        }
    }
}

}  // namespace ebin

struct ebin_dropout_plan_s {
    ebin_dropout_attrs at;
    int64_t ld_x, ld_r, ld_y;
    int64_t isz;
    uint32_t least;
    int64_t parts[2] = {};      // CTAs down the rows, for vectors of 16 bytes and for quads
    size_t workspace = 0;
};

using namespace ebin;

namespace {

int64_t span_of(int64_t rows, int64_t cols, int64_t ld) {
    return rows > 0 && cols > 0 ? (rows - 1) * ld + cols : 0;
}

template <class T, int V, bool VEC>
cudaError_t launch_dropout(const DropoutArgs &a, bool grad, int64_t parts, cudaStream_t s) {
    const dim3 grid((unsigned)div_up(a.n, 32 * V), (unsigned)parts);
    return grad ? launch_layer(k_dropout<T, V, VEC, true>, grid, kDropThreads, 0, s, 1, a)
                : launch_layer(k_dropout<T, V, VEC, false>, grid, kDropThreads, 0, s, 1, a);
}

template <class T>
cudaError_t launch_dropout_type(const DropoutArgs &a, bool grad, bool vec, int64_t parts,
                                cudaStream_t s) {
    return vec ? launch_dropout<T, 16 / sizeof(T), true>(a, grad, parts, s)
               : launch_dropout<T, 4, false>(a, grad, parts, s);
}

// Parts down the rows: forward about four waves of CTAs (one: 149 us), a gradient, whose
// parts each leave sums, two; at least one row of every warp each.
int64_t dropout_parts(int64_t m, int64_t n, int64_t V, bool gradient) {
    const int64_t strips = std::max<int64_t>(1, div_up(n, 32 * V));
    const int64_t want = std::max<int64_t>(1, div_up((gradient ? 8 : 20) * 152, strips));
    return std::max<int64_t>(1, std::min<int64_t>({want, div_up(m, kDropWarps), 65535}));
}

// The checks and arguments that both executions share.
ebin_status prepare_dropout(const ebin_dropout_plan_s &p, const void *x, const void *bias,
                            const void *residual, void *y, uint64_t seed, uint64_t offset,
                            const uint64_t *offset_device, DropoutArgs &a, bool &vec) {
    const ebin_dropout_attrs &at = p.at;
    if (!x || !y) return EBIN_ERR_INVALID_ARG;
    if (((uintptr_t)x | (uintptr_t)residual | (uintptr_t)y) % (uintptr_t)p.isz ||
        (bias && (uintptr_t)bias % ebin_dtype_size(at.dtype_bias)) || (uintptr_t)offset_device % 8)
        return EBIN_ERR_INVALID_ARG;
    const int64_t y_b = span_of(at.rows, at.n, p.ld_y) * p.isz;
    const bool one = at.rows <= 1;      // a single row has no stride
    // whether y may lie where it lies beside an input
    auto apart = [&](const void *in, int64_t ld) {
        const int64_t row = at.n * p.isz;
        return (in == y && (one || ld == p.ld_y)) ||
               !rows_share(in, row, ld * p.isz, y, row, p.ld_y * p.isz, at.rows);
    };
    if (!apart(x, p.ld_x) || (residual && !apart(residual, p.ld_r))) return EBIN_ERR_ALIAS;
    if ((bias && ranges_overlap(bias, at.n * (int64_t)ebin_dtype_size(at.dtype_bias), y, y_b)) ||
        (offset_device && ranges_overlap(offset_device, 8, y, y_b)))
        return EBIN_ERR_ALIAS;
    const int64_t V = 16 / p.isz;
    vec = at.n % V == 0 && (one || (p.ld_x % V == 0 && p.ld_y % V == 0 &&
                                    (!residual || p.ld_r % V == 0))) &&
          ((uintptr_t)x | (uintptr_t)residual | (uintptr_t)y) % 16 == 0;
    a = DropoutArgs{};
    a.x = x;
    a.residual = residual;
    a.bias = bias;
    a.y = y;
    a.ld_x = p.ld_x;
    a.ld_r = p.ld_r;
    a.ld_y = p.ld_y;
    a.m = at.rows;
    a.n = at.n;
    a.rows = div_up(at.rows, p.parts[vec ? 0 : 1]);
    a.bias_f32 = at.dtype_bias == EBIN_FLOAT32;
    a.drop = drop_args(p.least, seed, offset, offset_device);
    return EBIN_OK;
}

cudaError_t launch_dropout_typed(const ebin_dropout_plan_s &p, const DropoutArgs &a, bool vec,
                                 cudaStream_t s) {
    const bool grad = p.at.gradient != 0;
    const int64_t parts = p.parts[vec ? 0 : 1];
    if (p.at.dtype == EBIN_FLOAT32) return launch_dropout_type<float>(a, grad, vec, parts, s);
    if (p.at.dtype == EBIN_FLOAT16) return launch_dropout_type<__half>(a, grad, vec, parts, s);
    return launch_dropout_type<__nv_bfloat16>(a, grad, vec, parts, s);
}

}  // namespace

extern "C" ebin_status ebin_dropout_plan_create(const ebin_dropout_attrs *attrs,
                                                ebin_dropout_plan_t *out) {
    if (!attrs || !out) return EBIN_ERR_INVALID_ARG;
    *out = nullptr;
    const ebin_dropout_attrs &a = *attrs;
    if (a.dtype != EBIN_FLOAT16 && a.dtype != EBIN_BFLOAT16 && a.dtype != EBIN_FLOAT32)
        return EBIN_ERR_UNSUPPORTED_TYPE;
    if ((a.has_bias != 0 && a.has_bias != 1) || (a.has_residual != 0 && a.has_residual != 1) ||
        (a.gradient != 0 && a.gradient != 1) || (a.gradient && a.has_residual))
        return EBIN_ERR_INVALID_ATTR;
    if (a.has_bias && a.dtype_bias != a.dtype && a.dtype_bias != EBIN_FLOAT32)
        return EBIN_ERR_UNSUPPORTED_TYPE;
    uint32_t least;
    if (!drop_bound(a.p, &least)) return EBIN_ERR_INVALID_ATTR;
    const int64_t most = int64_t(1) << 30;
    if (a.rows < 0 || a.n < 0 || a.rows > most || a.n > most) return EBIN_ERR_INVALID_ARG;
    const int64_t ld[3] = {a.ld_x ? a.ld_x : a.n, a.ld_residual ? a.ld_residual : a.n,
                           a.ld_y ? a.ld_y : a.n};
    for (int64_t v : ld) {
        int64_t span;
        if (v < a.n || !product_fits(std::max<int64_t>(a.rows, 1), v, &span))
            return EBIN_ERR_INVALID_ARG;
    }
    auto *p = new (std::nothrow) ebin_dropout_plan_s;
    if (!p) return EBIN_ERR_INVALID_ARG;
    p->at = a;
    p->ld_x = ld[0];
    p->ld_r = ld[1];
    p->ld_y = ld[2];
    p->isz = (int64_t)ebin_dtype_size(a.dtype);
    p->least = least;
    if (a.rows > 0 && a.n > 0) {
        p->parts[0] = dropout_parts(a.rows, a.n, 16 / p->isz, a.gradient);
        p->parts[1] = dropout_parts(a.rows, a.n, 4, a.gradient);
        if (a.gradient && a.has_bias)
            p->workspace = sizeof(float) * (size_t)(std::max(p->parts[0], p->parts[1]) * a.n);
    }
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_dropout_plan_workspace(ebin_dropout_plan_t plan, size_t *bytes) {
    if (!plan || !bytes) return EBIN_ERR_INVALID_ARG;
    *bytes = plan->workspace;
    return EBIN_OK;
}

extern "C" void ebin_dropout_plan_release(ebin_dropout_plan_t plan) { delete plan; }

extern "C" ebin_status ebin_dropout_execute(ebin_dropout_plan_t plan, const void *x,
                                            const void *bias, const void *residual, void *y,
                                            uint64_t seed, uint64_t offset,
                                            const uint64_t *offset_device, void *stream) {
    if (!plan || plan->at.gradient) return EBIN_ERR_INVALID_ARG;
    const ebin_dropout_plan_s &p = *plan;
    if (p.at.rows == 0 || p.at.n == 0) return EBIN_OK;
    if (!p.at.has_bias) bias = nullptr;
    else if (!bias) return EBIN_ERR_INVALID_ARG;
    if (!p.at.has_residual) residual = nullptr;
    else if (!residual) return EBIN_ERR_INVALID_ARG;
    DropoutArgs a;
    bool vec;
    const ebin_status st = prepare_dropout(p, x, bias, residual, y, seed, offset, offset_device, a,
                                           vec);
    if (st != EBIN_OK) return st;
    return launch_dropout_typed(p, a, vec, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? EBIN_OK : EBIN_ERR_CUDA;
}

extern "C" ebin_status ebin_dropout_grad_execute(ebin_dropout_plan_t plan, const void *dy,
                                                 void *dx, float *dbias, void *workspace,
                                                 size_t workspace_bytes, uint64_t seed,
                                                 uint64_t offset, const uint64_t *offset_device,
                                                 void *stream) {
    if (!plan || !plan->at.gradient) return EBIN_ERR_INVALID_ARG;
    const ebin_dropout_plan_s &p = *plan;
    const ebin_dropout_attrs &at = p.at;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (at.n == 0) return EBIN_OK;
    if (!at.has_bias) dbias = nullptr;
    else if (!dbias || (uintptr_t)dbias % 4) return EBIN_ERR_INVALID_ARG;
    if (at.rows == 0) {
        if (dbias && cudaMemsetAsync(dbias, 0, sizeof(float) * at.n, s) != cudaSuccess)
            return EBIN_ERR_CUDA;
        return EBIN_OK;
    }
    if (dbias && (!workspace || workspace_bytes < p.workspace || (uintptr_t)workspace % 16))
        return EBIN_ERR_INVALID_ARG;
    DropoutArgs a;
    bool vec;
    const ebin_status st = prepare_dropout(p, dy, nullptr, nullptr, dx, seed, offset,
                                           offset_device, a, vec);
    if (st != EBIN_OK) return st;
    if (dbias) {
        const int64_t b = sizeof(float) * at.n, w = (int64_t)p.workspace;
        const void *others[3] = {dy, dx, offset_device};
        const int64_t sizes[3] = {span_of(at.rows, at.n, p.ld_x) * p.isz,
                                  span_of(at.rows, at.n, p.ld_y) * p.isz, offset_device ? 8 : 0};
        for (int i = 0; i < 3; ++i)
            if (ranges_overlap(dbias, b, others[i], sizes[i]) ||
                ranges_overlap(workspace, w, others[i], sizes[i]))
                return EBIN_ERR_ALIAS;
        if (ranges_overlap(dbias, b, workspace, w)) return EBIN_ERR_ALIAS;
        a.partial = static_cast<float *>(workspace);
    }
    if (launch_dropout_typed(p, a, vec, s) != cudaSuccess) return EBIN_ERR_CUDA;
    if (!dbias) return EBIN_OK;
    const float *part[2] = {a.partial, nullptr};
    const int64_t count[2] = {p.parts[vec ? 0 : 1], 0};
    float *sum[2] = {dbias, nullptr};
    return launch_sum_rows(part, count, sum, at.n, 1, s) == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}
