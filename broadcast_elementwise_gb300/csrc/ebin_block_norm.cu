// Plans of the norms around a block and their execution: attribute checks, the
// alias rule, kernel choice and launch, and the last step of the parameters'
// gradients.
#include <new>

#include "ebin_block.cuh"

namespace ebin {

constexpr int kSumColumns = 32, kSumRows = 32;   // of a CTA

// A parameter in the launch's element type.
__device__ __forceinline__ float sums_at(const BlockSumsArgs &a, const void *p, int64_t j, int f32,
                                         float none) {
    if (a.dtype == EBIN_FLOAT16) return block_param<__half>(p, j, f32, none);
    if (a.dtype == EBIN_BFLOAT16) return block_param<__nv_bfloat16>(p, j, f32, none);
    return block_param<float>(p, j, 1, none);
}

// The sums of a CTA's 32 columns, [kind][column], over `count` rows of them that lie
// `stride` apart from `first` on, each kind `pad` further.  256 threads take a kind that is
// wanted: eight lanes of four columns every 32nd row, then the 32 join in order: an order
// fixed by the count.
__device__ __forceinline__ void sums_columns(const BlockSumsArgs &a, const float *first,
                                             int64_t count, int64_t stride, int64_t col0,
                                             float (*s)[kSumRows][kSumColumns + 1],
                                             float (*total)[kSumColumns]) {
    const int lane = threadIdx.x & 7, row = threadIdx.x >> 3 & 31;
    int k = 0;   // this thread's kind: the bit of its rank
    for (int rank = threadIdx.x >> 8; k < 3; ++k)
        if (a.need >> k & 1 && rank-- == 0) break;
    const int64_t col = col0 + lane * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col < a.n) {   // the last vector ends in the padding
        const float *p = first + k * a.pad + col + row * stride;
#pragma unroll 8
        for (int64_t c = row; c < count; c += kSumRows, p += kSumRows * stride) {
            const float4 x = *reinterpret_cast<const float4 *>(p);
            v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
        }
    }
    float *const at = &s[k][row][lane * 4];
    at[0] = v.x;
    at[1] = v.y;
    at[2] = v.z;
    at[3] = v.w;
    __syncthreads();
    for (int j = threadIdx.x; j < 4 * kSumColumns; j += blockDim.x) {
        const int kind = j / kSumColumns, c = j % kSumColumns;
        float t = 0.0f;
        if (a.need >> kind & 1)
#pragma unroll
            for (int r = 0; r < kSumRows; ++r) t += s[kind][r][c];
        total[kind][c] = t;
    }
    __syncthreads();
}

// The parameters' gradients that all rows share, from the sums of all groups.  w:
// whether the sums carry the groups' gate and scale already.
__device__ __forceinline__ void sums_shared(const BlockSumsArgs &a, int64_t j, const float *t,
                                            bool weighed) {
    const float scale = weighed && a.mod_grouped ? 1.0f
        : 1.0f + sums_at(a, a.scale, j, a.mod_f32, 0.0f);
    const float gate = weighed && a.gate_grouped ? 1.0f : sums_at(a, a.gate, j, a.mod_f32, 1.0f);
    if (a.dw_pre) a.dw_pre[j] = scale * t[SUM_DZ_HH];
    if (a.db_pre) a.db_pre[j] = scale * t[SUM_DZ];
    if (a.dw_post) a.dw_post[j] = gate * t[SUM_E_YH];
    if (a.db_post) a.db_post[j] = gate * t[SUM_E];
    if (!a.mod_grouped) {
        if (a.dscale)
            a.dscale[j] = fmaf(t[SUM_DZ_HH], sums_at(a, a.w_pre, j, a.w_f32, 1.0f),
                               t[SUM_DZ] * sums_at(a, a.b_pre, j, a.w_f32, 0.0f));
        if (a.dshift) a.dshift[j] = t[SUM_DZ];
    }
    if (!a.gate_grouped && a.dgate)
        a.dgate[j] = fmaf(t[SUM_E_YH], sums_at(a, a.w_post, j, a.w_f32, 1.0f),
                          t[SUM_E] * sums_at(a, a.b_post, j, a.w_f32, 0.0f));
}

// One CTA per group and 32 columns: the group's parts joined; its gradients of gate, scale
// and shift; then, with one group, everything, else its share of what all rows
// have in common, into its first part's place.
__global__ void __launch_bounds__(1024) k_block_sums(const BlockSumsArgs a) {
    __shared__ float s[4][kSumRows][kSumColumns + 1], total[4][kSumColumns];
    const int64_t group = blockIdx.x / a.tiles, col0 = (blockIdx.x - group * a.tiles) * kSumColumns;
    layer_pdl_launch();
    layer_pdl_wait();
    float *const at = a.partial + group * a.parts * 4 * a.pad;
    sums_columns(a, at, a.parts, 4 * a.pad, col0, s, total);
    const int64_t j = col0 + threadIdx.x;
    if (threadIdx.x >= kSumColumns || j >= a.n) return;
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = total[k][threadIdx.x];
    if (a.groups == 1) {
        sums_shared(a, j, t, false);
        if (!a.mod_grouped && !a.gate_grouped) return;
    }
    if (a.mod_grouped) {
        if (a.dscale)
            a.dscale[group * a.n + j] =
                fmaf(t[SUM_DZ_HH], sums_at(a, a.w_pre, j, a.w_f32, 1.0f),
                     t[SUM_DZ] * sums_at(a, a.b_pre, j, a.w_f32, 0.0f));
        if (a.dshift) a.dshift[group * a.n + j] = t[SUM_DZ];
    }
    if (a.gate_grouped && a.dgate)
        a.dgate[group * a.n + j] =
            fmaf(t[SUM_E_YH], sums_at(a, a.w_post, j, a.w_f32, 1.0f),
                 t[SUM_E] * sums_at(a, a.b_post, j, a.w_f32, 0.0f));
    if (!a.second) return;
    const float scale = a.mod_grouped
        ? 1.0f + sums_at(a, a.scale, group * a.ld_scale + j, a.mod_f32, 0.0f) : 1.0f;
    const float gate = a.gate_grouped
        ? sums_at(a, a.gate, group * a.ld_gate + j, a.mod_f32, 1.0f) : 1.0f;
    at[SUM_DZ_HH * a.pad + j] = scale * t[SUM_DZ_HH];
    at[SUM_DZ * a.pad + j] = scale * t[SUM_DZ];
    at[SUM_E_YH * a.pad + j] = gate * t[SUM_E_YH];
    at[SUM_E * a.pad + j] = gate * t[SUM_E];
}

// The groups' shares joined.
__global__ void __launch_bounds__(1024) k_block_sums_all(const BlockSumsArgs a) {
    __shared__ float s[4][kSumRows][kSumColumns + 1], total[4][kSumColumns];
    const int64_t col0 = (int64_t)blockIdx.x * kSumColumns;
    layer_pdl_launch();
    layer_pdl_wait();
    sums_columns(a, a.partial, a.groups, 4 * a.pad * a.parts, col0, s, total);
    const int64_t j = col0 + threadIdx.x;
    if (threadIdx.x >= kSumColumns || j >= a.n) return;
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) t[k] = total[k][threadIdx.x];
    sums_shared(a, j, t, true);
}

}  // namespace ebin

struct ebin_block_norm_plan_s {
    ebin_block_norm_attrs at;      // its strides filled in
    int64_t isz, ssz, wsz, msz;    // bytes of an element of the four types
    uint32_t least;
    int64_t groups = 1, group_rows = 0;
    // the rows' units: a CTA's (of a gradient with a norm after the block, by whether it is the
    // full kernel's), and a gradient's teams'
    ebin::BlockUnits cta[2], team;
    size_t workspace = 0;
};

using namespace ebin;

namespace {

// A matrix or a vector in memory, as bytes.
struct Range {
    const void *p;
    int64_t bytes;
    int64_t ld;      // bytes between rows; 0: not a matrix that an output may be
    int64_t size;    // of an element
};

int64_t rows_bytes(int64_t rows, int64_t n, int64_t ld, int64_t size) {
    return rows > 0 && n > 0 ? ((rows - 1) * ld + n) * size : 0;
}

// Whether two ranges share nothing; of two matrices their rows of n elements count.
bool disjoint(const Range &x, const Range &y, int64_t rows, int64_t n) {
    if (!x.p || !y.p || !ranges_overlap(x.p, x.bytes, y.p, y.bytes)) return true;
    return x.ld > 0 && y.ld > 0 &&
           !rows_share(x.p, n * x.size, x.ld, y.p, n * y.size, y.ld, rows);
}

// Whether output y may lie where it lies beside input x.
bool apart(const Range &x, const Range &y, int64_t rows, int64_t n) {
    return disjoint(x, y, rows, n) ||
           (x.p == y.p && x.size == y.size && x.ld > 0 && y.ld > 0 && (rows <= 1 || x.ld == y.ld));
}

// Columns of a row of sums: whole vectors.
int64_t pad_of(int64_t n) { return div_up(n, 4) * 4; }

bool block_float(ebin_dtype t) {
    return t == EBIN_FLOAT32 || t == EBIN_FLOAT16 || t == EBIN_BFLOAT16;
}

// The arguments that both directions share, once they have been checked.
ebin_status prepare_block(const ebin_block_norm_plan_s &p, const ebin_block_norm_params &w,
                          BlockArgs &a) {
    const ebin_block_norm_attrs &at = p.at;
    const bool post = at.post != EBIN_NORM_NONE, pre = at.pre != EBIN_NORM_NONE;
    if ((w.gate && !at.has_branch) || (!post && (w.w_post || w.b_post)) ||
        (!pre && (w.w_pre || w.b_pre || w.scale || w.shift)) ||
        ((uintptr_t)w.gate | (uintptr_t)w.scale | (uintptr_t)w.shift) % (uintptr_t)p.msz ||
        ((uintptr_t)w.w_post | (uintptr_t)w.b_post | (uintptr_t)w.w_pre | (uintptr_t)w.b_pre) %
            (uintptr_t)p.wsz || (uintptr_t)w.offset_device % 8)
        return EBIN_ERR_INVALID_ARG;
    a = BlockArgs{};
    a.gate = w.gate;
    a.w_post = w.w_post;
    a.b_post = w.b_post;
    a.w_pre = w.w_pre;
    a.b_pre = w.b_pre;
    a.scale = w.scale;
    a.shift = w.shift;
    a.ld_gate = at.ld_gate;
    a.ld_scale = at.ld_scale;
    a.ld_shift = at.ld_shift;
    a.gate_rows = at.gate_rows ? at.gate_rows : at.rows;
    a.mod_rows = at.mod_rows ? at.mod_rows : at.rows;
    a.rows = at.rows;
    a.n = at.n;
    a.stream_scale = at.stream_scale;
    a.branch_scale = at.branch_scale;
    a.eps_post = at.epsilon_post;
    a.eps_pre = at.epsilon_pre;
    a.post = at.post;
    a.pre = at.pre;
    a.w_f32 = at.dtype_w == EBIN_FLOAT32;
    a.mod_f32 = at.dtype_mod == EBIN_FLOAT32;
    a.drop = drop_args(p.least, w.seed, w.offset, w.offset_device);
    a.cta = p.cta[0];
    a.team = p.team;
    a.groups = p.groups;
    a.group_rows = p.group_rows;
    return EBIN_OK;
}

// The small inputs that a call reads, as ranges.
int param_ranges(const ebin_block_norm_plan_s &p, const BlockArgs &a, Range *r) {
    const ebin_block_norm_attrs &at = p.at;
    const int64_t w = at.n * p.wsz;
    auto mod = [&](int64_t per, int64_t ld) {
        return rows_bytes(per ? at.rows / per : 1, at.n, ld, p.msz);
    };
    int c = 0;
    for (const void *q : {a.w_post, a.b_post, a.w_pre, a.b_pre})
        if (q) r[c++] = Range{q, w, 0, 0};
    if (a.gate) r[c++] = Range{a.gate, mod(at.gate_rows, at.ld_gate), 0, 0};
    if (a.scale) r[c++] = Range{a.scale, mod(at.mod_rows, at.ld_scale), 0, 0};
    if (a.shift) r[c++] = Range{a.shift, mod(at.mod_rows, at.ld_shift), 0, 0};
    if (p.least && a.drop.offset_device) r[c++] = Range{a.drop.offset_device, 8, 0, 0};
    return c;
}

cudaError_t launch_sums(const BlockSumsArgs &a, cudaStream_t s) {
    const int threads = 256 * __builtin_popcount(a.need);
    cudaError_t e = launch_layer(k_block_sums, dim3((unsigned)(a.tiles * a.groups)), threads, 0, s,
                                 1, a);
    if (e == cudaSuccess && a.second)
        e = launch_layer(k_block_sums_all, dim3((unsigned)a.tiles), threads, 0, s, 1, a);
    return e;
}

// Whether every buffer of a call lies on vectors: rows that are whole vectors, each
// starting on 16 bytes.
bool block_vectors(const ebin_block_norm_plan_s &p, const BlockArgs &a) {
    const int64_t V = p.ssz == 4 ? 4 : 8;   // columns of a vector
    if (a.n % V) return false;
    const void *all[13] = {a.x, a.y, a.dz, a.dh, a.h, a.z, a.gate, a.w_post, a.b_post, a.w_pre,
                           a.b_pre, a.scale, a.shift};
    for (const void *q : all)
        if ((uintptr_t)q % 16) return false;
    if (a.rows == 1) return true;
    const struct { const void *p; int64_t ld; } rows[9] = {
        {a.x, a.ld_x}, {a.y, a.ld_y}, {a.dz, a.ld_dz}, {a.dh, a.ld_dh}, {a.h, a.ld_h},
        {a.z, a.ld_z}, {a.gate, a.ld_gate}, {a.scale, a.ld_scale}, {a.shift, a.ld_shift}};
    for (const auto &r : rows)
        if (r.p && r.ld % V) return false;
    return true;
}

template <class T, class S>
cudaError_t launch_block_any(const BlockArgs &a, bool grad, cudaStream_t s) {
    if (grad)
        return launch_layer(k_block_any_grad<T, S>, dim3((unsigned)(a.groups * a.team.parts)),
                            kBlockAnyThreads, 0, s, 1, a);
    const int64_t grid = std::min<int64_t>(a.rows, 32ll * current_sm_count());
    return launch_layer(k_block_any<T, S>, dim3((unsigned)grid), kBlockAnyThreads, 0, s, 1, a);
}

// parts: the units of a group whose sums a gradient left.
cudaError_t launch_block(const ebin_block_norm_plan_s &p, const BlockArgs &a, bool grad,
                         int64_t *parts, cudaStream_t s) {
    const bool wide = p.ssz == 4, vec = block_vectors(p, a);
    cudaError_t e;
    *parts = 0;
#define EBIN_ROWS(dt, T, S)                                                                 \
    e = grad ? launch_block_rows_grad_##dt(a, vec, parts, s)                                 \
             : launch_block_rows_##dt(a, vec, parts, s);                                     \
    if (*parts > 0 || e != cudaSuccess) return e;                                            \
    *parts = a.team.parts;                                                                   \
    return launch_block_any<T, S>(a, grad, s)
    if (p.at.dtype == EBIN_FLOAT32) { EBIN_ROWS(0, float, float); }
    if (p.at.dtype == EBIN_FLOAT16) {
        if (wide) { EBIN_ROWS(3, __half, float); }
        EBIN_ROWS(1, __half, __half);
    }
    if (wide) { EBIN_ROWS(4, __nv_bfloat16, float); }
    EBIN_ROWS(2, __nv_bfloat16, __nv_bfloat16);
#undef EBIN_ROWS
}

// Of a group's rows, `parts` parts.
BlockUnits block_units(int64_t group_rows, int64_t parts) {
    BlockUnits u;
    u.rows = div_up(group_rows, parts);
    u.parts = div_up(group_rows, u.rows);
    return u;
}

// Units of a CTA an SM.  A count of parts is judged by when its last wave of 152 ends, a
// unit costing its teams' steps and what three more would (its tables, its sums).  Of a
// gradient's the least within 3.5 % of the best where a CTA has two teams or more: SMs left
// over are where the last sums begin.  us with RMS norms on both sides, bf16, against the best's:
// [8192,4096] 69.0 and 70.5, [10000,4096] 83.1 and 86.6, [12288,4096] 100.7 and 102.4,
// [16384,2048] 71.5 and 72.7, [24576,1536] 76.5 and 80.2, but [9000,3584] 70.9 and 69.1.  Within
// 2.5 % [10000,4096] 86.3 and [24576,1536] 80.4; within 5 % [16384,1152] 50.7 (48.6),
// [5000,4096] 48.0 (46.7) and [16388,1152] modulated 69.4 (66.9), steps of few.  With one team a
// step more costs more than that gives: [4096,8192] 74.9 and 73.0, [6553,5120] 84.8 and 83.1.
BlockUnits cta_units(int64_t groups, int64_t group_rows, int64_t n, int vpt, bool gradient) {
    const int64_t warps = std::max<int64_t>(1, div_up(div_up(n, 256), vpt));
    const int64_t teams = std::max<int64_t>(1, kUnitWarps / warps);
    const int64_t most = std::min<int64_t>(group_rows, div_up(3 * 152, groups));
    auto cost = [&](int64_t p) {
        return (double)div_up(groups * p, 152) *
               (double)(div_up(div_up(group_rows, p), teams) + 3);
    };
    double least = cost(1);
    for (int64_t p = 2; p <= most; ++p) least = std::min(least, cost(p));
    int64_t p = 1;
    while (cost(p) > (gradient && teams > 1 ? 1.035 : 1.0) * least) ++p;
    return block_units(group_rows, p);
}

// Units of teams: as many over all groups as 152 SMs hold teams of the row kernel at 128
// registers (a warp for two chunks of 256 columns), each with a row at least, and
// no more than 2^28 sums in the workspace where that leaves one.
BlockUnits team_units(int64_t groups, int64_t group_rows, int64_t n) {
    const int64_t warps = std::max<int64_t>(1, div_up(n, 512));
    const int64_t want = div_up(152 * std::max<int64_t>(1, 16 / warps), groups);
    const int64_t room = (int64_t(1) << 26) / (groups * std::max<int64_t>(n, 1));
    return block_units(group_rows,
                       std::max<int64_t>(1, std::min<int64_t>({want, group_rows, room})));
}

}  // namespace

extern "C" ebin_status ebin_block_norm_plan_create(const ebin_block_norm_attrs *attrs,
                                                   ebin_block_norm_plan_t *out) {
    if (!attrs || !out) return EBIN_ERR_INVALID_ARG;
    *out = nullptr;
    const ebin_block_norm_attrs &a = *attrs;
    if (!block_float(a.dtype) || (a.dtype_stream != a.dtype && a.dtype_stream != EBIN_FLOAT32) ||
        (a.dtype_w != a.dtype && a.dtype_w != EBIN_FLOAT32) ||
        (a.dtype_mod != a.dtype && a.dtype_mod != EBIN_FLOAT32))
        return EBIN_ERR_UNSUPPORTED_TYPE;
    uint32_t least;
    if (a.post < EBIN_NORM_NONE || a.post > EBIN_NORM_LAYER || a.pre < EBIN_NORM_NONE ||
        a.pre > EBIN_NORM_LAYER || (a.has_branch != 0 && a.has_branch != 1) ||
        (a.gradient != 0 && a.gradient != 1) || !(a.epsilon_post >= 0.0f) ||
        !std::isfinite(a.epsilon_post) || !(a.epsilon_pre >= 0.0f) ||
        !std::isfinite(a.epsilon_pre) || !std::isfinite(a.stream_scale) ||
        !std::isfinite(a.branch_scale) || !drop_bound(a.p, &least) ||
        (!a.has_branch && (a.post != EBIN_NORM_NONE || least != 0)))
        return EBIN_ERR_INVALID_ATTR;
    if (a.rows < 0 || a.n < 0 || a.rows > int64_t(1) << 30 || a.n > int64_t(1) << 24 ||
        a.gate_rows < 0 || a.mod_rows < 0 || (a.gate_rows && a.rows % a.gate_rows) ||
        (a.mod_rows && a.rows % a.mod_rows) ||
        (a.gate_rows && a.mod_rows && a.gate_rows != a.mod_rows))
        return EBIN_ERR_INVALID_ARG;
    auto *p = new (std::nothrow) ebin_block_norm_plan_s;
    if (!p) return EBIN_ERR_INVALID_ARG;
    p->at = a;
    ebin_block_norm_attrs &at = p->at;
    for (int64_t *ld : {&at.ld_x, &at.ld_y, &at.ld_h, &at.ld_z, &at.ld_gate, &at.ld_scale,
                        &at.ld_shift, &at.ld_dz, &at.ld_dh, &at.ld_dx, &at.ld_dy}) {
        int64_t span;
        if (*ld == 0) *ld = a.n;
        if (*ld < a.n || !product_fits(std::max<int64_t>(a.rows, 1), *ld, &span)) {
            delete p;
            return EBIN_ERR_INVALID_ARG;
        }
    }
    p->isz = (int64_t)ebin_dtype_size(a.dtype);
    p->ssz = (int64_t)ebin_dtype_size(a.dtype_stream);
    p->wsz = (int64_t)ebin_dtype_size(a.dtype_w);
    p->msz = (int64_t)ebin_dtype_size(a.dtype_mod);
    p->least = least;
    const int64_t per = std::max(a.gate_rows, a.mod_rows);
    if (a.rows > 0) {
        p->group_rows = per ? per : a.rows;
        p->groups = a.rows / p->group_rows;
        const bool grad = a.gradient != 0;
        p->cta[0] = cta_units(p->groups, p->group_rows, a.n,
                              grad ? kUnitGradVpt<false, true> : kUnitVpt, grad);
        p->cta[1] = grad && a.post != EBIN_NORM_NONE
            ? cta_units(p->groups, p->group_rows, a.n, kUnitGradVpt<true, true>, true) : p->cta[0];
        if (a.gradient) {
            if (p->groups * div_up(a.n, kSumColumns) > 0x7FFFFFFF) {   // CTAs of the last step
                delete p;
                return EBIN_ERR_INVALID_ARG;
            }
            p->team = team_units(p->groups, p->group_rows, a.n);
            // wider rows are no CTA's units
            const int64_t parts = a.n > kUnitColumns ? p->team.parts
                : std::max({p->cta[0].parts, p->cta[1].parts, p->team.parts});
            p->workspace = sizeof(float) * 4 * (size_t)(p->groups * parts * pad_of(a.n));
        }
    }
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_block_norm_plan_workspace(ebin_block_norm_plan_t plan, size_t *bytes) {
    if (!plan || !bytes) return EBIN_ERR_INVALID_ARG;
    *bytes = plan->workspace;
    return EBIN_OK;
}

extern "C" void ebin_block_norm_plan_release(ebin_block_norm_plan_t plan) { delete plan; }

extern "C" ebin_status ebin_block_norm_execute(ebin_block_norm_plan_t plan, const void *x,
                                               const void *y,
                                               const ebin_block_norm_params *params, void *h,
                                               void *z, void *stream) {
    if (!plan || plan->at.gradient) return EBIN_ERR_INVALID_ARG;
    const ebin_block_norm_plan_s &p = *plan;
    const ebin_block_norm_attrs &at = p.at;
    if (at.rows == 0 || at.n == 0) return EBIN_OK;
    if (at.pre == EBIN_NORM_NONE) z = nullptr;
    if (!at.has_branch) y = nullptr;
    else if (!y) return EBIN_ERR_INVALID_ARG;
    if (!x || ((uintptr_t)x | (uintptr_t)h) % (uintptr_t)p.ssz ||
        ((uintptr_t)y | (uintptr_t)z) % (uintptr_t)p.isz)
        return EBIN_ERR_INVALID_ARG;
    BlockArgs a;
    const ebin_status st = prepare_block(p, params ? *params : ebin_block_norm_params{}, a);
    if (st != EBIN_OK) return st;
    Range in[10];
    int c = param_ranges(p, a, in);
    in[c++] = Range{x, rows_bytes(at.rows, at.n, at.ld_x, p.ssz), at.ld_x * p.ssz, p.ssz};
    in[c++] = Range{y, rows_bytes(at.rows, at.n, at.ld_y, p.isz), at.ld_y * p.isz, p.isz};
    const Range out[2] = {
        {h, rows_bytes(at.rows, at.n, at.ld_h, p.ssz), at.ld_h * p.ssz, p.ssz},
        {z, rows_bytes(at.rows, at.n, at.ld_z, p.isz), at.ld_z * p.isz, p.isz}};
    for (const Range &o : out)
        for (int i = 0; i < c; ++i)
            if (!apart(in[i], o, at.rows, at.n)) return EBIN_ERR_ALIAS;
    if (!disjoint(out[0], out[1], at.rows, at.n)) return EBIN_ERR_ALIAS;
    if (!h && !z) return EBIN_OK;
    a.x = x;
    a.y = y;
    a.h = h;
    a.z = z;
    a.ld_x = at.ld_x;
    a.ld_y = at.ld_y;
    a.ld_h = at.ld_h;
    a.ld_z = at.ld_z;
    if (!z) a.pre = EBIN_NORM_NONE;   // its sums are not wanted
    int64_t parts;
    return launch_block(p, a, false, &parts, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? EBIN_OK : EBIN_ERR_CUDA;
}

extern "C" ebin_status ebin_block_norm_grad_execute(ebin_block_norm_plan_t plan, const void *dz,
                                                    const void *dh, const void *h, const void *y,
                                                    const ebin_block_norm_params *params, void *dx,
                                                    void *dy, const ebin_block_norm_grads *grads,
                                                    void *workspace, size_t workspace_bytes,
                                                    void *stream) {
    if (!plan || !plan->at.gradient) return EBIN_ERR_INVALID_ARG;
    const ebin_block_norm_plan_s &p = *plan;
    const ebin_block_norm_attrs &at = p.at;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (at.n == 0) return EBIN_OK;
    const ebin_block_norm_grads g = grads ? *grads : ebin_block_norm_grads{};
    const ebin_block_norm_params w = params ? *params : ebin_block_norm_params{};
    const bool post = at.post != EBIN_NORM_NONE, pre = at.pre != EBIN_NORM_NONE;
    // a gradient of what does not enter the formula is refused
    if ((!at.has_branch && (g.gate || dy)) || (!post && (g.w_post || g.b_post)) ||
        (!pre && (g.w_pre || g.b_pre || g.scale || g.shift)))
        return EBIN_ERR_INVALID_ARG;
    struct Out { float *p; int64_t bytes; };
    const int64_t row = sizeof(float) * at.n;
    const int64_t gate_bytes = row * (at.gate_rows ? at.rows / at.gate_rows : 1);
    const int64_t mod_bytes = row * (at.mod_rows ? at.rows / at.mod_rows : 1);
    const Out sums[7] = {{g.gate, gate_bytes}, {g.scale, mod_bytes}, {g.shift, mod_bytes},
                         {g.w_post, row}, {g.b_post, row}, {g.w_pre, row}, {g.b_pre, row}};
    bool wanted = false;
    for (const Out &o : sums) {
        if ((uintptr_t)o.p % 4) return EBIN_ERR_INVALID_ARG;
        wanted |= o.p != nullptr;
    }
    if (at.rows == 0) {
        for (const Out &o : sums)
            if (o.p && o.bytes > 0 && cudaMemsetAsync(o.p, 0, (size_t)o.bytes, s) != cudaSuccess)
                return EBIN_ERR_CUDA;
        return EBIN_OK;
    }
    if (!pre) dz = h = nullptr;
    else if (!dz || !h) return EBIN_ERR_INVALID_ARG;
    if (!post && !g.gate) y = nullptr;
    else if (!y) return EBIN_ERR_INVALID_ARG;
    if (((uintptr_t)h | (uintptr_t)dh | (uintptr_t)dx) % (uintptr_t)p.ssz ||
        ((uintptr_t)y | (uintptr_t)dz | (uintptr_t)dy) % (uintptr_t)p.isz)
        return EBIN_ERR_INVALID_ARG;
    if (wanted && (!workspace || workspace_bytes < p.workspace || (uintptr_t)workspace % 16))
        return EBIN_ERR_INVALID_ARG;
    BlockArgs a;
    const ebin_status st = prepare_block(p, w, a);
    if (st != EBIN_OK) return st;
    a.shift = nullptr;
    Range in[12];
    int c = param_ranges(p, a, in);
    in[c++] = Range{dz, rows_bytes(at.rows, at.n, at.ld_dz, p.isz), at.ld_dz * p.isz, p.isz};
    in[c++] = Range{dh, rows_bytes(at.rows, at.n, at.ld_dh, p.ssz), at.ld_dh * p.ssz, p.ssz};
    in[c++] = Range{h, rows_bytes(at.rows, at.n, at.ld_h, p.ssz), at.ld_h * p.ssz, p.ssz};
    in[c++] = Range{y, rows_bytes(at.rows, at.n, at.ld_y, p.isz), at.ld_y * p.isz, p.isz};
    Range out[10] = {
        {dx, rows_bytes(at.rows, at.n, at.ld_dx, p.ssz), at.ld_dx * p.ssz, p.ssz},
        {dy, rows_bytes(at.rows, at.n, at.ld_dy, p.isz), at.ld_dy * p.isz, p.isz}};
    int o = 2;
    for (const Out &q : sums)
        if (q.p) out[o++] = Range{q.p, q.bytes, 0, 0};
    if (wanted) out[o++] = Range{workspace, (int64_t)p.workspace, 0, 0};
    for (int k = 0; k < o; ++k) {
        for (int i = 0; i < c; ++i)
            if (!apart(in[i], out[k], at.rows, at.n)) return EBIN_ERR_ALIAS;
        for (int i = 0; i < k; ++i)
            if (!disjoint(out[i], out[k], at.rows, at.n)) return EBIN_ERR_ALIAS;
    }
    a.x = h;
    a.y = y;
    a.dz = dz;
    a.dh = dh;
    a.h = dx;
    a.z = dy;
    a.ld_x = at.ld_h;
    a.ld_y = at.ld_y;
    a.ld_dz = at.ld_dz;
    a.ld_dh = at.ld_dh;
    a.ld_h = at.ld_dx;
    a.ld_z = at.ld_dy;
    a.partial = wanted ? static_cast<float *>(workspace) : nullptr;
    a.pad = pad_of(at.n);
    if (g.scale || g.w_pre) a.need |= 1 << SUM_DZ_HH;
    if (g.shift || g.b_pre || (g.scale && a.b_pre)) a.need |= 1 << SUM_DZ;
    if (g.gate || g.w_post) a.need |= 1 << SUM_E_YH;
    if (g.b_post || (g.gate && a.b_post)) a.need |= 1 << SUM_E;
    if (!wanted && !dx && !dy) return EBIN_OK;
    a.cta = p.cta[unit_grad_full(a.post, a.pre, a.need)];
    int64_t parts;
    if (launch_block(p, a, true, &parts, s) != cudaSuccess) return EBIN_ERR_CUDA;
    if (!wanted) return EBIN_OK;
    BlockSumsArgs b{};
    b.partial = a.partial;
    b.parts = parts;
    b.groups = p.groups;
    b.n = at.n;
    b.pad = a.pad;
    b.gate = a.gate;
    b.w_post = a.w_post;
    b.b_post = a.b_post;
    b.w_pre = a.w_pre;
    b.b_pre = a.b_pre;
    b.scale = a.scale;
    b.ld_gate = at.ld_gate;
    b.ld_scale = at.ld_scale;
    b.gate_grouped = at.gate_rows != 0;
    b.mod_grouped = at.mod_rows != 0;
    b.w_f32 = a.w_f32;
    b.mod_f32 = a.mod_f32;
    b.dtype = at.dtype;
    b.need = a.need;
    b.dgate = g.gate;
    b.dw_post = g.w_post;
    b.db_post = g.b_post;
    b.dw_pre = g.w_pre;
    b.db_pre = g.b_pre;
    b.dscale = g.scale;
    b.dshift = g.shift;
    // what all rows share, and the groups more than one
    b.second = p.groups > 1 && (g.w_post || g.b_post || g.w_pre || g.b_pre ||
                                (!b.gate_grouped && g.gate) ||
                                (!b.mod_grouped && (g.scale || g.shift)));
    b.tiles = div_up(at.n, kSumColumns);
    if (launch_sums(b, s) != cudaSuccess) return EBIN_ERR_CUDA;
    return EBIN_OK;
}
