// Product plans and their execution: attribute checks, the alias rule, kernel
// choice and launch.
#include <new>

#include "ebin_gemm.cuh"

struct ebin_gemm_plan_s {
    ebin_gemm_attrs at;
    int64_t lda, ldb, ldy, ldr, ldz;
    int64_t a_rows, a_cols, b_rows, b_cols;   // as stored
    size_t workspace = 0;
};

using namespace ebin;

namespace {

int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t isz) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * isz : 0;
}

template <class T, int ACT>
cudaError_t launch_any(const ebin_gemm_plan_s &p, const void *A, const void *B,
                       const GemmEpilogue &e, cudaStream_t s) {
    GemmAnyArgs g{};
    g.a = A;
    g.b = B;
    g.a_m = p.at.trans_a ? 1 : p.lda;
    g.a_k = p.at.trans_a ? p.lda : 1;
    g.b_k = p.at.trans_b ? 1 : p.ldb;
    g.b_n = p.at.trans_b ? p.ldb : 1;
    g.s = {p.at.m, p.at.n, p.at.k};
    g.e = e;
    const dim3 grid((unsigned)div_up(p.at.n, 64), (unsigned)div_up(p.at.m, 64));
    return launch_layer(k_gemm_any<T, ACT>, grid, 256, 0, s, 1, g);
}

template <class T>
cudaError_t launch_gemm(const ebin_gemm_plan_s &p, const void *A, const void *B,
                        const GemmEpilogue &e, cudaStream_t s) {
    switch (p.at.activation) {
    case EBIN_ACT_RELU: return launch_any<T, EBIN_ACT_RELU>(p, A, B, e, s);
    case EBIN_ACT_GELU: return launch_any<T, EBIN_ACT_GELU>(p, A, B, e, s);
    case EBIN_ACT_GELU_TANH: return launch_any<T, EBIN_ACT_GELU_TANH>(p, A, B, e, s);
    case EBIN_ACT_SILU: return launch_any<T, EBIN_ACT_SILU>(p, A, B, e, s);
    default: return launch_any<T, EBIN_ACT_NONE>(p, A, B, e, s);
    }
}

}  // namespace

extern "C" ebin_status ebin_gemm_plan_create(const ebin_gemm_attrs *attrs, ebin_gemm_plan_t *out) {
    if (!attrs || !out) return EBIN_ERR_INVALID_ARG;
    *out = nullptr;
    const ebin_gemm_attrs &a = *attrs;
    if (a.dtype != EBIN_FLOAT16 && a.dtype != EBIN_BFLOAT16) return EBIN_ERR_UNSUPPORTED_TYPE;
    for (int32_t f : {a.trans_a, a.trans_b, a.has_bias, a.has_residual, a.any_alignment})
        if (f != 0 && f != 1) return EBIN_ERR_INVALID_ATTR;
    if (a.activation < EBIN_ACT_NONE || a.activation > EBIN_ACT_SILU) return EBIN_ERR_INVALID_ATTR;
    if (a.has_bias && a.dtype_bias != a.dtype && a.dtype_bias != EBIN_FLOAT32)
        return EBIN_ERR_UNSUPPORTED_TYPE;
    const int64_t most = int64_t(1) << 30;
    if (a.m < 0 || a.n < 0 || a.k < 0 || a.m > most || a.n > most || a.k > most)
        return EBIN_ERR_INVALID_ARG;
    auto *p = new (std::nothrow) ebin_gemm_plan_s;
    if (!p) return EBIN_ERR_INVALID_ARG;
    p->at = a;
    p->a_rows = a.trans_a ? a.k : a.m;
    p->a_cols = a.trans_a ? a.m : a.k;
    p->b_rows = a.trans_b ? a.n : a.k;
    p->b_cols = a.trans_b ? a.k : a.n;
    p->lda = a.lda ? a.lda : p->a_cols;
    p->ldb = a.ldb ? a.ldb : p->b_cols;
    p->ldy = a.ldy ? a.ldy : a.n;
    p->ldr = a.ld_residual ? a.ld_residual : a.n;
    p->ldz = a.ld_preact ? a.ld_preact : a.n;
    const int64_t ld[5] = {p->lda, p->ldb, p->ldy, p->ldr, p->ldz};
    const int64_t rows[5] = {p->a_rows, p->b_rows, a.m, a.m, a.m};
    const int64_t cols[5] = {p->a_cols, p->b_cols, a.n, a.n, a.n};
    for (int i = 0; i < 5; ++i) {
        int64_t n;
        if (ld[i] < cols[i] || !product_fits(std::max<int64_t>(rows[i], 1), ld[i], &n)) {
            delete p;
            return EBIN_ERR_INVALID_ARG;
        }
    }
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_gemm_plan_workspace(ebin_gemm_plan_t plan, size_t *bytes) {
    if (!plan || !bytes) return EBIN_ERR_INVALID_ARG;
    *bytes = plan->workspace;
    return EBIN_OK;
}

extern "C" void ebin_gemm_plan_release(ebin_gemm_plan_t plan) { delete plan; }

extern "C" ebin_status ebin_gemm_execute(ebin_gemm_plan_t plan, const void *A, const void *B,
                                         const void *bias, const void *residual, void *Y,
                                         void *preact, void *workspace, size_t workspace_bytes,
                                         void *stream) {
    if (!plan) return EBIN_ERR_INVALID_ARG;
    const ebin_gemm_plan_s &p = *plan;
    const ebin_gemm_attrs &at = p.at;
    if (at.m == 0 || at.n == 0) return EBIN_OK;
    if (at.k == 0) A = B = nullptr;
    if (!at.has_bias) bias = nullptr;
    if (!at.has_residual) residual = nullptr;
    if (!Y || (at.k > 0 && (!A || !B)) || (at.has_bias && !bias) || (at.has_residual && !residual))
        return EBIN_ERR_INVALID_ARG;
    const uintptr_t elements = (uintptr_t)A | (uintptr_t)B | (uintptr_t)residual | (uintptr_t)Y |
                               (uintptr_t)preact;
    const uintptr_t bias_size = at.has_bias ? (uintptr_t)ebin_dtype_size(at.dtype_bias) : 1;
    if (elements % 2 || (uintptr_t)bias % bias_size) return EBIN_ERR_INVALID_ARG;
    if (!at.any_alignment && ((uintptr_t)A | (uintptr_t)B) % 16) return EBIN_ERR_INVALID_ARG;
    if (p.workspace > 0 && (!workspace || workspace_bytes < p.workspace ||
                            (uintptr_t)workspace % 16 != 0))
        return EBIN_ERR_INVALID_ARG;
    struct Range { const void *p; int64_t n; };
    const Range out[3] = {{Y, matrix_bytes(at.m, at.n, p.ldy, 2)},
                          {preact, preact ? matrix_bytes(at.m, at.n, p.ldz, 2) : 0},
                          {workspace, (int64_t)p.workspace}};
    const Range in[4] = {{A, A ? matrix_bytes(p.a_rows, p.a_cols, p.lda, 2) : 0},
                         {B, B ? matrix_bytes(p.b_rows, p.b_cols, p.ldb, 2) : 0},
                         {bias, bias ? at.n * (int64_t)bias_size : 0},
                         {residual, residual ? matrix_bytes(at.m, at.n, p.ldr, 2) : 0}};
    for (int o = 0; o < 3; ++o) {
        for (int i = 0; i < 4; ++i)
            if (ranges_overlap(out[o].p, out[o].n, in[i].p, in[i].n) &&
                !(o == 0 && i == 3 && Y == residual && p.ldy == p.ldr))
                return EBIN_ERR_ALIAS;
        for (int q = 0; q < o; ++q)
            if (ranges_overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return EBIN_ERR_ALIAS;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    GemmEpilogue e{};
    e.bias = bias;
    e.residual = residual;
    e.y = Y;
    e.z = preact;
    e.ld_residual = p.ldr;
    e.ldy = p.ldy;
    e.ldz = p.ldz;
    e.bias_f32 = at.dtype_bias == EBIN_FLOAT32;
    e.act = at.activation;
    const cudaError_t st = at.dtype == EBIN_FLOAT16 ? launch_gemm<__half>(p, A, B, e, s)
                                                    : launch_gemm<__nv_bfloat16>(p, A, B, e, s);
    return st == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}
