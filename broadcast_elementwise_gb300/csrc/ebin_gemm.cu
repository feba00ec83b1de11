// Product plans and their execution: attribute checks, the alias rule, kernel
// choice and launch.
#include <new>

#include "ebin_gemm_tc.cuh"

struct ebin_gemm_plan_s {
    ebin_gemm_attrs at;
    int64_t lda, ldb, ldy, ldr, ldz;
    int64_t a_rows, a_cols, b_rows, b_cols;   // as stored
    int64_t copy_a = -1, copy_b = -1;         // workspace offsets of their copies, or -1
    size_t workspace = 0;
};

namespace ebin {

#define EBIN_DECLARE_TC(name)                                                             \
    cudaError_t name(const CUtensorMap &, const CUtensorMap &, const TcArgs &, int bn,    \
                     bool pair, int grid, int cluster, cudaStream_t);
EBIN_DECLARE_TC(launch_tc_f16)
EBIN_DECLARE_TC(launch_tc_bf16)
#undef EBIN_DECLARE_TC
// Clusters of so many CTAs of the split kernel that the current device holds at once.
int tc_clusters_f16(int bn, int cluster);
int tc_clusters_bf16(int bn, int cluster);

// Lay a matrix of 16-bit elements out anew, its rows on 16-byte boundaries.  A
// vector of eight elements comes from the two aligned vectors that hold them,
// shifted by the row's offset; the first and last of the matrix, whose aligned
// vectors reach past it, element by element.  What a row's last vector holds
// past the row is never read.  Bound by latency: one round of loads, all of a
// thread's on their way before the first is used ([1021,2049] and [1543,2049]
// together 12 us element by element, 3.6 us so).
struct RepackArgs {
    const uint16_t *src;
    uint4 *dst;
    int64_t rows, cols, ld;
    int64_t units, pitch;            // vectors of a row of dst, and from row to row
    FastDiv per_row;                 // by units
};

constexpr int kRepackVectors = 2;    // of a thread

__global__ void __launch_bounds__(256) k_repack(const RepackArgs a, const RepackArgs b) {
    layer_pdl_launch();
    const RepackArgs &r = blockIdx.y ? b : a;
    const int64_t total = r.rows * r.units;
    const bool narrow = total < (1ll << 31);
    const uintptr_t first = (uintptr_t)r.src;
    const uintptr_t last = first + 2 * (uintptr_t)((r.rows - 1) * r.ld + r.cols);
    layer_pdl_wait();
    for (int64_t i0 = (int64_t)blockIdx.x * (256 * kRepackVectors) + threadIdx.x; i0 < total;
         i0 += (int64_t)gridDim.x * (256 * kRepackVectors)) {
        uint4 v[kRepackVectors], n[kRepackVectors];
        int64_t to[kRepackVectors], c[kRepackVectors];
        uintptr_t at[kRepackVectors];
        bool whole[kRepackVectors];
#pragma unroll
        for (int k = 0; k < kRepackVectors; ++k) {
            const int64_t i = min(i0 + 256 * k, total - 1);   // one past the end repeats the last
            int64_t row, u;
            if (narrow) {
                uint32_t q, rest;
                r.per_row.split((uint32_t)i, q, rest);
                row = q;
                u = rest;
            } else {
                row = i / r.units;
                u = i - row * r.units;
            }
            c[k] = u * 8;
            to[k] = row * r.pitch + u;
            at[k] = (uintptr_t)(r.src + row * r.ld + c[k]);
            const uintptr_t low = at[k] & ~(uintptr_t)15;
            whole[k] = low >= first && low + 32 <= last;
            v[k] = n[k] = make_uint4(0, 0, 0, 0);
            if (whole[k]) {
                v[k] = __ldg(reinterpret_cast<const uint4 *>(low));
                n[k] = __ldg(reinterpret_cast<const uint4 *>(low) + 1);
            }
        }
#pragma unroll
        for (int k = 0; k < kRepackVectors; ++k) {
            uint32_t w[8] = {v[k].x, v[k].y, v[k].z, v[k].w, n[k].x, n[k].y, n[k].z, n[k].w};
            if (whole[k]) {
                const uint32_t shift = (uint32_t)(at[k] & 15);
                if (shift & 8) {
#pragma unroll
                    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
                }
                if (shift & 4) {
#pragma unroll
                    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
                }
                if (shift & 2) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
                }
            } else {
                const uint16_t *const x = reinterpret_cast<const uint16_t *>(at[k]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = c[k] + 2 * j < r.cols ? x[2 * j] : 0u;
                    const uint32_t hi = c[k] + 2 * j + 1 < r.cols ? x[2 * j + 1] : 0u;
                    w[j] = lo | hi << 16;
                }
            }
            if (i0 + 256 * k < total) r.dst[to[k]] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace ebin

using namespace ebin;

namespace {

int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld, int64_t isz) {
    return rows > 0 && cols > 0 ? ((rows - 1) * ld + cols) * isz : 0;
}

// Row pitch of an operand's copy: whole 128-byte lines, so that a copy's rows
// of 128 bytes do not straddle two (13.0 -> 8.9 us for [1021, 2049] x [1543, 2049]).
int64_t copy_pitch(int64_t cols) { return div_up(cols, 64) * 64; }

// cuTensorMapEncodeTiled, looked up through the runtime, or null.
using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (EncodeFn) nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// One operand of the product as the kernel sees it.
struct Operand {
    const void *p;
    int64_t rows, cols, ld;   // as stored
    int64_t copy;             // its copy's workspace offset, or -1
    bool mn;                  // dense across k
};

// The tensor map of an operand: boxes of 64 dense elements by `box` rows.
bool encode(const Operand &o, int box, bool bf16, CUtensorMap *map) {
    const EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)o.cols, (cuuint64_t)o.rows};
    // a single row has no step; any whole number of vectors serves
    const cuuint64_t strides[1] = {(cuuint64_t)(o.rows > 1 ? o.ld : copy_pitch(o.cols)) * 2};
    const cuuint32_t boxes[2] = {64, (cuuint32_t)(o.mn ? kTcBK : box)};
    const cuuint32_t steps[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
              const_cast<void *>(o.p), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool needs_copy(const Operand &o) {
    return (uintptr_t)o.p % 16 != 0 || (o.rows > 1 && o.ld % 8 != 0);
}

struct Shape {
    int bn;        // accumulator columns of a tile
    int split;     // CTAs that share a tile's k (1 for the paired kernel too)
    bool pair;     // 256 x 256 tiles on pairs of CTAs, P = A; else P = B on single CTAs
};

// Which tiles: the least of an estimate in nanoseconds.  A step of k takes a
// CTA its matrix instructions or its copies, whichever is longer (on a pair
// 1.05 ns a column; copies at 190 bytes a ns), and 24 ns that keep wide tiles,
// which move fewer bytes a product, ahead of a narrower one's last wave where
// that gains under a tenth (medians of runs in turn: [4096,4096] x [4096,8192] on
// 160 columns 149 us, on 256 150; 4096^3 on 256 columns 96 us, on 224 85); a tile's end
// costs 12 ns a column once, the sums of split tiles 1.5 us more.  On single CTAs a
// step takes 140 ns to 64 columns, 230 to 128 with every SM at it (operands from
// memory and, after the stroke, in the L2: [256,4096] x [4096,4096] on pairs of 64
// columns 13.4 / 12.5 us, on tiles of 128 split in two 15.0 / 13.4; [128,4096] x
// [4096,4096] on pairs of 64 13.2 / 12.4, on tiles of 128 split in four 13.1 / 10.7).
//   pair   256 rows of A by 64 to 256 columns, a CTA pair each, waves of pairs
//   split  128 columns of B by 16 to 128 rows of A, k cut in up to eight while
//          all clusters fit at once ([4,4096] x [4096,4096] from memory cut in eight,
//          two waves of clusters: 20.1 us; in four, one wave: 9.8; in two 10.2)
Shape gemm_shape(const ebin_gemm_attrs &at, int sms) {
    const bool bf16 = at.dtype == EBIN_BFLOAT16;
    const double kblocks = (double)div_up(at.k, kTcBK);
    Shape best{};
    double least = 0;
    auto consider = [&](const Shape &s, double ns) {
        if (best.bn == 0 || ns < least) {
            best = s;
            least = ns;
        }
    };
    Shape s{};
    s.bn = at.m <= 16 ? 16 : at.m <= 32 ? 32 : at.m <= 64 ? 64 : 128;
    const int64_t tiles = div_up(at.n, kTcRows) * div_up(at.m, s.bn);
    for (s.split = 1; s.split <= 8; s.split *= 2) {
        if (s.split > 1 && (kblocks < s.split * 4 ||
                            tiles > (bf16 ? tc_clusters_bf16 : tc_clusters_f16)(s.bn, s.split)))
            break;
        const double step = s.bn <= 64 ? 140 : 230;
        consider(s, div_up(tiles * s.split, sms) * (kblocks / s.split) * step + 12.0 * s.bn +
                        (s.split > 1 ? 1500 : 0));
    }
    if (at.m > 64) {
        s.split = 1;
        s.pair = true;
        for (int bn : {256, 224, 192, 160, 128, 96, 64}) {
            s.bn = bn;
            const int64_t waves = div_up(div_up(at.m, 2 * kTcRows) * div_up(at.n, bn), sms / 2);
            const double step = std::max(1.05 * bn, (16384 + 64.0 * bn) / 190) + 24;
            consider(s, waves * kblocks * step + 12.0 * bn);
        }
    }
    return best;
}

cudaError_t launch_gemm(const ebin_gemm_plan_s &p, const void *A, const void *B,
                        const GemmEpilogue &e, void *workspace, cudaStream_t s) {
    const ebin_gemm_attrs &at = p.at;
    Operand a{A, p.a_rows, p.a_cols, p.lda, p.copy_a, at.trans_a != 0};
    Operand b{B, p.b_rows, p.b_cols, p.ldb, p.copy_b, at.trans_b == 0};
    const bool bf16 = at.dtype == EBIN_BFLOAT16;
    if (at.k > 0) {
        RepackArgs r[2];
        int count = 0;
        int64_t most = 0;
        for (Operand *o : {&a, &b}) {
            if (!needs_copy(*o)) continue;
            char *dst = static_cast<char *>(workspace) + o->copy;
            const int64_t units = div_up(o->cols, 8);
            r[count++] = RepackArgs{static_cast<const uint16_t *>(o->p),
                                    reinterpret_cast<uint4 *>(dst), o->rows, o->cols, o->ld,
                                    units, copy_pitch(o->cols) / 8, fast_div((uint32_t)units)};
            most = std::max(most, o->rows * units);
            o->p = dst;
            o->ld = copy_pitch(o->cols);
        }
        if (count > 0) {
            const int64_t grid = std::min<int64_t>(
                div_up(most, 256 * kRepackVectors), 16ll * current_sm_count());
            const cudaError_t st = launch_layer(k_repack, dim3((unsigned)grid, (unsigned)count),
                                                256, 0, s, 1, r[0], r[count - 1]);
            if (st != cudaSuccess) return st;
        }
    }
    const Shape shape = gemm_shape(at, current_sm_count());
    const Operand &po = shape.pair ? a : b, &qo = shape.pair ? b : a;
    TcArgs t{};
    t.e = e;
    t.m = at.m;
    t.n = at.n;
    t.kblocks = (int)div_up(at.k, kTcBK);
    const int64_t p_rows = shape.pair ? at.m : at.n, q_rows = shape.pair ? at.n : at.m;
    const int64_t p_tiles = div_up(p_rows, kTcRows * (shape.pair ? 2 : 1));
    const int64_t q_tiles = div_up(q_rows, shape.bn);
    t.p_tiles = (int)p_tiles;
    t.q_tiles = (int)q_tiles;
    t.p_mn = po.mn;
    t.q_mn = qo.mn;
    t.q_box = shape.bn / (shape.pair ? 2 : 1);
    auto aligned = [&](const void *x, int64_t ld) { return (uintptr_t)x % 16 == 0 && ld % 8 == 0; };
    t.vec = aligned(e.y, e.ldy) && aligned(e.z, e.z ? e.ldz : 0) &&
            aligned(e.residual, e.residual ? e.ld_residual : 0) && (uintptr_t)e.bias % 16 == 0;
    if (t.vec && ((uintptr_t)e.y | (uintptr_t)e.z | (uintptr_t)e.residual) % 32 == 0 &&
        (e.ldy | (e.z ? e.ldz : 0) | (e.residual ? e.ld_residual : 0)) % 16 == 0)
        t.vec = 2;
    // two seconds, and the time that a long sum may take
    t.limit = 4000000000ll + 100000ll * t.kblocks;
    t.status = stream_status_word(s);
    if (!t.status) return cudaErrorMemoryAllocation;
    CUtensorMap maps[2] = {};
    if (at.k > 0 && (!encode(po, kTcRows, bf16, &maps[0]) || !encode(qo, t.q_box, bf16, &maps[1])))
        return cudaErrorInvalidValue;
    const int64_t tiles = p_tiles * q_tiles;
    const int cluster = shape.pair ? 2 : shape.split;
    const int64_t clusters = shape.pair ? std::min<int64_t>(tiles, current_sm_count() / 2) : tiles;
    if (tiles > 0x7FFFFFFF || clusters * cluster > 0x7FFFFFFF)
        return cudaErrorInvalidConfiguration;
    return (bf16 ? launch_tc_bf16 : launch_tc_f16)(
        maps[0], maps[1], t, shape.bn, shape.pair, (int)clusters * cluster, cluster, s);
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
    // copies of operands whose rows the tensor copies cannot take as they lie
    if (a.m > 0 && a.n > 0 && a.k > 0) {
        if (a.any_alignment || (p->a_rows > 1 && p->lda % 8 != 0)) {
            p->copy_a = (int64_t)p->workspace;
            p->workspace += (size_t)(p->a_rows * copy_pitch(p->a_cols) * 2);
        }
        if (a.any_alignment || (p->b_rows > 1 && p->ldb % 8 != 0)) {
            p->copy_b = (int64_t)p->workspace;
            p->workspace += (size_t)(p->b_rows * copy_pitch(p->b_cols) * 2);
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
    return launch_gemm(p, A, B, e, workspace, s) == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}
