// Heads plans and their execution (rotary positions, head norms with the
// rotation): attribute checks, the alias rule, kernel choice and launch; and
// the rotation tables.
#include <cmath>
#include <new>

#include "ebin_heads.cuh"

namespace ebin {

// The pairs of a table's columns: (axis' pairs, place among them) of each.
struct TableSections {
    uint16_t pairs[kHeadsMaxDim / 2], place[kHeadsMaxDim / 2];
};

struct TableArgs {
    int64_t first, positions;
    int32_t half, scaling;
    double log2_base;      // the base after its own scaling
    double factor, trained, slow, fast, amplitude;
    float *cos, *sin;
};

// One thread per frequency, its positions in steps of the grid's y: the
// frequency in binary64 once, then an angle, its cosine and its sine each.
template <bool AXES>
__global__ void __launch_bounds__(256)
k_rotary_table(const TableArgs a,
               const std::conditional_t<AXES, TableSections, HeadsOne> sections) {
    layer_pdl_launch();
    layer_pdl_wait();
    const int64_t n = a.positions * a.half;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / a.half;
        const int j = (int)(i - row * a.half);
        double part;
        if constexpr (AXES) part = (double)sections.place[j] / (double)sections.pairs[j];
        else part = (double)j / (double)a.half;
        double f = exp2(-a.log2_base * part);
        if (a.scaling == EBIN_ROTARY_SCALE_LINEAR) f /= a.factor;
        if (a.scaling == EBIN_ROTARY_SCALE_BY_PARTS) {
            const double turns = a.trained * f / 6.283185307179586476925;
            const double g = fmin(fmax((turns - a.slow) / (a.fast - a.slow), 0.0), 1.0);
            f *= g + (1.0 - g) / a.factor;
        }
        double s, c;
        sincos((double)(a.first + row) * f, &s, &c);
        a.cos[i] = (float)(c * a.amplitude);
        a.sin[i] = (float)(s * a.amplitude);
    }
}

}  // namespace ebin

struct ebin_heads_plan_s {
    ebin_heads_attrs at;
    int64_t rows = 0;          // batch * tokens
    int64_t isz = 0;
    int64_t span[6] = {};      // storage extent in elements: q, k, dq, dk, q_out, k_out
    bool empty = false;
    size_t workspace = 0;
    bool several = false;      // the positions have axes
    int64_t axes_count = 1;
    ebin::HeadsAxes axes = {};
};

using namespace ebin;

namespace {

const ebin_heads_view &view_of(const ebin_heads_attrs &a, int i) {
    const ebin_heads_view *v[6] = {&a.q, &a.k, &a.dq, &a.dk, &a.q_out, &a.k_out};
    return *v[i];
}

int heads_of(const ebin_heads_attrs &a, int i) { return i % 2 ? a.k_heads : a.q_heads; }

// Largest offset + 1 of a view, or -1 when it reaches 2^60 elements.
int64_t heads_span(const ebin_heads_attrs &a, const ebin_heads_view &v, int heads) {
    const int64_t n[3] = {a.batch, a.tokens, heads}, s[3] = {v.batch, v.token, v.head};
    int64_t last = a.head_dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 0) return 0;
        int64_t part;
        if (s[i] < 0 || !product_fits(n[i] - 1, s[i], &part) || part >= EBIN_MAX_ELEMENTS - last)
            return -1;
        last += part;
    }
    return last;
}

// Whether no two elements of an output view share an address: with the
// dimensions in order of their strides, each step passes what the smaller ones span.
bool heads_distinct(const ebin_heads_attrs &a, const ebin_heads_view &v, int heads) {
    int64_t n[3] = {a.batch, a.tokens, heads}, s[3] = {v.batch, v.token, v.head};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) {
                std::swap(s[i], s[j]);
                std::swap(n[i], n[j]);
            }
    int64_t span = a.head_dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < span) return false;
        span += (n[i] - 1) * s[i];
    }
    return true;
}

struct Placed {
    const char *p;
    const ebin_heads_view *v;
    int heads;
    int64_t span;   // elements
};

// A step taken c times, lo <= c <= hi.
struct Walk {
    int64_t step, lo, hi;
};

// Whether some counts c put the sum of c step within `width` of `target`.  Walks in
// falling order of their steps, so that each level of nested strides leaves one or
// two counts to try; past `tries` the answer is yes.
bool walks_meet(const Walk *w, int n, int64_t target, int64_t width, int &tries) {
    if (--tries < 0) return true;
    int64_t lo = 0, hi = 0;   // what the walks after the first can add
    for (int i = 1; i < n; ++i) {
        lo += w[i].lo * w[i].step;
        hi += w[i].hi * w[i].step;
    }
    if (n == 0) return target > -width && target < width;
    // c step lies in (target - hi - width, target - lo + width)
    const int64_t from = target - hi - width, to = target - lo + width, s = w->step;
    const int64_t first = from >= 0 ? from / s + 1 : -((-from - 1) / s);
    const int64_t last = to > 0 ? (to - 1) / s : -((-to) / s) - 1;
    for (int64_t c = std::max(first, w->lo); c <= std::min(last, w->hi); ++c)
        if (walks_meet(w + 1, n - 1, target - c * s, width, tries)) return true;
    return false;
}

// Whether two views share an element (true when the search for one gets too
// long).  Rows of head_dim elements of x and y share one when their starts are
// less than head_dim apart: y's first start less x's is then within head_dim
// of a sum of x's steps forward and y's back.
bool heads_share(const ebin_heads_attrs &a, const Placed &x, const Placed &y, int64_t isz) {
    if (!ranges_overlap(x.p, x.span * isz, y.p, y.span * isz)) return false;
    const int64_t d = (int64_t)((intptr_t)y.p - (intptr_t)x.p);
    if (d % isz != 0) return true;
    const int64_t nx[3] = {a.batch, a.tokens, x.heads}, ny[3] = {a.batch, a.tokens, y.heads};
    const int64_t sx[3] = {x.v->batch, x.v->token, x.v->head};
    const int64_t sy[3] = {y.v->batch, y.v->token, y.v->head};
    Walk w[6];
    int n = 0;
    auto add = [&](int64_t step, int64_t lo, int64_t hi) {
        if (step == 0 || lo == hi) return;   // goes nowhere
        for (int i = 0; i < n; ++i)
            if (w[i].step == step) {
                w[i].lo += lo;
                w[i].hi += hi;
                return;
            }
        w[n++] = Walk{step, lo, hi};
    };
    for (int i = 0; i < 3; ++i) {
        add(sx[i], 0, nx[i] - 1);
        add(sy[i], 1 - ny[i], 0);
    }
    std::sort(w, w + n, [](const Walk &p, const Walk &q) { return p.step > q.step; });
    int tries = 256;
    return walks_meet(w, n, d / isz, a.head_dim, tries);
}

bool same_view(const ebin_heads_attrs &a, const Placed &x, const Placed &y) {
    return x.p == y.p && x.heads == y.heads && (a.batch <= 1 || x.v->batch == y.v->batch) &&
           (a.tokens <= 1 || x.v->token == y.v->token) &&
           (x.heads <= 1 || x.v->head == y.v->head);
}

int64_t type_size(ebin_dtype t) { return (int64_t)ebin_dtype_size(t); }

bool layer_float(ebin_dtype t) {
    return t == EBIN_FLOAT32 || t == EBIN_FLOAT16 || t == EBIN_BFLOAT16;
}

// CTAs of one tensor whose weight-gradient sums the workspace holds at most.
constexpr int64_t kHeadsMaxPartials = 1024;

int64_t any_ctas(const ebin_heads_plan_s &p, int which, int mode) {
    const int64_t rows = p.rows * heads_of(p.at, which);
    const int64_t ctas = std::max<int64_t>(1, div_up(rows, kHeadsThreads / 32));
    // the gradient's CTAs each add one row to the final sum: about eight per SM
    const int64_t most = mode == HEADS_NORM_GRAD
        ? std::min<int64_t>(kHeadsMaxPartials, 4ll * current_sm_count()) : 0x7FFFFFFF;
    return std::min(ctas, most);
}

template <class T, class AX>
cudaError_t launch_any(const ebin_heads_plan_s &p, const HeadsArgs &a, const AX &ax, int mode,
                       int64_t *ctas, cudaStream_t s) {
    ctas[0] = any_ctas(p, 0, mode);
    ctas[1] = any_ctas(p, 1, mode);
    const int64_t gx = std::max(ctas[0], ctas[1]);
    ctas[0] = ctas[1] = gx;
    const dim3 grid((unsigned)gx, p.at.k_heads > 0 ? 2 : 1);
    const int il = p.at.layout == EBIN_ROTARY_INTERLEAVED;
    if (mode == HEADS_ROTATE)
        return launch_layer(k_heads_any<T, HEADS_ROTATE, AX>, grid, kHeadsThreads, 0, s, 1, a, ax,
                            il);
    if (mode == HEADS_NORM)
        return launch_layer(k_heads_any<T, HEADS_NORM, AX>, grid, kHeadsThreads, 0, s, 1, a, ax,
                            il);
    const size_t smem = sizeof(float) * (kHeadsThreads / 32) * a.dim;   // <= 32 KB
    return launch_layer(k_heads_any<T, HEADS_NORM_GRAD, AX>, grid, kHeadsThreads, smem, s, 1, a, ax,
                        il);
}

// The vector path's layout of a head, or false where it does not apply: rows
// that are not whole 16-byte vectors on 16-byte boundaries, heads of more than 64
// vectors, and an empty table (a token outside the table reads its first row's
// angles there, and drops them).
template <class AX>
bool heads_vectors(const ebin_heads_plan_s &p, const HeadsArgs &a, const AX &, bool grad,
                   HeadsVecArgs &v, int &kind) {
    const int64_t V = 16 / p.isz, D = a.dim;
    if (D % V != 0 || (a.half > 0 && a.table == 0)) return false;
    kind = p.at.layout == EBIN_ROTARY_INTERLEAVED ? (AX::kSeveral ? HEADS_SPREAD : HEADS_PAIRS)
         : a.half % V == 0 ? HEADS_HALF : HEADS_ODD;
    auto fits = [&](const HeadsTensor &t, int heads) {
        return (uintptr_t)t.p % 16 == 0 && (p.at.batch <= 1 || t.sb % V == 0) &&
               (p.at.tokens <= 1 || t.st % V == 0) && (heads <= 1 || t.sh % V == 0);
    };
    for (int w = 0; w < 2; ++w) {
        const int h = heads_of(p.at, w);
        if (h > 0 && !(fits(a.x[w], h) && fits(a.y[w], h) && (!grad || fits(a.dy[w], h))))
            return false;
    }
    const int64_t most = 0x7FFFFFFF;
    v = HeadsVecArgs{};
    for (int w = 0; w < 2; ++w) {
        const HeadsTensor *from[3] = {&a.x[w], &a.dy[w], &a.y[w]};
        HeadsNear *to[3] = {&v.x[w], &v.dy[w], &v.y[w]};
        for (int i = 0; i < 3; ++i) {
            if (heads_of(p.at, w) == 0 || (i == 1 && !grad)) continue;
            if (from[i]->st > most || from[i]->sh > most) return false;
            *to[i] = HeadsNear{from[i]->p, from[i]->sb, (int32_t)from[i]->st,
                               (int32_t)from[i]->sh};
        }
        const uint32_t parts = (uint32_t)div_up(a.heads[w], AX::kRingHeads);
        v.heads[w] = fast_div(std::max(1u, parts));
        v.heads[w].n = parts;
    }
    v.tokens = fast_div((uint32_t)a.tokens);
    v.rot_units = (int)(a.half / V);
    v.units = kind != HEADS_HALF ? (int)div_up(D / V, 2)
                                 : v.rot_units + (int)div_up((D - 2 * a.half) / V, 2);
    if (v.units > 32) return false;
    while ((1 << v.log_lanes) < v.units) ++v.log_lanes;
    // the launch's threads, and an item past the last step, are counted in 32 bits
    // (26 million tokens of 40 heads of 128 in 16 bits)
    const int64_t items = div_up(a.heads[0], 4) + div_up(a.heads[1], 4);
    if (p.rows > most >> v.log_lanes || (p.rows << v.log_lanes) > most / std::max<int64_t>(1, items))
        return false;
    v.weight_vec = ((uintptr_t)a.w[0] | (uintptr_t)a.w[1]) % 16 == 0;
    v.table_vec = a.half % 4 == 0 && ((uintptr_t)a.cos | (uintptr_t)a.sin) % 16 == 0;
    return true;
}

// CTAs of a kernel that fit an SM at once.
template <auto KERNEL> int heads_resident(size_t smem) {
    static const int n = [smem] {
        int b = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, KERNEL, kHeadsThreads, smem) !=
                cudaSuccess || b < 1) {
            cudaGetLastError();
            b = 1;
        }
        return b;
    }();
    return n;
}

template <class T, int KIND, int MODE, int HPT, class AX>
cudaError_t launch_vec(const HeadsArgs &a, HeadsVecArgs v, const AX &ax, cudaStream_t s) {
    v.q_items = (uint32_t)div_up(a.heads[0], HPT);
    v.per_token = fast_div(v.q_items + (uint32_t)div_up(a.heads[1], HPT));
    v.items = (uint32_t)a.rows * v.per_token.n;
    const int64_t grid = div_up((int64_t)v.items << v.log_lanes, kHeadsThreads);
    const size_t smem = KIND == HEADS_ODD
        ? sizeof(T) * (kHeadsThreads >> v.log_lanes) * HPT * a.dim : 0;   // at most 32 KB
    return launch_layer(k_heads_vec<T, KIND, MODE, HPT, AX>, dim3((unsigned)grid), kHeadsThreads,
                        smem, s, 1, a, v, ax);
}

template <class T, int KIND, class AX>
cudaError_t launch_ring(const HeadsArgs &a, HeadsVecArgs v, const AX &ax, cudaStream_t s) {
    const HeadsVecArgs plain = v;
    v.q_items = (uint32_t)div_up(a.heads[0], AX::kRingHeads);
    v.per_token = fast_div(v.q_items + (uint32_t)div_up(a.heads[1], AX::kRingHeads));
    v.items = (uint32_t)a.rows * v.per_token.n;
    constexpr size_t smem = HeadsRing<T, KIND, false, AX>::kBytes + (KIND == HEADS_ODD ? 8192 : 0);
    const cudaError_t opted = allow_smem<k_heads_ring<T, KIND, AX>>(smem);
    if (opted != cudaSuccess) return opted;
    const int64_t wave =
        (int64_t)heads_resident<k_heads_ring<T, KIND, AX>>(smem) * current_sm_count();
    // Under three items a group the walk is too short to pay for itself (norm
    // [3,1021,15,96] f32, 1.3 items: 11.5 us against 8.2 by a CTA an item; [2,4096,40,128]
    // bf16, 5.6 items: 29.0 against 32.2).
    if (((int64_t)v.items << v.log_lanes) < 3 * wave * kHeadsThreads)
        return launch_vec<T, KIND, HEADS_NORM, 4>(a, plain, ax, s);
    return launch_layer(k_heads_ring<T, KIND, AX>, dim3((unsigned)wave), kHeadsThreads, smem, s, 1,
                        a, v, ax);
}

template <class T, int KIND, class AX>
cudaError_t launch_vec_grad(const HeadsArgs &a, HeadsVecArgs v, const AX &ax, int64_t *ctas,
                            cudaStream_t s) {
    // the ring, one group's weights (two vectors a lane) and, HEADS_ODD, the groups'
    // rows: at most 4 KB and 8 KB of them; the sums at the end fit the ring
    constexpr size_t most =
        HeadsRing<T, KIND, true, AX>::kBytes + 4096 + (KIND == HEADS_ODD ? 8192 : 0);
    const cudaError_t opted = allow_smem<k_heads_vec_grad<T, KIND, AX>>(most);
    if (opted != cudaSuccess) return opted;
    // one wave of CTAs, shared between q and k by their rows
    const int per = kHeadsThreads >> v.log_lanes;
    const int64_t all = std::min<int64_t>(
        (int64_t)heads_resident<k_heads_vec_grad<T, KIND, AX>>(most) * current_sm_count(),
        kHeadsMaxPartials);
    const int64_t heads = a.heads[0] + a.heads[1];
    for (int w = 0; w < 2; ++w) {
        const int64_t items = div_up(a.rows * div_up(a.heads[w], AX::kRingHeads), per);
        const int64_t share = std::max<int64_t>(1, all * a.heads[w] / heads);
        v.ctas[w] = (int)std::min(items, share);
        ctas[w] = v.ctas[w];
    }
    return launch_layer(k_heads_vec_grad<T, KIND, AX>, dim3((unsigned)(v.ctas[0] + v.ctas[1])),
                        kHeadsThreads, most, s, 1, a, v, ax);
}

template <class T, int KIND, class AX>
cudaError_t launch_vec_mode(const HeadsArgs &a, const HeadsVecArgs &v, const AX &ax, int mode,
                            int64_t *ctas, cudaStream_t s) {
    if (mode == HEADS_NORM_GRAD) return launch_vec_grad<T, KIND>(a, v, ax, ctas, s);
    // Few rows: one head per item spreads them over the SMs.  Many: four heads
    // share the token's position, cosines, sines and weights (tokens of 32 and 8
    // heads of 128 bf16, one head an item against four: rotation of 64 1.8 and 2.2
    // us, 512 2.8 and 3.6, 1024 4.2 and 3.9, 4096 14.2 and 10.4; norms alike).
    const bool few = (a.rows * (a.heads[0] + a.heads[1]) << v.log_lanes) <
                     2048ll * current_sm_count();
    if (mode == HEADS_ROTATE)
        return few ? launch_vec<T, KIND, HEADS_ROTATE, 1>(a, v, ax, s)
                   : launch_vec<T, KIND, HEADS_ROTATE, 4>(a, v, ax, s);
    return few ? launch_vec<T, KIND, HEADS_NORM, 1>(a, v, ax, s)
               : launch_ring<T, KIND>(a, v, ax, s);
}

template <class T, class AX>
cudaError_t launch_heads(const ebin_heads_plan_s &p, const HeadsArgs &a, const AX &ax, int mode,
                         int64_t *ctas, cudaStream_t s) {
    HeadsVecArgs v;
    int kind = 0;
    if (!heads_vectors(p, a, ax, mode == HEADS_NORM_GRAD, v, kind))
        return launch_any<T>(p, a, ax, mode, ctas, s);
    if (kind == HEADS_HALF) return launch_vec_mode<T, HEADS_HALF>(a, v, ax, mode, ctas, s);
    if (kind == HEADS_PAIRS || kind == HEADS_SPREAD)
        return launch_vec_mode<T, AX::kSeveral ? HEADS_SPREAD : HEADS_PAIRS>(a, v, ax, mode, ctas,
                                                                            s);
    return launch_vec_mode<T, HEADS_ODD>(a, v, ax, mode, ctas, s);
}

template <class AX>
cudaError_t launch_axes(const ebin_heads_plan_s &p, const HeadsArgs &a, const AX &ax, int mode,
                        int64_t *ctas, cudaStream_t s) {
    if (p.at.dtype == EBIN_FLOAT32) return launch_heads<float>(p, a, ax, mode, ctas, s);
    if (p.at.dtype == EBIN_FLOAT16) return launch_heads<__half>(p, a, ax, mode, ctas, s);
    return launch_heads<__nv_bfloat16>(p, a, ax, mode, ctas, s);
}

cudaError_t launch_typed(const ebin_heads_plan_s &p, const HeadsArgs &a, int mode, int64_t *ctas,
                         cudaStream_t s) {
    return p.several ? launch_axes(p, a, p.axes, mode, ctas, s)
                     : launch_axes(p, a, HeadsOne{}, mode, ctas, s);
}

// Elements of the positions' storage.
int64_t positions_span(const ebin_heads_plan_s &p) {
    int64_t n = (p.at.batch - 1) * p.at.position_strides[0] +
                (p.at.tokens - 1) * p.at.position_strides[1] + 1;
    if (p.several) n += (p.axes_count - 1) * p.axes.ps_a;
    return n;
}

HeadsTensor tensor_of(const ebin_heads_attrs &a, int i, const void *p) {
    const ebin_heads_view &v = view_of(a, i);
    return HeadsTensor{p, v.batch, v.token, v.head};
}

// The checks and arguments that both executions share.  in / out: pointers of
// (q, k, dq, dk) and (q_out, k_out).
ebin_status prepare_heads(const ebin_heads_plan_s &p, const void *const in[4],
                          const float *cos, const float *sin, const void *pos, const void *wq,
                          const void *wk, void *const out[2], bool grad, HeadsArgs &a) {
    const ebin_heads_attrs &at = p.at;
    if (at.rotary_dim > 0 && ((at.table_positions > 0 && (!cos || !sin)) ||
                              (at.position_type && !pos)))
        return EBIN_ERR_INVALID_ARG;
    const int inputs = grad ? 4 : 2;
    for (int w = 0; w < 2; ++w) {
        if (heads_of(at, w) == 0) continue;
        if (!in[w] || !out[w] || (grad && !in[2 + w])) return EBIN_ERR_INVALID_ARG;
        const uintptr_t mis = (uintptr_t)in[w] | (uintptr_t)out[w] |
                              (grad ? (uintptr_t)in[2 + w] : 0);
        if (mis % (uintptr_t)p.isz) return EBIN_ERR_INVALID_ARG;
    }
    // every buffer on its own element's boundary
    const uintptr_t ps = at.position_type ? (uintptr_t)type_size((ebin_dtype)at.position_type) : 1;
    if (at.rotary_dim > 0 && (((uintptr_t)cos | (uintptr_t)sin) % 4 || (uintptr_t)pos % ps))
        return EBIN_ERR_INVALID_ARG;
    if (at.norm != EBIN_NORM_NONE &&
        ((uintptr_t)wq | (uintptr_t)wk) % (uintptr_t)type_size(at.dtype_w))
        return EBIN_ERR_INVALID_ARG;
    const int64_t table_bytes = at.table_positions * (at.rotary_dim / 2) * 4;
    const int64_t w_bytes = at.head_dim * type_size(at.dtype_w);
    for (int w = 0; w < 2; ++w) {
        if (heads_of(at, w) == 0) continue;
        const Placed y{(const char *)out[w], &view_of(at, 4 + w), heads_of(at, w), p.span[4 + w]};
        const int64_t y_bytes = y.span * p.isz;
        for (int i = 0; i < inputs; ++i) {
            if (heads_of(at, i) == 0) continue;
            const Placed x{(const char *)in[i], &view_of(at, i), heads_of(at, i), p.span[i]};
            if (i % 2 == w && same_view(at, x, y)) continue;   // in place
            if (heads_share(at, x, y, p.isz)) return EBIN_ERR_ALIAS;
        }
        if (w == 0 && at.k_heads > 0) {
            const Placed y2{(const char *)out[1], &at.k_out, at.k_heads, p.span[5]};
            if (heads_share(at, y, y2, p.isz)) return EBIN_ERR_ALIAS;
        }
        if (at.rotary_dim > 0 && (ranges_overlap(cos, table_bytes, y.p, y_bytes) ||
                                  ranges_overlap(sin, table_bytes, y.p, y_bytes)))
            return EBIN_ERR_ALIAS;
        if (at.norm != EBIN_NORM_NONE &&
            ((wq && ranges_overlap(wq, w_bytes, y.p, y_bytes)) ||
             (wk && ranges_overlap(wk, w_bytes, y.p, y_bytes))))
            return EBIN_ERR_ALIAS;
        if (at.rotary_dim > 0 && at.position_type) {
            const int64_t ps = type_size((ebin_dtype)at.position_type);
            if (ranges_overlap(pos, positions_span(p) * ps, y.p, y_bytes)) return EBIN_ERR_ALIAS;
        }
    }
    a = HeadsArgs{};
    for (int w = 0; w < 2; ++w) {
        a.x[w] = tensor_of(at, w, in[w]);
        a.dy[w] = tensor_of(at, 2 + w, in[2 + w]);
        a.y[w] = tensor_of(at, 4 + w, out[w]);
    }
    a.w[0] = at.norm ? wq : nullptr;
    a.w[1] = at.norm ? wk : nullptr;
    a.cos = cos;
    a.sin = sin;
    a.pos = pos;
    a.ps_b = at.position_strides[0];
    a.ps_t = at.position_strides[1];
    a.table = at.table_positions;
    a.tokens = at.tokens;
    a.rows = p.rows;
    a.heads[0] = at.q_heads;
    a.heads[1] = at.k_heads;
    a.dim = at.head_dim;
    a.half = at.rotary_dim / 2;
    a.pos_size = at.position_type ? (int)type_size((ebin_dtype)at.position_type) : 0;
    a.w_f32 = at.dtype_w == EBIN_FLOAT32;
    a.eps = at.epsilon;
    a.sign = at.gradient ? -1.0f : 1.0f;
    a.status = nullptr;
    return EBIN_OK;
}

// The stream's status word, once nothing is left to refuse (a rotation's
// positions are checked on the device).
bool attach_status(const ebin_heads_plan_s &p, cudaStream_t s, HeadsArgs &a) {
    if (p.at.rotary_dim == 0) return true;
    a.status = stream_status_word(s);
    return a.status != nullptr;
}

}  // namespace

namespace {

// Checks axes and gives each pair its axis and its place among the axis' pairs.
ebin_status axes_of_pairs(const ebin_rotary_axes &x, int rotary_dim, uint8_t *axis,
                          uint16_t *place) {
    if (x.count < 1 || x.count > kHeadsMaxAxes ||
        (x.order != EBIN_AXES_BLOCKS && x.order != EBIN_AXES_DEALT))
        return EBIN_ERR_INVALID_ATTR;
    int64_t pairs = 0;
    int most = 0;
    for (int i = 0; i < x.count; ++i) {
        if (x.sections[i] < 0) return EBIN_ERR_INVALID_ATTR;
        pairs += x.sections[i];
        most = std::max(most, x.sections[i]);
    }
    if (pairs < 1 || pairs > kHeadsMaxDim / 2 || 2 * pairs != rotary_dim)
        return EBIN_ERR_INVALID_ATTR;
    int j = 0;
    auto give = [&](int i, int k) {
        axis[j] = (uint8_t)i;
        place[j++] = (uint16_t)k;
    };
    if (x.order == EBIN_AXES_BLOCKS) {
        for (int i = 0; i < x.count; ++i)
            for (int k = 0; k < x.sections[i]; ++k) give(i, k);
    } else {
        for (int k = 0; k < most; ++k)
            for (int i = 0; i < x.count; ++i)
                if (k < x.sections[i]) give(i, k);
    }
    return EBIN_OK;
}

ebin_status rotary_table(const ebin_rotary_attrs *attrs, const ebin_rotary_axes *axes,
                         int64_t first_position, int64_t positions, float *cos, float *sin,
                         void *stream) {
    if (!attrs || first_position < 0 || positions < 0) return EBIN_ERR_INVALID_ARG;
    const ebin_rotary_attrs &t = *attrs;
    if (t.rotary_dim < 2 || t.rotary_dim > 65536 || t.rotary_dim % 2 != 0 ||
        t.scaling < EBIN_ROTARY_SCALE_NONE || t.scaling > EBIN_ROTARY_SCALE_BY_PARTS ||
        !(t.base > 0) || !std::isfinite(t.base) || !(t.amplitude > 0) ||
        !std::isfinite(t.amplitude))
        return EBIN_ERR_INVALID_ATTR;
    if (t.scaling != EBIN_ROTARY_SCALE_NONE && (!(t.factor >= 1) || !std::isfinite(t.factor)))
        return EBIN_ERR_INVALID_ATTR;
    if (t.scaling == EBIN_ROTARY_SCALE_BASE && t.rotary_dim <= 2) return EBIN_ERR_INVALID_ATTR;
    if (t.scaling == EBIN_ROTARY_SCALE_BY_PARTS &&
        (!(t.trained_length > 0) || !std::isfinite(t.trained_length) ||
         !(t.fast_turns > t.slow_turns) || !std::isfinite(t.fast_turns) ||
         !std::isfinite(t.slow_turns)))
        return EBIN_ERR_INVALID_ATTR;
    TableSections sections{};
    if (axes) {
        // each axis has a base of its own width
        if (t.scaling == EBIN_ROTARY_SCALE_BASE) return EBIN_ERR_INVALID_ATTR;
        uint8_t axis[kHeadsMaxDim / 2];
        const ebin_status st = axes_of_pairs(*axes, t.rotary_dim, axis, sections.place);
        if (st != EBIN_OK) return st;
        for (int j = 0; j < t.rotary_dim / 2; ++j)
            sections.pairs[j] = (uint16_t)axes->sections[axis[j]];
    }
    int64_t n;
    if (!product_fits(positions, t.rotary_dim / 2, &n) ||
        first_position > (int64_t(1) << 53) - positions)
        return EBIN_ERR_INVALID_ARG;
    if (n == 0) return EBIN_OK;
    if (!cos || !sin || ((uintptr_t)cos | (uintptr_t)sin) % 4 != 0) return EBIN_ERR_INVALID_ARG;
    if (ranges_overlap(cos, n * 4, sin, n * 4)) return EBIN_ERR_ALIAS;
    TableArgs a{};
    a.first = first_position;
    a.positions = positions;
    a.half = t.rotary_dim / 2;
    a.scaling = t.scaling;
    const double r = t.rotary_dim;
    a.log2_base = std::log2(t.base);
    if (t.scaling == EBIN_ROTARY_SCALE_BASE) a.log2_base += std::log2(t.factor) * r / (r - 2);
    a.factor = t.factor;
    a.trained = t.trained_length;
    a.slow = t.slow_turns;
    a.fast = t.fast_turns;
    a.amplitude = t.amplitude;
    a.cos = cos;
    a.sin = sin;
    const int64_t grid = std::min<int64_t>(div_up(n, 256), 16ll * current_sm_count());
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        axes ? launch_layer(k_rotary_table<true>, dim3((unsigned)grid), 256, 0, s, 1, a, sections)
             : launch_layer(k_rotary_table<false>, dim3((unsigned)grid), 256, 0, s, 1, a,
                            HeadsOne{});
    return e == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}

}  // namespace

extern "C" ebin_status ebin_rotary_table(const ebin_rotary_attrs *attrs, int64_t first_position,
                                         int64_t positions, float *cos, float *sin,
                                         void *stream) {
    return rotary_table(attrs, nullptr, first_position, positions, cos, sin, stream);
}

extern "C" ebin_status ebin_rotary_table_axes(const ebin_rotary_attrs *attrs,
                                              const ebin_rotary_axes *axes,
                                              int64_t first_position, int64_t positions,
                                              float *cos, float *sin, void *stream) {
    if (!axes) return EBIN_ERR_INVALID_ARG;
    return rotary_table(attrs, axes, first_position, positions, cos, sin, stream);
}

extern "C" ebin_status ebin_heads_plan_create(const ebin_heads_attrs *attrs,
                                              ebin_heads_plan_t *out) {
    if (!attrs || !out) return EBIN_ERR_INVALID_ARG;
    *out = nullptr;
    const ebin_heads_attrs &a = *attrs;
    if (!layer_float(a.dtype)) return EBIN_ERR_UNSUPPORTED_TYPE;
    if ((a.norm != EBIN_NORM_NONE && a.norm != EBIN_NORM_RMS) ||
        (a.layout != EBIN_ROTARY_HALF && a.layout != EBIN_ROTARY_INTERLEAVED) ||
        (a.gradient != 0 && a.gradient != 1))
        return EBIN_ERR_INVALID_ATTR;
    if (a.norm != EBIN_NORM_NONE) {
        if (a.dtype_w != a.dtype && a.dtype_w != EBIN_FLOAT32) return EBIN_ERR_UNSUPPORTED_TYPE;
        if (!(a.epsilon >= 0.0f) || !std::isfinite(a.epsilon)) return EBIN_ERR_INVALID_ATTR;
    }
    if (a.position_type != 0 && a.position_type != EBIN_INT32 && a.position_type != EBIN_INT64)
        return EBIN_ERR_INVALID_ATTR;
    if (a.batch < 0 || a.tokens < 0 || a.q_heads < 0 || a.k_heads < 0 || a.head_dim < 1 ||
        a.head_dim > kHeadsMaxDim || a.table_positions < 0)
        return EBIN_ERR_INVALID_ARG;
    if (a.rotary_dim < 0 || a.rotary_dim > a.head_dim || a.rotary_dim % 2 != 0)
        return EBIN_ERR_INVALID_ATTR;
    int64_t rows, n;
    if (!product_fits(a.batch, a.tokens, &rows) ||
        !product_fits(rows, std::max<int64_t>(1, std::max(a.q_heads, a.k_heads)), &n) ||
        !product_fits(n, a.head_dim, &n) ||
        !product_fits(a.table_positions, std::max(1, a.rotary_dim), &n))
        return EBIN_ERR_INVALID_ARG;
    if (a.position_type) {
        int64_t p0, p1;
        if (a.position_strides[0] < 0 || a.position_strides[1] < 0 ||
            !product_fits(std::max<int64_t>(a.batch, 1) - 1, a.position_strides[0], &p0) ||
            !product_fits(std::max<int64_t>(a.tokens, 1) - 1, a.position_strides[1], &p1) ||
            p0 >= EBIN_MAX_ELEMENTS - p1)
            return EBIN_ERR_INVALID_ARG;
    }
    const bool grad = a.norm != EBIN_NORM_NONE && a.gradient;
    int64_t span[6] = {};
    for (int i = 0; i < 6; ++i) {
        if ((i == 2 || i == 3) && !grad) continue;
        span[i] = heads_span(a, view_of(a, i), heads_of(a, i));
        if (span[i] < 0) return EBIN_ERR_INVALID_ARG;
    }
    for (int i = 4; i < 6; ++i)
        if (span[i] > 0 && !heads_distinct(a, view_of(a, i), heads_of(a, i)))
            return EBIN_ERR_INVALID_ARG;
    auto *p = new (std::nothrow) ebin_heads_plan_s;
    if (!p) return EBIN_ERR_INVALID_ARG;
    p->at = a;
    p->rows = rows;
    p->isz = type_size(a.dtype);
    std::memcpy(p->span, span, sizeof(span));
    p->empty = span[4] == 0 && span[5] == 0;
    if (grad && !p->empty) p->workspace = sizeof(float) * 2 * kHeadsMaxPartials * a.head_dim;
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_heads_plan_create_axes(const ebin_heads_attrs *attrs,
                                                   const ebin_rotary_axes *axes,
                                                   ebin_heads_plan_t *out) {
    if (out) *out = nullptr;
    if (!attrs || !axes || !out) return EBIN_ERR_INVALID_ARG;
    uint8_t axis[kHeadsMaxDim / 2];
    uint16_t place[kHeadsMaxDim / 2];
    ebin_heads_plan_t p = nullptr;
    ebin_status st = ebin_heads_plan_create(attrs, &p);
    if (st == EBIN_OK) st = axes_of_pairs(*axes, attrs->rotary_dim, axis, place);
    if (st == EBIN_OK && !attrs->position_type) st = EBIN_ERR_INVALID_ATTR;
    int64_t far;
    if (st == EBIN_OK && (axes->position_stride < 0 ||
                          !product_fits(kHeadsMaxAxes, axes->position_stride, &far) ||
                          !product_fits(std::max<int64_t>(attrs->batch, 1),
                                        attrs->position_strides[0], &far) ||
                          !product_fits(std::max<int64_t>(attrs->tokens, 1),
                                        attrs->position_strides[1], &far) ||
                          attrs->table_positions > 0x7FFFFFFF))   // rows are kept in 32 bits
        st = EBIN_ERR_INVALID_ARG;
    if (st != EBIN_OK) {
        ebin_heads_plan_release(p);
        return st;
    }
    p->several = true;
    p->axes_count = axes->count;
    p->axes.ps_a = axes->position_stride;
    for (int j = 0; j < attrs->rotary_dim / 2; ++j) {
        p->axes.of_pair[j / 16] |= (uint32_t)axis[j] << (2 * (j % 16));
        p->axes.used |= 1 << axis[j];
    }
    *out = p;
    return EBIN_OK;
}

extern "C" ebin_status ebin_heads_plan_workspace(ebin_heads_plan_t plan, size_t *bytes) {
    if (!plan || !bytes) return EBIN_ERR_INVALID_ARG;
    *bytes = plan->workspace;
    return EBIN_OK;
}

extern "C" void ebin_heads_plan_release(ebin_heads_plan_t plan) { delete plan; }

extern "C" ebin_status ebin_heads_execute(ebin_heads_plan_t plan, const void *q, const void *k,
                                          const float *cos, const float *sin,
                                          const void *positions, const void *wq, const void *wk,
                                          void *q_out, void *k_out, void *stream) {
    if (!plan || (plan->at.norm != EBIN_NORM_NONE && plan->at.gradient))
        return EBIN_ERR_INVALID_ARG;
    if (plan->empty) return EBIN_OK;
    const void *const in[4] = {q, k, nullptr, nullptr};
    void *const out[2] = {q_out, k_out};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    HeadsArgs a;
    const ebin_status st = prepare_heads(*plan, in, cos, sin, positions, wq, wk, out, false, a);
    if (st != EBIN_OK) return st;
    if (!attach_status(*plan, s, a)) return EBIN_ERR_CUDA;
    int64_t ctas[2];
    const int mode = plan->at.norm == EBIN_NORM_NONE ? HEADS_ROTATE : HEADS_NORM;
    return launch_typed(*plan, a, mode, ctas, s) == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}

extern "C" ebin_status ebin_heads_grad_execute(ebin_heads_plan_t plan, const void *dq,
                                               const void *dk, const void *q, const void *k,
                                               const float *cos, const float *sin,
                                               const void *positions, const void *wq,
                                               const void *wk, void *dq_out, void *dk_out,
                                               float *dwq, float *dwk, void *workspace,
                                               size_t workspace_bytes, void *stream) {
    if (!plan || plan->at.norm == EBIN_NORM_NONE || !plan->at.gradient)
        return EBIN_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const ebin_heads_plan_s &p = *plan;
    float *const dw[2] = {dwq, dwk};
    if (p.empty) {   // no rows: the sums are empty
        for (int w = 0; w < 2; ++w)
            if (dw[w] && cudaMemsetAsync(dw[w], 0, sizeof(float) * p.at.head_dim, s) != cudaSuccess)
                return EBIN_ERR_CUDA;
        return EBIN_OK;
    }
    if (!workspace || workspace_bytes < p.workspace || (uintptr_t)workspace % 16 != 0 ||
        ((uintptr_t)dwq | (uintptr_t)dwk) % 4 != 0)
        return EBIN_ERR_INVALID_ARG;
    const void *const in[4] = {q, k, dq, dk};
    void *const out[2] = {dq_out, dk_out};
    HeadsArgs a;
    const ebin_status st = prepare_heads(p, in, cos, sin, positions, wq, wk, out, true, a);
    if (st != EBIN_OK) return st;
    // the small buffers and the workspace overlap nothing that is read or written
    const int64_t dw_bytes = sizeof(float) * p.at.head_dim;
    const int64_t pos_bytes = p.at.position_type && p.at.rotary_dim
        ? positions_span(p) * type_size((ebin_dtype)p.at.position_type) : 0;
    struct Range { const void *p; int64_t n; };
    const int64_t table_bytes = p.at.table_positions * (p.at.rotary_dim / 2) * 4;
    const int64_t w_bytes = p.at.head_dim * type_size(p.at.dtype_w);
    const Range others[11] = {{in[0], p.span[0] * p.isz}, {in[1], p.span[1] * p.isz},
                              {in[2], p.span[2] * p.isz}, {in[3], p.span[3] * p.isz},
                              {out[0], p.span[4] * p.isz}, {out[1], p.span[5] * p.isz},
                              {cos, cos ? table_bytes : 0}, {sin, sin ? table_bytes : 0},
                              {positions, positions ? pos_bytes : 0},
                              {wq, wq ? w_bytes : 0}, {wk, wk ? w_bytes : 0}};
    for (const Range &r : others) {
        if (ranges_overlap(workspace, (int64_t)p.workspace, r.p, r.n)) return EBIN_ERR_ALIAS;
        for (int w = 0; w < 2; ++w)
            if (dw[w] && ranges_overlap(dw[w], dw_bytes, r.p, r.n)) return EBIN_ERR_ALIAS;
    }
    for (int w = 0; w < 2; ++w)
        if (dw[w] && ranges_overlap(dw[w], dw_bytes, workspace, (int64_t)p.workspace))
            return EBIN_ERR_ALIAS;
    if (dwq && dwk && ranges_overlap(dwq, dw_bytes, dwk, dw_bytes)) return EBIN_ERR_ALIAS;

    if (!attach_status(p, s, a)) return EBIN_ERR_CUDA;
    a.partial[0] = static_cast<float *>(workspace);
    a.partial[1] = a.partial[0] + kHeadsMaxPartials * p.at.head_dim;
    int64_t ctas[2];
    if (launch_typed(p, a, HEADS_NORM_GRAD, ctas, s) != cudaSuccess) return EBIN_ERR_CUDA;
    if (!dwq && !dwk) return EBIN_OK;
    const float *partial[2] = {a.partial[0], a.partial[1]};
    const int64_t count[2] = {heads_of(p.at, 0) > 0 ? ctas[0] : 0,
                              heads_of(p.at, 1) > 0 ? ctas[1] : 0};
    return launch_sum_rows(partial, count, dw, p.at.head_dim, 2, s) == cudaSuccess ? EBIN_OK : EBIN_ERR_CUDA;
}
