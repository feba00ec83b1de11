// The row kernels of the norms around a block, one pair of element types in each
// compilation (-DEBIN_DT=0 .. 4).
#include "ebin_block_unit.cuh"

namespace ebin {

#if EBIN_DT == 0
using T = float;
using S = float;
#elif EBIN_DT == 1
using T = __half;
using S = __half;
#elif EBIN_DT == 2
using T = __nv_bfloat16;
using S = __nv_bfloat16;
#elif EBIN_DT == 3
using T = __half;
using S = float;
#else
using T = __nv_bfloat16;
using S = float;
#endif


// Shared memory of an SM, what a CTA takes of it besides its rows, and the most
// that a CTA's rows may take.
constexpr size_t kSmSmem = 228 * 1024, kCtaSmem = 3 * 1024, kRowsSmem = 224 * 1024;

template <auto KERNEL>
static cudaError_t launch_rows(const BlockArgs &a, const RowsGeom &g, int64_t grid, size_t smem,
                        cudaStream_t s) {
    const cudaError_t e = allow_smem<KERNEL>(kRowsSmem);
    if (e != cudaSuccess) return e;
    return launch_layer(KERNEL, dim3((unsigned)grid), g.warps * g.teams * 32, smem, s, 1, a, g);
}

// Rows in flight: up to three, where the CTAs that an SM holds by their threads
// leave room beside `more` bytes; 0: not even one fits.
static int rows_slots(size_t row_bytes, size_t more, int ctas) {
    const size_t share = kSmSmem / ctas - kCtaSmem;
    int slots = share > more ? (int)((share - more) / row_bytes) : 0;
    if (slots < 1 && row_bytes + more <= kRowsSmem) slots = 1;
    return std::min(slots, 3);
}

static RowsGeom rows_geom(const BlockArgs &a, int chunks, int vpt) {
    RowsGeom g{};
    g.warps = (int)div_up(chunks, vpt);
    g.joins = 1;
    while (g.joins < g.warps) g.joins *= 2;
    g.teams = g.warps == 1 ? 4 : 1;
    g.slots = 1;
    g.gate = fast_div((uint32_t)a.gate_rows);
    g.mod = fast_div((uint32_t)a.mod_rows);
    return g;
}


// Bytes of a CTA's rows of a tensor of E's in shared memory.
template <class E> static size_t unit_bytes(const RowsGeom &g, int vpt, bool vec) {
    using Lane = UnitLane<T, S, true>;
    return vec ? (size_t)vpt * Lane::vectors<E>() * kUnitThreads * 16
               : (size_t)vpt * g.warps * g.teams * Lane::buffer<E>();
}

#define EBIN_CAT(a, b) a##b
#define EBIN_NAME(f, dt) EBIN_CAT(f, dt)

// Whether a CTA an SM takes a unit: rows of at most 8192 columns, and enough of them in a
// unit.  Forward two for each team and two waves of a row a CTA at least (a step of few
// rows spreads over more SMs a row a team); a gradient, whose units each leave sums, half
// its teams' unless there is but one group.
static bool cta_takes(const BlockArgs &a, int chunks, int vpt, bool grad) {
    if (a.n > kUnitColumns) return false;
    const int64_t teams = kUnitWarps / div_up(chunks, vpt);
    return grad ? a.groups == 1 || 2 * a.cta.rows >= teams
                : a.rows > 304 && a.cta.rows >= 2 * teams;
}

// Its geometry, but for what lies in shared memory.
static RowsGeom unit_geom(const BlockArgs &a, int chunks, int vpt) {
    RowsGeom g = rows_geom(a, chunks, vpt);
    g.teams = kUnitWarps / g.warps;
    g.units = a.groups * a.cta.parts;
    g.table = g.warps * vpt * 64;
    return g;
}

cudaError_t EBIN_NAME(launch_block_rows_, EBIN_DT)(const BlockArgs &a, bool vec, int64_t *parts,
                                                   cudaStream_t s) {
    *parts = 0;
    const int chunks = (int)div_up(a.n, kChunk);
    if (chunks > 128) return cudaSuccess;
    const bool layer = a.post == EBIN_NORM_LAYER || a.pre == EBIN_NORM_LAYER;
    const int s_vectors = sizeof(S) == 4 ? 2 : 1, t_vectors = sizeof(T) == 4 ? 2 : 1;
    // Off the vectors the shifts pay for 16-bit rows of more than 2048 columns ([8191,4097]
    // bf16 122 us, a team a row 198; [20000,1543] f16 with dropout 151 and 136; [4095,2050] f32
    // 44 and 36).
    constexpr bool shifts = sizeof(S) == 2;
    if ((vec || (shifts && chunks > 8)) && cta_takes(a, chunks, kUnitVpt, false)) {
        RowsGeom g = unit_geom(a, chunks, kUnitVpt);
        const bool scaled = a.branch_scale != 1.0f || a.drop.least;
        if (a.y && (a.gate || a.w_post || a.b_post || scaled)) g.tables |= TABLE_Y;
        if (a.b_post) g.tables |= TABLE_Y_ADD;
        if (a.z && (a.scale || a.w_pre)) g.tables |= TABLE_H;
        if (a.z && (a.shift || a.b_pre)) g.tables |= TABLE_H_ADD;
        const size_t tables = 16 * (size_t)g.table * __builtin_popcount(g.tables);
        const size_t row = unit_bytes<S>(g, kUnitVpt, vec) +
                           (a.y ? unit_bytes<T>(g, kUnitVpt, vec) : 0);
        g.slot_bytes = (int)row;
        g.slots = rows_slots(row, tables, 1);
        if (g.slots > 0) {
            *parts = a.cta.parts;
            const size_t smem = tables + g.slots * row;
            if constexpr (shifts)
                if (!vec) return launch_rows<k_block_unit<T, S, true, true>>(a, g, g.units, smem, s);
            return layer ? launch_rows<k_block_unit<T, S, true, false>>(a, g, g.units, smem, s)
                         : launch_rows<k_block_unit<T, S, false, false>>(a, g, g.units, smem, s);
        }
    }
    const int vpt = chunks > 32 ? 4 : 1;
    RowsGeom g = rows_geom(a, chunks, vpt);
    const int threads = g.warps * g.teams * 32;
    const int per_sm = std::min(1024 / threads, 16);
    size_t smem = 0;
    if (vec) {
        const size_t row = (size_t)threads * vpt * 16 * (s_vectors + t_vectors);
        g.slots = rows_slots(row, 0, per_sm);
        smem = g.slots * row;
        vec = g.slots > 0;   // rows too wide for shared memory are read where they lie
    }
    const int64_t grid = std::min<int64_t>(div_up(a.rows, g.teams),
                                           (int64_t)per_sm * current_sm_count());
    *parts = 1;
#define EBIN_ROWS(VPT)                                                                       \
    if (!vec) return launch_rows<k_block_rows<T, S, VPT, false, true>>(a, g, grid, smem, s);  \
    return layer ? launch_rows<k_block_rows<T, S, VPT, true, true>>(a, g, grid, smem, s)      \
                 : launch_rows<k_block_rows<T, S, VPT, true, false>>(a, g, grid, smem, s)
    if (vpt == 1) { EBIN_ROWS(1); }
    EBIN_ROWS(4);
#undef EBIN_ROWS
}

cudaError_t EBIN_NAME(launch_block_rows_grad_, EBIN_DT)(const BlockArgs &a, bool vec, int64_t *parts,
                                                        cudaStream_t s) {
    *parts = 0;
    const int chunks = (int)div_up(a.n, kChunk);
    if (chunks > 64) return cudaSuccess;
    const bool full = unit_grad_full(a.post, a.pre, a.need);
    const bool has[2] = {a.scale || a.w_pre,
                         a.gate || a.w_post || a.branch_scale != 1.0f || a.drop.least};
    const bool there[4] = {a.x != nullptr, a.dz != nullptr, a.dh != nullptr, a.y != nullptr};
    const int s_vectors = sizeof(S) == 4 ? 2 : 1, t_vectors = sizeof(T) == 4 ? 2 : 1;
    const bool post = a.post != EBIN_NORM_NONE;
    const int unit_vpt = !full ? kUnitGradVpt<false, false>
                       : post ? kUnitGradVpt<true, true> : kUnitGradVpt<true, false>;
    if (a.pre != EBIN_NORM_NONE && div_up(chunks, unit_vpt) <= kUnitWarps &&
        cta_takes(a, chunks, unit_vpt, true)) {
        RowsGeom g = unit_geom(a, chunks, unit_vpt);
        const size_t tables = 2 * 16 * (size_t)g.table;
        const size_t row = 2 * unit_bytes<S>(g, unit_vpt, vec) +
                           (a.y ? 2 : 1) * unit_bytes<T>(g, unit_vpt, vec);
        g.slot_bytes = (int)row;
        g.slots = rows_slots(row, tables, 1);
        if (g.slots > 0) {
            // the teams' sums at the end
            const size_t sums = g.teams > 1 ? (size_t)(full ? 4 : 2) * unit_vpt *
                                                  32 * g.warps * 32 : 0;
            const size_t smem = std::max(tables + g.slots * row, sums);
            *parts = a.cta.parts;
#define EBIN_UNIT(FULL, POST)                                                                \
    return vec ? launch_rows<k_block_unit_grad<T, S, FULL, POST, false>>(a, g, g.units, smem, s) \
               : launch_rows<k_block_unit_grad<T, S, FULL, POST, true>>(a, g, g.units, smem, s)
            if (full && post) { EBIN_UNIT(true, true); }
            if (full) { EBIN_UNIT(true, false); }
            if (post) { EBIN_UNIT(false, true); }
            EBIN_UNIT(false, false);
#undef EBIN_UNIT
        }
    }
    const int vpt = chunks > 32 ? 4 : 2;
    RowsGeom g = rows_geom(a, chunks, vpt);
    g.units = a.groups * a.team.parts;
    const int threads = g.warps * g.teams * 32;
    for (int f = 0; f < 2; ++f) {
        g.factor[f] = has[f] ? g.factors : -1;
        if (has[f]) g.factors += 2 * vpt;
    }
    const size_t factors = (size_t)threads * 16 * g.factors;
    size_t smem = factors;
    if (vec) {
        // As much of a row as fits beside the factors, what is read most often first: all of it
        // but for the widest ([2048,16384] bf16 with norms on both sides: h and dz, 196 us; without
        // shared memory, element by element, 560).
        const int order[4] = {0, 1, 3, 2};
        for (int k : order) {
            const int more = vpt * (k % 2 ? t_vectors : s_vectors);
            const bool fits = (size_t)(g.vectors + more) * 16 * threads + factors <= kRowsSmem;
            g.at[k] = there[k] && fits ? g.vectors : -1;
            if (g.at[k] >= 0) g.vectors += more;
        }
        const size_t row = (size_t)g.vectors * 16 * threads;
        if (row > 0)
            g.slots = rows_slots(row, factors, std::min(std::max(1, 512 / threads), 16));
        smem += g.slots * row;
    }
    const int64_t grid = div_up(g.units, g.teams);
    *parts = a.team.parts;
    if (vpt == 4)
        return vec ? launch_rows<k_block_rows_grad<T, S, 4, true, true>>(a, g, grid, smem, s)
                   : launch_rows<k_block_rows_grad<T, S, 4, false, true>>(a, g, grid, smem, s);
    return vec ? launch_rows<k_block_rows_grad<T, S, 2, true, false>>(a, g, grid, smem, s)
               : launch_rows<k_block_rows_grad<T, S, 2, false, false>>(a, g, grid, smem, s);
}

}  // namespace ebin
