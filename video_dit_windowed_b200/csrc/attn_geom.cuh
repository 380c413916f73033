// attn_geom.cuh -- which keys a query row sees, and which queries see a key:
// the windows, global tokens and aligned ranges of atlas_attn_layout, for the
// differential attention's row-sum and fp32 kernels. All counts are per problem. Ranges from
// offset arrays are clamped, so any contents keep every access in bounds; a
// detail row always sees its own key.
#pragma once

#include <stdint.h>

#include "atlas_internal.cuh"

namespace atlas {

struct AttnGeom {
    int64_t N, L, G, batch, n_win;
    int32_t heads;
    const int32_t *win_off, *gwin_off;
};

inline AttnGeom attn_geom_of(const AttnArgs &a) {
    AttnGeom g;
    g.N = a.n_detail;
    g.L = a.n_detail > 0 ? a.window_len : 1;
    g.G = a.n_global;
    g.batch = a.batch;
    g.n_win = a.win_off ? a.n_win : a.n_gwin;
    g.heads = a.heads;
    g.win_off = a.win_off;
    g.gwin_off = a.gwin_off;
    return g;
}

namespace geo {

__device__ __forceinline__ int64_t clamp64(int64_t x, int64_t lo, int64_t hi) {
    return x < lo ? lo : (x > hi ? hi : x);
}

// The last of n offsets that is <= x.
__device__ __forceinline__ int64_t last_below(const int32_t *off, int64_t n, int64_t x) {
    int64_t a = 0, c = n - 1;
    while (a < c) {
        const int64_t mid = (a + c + 1) / 2;
        if (__ldg(off + mid) <= x) a = mid; else c = mid - 1;
    }
    return a;
}

// The window of detail row x and its rows [lo, hi).
__device__ __forceinline__ int64_t window_at(const AttnGeom &g, int64_t x, int64_t &lo,
                                             int64_t &hi) {
    if (g.win_off == nullptr) {
        const int64_t w = x / g.L;
        lo = w * g.L;
        hi = lo + g.L;
        return w;
    }
    const int64_t w = last_below(g.win_off, g.n_win, x);
    lo = clamp64(__ldg(g.win_off + w), 0, x);
    hi = clamp64(__ldg(g.win_off + w + 1), x + 1, g.N);
    return w;
}

// Global keys [lo, hi) of the queries of window w.
__device__ __forceinline__ void global_keys(const AttnGeom &g, int64_t w, int64_t &lo,
                                            int64_t &hi) {
    lo = 0;
    hi = g.G;
    if (g.gwin_off != nullptr) {
        lo = clamp64(__ldg(g.gwin_off + w), 0, g.G);
        hi = clamp64(__ldg(g.gwin_off + w + 1), lo, g.G);
    }
}

// Detail queries [lo, hi) that see global key x.
__device__ __forceinline__ void global_queries(const AttnGeom &g, int64_t x, int64_t &lo,
                                               int64_t &hi) {
    lo = 0;
    hi = g.N;
    if (g.gwin_off == nullptr || g.N == 0) return;
    const int64_t w = last_below(g.gwin_off, g.n_win, x);
    int64_t g0, g1;
    global_keys(g, w, g0, g1);
    lo = hi = 0;
    if (x < g0 || x >= g1) return;
    lo = g.win_off ? clamp64(__ldg(g.win_off + w), 0, g.N) : w * g.L;
    hi = g.win_off ? clamp64(__ldg(g.win_off + w + 1), lo, g.N) : lo + g.L;
}

// Row `row` of the stacked tensors, detail rows of all problems first.
struct RowAt {
    bool detail;
    int64_t b, local, row;   // problem; row in it; row in its tensor
};
__device__ __forceinline__ RowAt row_at(const AttnGeom &g, int64_t row) {
    RowAt r;
    const int64_t nd = g.batch * g.N;
    r.detail = row < nd;
    r.row = r.detail ? row : row - nd;
    r.b = r.row / (r.detail ? g.N : g.G);
    r.local = r.row - r.b * (r.detail ? g.N : g.G);
    return r;
}

}  // namespace geo
}  // namespace atlas
