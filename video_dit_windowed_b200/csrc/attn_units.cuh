// attn_units.cuh -- work units of the differential attention's tcgen05 kernels:
// 128 query rows (forward, dQ) or 128 key rows (dK/dV) of one head of one
// problem, with the ranges of rows they meet.
//
// Windows of at least 128 rows get units of their own: a fixed number of slots
// per window, the last one partly filled, slots past a shorter window's end
// empty, so a unit never meets a neighbouring window's rows. Shorter windows pack
// 128 consecutive rows, which meet the union of their windows, cut by per-row
// masks. Ranges from offset arrays are clamped, so any contents keep every access
// in bounds; a detail row always sees its own key.
#pragma once

#include <stdint.h>

#include "atlas_internal.cuh"
#include "sm100_diff.cuh"

namespace atlas {
namespace units {

constexpr int kRows = 128;   // rows of a unit

struct Shape {
    int32_t N, L, G, heads, batch;   // N, G: rows of ONE problem
    int32_t n_win;
    const int32_t *win_off, *gwin_off;
    int32_t tiles_d, tiles_g;        // 128-row tiles of one problem's rows
    int32_t upw;                     // slots per window; 0: packed; -1: from the offsets
    int32_t n_long;                  // dK/dV: units over global keys, scheduled first
    int32_t n_split;                 // and the parts that each one's queries are cut into
};

// The unit form and counts, the same in every thread of every CTA.
struct Sched {
    int32_t upw, n_dunits, per_prob, n_units;
};

// max_len: the longest window (clamped ranges of the offsets), when upw < 0.
// Slots stay within three times the packed count: offsets that mix a long
// window with many short ones would otherwise make mostly empty units.
__device__ __forceinline__ Sched make_sched(const Shape &p, int32_t max_len) {
    Sched S;
    S.upw = p.upw;
    if (S.upw < 0) {
        const int64_t upw = (max_len + kRows - 1) / kRows;
        const int64_t n = static_cast<int64_t>(p.n_win) * upw;
        const bool ok = max_len >= kRows && n <= 3 * static_cast<int64_t>(p.tiles_d) &&
                        (n + p.tiles_g) * p.batch * p.heads <= INT32_MAX;
        S.upw = ok ? static_cast<int32_t>(upw) : 0;
    }
    const int32_t n_win = p.win_off != nullptr ? p.n_win : (p.L > 0 ? p.N / p.L : 0);
    S.n_dunits = S.upw > 0 ? n_win * S.upw : p.tiles_d;
    S.per_prob = S.n_dunits + p.tiles_g;
    S.n_units = S.per_prob * p.batch * p.heads + (p.n_split - 1) * p.n_long;
    return S;
}

__device__ __forceinline__ int32_t last_below(const int32_t *off, int32_t n, int32_t x) {
    int32_t lo = 0, hi = n - 1;
    while (lo < hi) {
        const int32_t mid = (lo + hi + 1) >> 1;
        if (__ldg(off + mid) <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}
__device__ __forceinline__ int32_t window_of(const Shape &p, int32_t x) {
    return p.win_off == nullptr ? x / p.L : last_below(p.win_off, p.n_win, x);
}
// Row range of window w, which holds row x.
__device__ __forceinline__ int32_t window_start(const Shape &p, int32_t w, int32_t x) {
    return p.win_off == nullptr ? w * p.L : min(max(__ldg(p.win_off + w), 0), x);
}
__device__ __forceinline__ int32_t window_end(const Shape &p, int32_t w, int32_t x) {
    return p.win_off == nullptr ? min(p.N, (w + 1) * p.L)
                                : max(min(__ldg(p.win_off + w + 1), p.N), x + 1);
}
// Rows of window w without a row to hold.
__device__ __forceinline__ void window_rows(const Shape &p, int32_t w, int32_t &lo, int32_t &hi) {
    if (p.win_off == nullptr) {
        lo = w * p.L;
        hi = min(p.N, lo + p.L);
    } else {
        lo = min(max(__ldg(p.win_off + w), 0), p.N);
        hi = min(max(__ldg(p.win_off + w + 1), lo), p.N);
    }
}
__device__ __forceinline__ void global_keys(const Shape &p, int32_t w, int32_t &lo, int32_t &hi) {
    lo = 0;
    hi = p.G;
    if (p.gwin_off != nullptr) {
        lo = min(max(__ldg(p.gwin_off + w), 0), p.G);
        hi = min(max(__ldg(p.gwin_off + w + 1), lo), p.G);
    }
}
// Aligned variant: the window whose global range holds global row g (-1: none).
__device__ __forceinline__ int32_t window_of_global(const Shape &p, int32_t g) {
    const int32_t w = last_below(p.gwin_off, p.n_win, g);
    int32_t lo, hi;
    global_keys(p, w, lo, hi);
    return lo <= g && g < hi ? w : -1;
}

// A work unit: rows r0 .. rend-1 (within problem b) of one head; the streamed
// rows: n_a tiles of TILE detail rows from a0 (up to a_end), then n_b tiles of
// global rows from b0 (up to b_end). win >= 0: all rows meet the same ranges.
// n_a + n_b == 0: an empty slot.
struct Unit {
    int32_t head, b, detail, r0, rend, a0, n_a, a_end, b0, n_b, b_end, win;
    int32_t part;   // of a split unit
};

template <int TILE>
__device__ __forceinline__ int32_t tiles(int32_t n) { return (n + TILE - 1) / TILE; }

// Slot lu of one problem's detail rows, window form; the window's rows are
// streamed and, for queries, its global keys.
template <int TILE>
__device__ __forceinline__ void window_unit(const Shape &p, const Sched &S, int32_t lu,
                                            bool queries, Unit &U) {
    const int32_t w = lu / S.upw, sub = lu - w * S.upw;
    int32_t s, e;
    window_rows(p, w, s, e);
    U.win = w;
    U.r0 = s + sub * kRows;
    U.rend = min(U.r0 + kRows, e);
    U.a0 = s;
    U.a_end = e;
    U.n_a = tiles<TILE>(e - s);
    U.b0 = U.n_b = U.b_end = 0;
    if (queries) {
        global_keys(p, w, U.b0, U.b_end);
        U.n_b = tiles<TILE>(U.b_end - U.b0);
    }
    if (U.rend <= U.r0) U.n_a = U.n_b = 0;
}

// Packed detail rows or global rows, tile lu of one problem (forward, dQ).
template <int TILE>
__device__ __forceinline__ Unit query_unit(const Shape &p, const Sched &S, int32_t u) {
    Unit U;
    U.win = -1;
    U.part = 0;
    U.head = u / (S.per_prob * p.batch);
    int32_t lu = u - U.head * S.per_prob * p.batch;
    U.b = lu / S.per_prob;
    lu -= U.b * S.per_prob;
    U.detail = lu < S.n_dunits;
    if (U.detail && S.upw > 0) {
        window_unit<TILE>(p, S, lu, true, U);
        return U;
    }
    U.r0 = (U.detail ? lu : lu - S.n_dunits) * kRows;
    U.rend = min(U.r0 + kRows, U.detail ? p.N : p.G);
    U.n_a = U.a0 = U.a_end = 0;
    int32_t g0 = 0, g1 = p.G;
    if (U.detail) {
        const int32_t last = U.rend - 1, w0 = window_of(p, U.r0), w1 = window_of(p, last);
        U.a0 = window_start(p, w0, U.r0);
        U.a_end = window_end(p, w1, last);
        U.n_a = tiles<TILE>(U.a_end - U.a0);
        if (p.gwin_off != nullptr) {
            int32_t unused;
            global_keys(p, w0, g0, unused);
            global_keys(p, w1, unused, g1);
            g1 = max(g1, g0);
        }
    }
    U.b0 = g0;
    U.b_end = g1;
    U.n_b = tiles<TILE>(g1 - g0);
    return U;
}

// Key rows and the queries that see them (dK/dV). Units over global keys come
// first: they stream every query that sees them, in n_split parts.
template <int TILE>
__device__ __forceinline__ Unit key_unit(const Shape &p, const Sched &S, int32_t u) {
    Unit U;
    U.win = -1;
    const bool global_keys_unit = u < p.n_long * p.n_split;
    const int32_t span = global_keys_unit ? p.tiles_g : S.n_dunits;
    const int32_t v = global_keys_unit ? u / p.n_split : u - p.n_long * p.n_split;
    U.part = global_keys_unit ? u - v * p.n_split : 0;
    U.head = v / (span * p.batch);
    int32_t lv = v - U.head * span * p.batch;
    U.b = lv / span;
    lv -= U.b * span;
    U.detail = !global_keys_unit;
    if (U.detail && S.upw > 0) {
        window_unit<TILE>(p, S, lv, false, U);
        return U;
    }
    U.r0 = lv * kRows;
    U.rend = min(U.r0 + kRows, U.detail ? p.N : p.G);
    const int32_t last = U.rend - 1;
    U.b0 = U.b_end = U.n_b = 0;
    if (U.detail) {
        const int32_t w0 = window_of(p, U.r0), w1 = window_of(p, last);
        U.a0 = window_start(p, w0, U.r0);
        U.a_end = window_end(p, w1, last);
    } else {
        int32_t q0 = 0, q1 = p.N;
        if (p.gwin_off != nullptr && p.N > 0) {
            // windows whose global ranges hold the first and the last key
            int32_t wa = -1, wb = -1;
            for (int32_t g = U.r0; g <= last && wa < 0; ++g) wa = window_of_global(p, g);
            for (int32_t g = last; g >= U.r0 && wb < 0; --g) wb = window_of_global(p, g);
            if (wa < 0) {
                q0 = q1 = 0;
            } else {
                int32_t unused;
                window_rows(p, wa, q0, unused);
                window_rows(p, wb, unused, q1);
                q1 = max(q1, q0);
            }
        }
        U.a0 = q0;
        U.a_end = q1;
        U.b_end = p.G;
        U.n_b = tiles<TILE>(p.G);
    }
    U.n_a = tiles<TILE>(U.a_end - U.a0);
    if (!U.detail && p.n_split > 1) {
        // tiles [t0, t1) of the n_a + n_b
        const int32_t n = U.n_a + U.n_b;
        const int32_t t0 = static_cast<int32_t>(static_cast<int64_t>(n) * U.part / p.n_split);
        const int32_t t1 = static_cast<int32_t>(static_cast<int64_t>(n) * (U.part + 1) / p.n_split);
        const int32_t a = max(min(t1, U.n_a) - min(t0, U.n_a), 0);
        U.a0 += min(t0, U.n_a) * TILE;
        U.b0 += max(t0 - U.n_a, 0) * TILE;
        U.n_a = a;
        U.n_b = t1 - t0 - a;
    }
    return U;
}

// Streamed tile j of U: its first row (within the problem), and the rows behind
// it that the unit meets.
template <int TILE>
__device__ __forceinline__ int32_t tile_row(const Unit &U, int32_t j) {
    return j < U.n_a ? U.a0 + j * TILE : U.b0 + (j - U.n_a) * TILE;
}
template <int TILE>
__device__ __forceinline__ int32_t tile_rows(const Unit &U, int32_t j) {
    return (j < U.n_a ? U.a_end : U.b_end) - tile_row<TILE>(U, j);
}

// The rows that row r of unit U may meet: detail [da, db), global [ga, gb).
__device__ __forceinline__ void query_ranges(const Shape &p, const Unit &U, int32_t r, int32_t &da,
                                             int32_t &db, int32_t &ga, int32_t &gb) {
    da = U.a0;
    db = U.a_end;
    ga = U.b0;
    gb = U.b_end;
    if (!U.detail || U.win >= 0) return;
    const int32_t x = min(r, p.N - 1), w = window_of(p, x);
    da = window_start(p, w, x);
    db = window_end(p, w, x);
    global_keys(p, w, ga, gb);
}
__device__ __forceinline__ void key_ranges(const Shape &p, const Unit &U, int32_t r, int32_t &da,
                                           int32_t &db, int32_t &ga, int32_t &gb) {
    da = U.a0;
    db = U.a_end;
    ga = U.b0;
    gb = U.b_end;
    if (U.win >= 0) return;
    if (U.detail) {
        const int32_t x = min(r, p.N - 1), w = window_of(p, x);
        da = window_start(p, w, x);
        db = window_end(p, w, x);
    } else if (p.gwin_off != nullptr) {
        const int32_t w = p.N > 0 ? window_of_global(p, min(r, p.G - 1)) : -1;
        da = db = 0;
        if (w >= 0) window_rows(p, w, da, db);
    }
}

// Whether the queries of detail key r's window see no global key.
__device__ __forceinline__ bool no_global_key(const Shape &p, const Unit &U, int32_t r) {
    int32_t ga, gb;
    global_keys(p, U.win >= 0 ? U.win : window_of(p, min(r, p.N - 1)), ga, gb);
    return ga == gb;
}

// The fields that the tile functions above read, as uniform values of a
// converged warp.
__device__ __forceinline__ void make_uniform(Unit &U) {
    U.a0 = ptx::uniform(U.a0);
    U.a_end = ptx::uniform(U.a_end);
    U.n_a = ptx::uniform(U.n_a);
    U.b0 = ptx::uniform(U.b0);
    U.b_end = ptx::uniform(U.b_end);
    U.n_b = ptx::uniform(U.n_b);
}

// The longest window of the offsets (clamped), into *out (0 before), by all
// threads of a CTA; the caller synchronises.
__device__ __forceinline__ void longest_window(const Shape &p, int32_t *out) {
    int32_t m = 0;
    for (int32_t w = threadIdx.x; w < p.n_win; w += blockDim.x) {
        int32_t s, e;
        window_rows(p, w, s, e);
        m = max(m, e - s);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) atomicMax(out, m);
}

// Host: the shape of a call and its units (an upper bound when the kernel
// chooses the form from the offsets, at least one per SM). False: too many.
inline bool make_shape(const AttnArgs &a, int sm_count, Shape *out, int64_t *n_units) {
    Shape p{};
    p.N = static_cast<int32_t>(a.n_detail);
    p.L = static_cast<int32_t>(a.n_detail > 0 ? a.window_len : 1);
    p.G = static_cast<int32_t>(a.n_global);
    p.heads = a.heads;
    p.batch = static_cast<int32_t>(a.batch);
    p.win_off = a.win_off;
    p.gwin_off = a.gwin_off;
    p.n_win = static_cast<int32_t>(a.win_off ? a.n_win : a.n_gwin);
    p.tiles_d = static_cast<int32_t>((a.n_detail + kRows - 1) / kRows);
    p.tiles_g = static_cast<int32_t>((a.n_global + kRows - 1) / kRows);
    const int64_t cells = a.batch * a.heads;
    int64_t n = (static_cast<int64_t>(p.tiles_d) + p.tiles_g) * cells;
    if (n > INT32_MAX) return false;
    if (p.N == 0) {
        p.upw = 0;
    } else if (p.win_off != nullptr) {
        p.upw = -1;
        n = n > sm_count ? n : sm_count;
    } else {
        p.upw = p.L >= kRows ? (p.L + kRows - 1) / kRows : 0;
        if (p.upw > 0) n = (static_cast<int64_t>(p.N / p.L) * p.upw + p.tiles_g) * cells;
        if (n > INT32_MAX) return false;
    }
    p.n_long = static_cast<int32_t>(p.tiles_g * cells);
    p.n_split = 1;
    *out = p;
    *n_units = n;
    return true;
}

}  // namespace units
}  // namespace atlas
