// diff_attn_simt.cu -- differential attention and its backward pass, fp32 I/O,
// exact fp32 products on the FMA pipe (formulas: diff_attn.cu).
//
// A block of 512 threads takes 64 rows of one head of one problem (queries, or
// keys for dK/dV) and streams the rows they meet in tiles of 64 through shared
// memory. Warp ty owns rows 4 ty .. 4 ty + 3: lane tx columns tx and tx + 32 of
// their scores, and D / 32 columns of their accumulators. Scores, weights and
// accumulators stay in registers; the weights pass through shared memory within
// the warp whose rows they are. The row pitch of D + 4 floats spreads the 32 rows
// that a warp reads side by side over the banks. Bound by latency, not by the FMA
// pipe or shared memory (2 x 3 heads of 3,600 + 1,000 rows, D = 128, training: 3.7
// ms; 256 threads with 4 x 4 scores each took 4.43 ms at 50 % issue, 4 x 2 over
// 32-row tiles 5.37 ms). dK/dV: the queries of a block over global keys are cut into
// parts where such blocks are few and long (diff_attn.cu, diff_split_plan; 2 heads of
// 10,672 rows and 6 global ones, D = 128, training: 3,814 us uncut, 378 cut).
// Masked pairs get weight 0. 0 * NaN would still reach a row, so streamed rows
// that enter a product by their weight are zeroed where they hold a non-finite
// value, and pairs that do see such a row get the weight NaN.
#include "attn_geom.cuh"

namespace atlas {
namespace {

constexpr int kThreads = 512;
constexpr int kRows = 64;     // rows of a block
constexpr int kTile = 64;     // streamed rows of a tile
constexpr int kJ = kTile / 32;   // score columns of a thread
constexpr int kPitchW = kTile + 4;
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float nan_f() { return __uint_as_float(0x7fffffffu); }

// The block's rows [r0, rend) of one problem, and the streamed rows: detail [a0,
// a1), then global [b0, b1), cut into tiles.
struct Span {
    int head;
    int64_t b;
    bool detail;
    int64_t r0, rend, a0, a1, b0, b1;
    int na, nb;
    __device__ __forceinline__ void cut() {
        na = static_cast<int>((a1 - a0 + kTile - 1) / kTile);
        nb = static_cast<int>((b1 - b0 + kTile - 1) / kTile);
    }
    __device__ __forceinline__ int64_t row(int j) const {
        return j < na ? a0 + static_cast<int64_t>(j) * kTile
                      : b0 + static_cast<int64_t>(j - na) * kTile;
    }
    __device__ __forceinline__ int rows(int j) const {
        const int64_t n = (j < na ? a1 : b1) - row(j);
        return n < kTile ? static_cast<int>(n) : kTile;
    }
};

// Blocks of global rows come first, in `parts` each: over keys they are the longest.
__device__ __forceinline__ Span rows_of_block(const AttnGeom &g, int parts, int &part) {
    Span s;
    s.head = blockIdx.y;
    const int64_t td = (g.N + kRows - 1) / kRows, tg = (g.G + kRows - 1) / kRows;
    const int64_t n_long = g.batch * tg * parts, x = blockIdx.x;
    s.detail = x >= n_long;
    const int64_t v = s.detail ? x - n_long : x / parts, span = s.detail ? td : tg;
    part = s.detail ? 0 : static_cast<int>(x - v * parts);
    s.b = v / span;
    s.r0 = (v - s.b * span) * kRows;
    const int64_t n = s.detail ? g.N : g.G;
    s.rend = s.r0 + kRows < n ? s.r0 + kRows : n;
    return s;
}

// Queries: the union of the rows' windows and global keys.
__device__ __forceinline__ Span query_span(const AttnGeom &g) {
    int unused_part;
    Span s = rows_of_block(g, 1, unused_part);
    s.a0 = s.a1 = s.b0 = 0;
    s.b1 = g.G;
    if (s.detail) {
        int64_t unused;
        const int64_t w0 = geo::window_at(g, s.r0, s.a0, unused);
        const int64_t w1 = geo::window_at(g, s.rend - 1, unused, s.a1);
        geo::global_keys(g, w0, s.b0, unused);
        geo::global_keys(g, w1, unused, s.b1);
        if (s.b1 < s.b0) s.b1 = s.b0;
    }
    s.cut();
    return s;
}

// Keys: the queries that see them, or (of global keys) one part of their tiles.
__device__ __forceinline__ Span key_span(const AttnGeom &g, int parts, int &part) {
    Span s = rows_of_block(g, parts, part);
    s.b0 = s.b1 = 0;
    int64_t lo, hi;
    if (s.detail) {
        geo::window_at(g, s.r0, s.a0, hi);
        geo::window_at(g, s.rend - 1, lo, s.a1);
    } else {
        s.a0 = s.a1 = 0;
        s.b1 = g.G;
        bool any = false;
        if (g.gwin_off == nullptr) {
            s.a1 = g.N;
        } else {
            for (int64_t x = s.r0; x < s.rend; ++x) {
                geo::global_queries(g, x, lo, hi);
                if (lo >= hi) continue;
                s.a0 = any && s.a0 < lo ? s.a0 : lo;
                s.a1 = any && s.a1 > hi ? s.a1 : hi;
                any = true;
            }
        }
    }
    s.cut();
    if (!s.detail && parts > 1) {
        const int64_t n = s.na + s.nb;
        const int t0 = static_cast<int>(n * part / parts), t1 = static_cast<int>(n * (part + 1) / parts);
        const int a = max(min(t1, s.na) - min(t0, s.na), 0);
        s.a0 += static_cast<int64_t>(min(t0, s.na)) * kTile;
        s.b0 += static_cast<int64_t>(max(t0 - s.na, 0)) * kTile;
        s.na = a;
        s.nb = t1 - t0 - a;
    }
    return s;
}

// The streamed rows a row of the block meets, relative to nothing: [da, db)
// detail, [ga, gb) global; empty past the block's rows.
struct Sees {
    int da, db, ga, gb;
    __device__ __forceinline__ bool at(bool detail, int64_t x) const {
        return detail ? x >= da && x < db : x >= ga && x < gb;
    }
};
__device__ __forceinline__ Sees query_sees(const AttnGeom &g, const Span &s, int64_t r) {
    Sees v{0, 0, 0, 0};
    if (r >= s.rend) return v;
    int64_t lo = 0, hi = 0, g0 = 0, g1 = g.G;
    if (s.detail) geo::global_keys(g, geo::window_at(g, r, lo, hi), g0, g1);
    v.da = static_cast<int>(lo);
    v.db = static_cast<int>(hi);
    v.ga = static_cast<int>(g0);
    v.gb = static_cast<int>(g1);
    return v;
}
__device__ __forceinline__ Sees key_sees(const AttnGeom &g, const Span &s, int64_t r) {
    Sees v{0, 0, 0, 0};
    if (r >= s.rend) return v;
    int64_t lo, hi;
    if (s.detail) geo::window_at(g, r, lo, hi);
    else geo::global_queries(g, r, lo, hi);
    v.da = static_cast<int>(lo);
    v.db = static_cast<int>(hi);
    v.gb = s.detail ? 0 : static_cast<int>(g.G);
    return v;
}

__device__ __forceinline__ bool finite4(const float4 &v) {
    return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w);
}

// ROWS rows of D floats into shared memory, rows past `n` as zeros. SCRUB: rows
// with a non-finite value as zeros too, and marked in bad.
template <int HD, int ROWS, bool SCRUB>
__device__ __forceinline__ void load_rows(float *dst, const float *src, int64_t stride, int n,
                                          uint8_t *bad) {
    constexpr int kLanes = HD / 4, kPer = 32 / kLanes;   // lanes of a row, rows of a warp
    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    const int sub = lane / kLanes, c = (lane % kLanes) * 4;
#pragma unroll 4
    for (int r = warp * kPer + sub; r < ROWS; r += kThreads / 32 * kPer) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (r < n) v = __ldg(reinterpret_cast<const float4 *>(src + r * stride + c));
        if (SCRUB) {
            uint32_t any = __ballot_sync(0xffffffffu, !finite4(v));
            if (kPer > 1) any = (any >> (sub * kLanes)) & ((1u << (kLanes % 32)) - 1u);
            if (any) v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c == 0) bad[r] = any != 0;
        }
        *reinterpret_cast<float4 *>(dst + r * (HD + 4) + c) = v;
    }
}

__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float s) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, s))));
}

// s[i][j] = <a row 4 ty + i, b row tx + 32 j> over channels [d0, d1).
template <int HD>
__device__ __forceinline__ void scores(const float *a, const float *b, int d0, int d1,
                                       float (&s)[4][kJ]) {
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < kJ; ++j) s[i][j] = 0.f;
#pragma unroll 2
    for (int d = d0; d < d1; d += 4) {
        float4 x[4], y[kJ];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const float4 *>(a + (4 * ty + i) * (HD + 4) + d);
#pragma unroll
        for (int j = 0; j < kJ; ++j)
            y[j] = *reinterpret_cast<const float4 *>(b + (tx + 32 * j) * (HD + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < kJ; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
    }
}

// An accumulator of the thread's 4 rows: W = D / 32 columns from W tx on. The
// second map's channels are those of lanes 16 to 31.
template <int W>
struct alignas(4 * W) Cols {
    float x[W];
};
template <int HD>
struct Acc {
    static constexpr int kW = HD / 32;
    float v[4][kW];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < kW; ++c) v[i][c] = 0.f;
    }
    __device__ __forceinline__ void scale(int i, float f) {
#pragma unroll
        for (int c = 0; c < kW; ++c) v[i][c] *= f;
    }
};

// acc += w b: w [64][kPitchW] (weights of the thread's rows), b [64][D + 4].
template <int HD>
__device__ __forceinline__ void weighted(Acc<HD> &acc, const float *w, const float *b) {
    constexpr int W = Acc<HD>::kW;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        Cols<W> y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = *reinterpret_cast<const Cols<W> *>(b + (k + e) * (HD + 4) + W * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = *reinterpret_cast<const float4 *>(w + (4 * ty + i) * kPitchW + k);
#pragma unroll
            for (int c = 0; c < W; ++c)
                acc.v[i][c] = fmaf(x.w, y[3].x[c],
                                   fmaf(x.z, y[2].x[c],
                                        fmaf(x.y, y[1].x[c], fmaf(x.x, y[0].x[c], acc.v[i][c]))));
        }
    }
}

// Both maps' accumulators over the same b: each row of b is read once.
template <int HD>
__device__ __forceinline__ void weighted2(Acc<HD> &a0, Acc<HD> &a1, const float *w0,
                                          const float *w1, const float *b) {
    constexpr int W = Acc<HD>::kW;
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        Cols<W> y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            y[e] = *reinterpret_cast<const Cols<W> *>(b + (k + e) * (HD + 4) + W * tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x0 = *reinterpret_cast<const float4 *>(w0 + (4 * ty + i) * kPitchW + k);
            const float4 x1 = *reinterpret_cast<const float4 *>(w1 + (4 * ty + i) * kPitchW + k);
#pragma unroll
            for (int c = 0; c < W; ++c) {
                a0.v[i][c] = fmaf(x0.w, y[3].x[c],
                                  fmaf(x0.z, y[2].x[c],
                                       fmaf(x0.y, y[1].x[c], fmaf(x0.x, y[0].x[c], a0.v[i][c]))));
                a1.v[i][c] = fmaf(x1.w, y[3].x[c],
                                  fmaf(x1.z, y[2].x[c],
                                       fmaf(x1.y, y[1].x[c], fmaf(x1.x, y[0].x[c], a1.v[i][c]))));
            }
        }
    }
}

template <int HD>
__device__ __forceinline__ void store(float *out, const Acc<HD> &acc, int i, float f0, float f1) {
    constexpr int W = Acc<HD>::kW;
    const int tx = threadIdx.x % 32;
    Cols<W> v;
#pragma unroll
    for (int c = 0; c < W; ++c) v.x[c] = acc.v[i][c] * (tx >= 16 ? f1 : f0);
    *reinterpret_cast<Cols<W> *>(out + W * tx) = v;
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Ptr {
    const float *q[2], *k[2], *v[2], *go[2];   // [0] detail, [1] global
    float *o[2], *s[2], *dq[2], *dk[2], *dv[2];
    float *lse;                                // forward: output
    const float *delta, *lambda;
    int32_t n_lambda;
    float scale;
    float *split;                              // dK/dV: the parts' sums, with n_split > 1
    int32_t n_split;
};

template <int HD>
__global__ void __launch_bounds__(kThreads) diff_simt_kernel(const Ptr p, const AttnGeom g) {
    extern __shared__ float sm[];
    float *qs = sm, *ks = qs + kRows * (HD + 4), *vs = ks + kTile * (HD + 4),
          *w = vs + kTile * (HD + 4);
    __shared__ uint8_t bad[kTile];
    __shared__ Sees sees[kRows];
    const Span S = query_span(g);
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    load_rows<HD, kRows, false>(qs, p.q[side] + own, stride, static_cast<int>(S.rend - S.r0), nullptr);
    float m[2][4], l[2][4];
    Acc<HD> o[2];
    if (threadIdx.x < kRows) sees[threadIdx.x] = query_sees(g, S, S.r0 + threadIdx.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[0][i] = m[1][i] = kNegInf;
        l[0][i] = l[1][i] = 0.f;
    }
    o[0].zero();
    o[1].zero();
    for (int j = 0; j < S.na + S.nb; ++j) {
        const bool det = j < S.na;
        const int64_t x0 = S.row(j);
        const int64_t at = (S.b * (det ? g.N : g.G) + x0) * stride + S.head * HD;
        __syncthreads();
        load_rows<HD, kTile, false>(ks, p.k[det ? 0 : 1] + at, stride, S.rows(j), nullptr);
        load_rows<HD, kTile, true>(vs, p.v[det ? 0 : 1] + at, stride, S.rows(j), bad);
        __syncthreads();
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            float s[4][kJ];
            scores<HD>(qs, ks, map * (HD / 2), (map + 1) * (HD / 2), s);
            float *wm = w + map * kRows * kPitchW;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bool see[kJ];
                float top = m[map][i];
                const Sees mine = sees[4 * ty + i];
#pragma unroll
                for (int e = 0; e < kJ; ++e) {
                    see[e] = mine.at(det, x0 + tx + 32 * e);
                    s[i][e] = see[e] ? s[i][e] * p.scale : kNegInf;
                    top = fmaxf(top, s[i][e]);
                }
                top = row_max(top);
                const float ref = top == kNegInf ? 0.f : top;
                const float alpha = expf(m[map][i] - ref);
                m[map][i] = top;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < kJ; ++e) {
                    float pr = see[e] ? expf(s[i][e] - ref) : 0.f;
                    sum += pr;
                    if (see[e] && bad[tx + 32 * e]) pr = nan_f();
                    wm[(4 * ty + i) * kPitchW + tx + 32 * e] = pr;
                }
                l[map][i] = fmaf(l[map][i], alpha, sum);
                o[map].scale(i, alpha);
            }
        }
        __syncwarp();
        weighted2<HD>(o[0], o[1], w, w + kRows * kPitchW, vs);
    }
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : S.head];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = S.r0 + 4 * ty + i;
        const float l1 = row_sum(l[0][i]), l2 = row_sum(l[1][i]);
        if (r >= S.rend) continue;
        o[1].scale(i, 1.f / l2);
        o[0].scale(i, 1.f / l1);
#pragma unroll
        for (int c = 0; c < Acc<HD>::kW; ++c) o[0].v[i][c] = fmaf(-lam, o[1].v[i][c], o[0].v[i][c]);
        const int64_t off = own + (4 * ty + i) * stride;
        store<HD>(p.o[side] + off, o[0], i, 1.f, 1.f);
        if (p.s[side] != nullptr) store<HD>(p.s[side] + off, o[1], i, 1.f, 1.f);
        if (p.lse != nullptr && tx < 2) {
            const int64_t rows = g.N + g.G;
            p.lse[((S.b * g.heads + S.head) * 2 + tx) * rows + (S.detail ? r : g.N + r)] =
                tx == 0 ? m[0][i] + logf(l1) : m[1][i] + logf(l2);
        }
    }
}

template <int HD>
__global__ void __launch_bounds__(kThreads) diff_dq_simt_kernel(const Ptr p, const AttnGeom g) {
    extern __shared__ float sm[];
    float *qs = sm, *gs = qs + kRows * (HD + 4), *ks = gs + kRows * (HD + 4),
          *vs = ks + kTile * (HD + 4), *w = vs + kTile * (HD + 4);
    __shared__ uint8_t bad[kTile];
    __shared__ Sees sees[kRows];
    __shared__ float lse[2][kRows], del[2][kRows];
    const Span S = query_span(g);
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, rows = g.N + g.G;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    const int n = static_cast<int>(S.rend - S.r0);
    load_rows<HD, kRows, false>(qs, p.q[side] + own, stride, n, nullptr);
    load_rows<HD, kRows, false>(gs, p.go[side] + own, stride, n, nullptr);
    Acc<HD> dq;
    dq.zero();
    if (threadIdx.x < 2 * kRows) {
        const int map = threadIdx.x / kRows, i = threadIdx.x % kRows;
        const int64_t r = S.r0 + i;
        const int64_t col = ((S.b * g.heads + S.head) * 2 + map) * rows +
                            (S.detail ? 0 : g.N) + (r < S.rend ? r : S.r0);
        lse[map][i] = p.lse[col];
        del[map][i] = p.delta[col];
        if (map == 0) {
            Sees v = query_sees(g, S, r);
            // the one key of a query has P = 1 and dS = 0 (or NaN)
            if (v.db - v.da + v.gb - v.ga == 1 && !isnan(del[0][i])) v = Sees{0, 0, 0, 0};
            sees[i] = v;
        }
    }
    for (int j = 0; j < S.na + S.nb; ++j) {
        const bool det = j < S.na;
        const int64_t x0 = S.row(j);
        const int64_t at = (S.b * (det ? g.N : g.G) + x0) * stride + S.head * HD;
        __syncthreads();
        load_rows<HD, kTile, true>(ks, p.k[det ? 0 : 1] + at, stride, S.rows(j), bad);
        load_rows<HD, kTile, false>(vs, p.v[det ? 0 : 1] + at, stride, S.rows(j), nullptr);
        __syncthreads();
        float dp[4][kJ], s[4][kJ];
        scores<HD>(gs, vs, 0, HD, dp);
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            scores<HD>(qs, ks, map * (HD / 2), (map + 1) * (HD / 2), s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = 4 * ty + i;
                const Sees mine = sees[r];
                const float ls = lse[map][r], de = del[map][r];
#pragma unroll
                for (int e = 0; e < kJ; ++e) {
                    float ds = expf(fmaf(s[i][e], p.scale, -ls)) * (dp[i][e] - de);
                    if (bad[tx + 32 * e]) ds = nan_f();
                    if (!mine.at(det, x0 + tx + 32 * e)) ds = 0.f;
                    w[(map * kRows + r) * kPitchW + tx + 32 * e] = ds;
                }
            }
        }
        __syncwarp();
        weighted<HD>(dq, w + (tx >= 16 ? kRows * kPitchW : 0), ks);
    }
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : S.head];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (S.r0 + 4 * ty + i < S.rend)
            store<HD>(p.dq[side] + own + (4 * ty + i) * stride, dq, i, p.scale, -lam * p.scale);
}

template <int HD>
__global__ void __launch_bounds__(kThreads) diff_dkdv_simt_kernel(const Ptr p, const AttnGeom g) {
    extern __shared__ float sm[];
    float *ks = sm, *vs = ks + kRows * (HD + 4), *qs = vs + kRows * (HD + 4),
          *gs = qs + kTile * (HD + 4), *w = gs + kTile * (HD + 4);
    __shared__ float lse[2][kTile], del[2][kTile];
    __shared__ uint8_t bad[2][kTile];
    int part;
    const Span S = key_span(g, p.n_split, part);
    const int tx = threadIdx.x % 32, ty = threadIdx.x / 32, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, rows = g.N + g.G;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    const int n = static_cast<int>(S.rend - S.r0);
    load_rows<HD, kRows, false>(ks, p.k[side] + own, stride, n, nullptr);
    load_rows<HD, kRows, false>(vs, p.v[side] + own, stride, n, nullptr);
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : S.head];
    __shared__ Sees sees[kRows];
    __shared__ uint8_t lone[kRows];   // the key's queries see no other: 1 detail, 2 global ones
    if (threadIdx.x < kRows) {
        const Sees v = key_sees(g, S, S.r0 + threadIdx.x);
        sees[threadIdx.x] = v;
        uint8_t alone = !S.detail && g.G == 1 ? 2 : 0;
        if (S.detail && v.db - v.da == 1) {
            int64_t lo, hi, g0 = 0, g1 = g.G;
            geo::global_keys(g, geo::window_at(g, S.r0 + threadIdx.x, lo, hi), g0, g1);
            if (g0 == g1) alone = 1;
        }
        lone[threadIdx.x] = alone;
    }
    Acc<HD> dk, dv;
    dk.zero();
    dv.zero();
    for (int j = 0; j < S.na + S.nb; ++j) {
        const bool det = j < S.na;
        const int64_t x0 = S.row(j);
        const int64_t at = (S.b * (det ? g.N : g.G) + x0) * stride + S.head * HD;
        const int nt = S.rows(j);
        __syncthreads();
        load_rows<HD, kTile, true>(qs, p.q[det ? 0 : 1] + at, stride, nt, bad[0]);
        load_rows<HD, kTile, true>(gs, p.go[det ? 0 : 1] + at, stride, nt, bad[1]);
        for (int t = threadIdx.x; t < 2 * kTile; t += kThreads) {
            const int map = t / kTile, c = t % kTile;
            const int64_t col = ((S.b * g.heads + S.head) * 2 + map) * rows + (det ? 0 : g.N) + x0 + c;
            lse[map][c] = c < nt ? p.lse[col] : 0.f;
            del[map][c] = c < nt ? p.delta[col] : 0.f;
        }
        __syncthreads();
        float dp[4][kJ], s[4][kJ], wt[4][kJ];
        scores<HD>(vs, gs, 0, HD, dp);
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            scores<HD>(ks, qs, map * (HD / 2), (map + 1) * (HD / 2), s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Sees mine = sees[4 * ty + i];
                const bool alone = lone[4 * ty + i] & (det ? 1 : 2);
#pragma unroll
                for (int e = 0; e < kJ; ++e) {
                    const int c = tx + 32 * e;
                    float pr = expf(fmaf(s[i][e], p.scale, -lse[map][c]));
                    // a query with a non-finite value (its D is NaN; a row of zeros
                    // here) gives NaN to the keys it sees
                    if (bad[0][c] || bad[1][c]) pr = nan_f();
                    const bool see = mine.at(det, x0 + c);
                    float ds = see ? pr * (dp[i][e] - del[map][c]) : 0.f;
                    if (alone && !isnan(del[map][c])) ds = 0.f;   // of a query with one key
                    wt[i][e] = map == 0 ? pr : (see ? fmaf(-lam, pr, wt[i][e]) : 0.f);
                    w[((1 + map) * kRows + 4 * ty + i) * kPitchW + c] = ds;
                    if (map == 1) w[(4 * ty + i) * kPitchW + c] = wt[i][e];
                }
            }
        }
        __syncwarp();
        weighted<HD>(dv, w, gs);
        weighted<HD>(dk, w + (tx >= 16 ? 2 : 1) * kRows * kPitchW, qs);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (S.r0 + 4 * ty + i >= S.rend) continue;
        const int64_t off = own + (4 * ty + i) * stride;
        if (!S.detail && p.n_split > 1) {
            float *sums = p.split + (((static_cast<int64_t>(part) * g.batch + S.b) * g.heads + S.head) *
                                         g.G + S.r0 + 4 * ty + i) * (2 * HD);
            store<HD>(sums, dv, i, 1.f, 1.f);
            store<HD>(sums + HD, dk, i, 1.f, 1.f);
            continue;
        }
        store<HD>(p.dk[side] + off, dk, i, p.scale, -lam * p.scale);
        store<HD>(p.dv[side] + off, dv, i, 1.f, 1.f);
    }
}

Ptr ptr_of(const DiffArgs &d) {
    const AttnArgs &a = d.attn;
    Ptr p{};
    p.q[0] = static_cast<const float *>(a.q_d);
    p.q[1] = static_cast<const float *>(a.q_g);
    p.k[0] = static_cast<const float *>(a.k_d);
    p.k[1] = static_cast<const float *>(a.k_g);
    p.v[0] = static_cast<const float *>(a.v_d);
    p.v[1] = static_cast<const float *>(a.v_g);
    p.o[0] = static_cast<float *>(a.o_d);
    p.o[1] = static_cast<float *>(a.o_g);
    p.s[0] = static_cast<float *>(d.s_d);
    p.s[1] = static_cast<float *>(d.s_g);
    p.lse = a.lse;
    p.lambda = d.lambda;
    p.n_lambda = d.n_lambda;
    p.scale = a.scale;
    p.n_split = 1;
    return p;
}

// Shared memory in floats: resident and streamed rows, weights.
template <int HD>
constexpr size_t floats(int resident, int weights) {
    return static_cast<size_t>(resident * kRows + 2 * kTile) * (HD + 4) + weights * kRows * kPitchW;
}

template <typename K>
atlas_status launch(K kernel, const char *name, const Ptr &p, const AttnArgs &a, size_t n_floats,
                    cudaStream_t stream) {
    const size_t smem = n_floats * sizeof(float);
    if (!set_smem_limit(reinterpret_cast<const void *>(kernel), static_cast<int>(smem)))
        return ATLAS_ERR_CUDA;
    const int64_t blocks = a.batch * ((a.n_detail + kRows - 1) / kRows +
                                      (a.n_global + kRows - 1) / kRows * p.n_split);
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(a.heads));
    if (log_enabled())
        log_launch(name, static_cast<int>(grid.x * grid.y), kThreads, smem, "head_dim %d rows %lld heads %d",
                   a.head_dim, static_cast<long long>(a.batch * (a.n_detail + a.n_global)), a.heads);
    kernel<<<grid, kThreads, smem, stream>>>(p, attn_geom_of(a));
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

template <int HD>
atlas_status bwd_hd(const DiffBwdArgs &b, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    Ptr p = ptr_of(b.fwd);
    p.go[0] = static_cast<const float *>(b.do_d);
    p.go[1] = static_cast<const float *>(b.do_g);
    p.delta = b.delta;
    p.dq[0] = static_cast<float *>(b.dq_d);
    p.dq[1] = static_cast<float *>(b.dq_g);
    p.dk[0] = static_cast<float *>(b.dk_d);
    p.dk[1] = static_cast<float *>(b.dk_g);
    p.dv[0] = static_cast<float *>(b.dv_d);
    p.dv[1] = static_cast<float *>(b.dv_g);
    atlas_status st = launch(diff_dq_simt_kernel<HD>, "diff_dq_simt_kernel", p, a, floats<HD>(2, 2), stream);
    if (st != ATLAS_OK) return st;
    p.n_split = diff_split_plan(a.batch, a.n_detail, a.n_global, a.heads, 4);
    p.split = b.split;
    st = launch(diff_dkdv_simt_kernel<HD>, "diff_dkdv_simt_kernel", p, a, floats<HD>(2, 3), stream);
    return st != ATLAS_OK || p.n_split == 1 ? st : launch_diff_split_join(b, p.n_split, stream);
}

}  // namespace

atlas_status launch_diff_attn_simt_f32(const DiffArgs &d, cudaStream_t stream) {
    const Ptr p = ptr_of(d);
    return d.attn.head_dim == 128
               ? launch(diff_simt_kernel<128>, "diff_simt_kernel", p, d.attn, floats<128>(1, 2), stream)
               : launch(diff_simt_kernel<64>, "diff_simt_kernel", p, d.attn, floats<64>(1, 2), stream);
}

atlas_status launch_diff_bwd_simt_f32(const DiffBwdArgs &b, cudaStream_t stream) {
    return b.fwd.attn.head_dim == 128 ? bwd_hd<128>(b, stream) : bwd_hd<64>(b, stream);
}

}  // namespace atlas
