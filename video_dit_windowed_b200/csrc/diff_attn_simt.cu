// diff_attn_simt.cu -- differential attention and its backward pass, fp32 I/O,
// exact fp32 products on the FMA pipe (formulas: diff_attn.cu).
//
// A block of 256 threads takes 64 rows of one head of one problem (queries, or
// keys for dK/dV) and streams the rows they meet in tiles of 32 through shared
// memory. Threads form 16 x 16: thread (ty, tx) owns rows 4 ty .. 4 ty + 3; of a
// 64 x 32 score tile columns tx and tx + 16; of an accumulator columns 4 tx .. +3
// (and + 64). Scores, weights and accumulators stay in registers; the weights
// pass through shared memory within a half-warp only, whose rows they are. At 64
// FMAs per 8 to 12 shared-memory accesses the FMA pipe bounds a long call; a
// short one its chain of tiles. Row pitch D + 4 floats: the 16 rows that a
// half-warp reads side by side fall into different banks.
// Masked pairs get weight 0. 0 * NaN would still reach a row, so streamed rows
// that enter a product by their weight are zeroed where they hold a non-finite
// value, and pairs that do see such a row get the weight NaN.
#include "attn_geom.cuh"

namespace atlas {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 64;     // rows of a block
constexpr int kTile = 32;     // streamed rows of a tile
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

__device__ __forceinline__ Span rows_of_block(const AttnGeom &g) {
    Span s;
    s.head = blockIdx.y;
    const int64_t td = (g.N + kRows - 1) / kRows, tg = (g.G + kRows - 1) / kRows;
    s.b = blockIdx.x / (td + tg);
    const int64_t t = blockIdx.x - s.b * (td + tg);
    s.detail = t < td;
    s.r0 = (s.detail ? t : t - td) * kRows;
    const int64_t n = s.detail ? g.N : g.G;
    s.rend = s.r0 + kRows < n ? s.r0 + kRows : n;
    return s;
}

// Queries: the union of the rows' windows and global keys.
__device__ __forceinline__ Span query_span(const AttnGeom &g) {
    Span s = rows_of_block(g);
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

// Keys: the queries that see them.
__device__ __forceinline__ Span key_span(const AttnGeom &g) {
    Span s = rows_of_block(g);
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

// s[i][j] = <a row 4 ty + i, b row tx + 16 j> over channels [d0, d1).
template <int HD>
__device__ __forceinline__ void scores(const float *a, const float *b, int d0, int d1,
                                       float (&s)[4][2]) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][0] = s[i][1] = 0.f;
#pragma unroll 4
    for (int d = d0; d < d1; d += 4) {
        float4 x[4], y[2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const float4 *>(a + (4 * ty + i) * (HD + 4) + d);
#pragma unroll
        for (int j = 0; j < 2; ++j)
            y[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * (HD + 4) + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) s[i][j] = dot4(x[i], y[j], s[i][j]);
    }
}

// An accumulator of the thread's 4 rows: columns 4 tx .. +3 (+ 64 for D = 128).
template <int HD>
struct Acc {
    static constexpr int kC = HD / 64;
    float4 v[4][kC];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < kC; ++c) v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __device__ __forceinline__ void scale(int i, float f) {
#pragma unroll
        for (int c = 0; c < kC; ++c) {
            v[i][c].x *= f;
            v[i][c].y *= f;
            v[i][c].z *= f;
            v[i][c].w *= f;
        }
    }
};
__device__ __forceinline__ void fma4(float4 &a, float f, const float4 &b) {
    a.x = fmaf(f, b.x, a.x);
    a.y = fmaf(f, b.y, a.y);
    a.z = fmaf(f, b.z, a.z);
    a.w = fmaf(f, b.w, a.w);
}

// acc += w b: w [64][kPitchW] (weights of the thread's rows), b [32][D + 4].
// MAPS: column block c takes the weights of its map (w0 map 1, w1 map 2).
template <int HD, bool MAPS>
__device__ __forceinline__ void weighted(Acc<HD> &acc, const float *w0, const float *w1,
                                         const float *b) {
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        float4 y[4][Acc<HD>::kC];
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int c = 0; c < Acc<HD>::kC; ++c)
                y[e][c] = *reinterpret_cast<const float4 *>(b + (k + e) * (HD + 4) + 4 * tx + 64 * c);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < Acc<HD>::kC; ++c) {
                const bool second = MAPS && (HD == 128 ? c == 1 : tx >= 8);
                const float4 x = *reinterpret_cast<const float4 *>((second ? w1 : w0) +
                                                                   (4 * ty + i) * kPitchW + k);
                fma4(acc.v[i][c], x.x, y[0][c]);
                fma4(acc.v[i][c], x.y, y[1][c]);
                fma4(acc.v[i][c], x.z, y[2][c]);
                fma4(acc.v[i][c], x.w, y[3][c]);
            }
    }
}

template <int HD>
__device__ __forceinline__ void store(float *out, const Acc<HD> &acc, int i, float f0, float f1) {
    const int tx = threadIdx.x % 16;
#pragma unroll
    for (int c = 0; c < Acc<HD>::kC; ++c) {
        const float f = (HD == 128 ? c == 1 : tx >= 8) ? f1 : f0;
        float4 v = acc.v[i][c];
        v.x *= f;
        v.y *= f;
        v.z *= f;
        v.w *= f;
        *reinterpret_cast<float4 *>(out + 4 * tx + 64 * c) = v;
    }
}

__device__ __forceinline__ float half_max(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float half_sum(float v) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct Ptr {
    const float *q[2], *k[2], *v[2], *go[2];   // [0] detail, [1] global
    float *o[2], *s[2], *dq[2], *dk[2], *dv[2];
    float *lse;                                // forward: output
    const float *delta, *lambda;
    int32_t n_lambda;
    float scale;
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 2) diff_simt_kernel(const Ptr p, const AttnGeom g) {
    extern __shared__ float sm[];
    float *qs = sm, *ks = qs + kRows * (HD + 4), *vs = ks + kTile * (HD + 4),
          *w = vs + kTile * (HD + 4);
    __shared__ uint8_t bad[kTile];
    const Span S = query_span(g);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    load_rows<HD, kRows, false>(qs, p.q[side] + own, stride, static_cast<int>(S.rend - S.r0), nullptr);
    Sees sees[4];
    float m[2][4], l[2][4];
    Acc<HD> o[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        sees[i] = query_sees(g, S, S.r0 + 4 * ty + i);
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
            float s[4][2];
            scores<HD>(qs, ks, map * (HD / 2), (map + 1) * (HD / 2), s);
            float *wm = w + map * kRows * kPitchW;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                bool see[2];
                float top = m[map][i];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    see[e] = sees[i].at(det, x0 + tx + 16 * e);
                    s[i][e] = see[e] ? s[i][e] * p.scale : kNegInf;
                    top = fmaxf(top, s[i][e]);
                }
                top = half_max(top);
                const float ref = top == kNegInf ? 0.f : top;
                const float alpha = expf(m[map][i] - ref);
                m[map][i] = top;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float pr = see[e] ? expf(s[i][e] - ref) : 0.f;
                    sum += pr;
                    if (see[e] && bad[tx + 16 * e]) pr = nan_f();
                    wm[(4 * ty + i) * kPitchW + tx + 16 * e] = pr;
                }
                l[map][i] = fmaf(l[map][i], alpha, sum);
                o[map].scale(i, alpha);
            }
        }
        __syncwarp();
        weighted<HD, false>(o[0], w, w, vs);
        weighted<HD, false>(o[1], w + kRows * kPitchW, w, vs);
    }
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : S.head];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = S.r0 + 4 * ty + i;
        const float l1 = half_sum(l[0][i]), l2 = half_sum(l[1][i]);
        if (r >= S.rend) continue;
        o[1].scale(i, 1.f / l2);
        o[0].scale(i, 1.f / l1);
#pragma unroll
        for (int c = 0; c < Acc<HD>::kC; ++c) fma4(o[0].v[i][c], -lam, o[1].v[i][c]);
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
    const Span S = query_span(g);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, rows = g.N + g.G;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    const int n = static_cast<int>(S.rend - S.r0);
    load_rows<HD, kRows, false>(qs, p.q[side] + own, stride, n, nullptr);
    load_rows<HD, kRows, false>(gs, p.go[side] + own, stride, n, nullptr);
    Sees sees[4];
    float lse[2][4], del[2][4];
    Acc<HD> dq;
    dq.zero();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = S.r0 + 4 * ty + i;
        sees[i] = query_sees(g, S, r);
        const int64_t col = (S.b * g.heads + S.head) * 2 * rows +
                            (S.detail ? 0 : g.N) + (r < S.rend ? r : S.r0);
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            lse[map][i] = p.lse[col + map * rows];
            del[map][i] = p.delta[col + map * rows];
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
        float dp[4][2], s[4][2];
        scores<HD>(gs, vs, 0, HD, dp);
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            scores<HD>(qs, ks, map * (HD / 2), (map + 1) * (HD / 2), s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float ds = expf(fmaf(s[i][e], p.scale, -lse[map][i])) * (dp[i][e] - del[map][i]);
                    if (bad[tx + 16 * e]) ds = nan_f();
                    if (!sees[i].at(det, x0 + tx + 16 * e)) ds = 0.f;
                    w[(map * kRows + 4 * ty + i) * kPitchW + tx + 16 * e] = ds;
                }
        }
        __syncwarp();
        weighted<HD, true>(dq, w, w + kRows * kPitchW, ks);
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
    const Span S = key_span(g);
    const int tx = threadIdx.x % 16, ty = threadIdx.x / 16, side = S.detail ? 0 : 1;
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, rows = g.N + g.G;
    const int64_t own = (S.b * (S.detail ? g.N : g.G) + S.r0) * stride + S.head * HD;
    const int n = static_cast<int>(S.rend - S.r0);
    load_rows<HD, kRows, false>(ks, p.k[side] + own, stride, n, nullptr);
    load_rows<HD, kRows, false>(vs, p.v[side] + own, stride, n, nullptr);
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : S.head];
    Sees sees[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sees[i] = key_sees(g, S, S.r0 + 4 * ty + i);
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
        if (threadIdx.x < 2 * kTile) {
            const int map = threadIdx.x / kTile, c = threadIdx.x % kTile;
            const int64_t col = ((S.b * g.heads + S.head) * 2 + map) * rows + (det ? 0 : g.N) + x0 + c;
            lse[map][c] = c < nt ? p.lse[col] : 0.f;
            del[map][c] = c < nt ? p.delta[col] : 0.f;
        }
        __syncthreads();
        float dp[4][2], s[4][2], wt[4][2];
        scores<HD>(vs, gs, 0, HD, dp);
#pragma unroll
        for (int map = 0; map < 2; ++map) {
            scores<HD>(ks, qs, map * (HD / 2), (map + 1) * (HD / 2), s);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int c = tx + 16 * e;
                    float pr = expf(fmaf(s[i][e], p.scale, -lse[map][c]));
                    // a query with a non-finite value (its D is NaN; a row of zeros
                    // here) gives NaN to the keys it sees
                    if (bad[0][c] || bad[1][c]) pr = nan_f();
                    const bool see = sees[i].at(det, x0 + c);
                    const float ds = see ? pr * (dp[i][e] - del[map][c]) : 0.f;
                    wt[i][e] = map == 0 ? pr : (see ? fmaf(-lam, pr, wt[i][e]) : 0.f);
                    w[((1 + map) * kRows + 4 * ty + i) * kPitchW + c] = ds;
                    if (map == 1) w[(4 * ty + i) * kPitchW + c] = wt[i][e];
                }
        }
        __syncwarp();
        weighted<HD, false>(dv, w, w, gs);
        weighted<HD, true>(dk, w + kRows * kPitchW, w + 2 * kRows * kPitchW, qs);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (S.r0 + 4 * ty + i >= S.rend) continue;
        const int64_t off = own + (4 * ty + i) * stride;
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
    const int64_t blocks = a.batch * ((a.n_detail + kRows - 1) / kRows + (a.n_global + kRows - 1) / kRows);
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
    const atlas_status st = launch(diff_dq_simt_kernel<HD>, "diff_dq_simt_kernel", p, a,
                                   floats<HD>(2, 2), stream);
    return st != ATLAS_OK ? st : launch(diff_dkdv_simt_kernel<HD>, "diff_dkdv_simt_kernel", p, a,
                                        floats<HD>(2, 3), stream);
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
