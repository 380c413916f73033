// diff_attn.cu -- differential attention: the weight lambda and its gradient,
// the backward pass' row sums, and SIMT kernels of the attention.
//
// With s_m = scale <q_m, k_m> of the two maps of a head (the halves of its
// channels) over a row's allowed keys:
//   o = (P_1 - lambda P_2) v,  P_m = softmax(s_m),
//   lambda = exp<q1,k1> - exp<q2,k2> + lambda_init  (learned vectors).
// Backward, with dP = <do, v>, o_2 = P_2 v and D_m = <do, o_m>:
//   dS_1 = P_1 (dP - D_1),  dS_2 = -lambda P_2 (dP - D_2),
//   dq_m = scale dS_m k_m,  dk_m = scale dS_m^T q_m,
//   dv = (P_1 - lambda P_2)^T do,  dlambda = -sum D_2.
#include <cuda_bf16.h>

#include "attn_geom.cuh"

namespace atlas {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// ---------------------------------------------------------------------------
// lambda: one warp per entry. A few hundred values: the launch is its cost.
// ---------------------------------------------------------------------------
struct LambdaPtr {
    const void *v[4];   // q1, k1, q2, k2 [n, d]
    void *dv[4];
    const float *dlambda;
    float *lambda;
    float init;
    int32_t n, d;
};

template <typename T>
__device__ __forceinline__ float lambda_exp(const LambdaPtr &p, int pair, int64_t row) {
    const int lane = threadIdx.x & 31;
    const T *a = static_cast<const T *>(p.v[2 * pair]) + row * p.d;
    const T *b = static_cast<const T *>(p.v[2 * pair + 1]) + row * p.d;
    float dot = 0.f;
    for (int i = lane; i < p.d; i += 32) dot = fmaf(to_f(a[i]), to_f(b[i]), dot);
    return expf(warp_sum(dot));
}

template <typename T, bool BWD>
__global__ void __launch_bounds__(kWarps * 32) lambda_kernel(const LambdaPtr p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (row >= p.n) return;
    const float e1 = lambda_exp<T>(p, 0, row), e2 = lambda_exp<T>(p, 1, row);
    if (!BWD) {
        if (lane == 0) p.lambda[row] = e1 - e2 + p.init;
        return;
    }
    const float g[2] = {p.dlambda[row] * e1, -p.dlambda[row] * e2};
#pragma unroll
    for (int v = 0; v < 4; ++v) {   // d<a,b>/da = b
        const T *other = static_cast<const T *>(p.v[v ^ 1]) + row * p.d;
        T *out = static_cast<T *>(p.dv[v]) + row * p.d;
        for (int i = lane; i < p.d; i += 32) out[i] = from_f<T>(g[v / 2] * to_f(other[i]));
    }
}

// ---------------------------------------------------------------------------
// Row sums of the backward pass: D_2 = <do, s>, D_1 = <do, o> + lambda D_2
// (o + lambda s is the first map's output), fp32 [batch, heads, 2, N+G]. Both are
// NaN where the row's lse is not finite (as <do, .> is where do is not), so a NaN
// here marks every query row that holds a non-finite value: the tensor-core
// kernel tells such a row from its neighbours in a tile by it.
// ---------------------------------------------------------------------------
template <typename T>
struct DeltaPtr {
    const T *o_d, *s_d, *do_d, *o_g, *s_g, *do_g;
    const float *lambda, *lse;
    int32_t n_lambda;
    float *delta;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kWarps * 32) diff_delta_kernel(const DeltaPtr<T> p,
                                                                 const AttnGeom g) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    const int head = blockIdx.y;
    if (row >= g.batch * (g.N + g.G)) return;
    const geo::RowAt at = geo::row_at(g, row);
    const int64_t off = (at.row * g.heads + head) * HD;
    const T *o = (at.detail ? p.o_d : p.o_g) + off, *s = (at.detail ? p.s_d : p.s_g) + off,
            *d = (at.detail ? p.do_d : p.do_g) + off;
    float sum_o = 0.f, sum_s = 0.f;
#pragma unroll
    for (int e = 0; e < HD / 32; ++e) {
        const float w = to_f(d[lane + 32 * e]);
        sum_o = fmaf(w, to_f(o[lane + 32 * e]), sum_o);
        sum_s = fmaf(w, to_f(s[lane + 32 * e]), sum_s);
    }
    sum_o = warp_sum(sum_o);
    sum_s = warp_sum(sum_s);
    if (lane == 0) {
        const float lam = p.lambda[p.n_lambda == 1 ? 0 : head];
        const int64_t rows = g.N + g.G;
        const int64_t col = (at.b * g.heads + head) * 2 * rows +
                            (at.detail ? at.local : g.N + at.local);
        const float d1 = fmaf(lam, sum_s, sum_o);
        // 0 for finite values, NaN otherwise
        const float mark = 0.f * p.lse[col] + 0.f * p.lse[col + rows] + 0.f * d1 + 0.f * sum_s;
        p.delta[col] = d1 + mark;
        p.delta[col + rows] = sum_s + mark;
    }
}

// dlambda = -sum of D_2 over a head's rows: kDiffLambdaParts partial sums per
// head, then one block joins them. Both orders are fixed.
__global__ void __launch_bounds__(256) dlambda_part_kernel(const float *delta, float *part,
                                                           int64_t batch, int32_t heads,
                                                           int64_t rows) {
    __shared__ float sums[8];
    const int head = blockIdx.y;
    const int64_t total = batch * rows;
    float acc = 0.f;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
         i += static_cast<int64_t>(kDiffLambdaParts) * 256) {
        const int64_t b = i / rows;
        acc += delta[((b * heads + head) * 2 + 1) * rows + (i - b * rows)];
    }
    acc = warp_sum(acc);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x / 32] = acc;
    __syncthreads();
    if (threadIdx.x == 0) {
        float s = 0.f;
        for (int i = 0; i < 8; ++i) s += sums[i];
        part[static_cast<int64_t>(head) * kDiffLambdaParts + blockIdx.x] = s;
    }
}

// One warp per lambda: a head's partial sums, or every head's.
__global__ void __launch_bounds__(32) dlambda_join_kernel(const float *part, float *dlambda,
                                                          int32_t per_lambda) {
    double acc = 0.0;
    const float *src = part + static_cast<int64_t>(blockIdx.x) * per_lambda;
    for (int32_t i = threadIdx.x; i < per_lambda; i += 32) acc += src[i];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    if (threadIdx.x == 0) dlambda[blockIdx.x] = static_cast<float>(-acc);
}

// ---------------------------------------------------------------------------
// SIMT attention: one warp per (row, head), exact fp32 products, online softmax
// of both maps. A lane's channels lane + 32 e belong to map e / (HD / 64).
// ---------------------------------------------------------------------------
template <typename T>
struct FwdPtr {
    const T *q_d, *k_d, *v_d, *q_g, *k_g, *v_g;
    T *o_d, *o_g, *s_d, *s_g;
    const float *lambda;
    int32_t n_lambda;
    float *lse;
    float scale;
};

template <int HD>
struct Row {
    static constexpr int kE = HD / 32, kMap = HD / 64;
    float x[kE];
    template <typename T>
    __device__ __forceinline__ void load(const T *p) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = to_f(p[lane + 32 * e]);
    }
    template <typename T>
    __device__ __forceinline__ void store(T *p, float f) const {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int e = 0; e < kE; ++e) p[lane + 32 * e] = from_f<T>(x[e] * f);
    }
    // <x, y> of map m, and of the whole row.
    __device__ __forceinline__ float dot(const Row &y, int m) const {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kMap; ++e) s = fmaf(x[m * kMap + e], y.x[m * kMap + e], s);
        return warp_sum(s);
    }
    __device__ __forceinline__ float dot(const Row &y) const {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e) s = fmaf(x[e], y.x[e], s);
        return warp_sum(s);
    }
    __device__ __forceinline__ void add(float f, const Row &y) {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = fmaf(f, y.x[e], x[e]);
    }
    // x += (f1, f2) y, a factor for each map.
    __device__ __forceinline__ void add(float f1, float f2, const Row &y) {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] = fmaf(e < kMap ? f1 : f2, y.x[e], x[e]);
    }
    __device__ __forceinline__ void times(float f) {
#pragma unroll
        for (int e = 0; e < kE; ++e) x[e] *= f;
    }
    __device__ __forceinline__ void zero() { times(0.f); }
};

template <typename T, int HD>
__global__ void __launch_bounds__(kWarps * 32) diff_simt_kernel(const FwdPtr<T> p,
                                                                const AttnGeom g) {
    const int lane = threadIdx.x & 31, head = blockIdx.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (row >= g.batch * (g.N + g.G)) return;
    const geo::RowAt at = geo::row_at(g, row);
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, off = at.row * stride + head * HD;
    Row<HD> q, o[2], k, v;
    q.load((at.detail ? p.q_d : p.q_g) + off);
#pragma unroll
    for (int e = 0; e < Row<HD>::kE; ++e) o[0].x[e] = o[1].x[e] = 0.f;
    float m[2] = {-__builtin_huge_valf(), -__builtin_huge_valf()}, l[2] = {0.f, 0.f};
    auto keys = [&](const T *kp, const T *vp, int64_t k0, int64_t k1) {
        for (int64_t j = k0; j < k1; ++j) {
            k.load(kp + j * stride);
            v.load(vp + j * stride);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float s = q.dot(k, i) * p.scale;
                const float m_new = fmaxf(m[i], s);
                const float corr = expf(m[i] - m_new), pr = expf(s - m_new);
                l[i] = fmaf(l[i], corr, pr);
                o[i].times(corr);
                o[i].add(pr, v);
                m[i] = m_new;
            }
        }
    };
    int64_t g_lo = 0, g_hi = g.G;
    if (at.detail) {
        int64_t lo, hi;
        const int64_t w = geo::window_at(g, at.local, lo, hi);
        geo::global_keys(g, w, g_lo, g_hi);
        keys(p.k_d + at.b * g.N * stride + head * HD, p.v_d + at.b * g.N * stride + head * HD, lo,
             hi);
    }
    keys(p.k_g + at.b * g.G * stride + head * HD, p.v_g + at.b * g.G * stride + head * HD, g_lo,
         g_hi);
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : head];
    o[1].times(1.f / l[1]);
    T *s_out = at.detail ? p.s_d : p.s_g;
    if (s_out != nullptr) o[1].store(s_out + off, 1.f);
    o[0].times(1.f / l[0]);
    o[0].add(-lam, o[1]);
    o[0].store((at.detail ? p.o_d : p.o_g) + off, 1.f);
    if (p.lse != nullptr && lane < 2) {
        const int64_t rows = g.N + g.G;
        p.lse[((at.b * g.heads + head) * 2 + lane) * rows + (at.detail ? at.local : g.N + at.local)] =
            lane == 0 ? m[0] + logf(l[0]) : m[1] + logf(l[1]);
    }
}

template <typename T>
struct BwdPtr {
    const T *q_d, *k_d, *v_d, *do_d, *q_g, *k_g, *v_g, *do_g;
    const float *lse, *delta, *lambda;
    int32_t n_lambda;
    T *dq_d, *dk_d, *dv_d, *dq_g, *dk_g, *dv_g;
    float scale;
};

template <typename T, int HD>
__global__ void __launch_bounds__(kWarps * 32) diff_dq_simt_kernel(const BwdPtr<T> p,
                                                                   const AttnGeom g) {
    const int head = blockIdx.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (row >= g.batch * (g.N + g.G)) return;
    const geo::RowAt at = geo::row_at(g, row);
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, off = at.row * stride + head * HD;
    const int64_t rows = g.N + g.G;
    const int64_t col = (at.b * g.heads + head) * 2 * rows + (at.detail ? at.local : g.N + at.local);
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : head];
    const float lse1 = p.lse[col], lse2 = p.lse[col + rows];
    const float d1 = p.delta[col], d2 = p.delta[col + rows];
    Row<HD> q, go, dq, k, v;
    q.load((at.detail ? p.q_d : p.q_g) + off);
    go.load((at.detail ? p.do_d : p.do_g) + off);
#pragma unroll
    for (int e = 0; e < Row<HD>::kE; ++e) dq.x[e] = 0.f;
    auto keys = [&](const T *kp, const T *vp, int64_t k0, int64_t k1) {
        for (int64_t j = k0; j < k1; ++j) {
            k.load(kp + j * stride);
            v.load(vp + j * stride);
            const float dp = go.dot(v);
            const float p1 = expf(q.dot(k, 0) * p.scale - lse1);
            const float p2 = expf(q.dot(k, 1) * p.scale - lse2);
            dq.add(p1 * (dp - d1), -lam * (p2 * (dp - d2)), k);
        }
    };
    int64_t g_lo = 0, g_hi = g.G;
    if (at.detail) {
        int64_t lo, hi;
        const int64_t w = geo::window_at(g, at.local, lo, hi);
        geo::global_keys(g, w, g_lo, g_hi);
        keys(p.k_d + at.b * g.N * stride + head * HD, p.v_d + at.b * g.N * stride + head * HD, lo,
             hi);
    }
    keys(p.k_g + at.b * g.G * stride + head * HD, p.v_g + at.b * g.G * stride + head * HD, g_lo,
         g_hi);
    dq.store((at.detail ? p.dq_d : p.dq_g) + off, p.scale);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kWarps * 32) diff_dkdv_simt_kernel(const BwdPtr<T> p,
                                                                     const AttnGeom g) {
    const int head = blockIdx.y;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
    if (row >= g.batch * (g.N + g.G)) return;
    const geo::RowAt at = geo::row_at(g, row);
    const int64_t stride = static_cast<int64_t>(g.heads) * HD, off = at.row * stride + head * HD;
    const int64_t rows = g.N + g.G, base = (at.b * g.heads + head) * 2 * rows;
    const float lam = p.lambda[p.n_lambda == 1 ? 0 : head];
    Row<HD> k, v, dk, dv, q, go;
    k.load((at.detail ? p.k_d : p.k_g) + off);
    v.load((at.detail ? p.v_d : p.v_g) + off);
#pragma unroll
    for (int e = 0; e < Row<HD>::kE; ++e) dk.x[e] = dv.x[e] = 0.f;
    auto queries = [&](const T *qp, const T *gp, int64_t col0, int64_t q0, int64_t q1) {
        for (int64_t i = q0; i < q1; ++i) {
            q.load(qp + i * stride);
            go.load(gp + i * stride);
            const int64_t col = base + col0 + i;
            const float dp = go.dot(v);
            const float p1 = expf(q.dot(k, 0) * p.scale - p.lse[col]);
            const float p2 = expf(q.dot(k, 1) * p.scale - p.lse[col + rows]);
            dk.add(p1 * (dp - p.delta[col]), -lam * (p2 * (dp - p.delta[col + rows])), q);
            dv.add(p1 - lam * p2, go);
        }
    };
    int64_t lo, hi;
    if (at.detail) geo::window_at(g, at.local, lo, hi);
    else geo::global_queries(g, at.local, lo, hi);
    queries(p.q_d + at.b * g.N * stride + head * HD, p.do_d + at.b * g.N * stride + head * HD, 0, lo,
            hi);
    if (!at.detail)
        queries(p.q_g + at.b * g.G * stride + head * HD, p.do_g + at.b * g.G * stride + head * HD,
                g.N, 0, g.G);
    dk.store((at.detail ? p.dk_d : p.dk_g) + off, p.scale);
    dv.store((at.detail ? p.dv_d : p.dv_g) + off, 1.f);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
atlas_status launched() {
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

dim3 row_grid(const AttnArgs &a) {
    const int64_t rows = a.batch * (a.n_detail + a.n_global);
    return dim3(static_cast<unsigned>((rows + kWarps - 1) / kWarps),
                static_cast<unsigned>(a.heads));
}

void log_rows(const char *kernel, const AttnArgs &a) {
    if (log_enabled())
        log_launch(kernel, static_cast<int>(row_grid(a).x * row_grid(a).y), kWarps * 32, 0,
                   "head_dim %d rows %lld heads %d", a.head_dim,
                   static_cast<long long>(a.batch * (a.n_detail + a.n_global)), a.heads);
}

template <typename T, int HD>
atlas_status fwd_simt(const DiffArgs &d, cudaStream_t stream) {
    const AttnArgs &a = d.attn;
    FwdPtr<T> p;
    p.q_d = static_cast<const T *>(a.q_d);
    p.k_d = static_cast<const T *>(a.k_d);
    p.v_d = static_cast<const T *>(a.v_d);
    p.q_g = static_cast<const T *>(a.q_g);
    p.k_g = static_cast<const T *>(a.k_g);
    p.v_g = static_cast<const T *>(a.v_g);
    p.o_d = static_cast<T *>(a.o_d);
    p.o_g = static_cast<T *>(a.o_g);
    p.s_d = static_cast<T *>(d.s_d);
    p.s_g = static_cast<T *>(d.s_g);
    p.lambda = d.lambda;
    p.n_lambda = d.n_lambda;
    p.lse = a.lse;
    p.scale = a.scale;
    log_rows("diff_simt_kernel", a);
    diff_simt_kernel<T, HD><<<row_grid(a), kWarps * 32, 0, stream>>>(p, attn_geom_of(a));
    return launched();
}

template <typename T, int HD>
atlas_status delta_hd(const DiffBwdArgs &b, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    DeltaPtr<T> p;
    p.o_d = static_cast<const T *>(a.o_d);
    p.s_d = static_cast<const T *>(b.fwd.s_d);
    p.do_d = static_cast<const T *>(b.do_d);
    p.o_g = static_cast<const T *>(a.o_g);
    p.s_g = static_cast<const T *>(b.fwd.s_g);
    p.do_g = static_cast<const T *>(b.do_g);
    p.lambda = b.fwd.lambda;
    p.n_lambda = b.fwd.n_lambda;
    p.lse = a.lse;
    p.delta = b.delta;
    log_rows("diff_delta_kernel", a);
    diff_delta_kernel<T, HD><<<row_grid(a), kWarps * 32, 0, stream>>>(p, attn_geom_of(a));
    return launched();
}

template <typename T, int HD>
atlas_status bwd_simt(const DiffBwdArgs &b, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    BwdPtr<T> p;
    p.q_d = static_cast<const T *>(a.q_d);
    p.k_d = static_cast<const T *>(a.k_d);
    p.v_d = static_cast<const T *>(a.v_d);
    p.do_d = static_cast<const T *>(b.do_d);
    p.q_g = static_cast<const T *>(a.q_g);
    p.k_g = static_cast<const T *>(a.k_g);
    p.v_g = static_cast<const T *>(a.v_g);
    p.do_g = static_cast<const T *>(b.do_g);
    p.lse = a.lse;
    p.delta = b.delta;
    p.lambda = b.fwd.lambda;
    p.n_lambda = b.fwd.n_lambda;
    p.dq_d = static_cast<T *>(b.dq_d);
    p.dk_d = static_cast<T *>(b.dk_d);
    p.dv_d = static_cast<T *>(b.dv_d);
    p.dq_g = static_cast<T *>(b.dq_g);
    p.dk_g = static_cast<T *>(b.dk_g);
    p.dv_g = static_cast<T *>(b.dv_g);
    p.scale = a.scale;
    const AttnGeom g = attn_geom_of(a);
    log_rows("diff_dq_simt_kernel", a);
    diff_dq_simt_kernel<T, HD><<<row_grid(a), kWarps * 32, 0, stream>>>(p, g);
    log_rows("diff_dkdv_simt_kernel", a);
    diff_dkdv_simt_kernel<T, HD><<<row_grid(a), kWarps * 32, 0, stream>>>(p, g);
    return launched();
}

}  // namespace

atlas_status launch_diff_lambda(const DiffLambdaArgs &a, bool bwd, cudaStream_t stream) {
    LambdaPtr p;
    for (int i = 0; i < 4; ++i) {
        p.v[i] = a.v[i];
        p.dv[i] = a.dv[i];
    }
    p.dlambda = a.dlambda;
    p.lambda = a.lambda;
    p.init = static_cast<float>(a.init);
    p.n = a.n;
    p.d = a.d;
    const unsigned grid = (static_cast<unsigned>(a.n) + kWarps - 1) / kWarps;
    if (log_enabled())
        log_launch(bwd ? "lambda_kernel<bwd>" : "lambda_kernel", static_cast<int>(grid), kWarps * 32,
                   0, "n %d d %d elem_bytes %d", a.n, a.d, a.elem_bytes);
    if (a.elem_bytes == 2) {
        if (bwd) lambda_kernel<__nv_bfloat16, true><<<grid, kWarps * 32, 0, stream>>>(p);
        else lambda_kernel<__nv_bfloat16, false><<<grid, kWarps * 32, 0, stream>>>(p);
    } else {
        if (bwd) lambda_kernel<float, true><<<grid, kWarps * 32, 0, stream>>>(p);
        else lambda_kernel<float, false><<<grid, kWarps * 32, 0, stream>>>(p);
    }
    return launched();
}

atlas_status launch_diff_attn_simt(const DiffArgs &d, cudaStream_t stream) {
    if (d.elem_bytes == 2)
        return d.attn.head_dim == 128 ? fwd_simt<__nv_bfloat16, 128>(d, stream)
                                      : fwd_simt<__nv_bfloat16, 64>(d, stream);
    return d.attn.head_dim == 128 ? fwd_simt<float, 128>(d, stream)
                                  : fwd_simt<float, 64>(d, stream);
}

atlas_status launch_diff_bwd_delta(const DiffBwdArgs &b, cudaStream_t stream) {
    if (b.fwd.elem_bytes == 2)
        return b.fwd.attn.head_dim == 128 ? delta_hd<__nv_bfloat16, 128>(b, stream)
                                          : delta_hd<__nv_bfloat16, 64>(b, stream);
    return b.fwd.attn.head_dim == 128 ? delta_hd<float, 128>(b, stream)
                                      : delta_hd<float, 64>(b, stream);
}

atlas_status launch_diff_dlambda(const DiffBwdArgs &b, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    const int64_t rows = a.n_detail + a.n_global;
    const dim3 grid(kDiffLambdaParts, static_cast<unsigned>(a.heads));
    dlambda_part_kernel<<<grid, 256, 0, stream>>>(b.delta, b.part, a.batch, a.heads, rows);
    const int32_t n = b.fwd.n_lambda;
    dlambda_join_kernel<<<n, 32, 0, stream>>>(b.part, b.dlambda,
                                              kDiffLambdaParts * (n == 1 ? a.heads : 1));
    return launched();
}

atlas_status launch_diff_bwd_simt(const DiffBwdArgs &b, cudaStream_t stream) {
    if (b.fwd.elem_bytes == 2)
        return b.fwd.attn.head_dim == 128 ? bwd_simt<__nv_bfloat16, 128>(b, stream)
                                          : bwd_simt<__nv_bfloat16, 64>(b, stream);
    return b.fwd.attn.head_dim == 128 ? bwd_simt<float, 128>(b, stream)
                                      : bwd_simt<float, 64>(b, stream);
}

}  // namespace atlas
