// diff_attn.cu -- differential attention: the weight lambda and its gradient,
// and the backward pass' row sums (the attention itself: diff_attn_tc.cu,
// diff_attn_bwd_tc.cu, diff_attn_simt.cu).
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
    const int64_t rows = g.N + g.G;
    const int64_t col = (at.b * g.heads + head) * 2 * rows +
                        (at.detail ? at.local : g.N + at.local);
    if (lane == 0) {
        const float d1 = fmaf(p.lambda[p.n_lambda == 1 ? 0 : head], sum_s, sum_o);
        // 0 for finite values, NaN otherwise
        const float mark = 0.f * p.lse[col] + 0.f * p.lse[col + rows] + 0.f * d1 + 0.f * sum_s;
        p.delta[col] = d1 + mark;
        p.delta[col + rows] = sum_s + mark;
    }
}

// bf16 rows of at most kFewKeys keys again: o and s were rounded to 8 bits, and where
// few keys share the weight dP - D, the other keys' weights times differences, is
// often far smaller than D, so those rows' D is summed from P and dP themselves
// (two keys, D = 128: dq's error 0.59% with the stored outputs; eight: 0.28%).
// A block per window (and one for the global rows), a warp per row: as a test in the
// kernel above it cost every row the search of its window (6 -> 25 us for 2 x 4 heads
// of 2,641 rows with offsets).
constexpr int kFewKeys = kWarps;

struct FewPtr {
    const __nv_bfloat16 *q[2], *k[2], *v[2], *go[2];   // [0] detail, [1] global
    const float *lse;
    float *delta;
    float scale;
};

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) diff_few_keys_kernel(const FewPtr p,
                                                                    const AttnGeom g,
                                                                    int64_t n_win) {
    const int lane = threadIdx.x & 31, slot = threadIdx.x / 32, head = blockIdx.y;
    const int64_t b = blockIdx.x / (n_win + 1), w = blockIdx.x - b * (n_win + 1);
    const bool detail = w < n_win;
    int64_t a0 = 0, a1 = 0, b0 = 0, b1 = g.G;
    if (detail) {
        a0 = g.win_off ? geo::clamp64(__ldg(g.win_off + w), 0, g.N) : w * g.L;
        a1 = g.win_off ? geo::clamp64(__ldg(g.win_off + w + 1), a0, g.N) : a0 + g.L;
        geo::global_keys(g, w, b0, b1);
    }
    if (a1 - a0 + b1 - b0 > kFewKeys || slot >= (detail ? a1 - a0 : b1 - b0)) return;
    const int n_a = static_cast<int>(a1 - a0), n = n_a + static_cast<int>(b1 - b0);
    const int64_t rows = g.N + g.G, local = (detail ? a0 : b0) + slot;
    const int64_t off = ((b * (detail ? g.N : g.G) + local) * g.heads + head) * HD;
    const int64_t col = (b * g.heads + head) * 2 * rows + (detail ? local : g.N + local);
    const __nv_bfloat16 *q = p.q[detail ? 0 : 1] + off, *d = p.go[detail ? 0 : 1] + off;
    const float l1 = p.lse[col], l2 = p.lse[col + rows];
    float d1 = 0.f, d2 = 0.f;
    for (int j = 0; j < n; ++j) {
        const int side = j < n_a ? 0 : 1;
        const int64_t row = b * (side ? g.G : g.N) + (side ? b0 + j - n_a : a0 + j);
        const __nv_bfloat16 *k = p.k[side] + (row * g.heads + head) * HD;
        const __nv_bfloat16 *v = p.v[side] + (row * g.heads + head) * HD;
        float s[2] = {0.f, 0.f}, dp = 0.f;
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
            const int c = lane + 32 * e;
            s[e / (HD / 64)] = fmaf(to_f(q[c]), to_f(k[c]), s[e / (HD / 64)]);
            dp = fmaf(to_f(d[c]), to_f(v[c]), dp);
        }
        dp = warp_sum(dp);
        d1 = fmaf(expf(fmaf(warp_sum(s[0]), p.scale, -l1)), dp, d1);
        d2 = fmaf(expf(fmaf(warp_sum(s[1]), p.scale, -l2)), dp, d2);
    }
    if (lane == 0) {   // (NaN marks stay)
        p.delta[col] = d1 + 0.f * p.delta[col];
        p.delta[col + rows] = d2 + 0.f * p.delta[col + rows];
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

// Global rows' dV and dK from the parts' sums: one thread per four channels of a
// (row, head), parts added in order.
template <typename T>
struct JoinPtr {
    const float *split, *lambda;
    T *dv, *dk;
    int64_t batch, rows;
    int32_t heads, n_lambda, parts;
    float scale;
};

template <typename T, int HD>
__global__ void __launch_bounds__(256) diff_split_join_kernel(const JoinPtr<T> p) {
    constexpr int kVecs = 2 * HD / 4;
    const int64_t cells = p.batch * p.heads;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= cells * p.rows * kVecs) return;
    const int64_t at = i / kVecs;   // (cell, row)
    const int c = static_cast<int>(i - at * kVecs) * 4;
    const int64_t cell = at / p.rows, row = at - cell * p.rows;
    const int64_t b = cell / p.heads, head = cell - b * p.heads;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int part = 0; part < p.parts; ++part) {
        const float4 x = __ldcs(reinterpret_cast<const float4 *>(
            p.split + (part * cells * p.rows + at) * (2 * HD) + c));
        s.x += x.x;
        s.y += x.y;
        s.z += x.z;
        s.w += x.w;
    }
    const bool dv = c < HD;
    const int ch = dv ? c : c - HD;
    const float f = dv ? 1.f
                       : (ch < HD / 2 ? p.scale
                                      : -p.scale * __ldg(p.lambda + (p.n_lambda == 1 ? 0 : head)));
    T *out = (dv ? p.dv : p.dk) + ((b * p.rows + row) * p.heads + head) * HD + ch;
    out[0] = from_f<T>(s.x * f);
    out[1] = from_f<T>(s.y * f);
    out[2] = from_f<T>(s.z * f);
    out[3] = from_f<T>(s.w * f);
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

// Launched where rows with few keys are possible.
template <int HD>
atlas_status few_hd(const DiffBwdArgs &b, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    const bool global_rows = a.n_global > 0 && a.n_global <= kFewKeys;
    const bool detail_rows = a.n_detail > 0 && (a.win_off || a.window_len <= kFewKeys) &&
                             (a.n_global <= kFewKeys || a.gwin_off);
    if (!global_rows && !detail_rows) return ATLAS_OK;
    const int64_t n_win = !detail_rows ? 0 : a.win_off ? a.n_win : a.n_detail / a.window_len;
    FewPtr p;
    p.q[0] = static_cast<const __nv_bfloat16 *>(a.q_d);
    p.q[1] = static_cast<const __nv_bfloat16 *>(a.q_g);
    p.k[0] = static_cast<const __nv_bfloat16 *>(a.k_d);
    p.k[1] = static_cast<const __nv_bfloat16 *>(a.k_g);
    p.v[0] = static_cast<const __nv_bfloat16 *>(a.v_d);
    p.v[1] = static_cast<const __nv_bfloat16 *>(a.v_g);
    p.go[0] = static_cast<const __nv_bfloat16 *>(b.do_d);
    p.go[1] = static_cast<const __nv_bfloat16 *>(b.do_g);
    p.lse = a.lse;
    p.delta = b.delta;
    p.scale = a.scale;
    const int64_t blocks = a.batch * (n_win + 1);
    if (blocks > INT32_MAX) return ATLAS_ERR_SHAPE;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(a.heads));
    if (log_enabled())
        log_launch("diff_few_keys_kernel", static_cast<int>(grid.x * grid.y), kWarps * 32, 0,
                   "head_dim %d windows %lld heads %d", HD, static_cast<long long>(n_win), a.heads);
    diff_few_keys_kernel<HD><<<grid, kWarps * 32, 0, stream>>>(p, attn_geom_of(a), n_win);
    return launched();
}

template <typename T, int HD>
atlas_status join_hd(const DiffBwdArgs &b, int parts, cudaStream_t stream) {
    const AttnArgs &a = b.fwd.attn;
    JoinPtr<T> p;
    p.split = b.split;
    p.lambda = b.fwd.lambda;
    p.dv = static_cast<T *>(b.dv_g);
    p.dk = static_cast<T *>(b.dk_g);
    p.batch = a.batch;
    p.rows = a.n_global;
    p.heads = a.heads;
    p.n_lambda = b.fwd.n_lambda;
    p.parts = parts;
    p.scale = a.scale;
    const int64_t vecs = a.batch * a.n_global * a.heads * (2 * HD / 4);
    diff_split_join_kernel<T, HD><<<static_cast<unsigned>((vecs + 255) / 256), 256, 0, stream>>>(p);
    return launched();
}

}  // namespace

// The count, up to 16 (bf16) or 64 (fp32), with the fewest tiles on the busiest of
// a B200's 148 SMs, a block's start and end taken as four tiles and the joining
// launch as eight. bf16 at 720p: with one head 40 units of 1,785 tiles kept 40 SMs
// busy for 2,423 us, cut into 11 parts 440 units take all of them 805 us; from four
// heads on the uncut units fill the SMs.
int diff_split_plan(int64_t batch, int64_t n_detail, int64_t n_global, int32_t heads,
                    int elem_bytes) {
    constexpr int64_t kSms = 148;
    const int64_t rows = elem_bytes == 2 ? 128 : 64;   // key rows of a block
    const int64_t tile = elem_bytes == 2 ? 48 : 64;    // streamed rows of a tile
    const int most = elem_bytes == 2 ? 16 : 64;
    const int64_t units = (n_global + rows - 1) / rows * batch * heads;
    const int64_t len = (n_detail + n_global + tile - 1) / tile;
    if (units == 0 || units > 16 * kSms) return 1;
    const int64_t whole = (units + kSms - 1) / kSms * (len + 4);
    int best = 1;
    int64_t least = whole;
    for (int s = 2; s <= most; ++s) {
        const int64_t load = (units * s + kSms - 1) / kSms * ((len + s - 1) / s + 4) + 8;
        if (load < least) {
            best = s;
            least = load;
        }
    }
    return 10 * least < 9 * whole ? best : 1;
}

atlas_status launch_diff_split_join(const DiffBwdArgs &b, int parts, cudaStream_t stream) {
    if (b.fwd.elem_bytes == 2)
        return b.fwd.attn.head_dim == 128 ? join_hd<__nv_bfloat16, 128>(b, parts, stream)
                                          : join_hd<__nv_bfloat16, 64>(b, parts, stream);
    return b.fwd.attn.head_dim == 128 ? join_hd<float, 128>(b, parts, stream)
                                      : join_hd<float, 64>(b, parts, stream);
}

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

atlas_status launch_diff_bwd_delta(const DiffBwdArgs &b, cudaStream_t stream) {
    if (b.fwd.elem_bytes == 2) {
        const bool wide = b.fwd.attn.head_dim == 128;
        const atlas_status st = wide ? delta_hd<__nv_bfloat16, 128>(b, stream)
                                     : delta_hd<__nv_bfloat16, 64>(b, stream);
        if (st != ATLAS_OK) return st;
        return wide ? few_hd<128>(b, stream) : few_hd<64>(b, stream);
    }
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

}  // namespace atlas
