// group_norm.cu -- group norm with an activation, channels last, and its
// gradients.
//
// Over the n = rows * channels/groups elements of a (sample, group):
//   xhat = (x - mean) rstd,  z = gamma xhat + beta,  y = act(z).
// Backward, with dz = dy act'(z), dh = dz gamma:
//   dx = rstd (dh - mean(dh) - xhat mean(dh xhat)),
//   dgamma = sum dz xhat,  dbeta = sum dz.
// HBM-bound throughout. Three forms, by what one sample's group needs:
//   heads     one row per sample and a group of 1, 2, 4, .. 32 16-byte vectors:
//             a group is that many lanes of a warp, its sums are shuffles, and
//             every element is read once;
//   resident  a sample's rows of some whole groups fit in shared memory: a block
//             reads them once and keeps them there between the sums and the
//             result;
//   split     anything longer: the sums' pass is cut into chunks of rows over the
//             whole GPU, partial sums per channel are joined by a second kernel,
//             and a third writes the result, walking the rows backwards so that
//             it starts with the rows that are still in L2.
// Measured: 80,640 tokens of 40 heads of 128, bf16, 314 us for 1.65 GB (5.3 TB/s,
// 80% of a copy); decoder latents 2 x 322,560 x 128, SiLU, forward and backward 308 us
// (0.83 GB: 2.7 TB/s; sums 35 and 84 us, results 73 and 101, joins 8 each); 3 x 1,001 x
// 60, fp32, 39 us, of which the forward's nine resident blocks are 28.
// Variances are sums of squared deviations: from the mean where the values are
// held (heads, resident), else from a pivot that a thread moves to the mean of its
// rows so far (split), joined in fp64, so that neither a large mean nor a first row
// unlike the others costs digits of the deviations.
#include <cuda_bf16.h>

#include <algorithm>

#include "atlas_internal.cuh"
#include "cube_geom.cuh"

namespace atlas {
namespace {

using geom::FastDiv;

constexpr int kThreads = 256;
constexpr uint32_t kAll = 0xffffffffu;
constexpr int kSms = 148;                    // of a B200: grids and workspaces are sized by it
constexpr int64_t kResidentBytes = 96 * 1024;
// Blocks of a split pass. Decoder latents (2 x 322,560 x 128), microseconds of the
// four passes: 2, 4, 8 and 16 blocks an SM 294, 299, 309 and 412: few blocks with
// long loops. Four fill the SMs at every register count.
constexpr int64_t kSplitBlocks = 4 * kSms;
// Rows that one thread of a split pass sums in fp32, at most: each sum is then within
// 1,024 * 2^-24 of its terms' magnitudes, however many samples fill the GPU by
// themselves. The parts it adds are 8 bytes a channel for 1,024 rows or more.
constexpr int64_t kThreadRows = 1024;
constexpr int64_t kPartBlocks = 4 * kSms;    // blocks of a backward pass that keep dgamma sums

struct Params {
    const void *x, *dy;
    void *out;                      // y or dx
    const float *gamma, *beta;
    float *stats;                   // (mean, rstd) of every (sample, group); may be NULL forward
    float *dgamma, *dbeta;
    int64_t samples, rows, channels;
    int32_t groups, cg, silu;
    float eps;
    int32_t width, per_block;       // heads, split: columns of a slice, rows at a time
    // resident: groups and channels of a slice, slices; threads per group
    int32_t slice_groups, slices, team;
    FastDiv by_cgv;
    // split: rows of a chunk, chunks of a sample
    int64_t chunk_rows;
    int32_t chunks;
    float2 *part;                   // partial sums (see each kernel)
    float2 *coef;                   // split: (mean, rstd), or the backward's two means
    int32_t n_parts;                // partial sums of dgamma and dbeta
};

template <typename T>
struct Io;
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ float get(const float &v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Io<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ float get(const __nv_bfloat16 &v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

// V consecutive values (16 bytes, or one).
template <typename T, int V>
struct Pack {
    T v[V];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (V > 1) *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(p);
        else v[0] = *p;
    }
    __device__ __forceinline__ void store(T *p) const {
        if constexpr (V > 1) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(v);
        else *p = v[0];
    }
    // The same for data that is not read again: first to leave L2.
    __device__ __forceinline__ void load_last(const T *p) {
        if constexpr (V > 1) *reinterpret_cast<uint4 *>(v) = __ldcs(reinterpret_cast<const uint4 *>(p));
        else v[0] = *p;
    }
    __device__ __forceinline__ void store_last(T *p) const {
        if constexpr (V > 1) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(v));
        else *p = v[0];
    }
    __device__ __forceinline__ float operator[](int i) const { return Io<T>::get(v[i]); }
    __device__ __forceinline__ void set(int i, float f) { v[i] = Io<T>::put(f); }
};
template <typename T, int V>
struct alignas(V > 1 ? 16 : sizeof(T)) Vec : Pack<T, V> {};

// The caller's statistics lie on a 4-byte boundary, not on a float2's.
__device__ __forceinline__ float2 stat_of(const Params &p, int64_t i) {
    return make_float2(__ldg(p.stats + 2 * i), __ldg(p.stats + 2 * i + 1));
}
__device__ __forceinline__ void put_stat(const Params &p, int64_t i, float mean, float rstd) {
    p.stats[2 * i] = mean;
    p.stats[2 * i + 1] = rstd;
}
__device__ __forceinline__ float gamma_of(const Params &p, int64_t c) {
    return p.gamma ? __ldg(p.gamma + c) : 1.f;
}
__device__ __forceinline__ float beta_of(const Params &p, int64_t c) {
    return p.beta ? __ldg(p.beta + c) : 0.f;
}
// 2^x, 2 ulp.
__device__ __forceinline__ float exp2f_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-z)). bf16 takes the fast exponential, whose relative error of 2^-21 +
// 2^-22 |z| is far inside the output's rounding wherever the value is not negligible
// beside the others. fp32 keeps the digits of small values too: -z log2(e) as a
// rounded product and, by fma, what it lacks; 2^(h + l) = 2^h (1 + l ln 2). Below z =
// -87 the quotient may be 0 (silu there: below 2^-119).
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-z));
    constexpr float kLog2e = 0x1.715476p+0f, kRest = 0x1.4ae0c0p-26f, kLn2 = 0x1.62e430p-1f;
    const float y = fminf(fmaxf(-z, -200.f), 200.f);   // (l of an infinite one would be NaN)
    const float h = y * kLog2e, l = fmaf(y, kRest, fmaf(y, kLog2e, -h));
    return __fdividef(1.f, fmaf(exp2f_fast(h), fmaf(l, kLn2, 1.f), 1.f));
}
// act(z), and dy act'(z).
template <typename T>
__device__ __forceinline__ float act(float z, int silu) { return silu ? z * sigmoid<T>(z) : z; }
template <typename T>
__device__ __forceinline__ float act_grad(float dy, float z, int silu) {
    if (!silu) return dy;
    const float s = sigmoid<T>(z);
    return dy * (s * fmaf(z, 1.f - s, 1.f));
}
// xhat and dz of one element.
struct Grad {
    float hat, dz;
};
template <typename T>
__device__ __forceinline__ Grad grad_of(float x, float dy, float2 st, float ga, float be, int silu) {
    Grad g;
    g.hat = (x - st.x) * st.y;
    g.dz = act_grad<T>(dy, fmaf(g.hat, ga, be), silu);
    return g;
}
// dh: its own rounding, so that a group of one value gives exactly 0.
__device__ __forceinline__ float dh_of(float dz, float ga) { return __fmul_rn(dz, ga); }

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
    for (int off = lanes / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    return v;
}

// ---------------------------------------------------------------------------
// Heads: rows == 1. Thread = one 16-byte column of a token; block = a slice of up
// to 256 columns (blockIdx.y), or several tokens when the rows are shorter; a
// thread keeps its column for all its tokens, so gamma, beta and its sums of
// dgamma and dbeta stay in registers.
// ---------------------------------------------------------------------------
template <typename T, int LANES, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_heads_kernel(const Params p) {
    constexpr int V = Io<T>::kVec, kFlight = BWD ? 2 : 4;
    const int nv = static_cast<int>(p.channels / V);
    const int width = p.width, per_block = p.per_block;   // tokens at a time
    const int sub = threadIdx.x / width;
    const int col = blockIdx.y * width + threadIdx.x - sub * width;
    const bool active = sub < per_block && col < nv;
    const int64_t ch = static_cast<int64_t>(col) * V, group = col / LANES;
    float ga[V], be[V], dga[V], dbe[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        ga[e] = active ? gamma_of(p, ch + e) : 0.f;
        be[e] = active ? beta_of(p, ch + e) : 0.f;
        dga[e] = dbe[e] = 0.f;
    }
    const float inv_n = 1.f / (LANES * V);
    const int64_t step = static_cast<int64_t>(gridDim.x) * per_block;
    const T *x = static_cast<const T *>(p.x), *dy = static_cast<const T *>(p.dy);
    for (int64_t s0 = static_cast<int64_t>(blockIdx.x) * per_block; s0 < p.samples;
         s0 += step * kFlight) {
        Vec<T, V> xv[kFlight], gv[kFlight];
        float2 st[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t s = s0 + f * step + sub;
            const bool on = active && s < p.samples;
            const int64_t at = (on ? s : 0) * p.channels + (on ? ch : 0);
            xv[f].load_last(x + at);
            if (BWD) {
                gv[f].load_last(dy + at);
                st[f] = stat_of(p, on ? s * p.groups + group : 0);
            }
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t s = s0 + f * step + sub;
            const bool on = active && s < p.samples;
            Vec<T, V> o;
            if (!BWD) {
                float sum = 0.f, sq = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) sum += xv[f][e];
                const float mean = lanes_sum(sum, LANES) * inv_n;
#pragma unroll
                for (int e = 0; e < V; ++e) sq = fmaf(xv[f][e] - mean, xv[f][e] - mean, sq);
                const float rstd = rsqrtf(fmaf(lanes_sum(sq, LANES), inv_n, p.eps));
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o.set(e, act<T>(fmaf((xv[f][e] - mean) * rstd, ga[e], be[e]), p.silu));
                if (on && p.stats != nullptr && col % LANES == 0)
                    put_stat(p, s * p.groups + group, mean, rstd);
            } else {
                float hat[V], dh[V], s1 = 0.f, s2 = 0.f;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const Grad g = grad_of<T>(xv[f][e], gv[f][e], st[f], ga[e], be[e], p.silu);
                    hat[e] = g.hat;
                    dh[e] = dh_of(g.dz, ga[e]);
                    s1 += dh[e];
                    s2 = fmaf(dh[e], g.hat, s2);
                    if (on) {
                        dga[e] = fmaf(g.dz, g.hat, dga[e]);
                        dbe[e] += g.dz;
                    }
                }
                const float m1 = lanes_sum(s1, LANES) * inv_n, m2 = lanes_sum(s2, LANES) * inv_n;
#pragma unroll
                for (int e = 0; e < V; ++e) o.set(e, st[f].y * (dh[e] - m1 - hat[e] * m2));
            }
            if (on) o.store_last(static_cast<T *>(p.out) + s * p.channels + ch);
        }
    }
    if (BWD && p.n_parts > 0) {
        // part [block][channel] of (dgamma, dbeta): the block's tokens in order
        __shared__ float2 sums[kThreads][V + 1];
#pragma unroll
        for (int e = 0; e < V; ++e) sums[threadIdx.x][e] = make_float2(dga[e], dbe[e]);
        __syncthreads();
        if (sub == 0 && col < nv) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float2 a = sums[threadIdx.x][e];
                for (int k = 1; k < per_block; ++k) {
                    a.x += sums[k * width + threadIdx.x][e].x;
                    a.y += sums[k * width + threadIdx.x][e].y;
                }
                p.part[blockIdx.x * p.channels + ch + e] = a;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Resident: block = a slice of whole groups (blockIdx.y) of one sample after
// another. A group's `team` threads (a power of two) hold its V-wide items
// (row, column) in turn, in shared memory of their own.
// ---------------------------------------------------------------------------
template <typename T, int V, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_resident_kernel(const Params p) {
    extern __shared__ uint8_t smem[];
    __shared__ float warp_sums[2][kThreads / 32];
    const int cgv = p.cg / V, team = p.team, g = threadIdx.x / team, lane = threadIdx.x % team;
    const int g0 = blockIdx.y * p.slice_groups, ng = min(p.slice_groups, p.groups - g0);
    const bool on = g < ng;
    const int64_t n_items = on ? p.rows * cgv : 0;
    const float n = static_cast<float>(p.rows * p.cg);   // (a division: exact for a constant)
    const int width = p.slice_groups * p.cg;   // channels of a slice
    T *xs = reinterpret_cast<T *>(smem);
    T *gs = xs + p.rows * width;               // BWD: dy
    float2 *acc = reinterpret_cast<float2 *>(
        smem + (2 * p.rows * width * sizeof(T) + 15) / 16 * 16);   // BWD: (dgamma, dbeta) [width]
    const int64_t ch0 = static_cast<int64_t>(g0) * p.cg;
    if (BWD)
        for (int c = threadIdx.x; c < width; c += kThreads) acc[c] = make_float2(0.f, 0.f);
    // Sum over a team, the same in all its threads (every thread calls).
    int which = 0;
    auto team_sum = [&](float v) -> float {
        v = lanes_sum(v, min(team, 32));
        if (team <= 32) return v;
        which ^= 1;   // the other buffer: one barrier a sum
        if ((threadIdx.x & 31) == 0) warp_sums[which][threadIdx.x / 32] = v;
        __syncthreads();
        float s = 0.f;
        const int first = threadIdx.x / team * (team / 32);
        for (int i = 0; i < team / 32; ++i) s += warp_sums[which][first + i];
        return s;
    };
    for (int64_t s = blockIdx.x; s < p.samples; s += gridDim.x) {
        const int64_t base = s * p.rows * p.channels + ch0;
        const T *x = static_cast<const T *>(p.x) + base, *dy = static_cast<const T *>(p.dy) + base;
        T *out = static_cast<T *>(p.out) + base;
        // item i of the group: row, then column; in the tensor and in the slice
        auto place = [&](int64_t i, int64_t &at, int &in, int &c) {
            const uint32_t r = p.by_cgv.div(static_cast<uint32_t>(i));
            c = g * p.cg + static_cast<int>(i - static_cast<int64_t>(r) * cgv) * V;
            at = r * p.channels + c;
            in = static_cast<int>(r) * width + c;
        };
        int64_t at;
        int in, c;
        const int64_t stat = s * p.groups + g0 + g;
        if (!BWD) {
            float sum = 0.f;
            for (int64_t i = lane; i < n_items; i += team) {
                place(i, at, in, c);
                Vec<T, V> v;
                v.load(x + at);
                v.store(xs + in);
#pragma unroll
                for (int e = 0; e < V; ++e) sum += v[e];
            }
            const float mean = team_sum(sum) / n;
            float sq = 0.f;
            for (int64_t i = lane; i < n_items; i += team) {
                place(i, at, in, c);
                Vec<T, V> v;
                v.load(xs + in);
#pragma unroll
                for (int e = 0; e < V; ++e) sq = fmaf(v[e] - mean, v[e] - mean, sq);
            }
            const float rstd = rsqrtf(team_sum(sq) / n + p.eps);
            for (int64_t i = lane; i < n_items; i += team) {
                place(i, at, in, c);
                Vec<T, V> v, o;
                v.load(xs + in);
#pragma unroll
                for (int e = 0; e < V; ++e)
                    o.set(e, act<T>(fmaf((v[e] - mean) * rstd, gamma_of(p, ch0 + c + e),
                                      beta_of(p, ch0 + c + e)), p.silu));
                o.store(out + at);
            }
            if (on && lane == 0 && p.stats != nullptr) put_stat(p, stat, mean, rstd);
        } else {
            const float2 st = on ? stat_of(p, stat) : make_float2(0.f, 0.f);
            float s1 = 0.f, s2 = 0.f;
            for (int64_t i = lane; i < n_items; i += team) {
                place(i, at, in, c);
                Vec<T, V> v, w;
                v.load(x + at);
                w.load(dy + at);
                v.store(xs + in);
                w.store(gs + in);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float ga = gamma_of(p, ch0 + c + e);
                    const Grad d = grad_of<T>(v[e], w[e], st, ga, beta_of(p, ch0 + c + e), p.silu);
                    s1 += dh_of(d.dz, ga);
                    s2 = fmaf(dh_of(d.dz, ga), d.hat, s2);
                }
            }
            const float m1 = team_sum(s1) / n, m2 = team_sum(s2) / n;
            for (int64_t i = lane; i < n_items; i += team) {
                place(i, at, in, c);
                Vec<T, V> v, w, o;
                v.load(xs + in);
                w.load(gs + in);
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float ga = gamma_of(p, ch0 + c + e);
                    const Grad d = grad_of<T>(v[e], w[e], st, ga, beta_of(p, ch0 + c + e), p.silu);
                    o.set(e, st.y * (dh_of(d.dz, ga) - m1 - d.hat * m2));
                }
                o.store(out + at);
            }
            if (p.n_parts > 0) {
                // dgamma, dbeta: thread = channel, rows in order
                __syncthreads();
                for (int k = threadIdx.x; k < ng * p.cg; k += kThreads) {
                    const float2 sk = stat_of(p, s * p.groups + g0 + k / p.cg);
                    const float ga = gamma_of(p, ch0 + k), be = beta_of(p, ch0 + k);
                    float2 a = acc[k];
                    for (int64_t r = 0; r < p.rows; ++r) {
                        const Grad d = grad_of<T>(Io<T>::get(xs[r * width + k]),
                                               Io<T>::get(gs[r * width + k]), sk, ga, be, p.silu);
                        a.x = fmaf(d.dz, d.hat, a.x);
                        a.y += d.dz;
                    }
                    acc[k] = a;
                }
                __syncthreads();
            }
        }
    }
    if (BWD && p.n_parts > 0) {
        __syncthreads();
        for (int c = threadIdx.x; c < ng * p.cg; c += kThreads)
            p.part[blockIdx.x * p.channels + ch0 + c] = acc[c];
    }
}

// ---------------------------------------------------------------------------
// Split: thread = one column of V channels for all rows of a chunk; block = a
// slice of up to 256 columns (blockIdx.y) of one chunk of a sample (blockIdx.x),
// several rows at a time when the rows are shorter.
// ---------------------------------------------------------------------------
struct Slot {
    int sub, col;
    bool active;
};
__device__ __forceinline__ Slot slot_of(const Params &p, int64_t nv) {
    Slot t;
    t.sub = threadIdx.x / p.width;
    t.col = blockIdx.y * p.width + threadIdx.x - t.sub * p.width;
    t.active = t.sub < p.per_block && t.col < nv;
    return t;
}

// Forward: part [sample][chunk][channel] = (mean, M2) of the chunk's rows. A thread
// sums deviations from a pivot, its first value of the channel, and their squares.
// M2 = sum d^2 - (sum d)^2 / n loses what a pivot far from the mean makes the two
// share, so after 4, 16, 64, .. rows the pivot moves to their mean: among n rows of
// which k have mean 0 (about the pivot), M2 is at least k/n of sum d^2, so no move and
// no end takes away more than two bits. Backward: (sum dz xhat, sum dz).
template <typename T, int V, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_split_sums_kernel(const Params p) {
    constexpr int kFlight = 4;
    __shared__ float2 sums[kThreads][V + 1];
    const Slot t = slot_of(p, p.channels / V);
    const int64_t ch = static_cast<int64_t>(t.col) * V;
    const int64_t s = blockIdx.x / p.chunks, chunk = blockIdx.x - s * p.chunks;
    const int64_t r0 = chunk * p.chunk_rows, r1 = min(r0 + p.chunk_rows, p.rows);
    const T *x = static_cast<const T *>(p.x) + s * p.rows * p.channels + ch;
    const T *dy = static_cast<const T *>(p.dy) + s * p.rows * p.channels + ch;
    float a[V], b[V];
#pragma unroll
    for (int e = 0; e < V; ++e) a[e] = b[e] = 0.f;
    if (t.active) {
        float ga[V], be[V];
        float2 st[V];   // forward: the pivot
        Vec<T, V> first;
        first.load(x + min(r0 + t.sub, r1 - 1) * p.channels);
        int64_t n = 0, move_at = kFlight;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            if (BWD) {
                ga[e] = gamma_of(p, ch + e);
                be[e] = beta_of(p, ch + e);
                st[e] = stat_of(p, s * p.groups + (ch + e) / p.cg);
            } else {
                st[e].x = first[e];
            }
        }
        for (int64_t r = r0 + t.sub; r < r1; r += kFlight * p.per_block) {
            Vec<T, V> v[kFlight], w[kFlight];
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                const int64_t rr = min(r + f * p.per_block, r1 - 1);
                v[f].load(x + rr * p.channels);
                if (BWD) w[f].load(dy + rr * p.channels);
            }
#pragma unroll
            for (int f = 0; f < kFlight; ++f) {
                if (r + f * p.per_block >= r1) continue;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    if (BWD) {
                        const Grad d = grad_of<T>(v[f][e], w[f][e], st[e], ga[e], be[e], p.silu);
                        a[e] = fmaf(d.dz, d.hat, a[e]);
                        b[e] += d.dz;
                    } else {
                        const float d = v[f][e] - st[e].x;
                        a[e] += d;
                        b[e] = fmaf(d, d, b[e]);
                    }
                }
                ++n;
            }
            if (!BWD && n == move_at) {
                const float fn = static_cast<float>(n), inv = 1.f / fn;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float to = fmaf(a[e], inv, st[e].x), by = to - st[e].x;
                    b[e] = fmaxf(fmaf(-by, 2.f * a[e] - fn * by, b[e]), 0.f);
                    a[e] = fmaf(-fn, by, a[e]);
                    st[e].x = to;
                }
                move_at *= 4;
            }
        }
        if (!BWD && n > 0) {   // to (mean, M2)
            const float inv = 1.f / static_cast<float>(n);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float d = a[e] * inv;
                b[e] = fmaxf(fmaf(-d, a[e], b[e]), 0.f);
                a[e] = st[e].x + d;
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) sums[threadIdx.x][e] = make_float2(a[e], b[e]);
    __syncthreads();
    // thread = channel of the slice
    for (int i = threadIdx.x; i < p.width * V; i += kThreads) {
        const int64_t c = static_cast<int64_t>(blockIdx.y) * p.width * V + i;
        if (c >= p.channels) break;
        float2 q = sums[i / V][i % V];
        if (BWD) {
            for (int k = 1; k < p.per_block; ++k) {
                q.x += sums[k * p.width + i / V][i % V].x;
                q.y += sums[k * p.width + i / V][i % V].y;
            }
        } else {
            // The threads' (mean, M2), about the first one's mean; thread k has
            // `each` rows, the first `more` threads one more.
            const int rows = static_cast<int>(r1 - r0), each = rows / p.per_block;
            const int more = rows - each * p.per_block, last = min(p.per_block, rows);
            const float inv = 1.f / static_cast<float>(rows);
            float d = 0.f, m2 = 0.f;
            for (int k = 1; k < last; ++k)
                d = fmaf(static_cast<float>(each + (k < more)),
                         sums[k * p.width + i / V][i % V].x - q.x, d);
            d *= inv;
            for (int k = 0; k < last; ++k) {
                const float2 w = sums[k * p.width + i / V][i % V];
                const float off = w.x - q.x - d;
                m2 += fmaf(static_cast<float>(each + (k < more)) * off, off, w.y);
            }
            q = make_float2(q.x + d, m2);
        }
        p.part[blockIdx.x * p.channels + c] = q;
    }
}

// Sum over the block in fp64, in a fixed order, in every thread.
__device__ __forceinline__ double block_sum(double v) {
    __shared__ double part[kThreads / 32];
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double s = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

// dgamma and dbeta of 32 channels from the parts: eight warps add every eighth
// part each, in order; lane = channel.
__device__ __forceinline__ void dgamma_sums(const Params &p, int64_t block) {
    __shared__ float2 sums[kThreads / 32][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int64_t c = block * 32 + lane;
    float2 a = make_float2(0.f, 0.f);
    if (c < p.channels) {
#pragma unroll 8
        for (int i = warp; i < p.n_parts; i += kThreads / 32) {
            const float2 q = p.part[i * p.channels + c];
            a.x += q.x;
            a.y += q.y;
        }
    }
    sums[warp][lane] = a;
    __syncthreads();
    if (warp != 0 || c >= p.channels) return;
    for (int i = 1; i < kThreads / 32; ++i) {
        a.x += sums[i][lane].x;
        a.y += sums[i][lane].y;
    }
    if (p.dgamma != nullptr) p.dgamma[c] = a.x;
    if (p.dbeta != nullptr) p.dbeta[c] = a.y;
}
__global__ void __launch_bounds__(kThreads) norm_dgamma_kernel(const Params p) {
    dgamma_sums(p, blockIdx.x);
}

// One block per (sample, group): the parts of its channels and chunks. Forward:
// coef = (mean, rstd), also into stats. Backward: the two means of dh; the blocks
// behind those sum dgamma and dbeta.
template <bool BWD>
__global__ void __launch_bounds__(kThreads) norm_split_join_kernel(const Params p) {
    const int64_t w = blockIdx.x;
    if (BWD && w >= p.samples * p.groups) {
        dgamma_sums(p, w - p.samples * p.groups);
        return;
    }
    const int64_t s = w / p.groups, c0 = (w - s * p.groups) * p.cg;
    const int64_t items = static_cast<int64_t>(p.chunks) * p.cg;
    const float2 *part = p.part + s * p.chunks * p.channels + c0;
    const double n = static_cast<double>(p.rows) * p.cg;
    double s1 = 0, s2 = 0;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < items; i += kThreads) {
        const int64_t chunk = i / p.cg, c = i - chunk * p.cg;
        const float2 q = part[chunk * p.channels + c];
        if (BWD) {
            const double ga = gamma_of(p, c0 + c);
            s1 += ga * q.y;
            s2 += ga * q.x;
        } else {
            s1 += static_cast<double>(min(p.chunk_rows, p.rows - chunk * p.chunk_rows)) * q.x;
        }
    }
    s1 = block_sum(s1) / n;
    if (BWD) {
        s2 = block_sum(s2) / n;
        if (threadIdx.x == 0) p.coef[w] = make_float2(static_cast<float>(s1), static_cast<float>(s2));
        return;
    }
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < items; i += kThreads) {
        const int64_t chunk = i / p.cg, c = i - chunk * p.cg;
        const float2 q = part[chunk * p.channels + c];
        const double d = q.x - s1;
        s2 += q.y + static_cast<double>(min(p.chunk_rows, p.rows - chunk * p.chunk_rows)) * d * d;
    }
    s2 = block_sum(s2) / n;
    if (threadIdx.x == 0) {
        const float2 st = make_float2(static_cast<float>(s1), rsqrtf(static_cast<float>(s2) + p.eps));
        p.coef[w] = st;
        if (p.stats != nullptr) put_stat(p, w, st.x, st.y);
    }
}

// The result, rows of all samples last to first. (fp32: three blocks an SM; left
// alone, the compiler takes 106 registers for eight rows' sigmoids side by side, two
// blocks: 400 x 20,000 x 32 without an activation 570 us, 540 with three; 2 x 322,560
// x 128 with SiLU 187, 196 with three.)
template <typename T, int V, bool BWD>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 && V > 1 ? 3 : 1)
norm_split_apply_kernel(const Params p) {
    constexpr int kFlight = BWD ? 4 : 8;
    const Slot t = slot_of(p, p.channels / V);
    if (!t.active) return;
    const int64_t ch = static_cast<int64_t>(t.col) * V;
    const int64_t block = gridDim.x - 1 - blockIdx.x;   // (sample, chunk)
    const int64_t s = block / p.chunks, chunk = block - s * p.chunks;
    const int64_t r0 = chunk * p.chunk_rows, r1 = min(r0 + p.chunk_rows, p.rows);
    const int64_t base = s * p.rows * p.channels + ch;
    const T *x = static_cast<const T *>(p.x) + base, *dy = static_cast<const T *>(p.dy) + base;
    T *out = static_cast<T *>(p.out) + base;
    float ga[V], be[V];
    float2 st[V], mm[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int64_t w = s * p.groups + (ch + e) / p.cg;
        ga[e] = gamma_of(p, ch + e);
        be[e] = beta_of(p, ch + e);
        st[e] = BWD ? stat_of(p, w) : p.coef[w];
        mm[e] = BWD ? p.coef[w] : make_float2(0.f, 0.f);
    }
    for (int64_t r = r1 - 1 - t.sub; r >= r0; r -= kFlight * p.per_block) {
        Vec<T, V> v[kFlight], w[kFlight];
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t rr = max(r - f * p.per_block, r0);
            v[f].load_last(x + rr * p.channels);
            if (BWD) w[f].load_last(dy + rr * p.channels);
        }
#pragma unroll
        for (int f = 0; f < kFlight; ++f) {
            const int64_t rr = r - f * p.per_block;
            if (rr < r0) continue;
            Vec<T, V> o;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (BWD) {
                    const Grad d = grad_of<T>(v[f][e], w[f][e], st[e], ga[e], be[e], p.silu);
                    o.set(e, st[e].y * (dh_of(d.dz, ga[e]) - mm[e].x - d.hat * mm[e].y));
                } else {
                    o.set(e, act<T>(fmaf((v[f][e] - st[e].x) * st[e].y, ga[e], be[e]), p.silu));
                }
            }
            o.store_last(out + rr * p.channels);
        }
    }
}

// ---------------------------------------------------------------------------
// Host side: the form of a call, its grids and workspace.
// ---------------------------------------------------------------------------
enum Form { kHeads, kResident, kSplit };

struct Plan {
    Form form;
    bool vec;                  // 16-byte columns
    int lanes;                 // heads
    int32_t slice_groups, slices, team;
    int64_t smem;              // resident
    int64_t chunk_rows;
    int32_t chunks;
    int32_t width, per_block;  // heads, split: columns of a slice, rows at a time
    int64_t grid, slices_y;    // of the main passes
    int32_t parts;             // backward: partial sums of dgamma and dbeta
    int64_t part_bytes, coef_bytes;
};

// nv columns in slices of at most a block's threads: the width of whole warps that
// leaves the fewest threads idle, several rows at a time where it is half a block or
// less (640 columns: 5 slices of 128, two rows, 314 us for the 40 heads above; 3 of
// 224, one row, 350). With very many columns the last slice does not matter.
void slice_columns(int64_t nv, Plan *p) {
    int64_t width = nv <= kThreads ? nv : kThreads, best = 0;
    if (nv > kThreads && nv <= 64 * kThreads)
        for (int64_t w = kThreads; w >= 64; w -= 32) {
            // threads in use, per 2^20
            const int64_t use = (nv << 20) / ((nv + w - 1) / w * w) * (kThreads / w * w) / kThreads;
            if (use > best) {
                best = use;
                width = w;
            }
        }
    p->slices_y = (nv + width - 1) / width;
    p->width = static_cast<int32_t>(width);
    p->per_block = kThreads / p->width;
}

Plan plan_of(const NormArgs &a, bool bwd) {
    Plan p{};
    const int64_t eb = a.elem_bytes, cg = a.channels / a.groups;
    const int vec = static_cast<int>(16 / eb);
    const bool aligned = a.channels % vec == 0;
    // Heads: the lanes of a group within a warp.
    if (a.rows == 1 && cg % vec == 0) {
        const int64_t lanes = cg / vec;
        if (lanes <= 32 && (lanes & (lanes - 1)) == 0) {
            p.form = kHeads;
            p.vec = true;
            p.lanes = static_cast<int>(lanes);
            slice_columns(a.channels / vec, &p);
            const int64_t tokens = (a.samples + p.per_block - 1) / p.per_block;
            // (forward, a slice: 2, 4, 5 and 8 blocks an SM 334, 314, 327 and 325 us)
            p.grid = std::min<int64_t>(tokens, bwd ? kPartBlocks : 4 * kSms);
            p.parts = static_cast<int32_t>(p.grid);
            p.part_bytes = bwd ? p.parts * a.channels * 8 : 0;
            return p;
        }
    }
    // Resident: the fewest groups whose rows are at least two sectors long (64
    // bytes), 16-byte aligned where the tensor allows it, and fill a block's
    // threads eight items deep; twice that while it stays within half of the
    // shared memory and two blocks an SM remain.
    const bool vec_items = aligned && cg % vec == 0;
    const int64_t per_group = a.rows * cg * eb * (bwd ? 2 : 1) + (bwd ? cg * 8 : 0);
    int64_t sg = 1;
    while (sg < a.groups && sg * cg * eb < 64) sg *= 2;
    while (sg < a.groups && 2 * sg <= kThreads && 2 * sg * per_group <= kResidentBytes / 2 &&
           a.samples * ((a.groups + 2 * sg - 1) / (2 * sg)) >= 2 * kSms)
        sg *= 2;
    sg = std::min<int64_t>(sg, a.groups);
    if (sg <= kThreads && sg * per_group + 16 <= kResidentBytes &&
        a.rows * (cg / (vec_items ? vec : 1)) < (1ll << 31)) {
        p.form = kResident;
        p.vec = vec_items;
        p.slice_groups = static_cast<int32_t>(sg);
        p.slices = static_cast<int32_t>((a.groups + sg - 1) / sg);
        p.team = 1;
        while (2 * p.team * sg <= kThreads) p.team *= 2;
        p.smem = sg * per_group + 16;
        const int64_t fill = (bwd ? kPartBlocks : 1 << 20);
        p.grid = std::min<int64_t>(a.samples, std::max<int64_t>(1, fill / p.slices));
        p.parts = static_cast<int32_t>(p.grid);
        p.part_bytes = bwd ? p.parts * a.channels * 8 : 0;
        p.slices_y = p.slices;
        if (p.slices <= 65535) return p;
    }
    // Split.
    p.form = kSplit;
    p.vec = aligned;
    slice_columns(a.channels / (aligned ? vec : 1), &p);
    const int64_t want = std::max<int64_t>(1, kSplitBlocks / (a.samples * p.slices_y));
    p.chunk_rows = std::min((a.rows + want - 1) / want, kThreadRows * p.per_block);
    p.chunks = static_cast<int32_t>((a.rows + p.chunk_rows - 1) / p.chunk_rows);
    p.grid = a.samples * p.chunks;
    p.parts = static_cast<int32_t>(p.grid);
    p.part_bytes = p.grid * a.channels * 8;
    p.coef_bytes = a.samples * a.groups * 8;
    return p;
}

template <typename T, int LANES>
void heads(const Params &p, dim3 grid, bool bwd, cudaStream_t s) {
    if (bwd) norm_heads_kernel<T, LANES, true><<<grid, kThreads, 0, s>>>(p);
    else norm_heads_kernel<T, LANES, false><<<grid, kThreads, 0, s>>>(p);
}

template <typename T, int V>
atlas_status resident(const Params &p, const Plan &plan, bool bwd, cudaStream_t s) {
    auto kernel = bwd ? norm_resident_kernel<T, V, true> : norm_resident_kernel<T, V, false>;
    if (!set_smem_limit(reinterpret_cast<const void *>(kernel), static_cast<int>(kResidentBytes)))
        return ATLAS_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(plan.grid), static_cast<unsigned>(plan.slices));
    kernel<<<grid, kThreads, static_cast<size_t>(plan.smem), s>>>(p);
    return ATLAS_OK;
}

template <typename T, int V>
void split(const Params &p, const Plan &plan, bool bwd, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(plan.grid), static_cast<unsigned>(plan.slices_y));
    const unsigned join = static_cast<unsigned>(p.samples * p.groups);
    if (bwd) {
        const unsigned more = p.n_parts > 0 ? static_cast<unsigned>((p.channels + 31) / 32) : 0;
        norm_split_sums_kernel<T, V, true><<<grid, kThreads, 0, s>>>(p);
        norm_split_join_kernel<true><<<join + more, kThreads, 0, s>>>(p);
        norm_split_apply_kernel<T, V, true><<<grid, kThreads, 0, s>>>(p);
    } else {
        norm_split_sums_kernel<T, V, false><<<grid, kThreads, 0, s>>>(p);
        norm_split_join_kernel<false><<<join, kThreads, 0, s>>>(p);
        norm_split_apply_kernel<T, V, false><<<grid, kThreads, 0, s>>>(p);
    }
}

template <typename T>
atlas_status launch(const Params &p, const Plan &plan, bool bwd, cudaStream_t s) {
    constexpr int V = Io<T>::kVec;
    if (plan.form == kHeads) {
        const dim3 grid(static_cast<unsigned>(plan.grid), static_cast<unsigned>(plan.slices_y));
        switch (plan.lanes) {
            case 1: heads<T, 1>(p, grid, bwd, s); break;
            case 2: heads<T, 2>(p, grid, bwd, s); break;
            case 4: heads<T, 4>(p, grid, bwd, s); break;
            case 8: heads<T, 8>(p, grid, bwd, s); break;
            case 16: heads<T, 16>(p, grid, bwd, s); break;
            default: heads<T, 32>(p, grid, bwd, s); break;
        }
        return ATLAS_OK;
    }
    if (plan.form == kResident)
        return plan.vec ? resident<T, V>(p, plan, bwd, s) : resident<T, 1>(p, plan, bwd, s);
    if (plan.vec) split<T, V>(p, plan, bwd, s);
    else split<T, 1>(p, plan, bwd, s);
    return ATLAS_OK;
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

}  // namespace

int64_t group_norm_workspace(const NormArgs &a, bool bwd) {
    const Plan plan = plan_of(a, bwd);
    return round16(plan.part_bytes) + round16(plan.coef_bytes);
}

atlas_status launch_group_norm(const NormArgs &a, bool bwd, cudaStream_t stream) {
    const Plan plan = plan_of(a, bwd);
    const int vec = 16 / a.elem_bytes;
    if (plan.slices_y > 65535) return ATLAS_ERR_SHAPE;
    Params p{};
    p.x = a.x;
    p.dy = a.dy;
    p.out = a.out;
    p.gamma = a.gamma;
    p.beta = a.beta;
    p.stats = a.stats;
    p.dgamma = a.dgamma;
    p.dbeta = a.dbeta;
    p.samples = a.samples;
    p.rows = a.rows;
    p.channels = a.channels;
    p.groups = a.groups;
    p.cg = static_cast<int32_t>(a.channels / a.groups);
    p.silu = a.act == ATLAS_ACT_SILU;
    p.eps = static_cast<float>(a.eps);
    p.width = plan.width;
    p.per_block = plan.per_block;
    p.slice_groups = plan.slice_groups;
    p.slices = plan.slices;
    p.team = plan.team;
    p.by_cgv = FastDiv(static_cast<uint32_t>(p.cg / (plan.vec ? vec : 1)));
    p.chunk_rows = plan.chunk_rows;
    p.chunks = plan.chunks;
    p.part = static_cast<float2 *>(a.workspace);
    p.coef = reinterpret_cast<float2 *>(static_cast<uint8_t *>(a.workspace) + round16(plan.part_bytes));
    const bool sums = bwd && (a.dgamma != nullptr || a.dbeta != nullptr);
    p.n_parts = sums ? plan.parts : 0;
    static const char *const names[] = {"norm_heads_kernel", "norm_resident_kernel",
                                        "norm_split_*_kernel"};
    if (log_enabled())
        log_launch(names[plan.form], static_cast<int>(plan.grid), kThreads,
                   static_cast<size_t>(plan.smem),
                   "%s elem_bytes %d samples %lld rows %lld channels %lld groups %d vec %d",
                   bwd ? "backward" : "forward", a.elem_bytes, static_cast<long long>(p.samples),
                   static_cast<long long>(p.rows), static_cast<long long>(p.channels), p.groups,
                   plan.vec);
    const atlas_status st = a.elem_bytes == 2 ? launch<__nv_bfloat16>(p, plan, bwd, stream)
                                              : launch<float>(p, plan, bwd, stream);
    if (st != ATLAS_OK) return st;
    if (sums && plan.form != kSplit)
        norm_dgamma_kernel<<<static_cast<unsigned>((a.channels + 31) / 32), kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace atlas
