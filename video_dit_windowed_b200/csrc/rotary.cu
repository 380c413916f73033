// rotary.cu -- rotary positions in the general form: interleaved and half
// layouts, part of the head, positions of the grid or given per token,
// frequencies scaled for long contexts, several tensors (row-strided slices of
// a fused projection among them) in one launch.
//
// For pair k of an axis segment of width d, at scaled position p of its token:
//   phi = p * omega_k,   y1 = m (x1 cos phi - x2 sin phi),
//                        y2 = m (x1 sin phi + x2 cos phi),
// (x1, x2) channels (2k, 2k+1) of the segment, or (k, k + d/2) in the half
// layout. The transpose (the gradient's map) is the same with -phi. The pass is
// HBM-bound: one read and one write of every element. A block takes tiles of
// whole rows. For each tile it first writes the rows' cos and sin to shared
// memory, once per (row, pair), for every head of the row: the angle in turns
// p * omega / pi is formed and reduced to [-1, 1] in fp64, which keeps positions
// of 2^31 at fp32 accuracy and needs no table in device memory, so the call
// allocates and caches nothing. Then it moves the rows:
//   interleaved  a pair lies inside one 16-byte vector: one vector per thread,
//                rotated in registers;
//   half         partners lie d/2 channels apart, at any 2-byte distance (the
//                splits 44/42/42 put them 44 and 42 bytes apart): a warp stages
//                whole heads in shared memory, rotates pair by pair there (lane
//                = pair, so neighbouring lanes touch neighbouring channels) and
//                writes them out as vectors.
// Measured, whole calls: Q, K, V of 40 heads at 720p, half layout, cube order, 885 us
// for 4.95 GB (5.6 TB/s, 86% of a copy); 1.61 GB at given positions 261 us (94%); two
// heads' Q and K of partial cubes, where the angles are half of the work, 432 us for
// 2.12 GB (75%).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "atlas_internal.cuh"
#include "cube_geom.cuh"

namespace atlas {
namespace {

using geom::FastDiv;
using geom::Geom;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxPairs = kRotaryMaxHeadDim / 2;
constexpr int kTileAngles = 2048;     // (row, pair) angles of a tile
constexpr int kMaxTileRows = 32;
constexpr int kStageBytes = 2048;     // half layout: one warp's staging buffer

struct Tensor {
    const uint8_t *src;
    uint8_t *dst;
    int64_t src_stride, dst_stride;   // bytes between rows
    int32_t heads, rotate;
    uint32_t row_jobs;                // 32-vector jobs of a row
    FastDiv by_jobs;
};

struct Params {
    Tensor t[kRotaryMaxTensors];
    uint32_t rows, total_rows;        // tokens of one problem, of all problems
    uint32_t tile_rows, n_tiles;
    int32_t n_tensors;
    uint32_t head_bytes, vph;         // bytes and 16-byte vectors of one head
    uint32_t n_pairs;                 // rotated pairs of a head
    uint32_t pitch;                   // the same, even: entries of a row's cos and sin
    uint32_t step_rows, step_pairs;   // kThreads = step_rows * n_pairs + step_pairs
    uint32_t pair_end[2];             // pairs of axis t; of axes t and h
    uint32_t seg_first[3], seg_half[3];   // first channel and pair count of an axis segment
    FastDiv by_rows, by_pairs, by_vph;
    int32_t vph_mask;                 // vph - 1 when it is a power of two, else -1
    Geom g;
    int32_t order, even;              // atlas_order; the cube divides the grid
    const int32_t *positions;
    int32_t n_axes;
    float magnitude, sign;
    double turn[kMaxPairs];           // scale * omega / pi of every pair
};

// A row of the tile: where it comes from, where it goes, its position.
struct Row {
    uint32_t src, dst;
    int32_t pos[3];
};

__device__ __forceinline__ uint4 ld_row(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void st_row(uint8_t *p, const uint4 &v) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};"
                 :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ Row row_of(const Params &p, uint32_t i) {
    const uint32_t b = p.by_rows.div(i), x = i - b * p.rows;
    uint32_t t, h, w, raster = x, src = x;
    if (p.order == ATLAS_ORDER_REORDER) {
        if (p.even) geom::cube_coords(p.g, x, t, h, w);
        else geom::cube_coords_general(p.g, x, t, h, w);
        raster = src = (t * p.g.H + h) * p.g.W + w;
    } else {
        geom::raster_coords(p.g, x, t, h, w);
        if (p.order == ATLAS_ORDER_UNORDER)
            src = p.even ? geom::cube_position(p.g, t, h, w)
                         : geom::cube_position_general(p.g, t, h, w);
    }
    Row r;
    r.src = b * p.rows + src;
    r.dst = i;
    r.pos[0] = static_cast<int32_t>(t);
    r.pos[1] = static_cast<int32_t>(h);
    r.pos[2] = static_cast<int32_t>(w);
    if (p.positions != nullptr) {
        const int64_t at = static_cast<int64_t>(b * p.rows + raster) * p.n_axes;
        r.pos[0] = __ldg(p.positions + at);
        r.pos[1] = p.n_axes > 1 ? __ldg(p.positions + at + 1) : 0;
        r.pos[2] = p.n_axes > 1 ? __ldg(p.positions + at + 2) : 0;
    }
    return r;
}

// m * (cos, sin) of pair k at the row's position. bf16 takes the MUFU's sine and
// cosine (absolute error 2^-21 on [-pi, pi], a thousandth of the output's rounding),
// fp32 sincospif: rows of two heads, whose angles are half of the work, took 505 us
// with it and 460 without.
template <int EB>
__device__ __forceinline__ float2 angle_of(const Params &p, const double *turn, const Row &r,
                                           uint32_t k) {
    const int32_t x = k < p.pair_end[0] ? r.pos[0] : (k < p.pair_end[1] ? r.pos[1] : r.pos[2]);
    double y = static_cast<double>(x) * turn[k];
    y = fma(-2.0, rint(0.5 * y), y);
    float s, c;
    if constexpr (EB == 2) __sincosf(static_cast<float>(y) * 3.14159265f, &s, &c);
    else sincospif(static_cast<float>(y), &s, &c);
    return make_float2(c * p.magnitude, s * p.magnitude * p.sign);
}

__device__ __forceinline__ float2 turned(float a, float b, float2 cs) {
    return make_float2(fmaf(a, cs.x, -(b * cs.y)), fmaf(a, cs.y, b * cs.x));
}

// The pairs of a 16-byte vector, from pair k0 on; pairs past the rotated part
// keep their bits. cs + k0 is 16-byte aligned, and the pitch even: the second entry
// of the last float4 is the row's own.
template <int EB>
__device__ __forceinline__ uint4 rotate_vec(uint4 v, const float2 *cs, uint32_t k0,
                                            uint32_t n_pairs) {
    constexpr int kPairs = 8 / EB;
    uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < kPairs; j += 2) {
        if (k0 + j >= n_pairs) break;
        const float4 q = *reinterpret_cast<const float4 *>(cs + k0 + j);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (k0 + j + e >= n_pairs) continue;
            const float2 c = e == 0 ? make_float2(q.x, q.y) : make_float2(q.z, q.w);
            if constexpr (EB == 2) {
                const float2 y = turned(__uint_as_float(u[j + e] << 16),
                                        __uint_as_float(u[j + e] & 0xffff0000u), c);
                const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
                u[j + e] = *reinterpret_cast<const uint32_t *>(&b);
            } else {
                const float2 y = turned(__uint_as_float(u[2 * (j + e)]),
                                        __uint_as_float(u[2 * (j + e) + 1]), c);
                u[2 * (j + e)] = __float_as_uint(y.x);
                u[2 * (j + e) + 1] = __float_as_uint(y.y);
            }
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

template <int EB>
__device__ __forceinline__ float ld_ch(const uint8_t *s, uint32_t c) {
    if constexpr (EB == 2)
        return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(s)[c]);
    else
        return reinterpret_cast<const float *>(s)[c];
}
template <int EB>
__device__ __forceinline__ void st_ch(uint8_t *s, uint32_t c, float v) {
    if constexpr (EB == 2)
        reinterpret_cast<__nv_bfloat16 *>(s)[c] = __float2bfloat16_rn(v);
    else
        reinterpret_cast<float *>(s)[c] = v;
}

template <int EB, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Params p) {
    __shared__ Row rows[kMaxTileRows];
    __shared__ alignas(16) float2 cs[kTileAngles];   // [row][pitch]
    __shared__ double turn[kMaxPairs];
    __shared__ alignas(16) uint8_t stage[HALF ? kWarps : 1][HALF ? kStageBytes : 16];
    const uint32_t tid = threadIdx.x, warp = tid / 32, lane = tid & 31;
    for (uint32_t k = tid; k < p.n_pairs; k += kThreads) turn[k] = p.turn[k];
    const uint32_t first_row = p.by_pairs.div(tid), first_pair = tid - first_row * p.n_pairs;
    for (uint32_t tile = blockIdx.x; tile < p.n_tiles; tile += gridDim.x) {
        const uint32_t first = tile * p.tile_rows;
        const uint32_t n = min(p.tile_rows, p.total_rows - first);
        __syncthreads();   // the previous tile's rows have been moved
        if (tid < n) rows[tid] = row_of(p, first + tid);
        __syncthreads();
        if (p.n_pairs > 0) {
            uint32_t r = first_row, k = first_pair;
            while (r < n) {
                cs[r * p.pitch + k] = angle_of<EB>(p, turn, rows[r], k);
                r += p.step_rows;
                k += p.step_pairs;
                if (k >= p.n_pairs) {
                    k -= p.n_pairs;
                    ++r;
                }
            }
        }
        __syncthreads();
        for (int32_t x = 0; x < p.n_tensors; ++x) {
            const Tensor &t = p.t[x];
            if (!HALF || !t.rotate) {
                // Jobs of one warp: 32 vectors of one row; kFlight of them in
                // flight.
                constexpr int kFlight = 4;
                const uint32_t per_row = t.heads * p.vph, jobs = n * t.row_jobs;
                for (uint32_t j0 = warp; j0 < jobs; j0 += kFlight * kWarps) {
                    uint4 v[kFlight];
                    uint32_t rr[kFlight], at[kFlight];
#pragma unroll
                    for (int f = 0; f < kFlight; ++f) {
                        const uint32_t j = j0 + f * kWarps;
                        rr[f] = t.by_jobs.div(j);
                        at[f] = (j - rr[f] * t.row_jobs) * 32 + lane;
                        if (j < jobs && at[f] < per_row)
                            v[f] = ld_row(t.src + rows[rr[f]].src * t.src_stride + at[f] * 16u);
                    }
#pragma unroll
                    for (int f = 0; f < kFlight; ++f) {
                        if (j0 + f * kWarps >= jobs || at[f] >= per_row) continue;
                        if (t.rotate) {
                            const uint32_t in = p.vph_mask >= 0 ? at[f] & p.vph_mask
                                                                : at[f] - p.by_vph.div(at[f]) * p.vph;
                            v[f] = rotate_vec<EB>(v[f], cs + rr[f] * p.pitch, in * (8 / EB), p.n_pairs);
                        }
                        st_row(t.dst + rows[rr[f]].dst * t.dst_stride + at[f] * 16u, v[f]);
                    }
                }
            } else {
                // Jobs of one warp: up to `chunk` heads of one row, the next one's
                // loads in flight while this one is rotated and stored.
                constexpr int kVecs = kStageBytes / 16 / 32;
                uint8_t *s = stage[warp];
                const uint32_t chunk = kStageBytes / p.head_bytes;
                const uint32_t per_row = (t.heads + chunk - 1) / chunk;
                const uint32_t jobs = n * per_row;
                uint4 v[kVecs];
                auto where = [&](uint32_t job, uint32_t &r, uint32_t &h0, uint32_t &nh) {
                    r = job / per_row;
                    h0 = (job - r * per_row) * chunk;
                    nh = min(chunk, static_cast<uint32_t>(t.heads) - h0);
                };
                auto fetch = [&](uint32_t job) {
                    uint32_t r, h0, nh;
                    where(job, r, h0, nh);
                    const uint8_t *src = t.src + rows[r].src * t.src_stride + h0 * p.head_bytes;
#pragma unroll
                    for (int f = 0; f < kVecs; ++f)
                        if (f * 32 + lane < nh * p.vph) v[f] = ld_row(src + (f * 32 + lane) * 16);
                };
                if (warp < jobs) fetch(warp);
                for (uint32_t job = warp; job < jobs; job += kWarps) {
                    uint32_t r, h0, nh;
                    where(job, r, h0, nh);
                    const uint32_t nv = nh * p.vph;
#pragma unroll
                    for (int f = 0; f < kVecs; ++f)
                        if (f * 32 + lane < nv)
                            *reinterpret_cast<uint4 *>(s + (f * 32 + lane) * 16) = v[f];
                    __syncwarp();
                    if (job + kWarps < jobs) fetch(job + kWarps);
                    for (uint32_t k = lane; k < p.n_pairs; k += 32) {
                        const float2 c = cs[r * p.pitch + k];
                        const int a = k < p.pair_end[0] ? 0 : (k < p.pair_end[1] ? 1 : 2);
                        const uint32_t c1 = p.seg_first[a] + k - (a == 0 ? 0 : p.pair_end[a - 1]);
                        const uint32_t c2 = c1 + p.seg_half[a];
#pragma unroll 4
                        for (uint32_t h = 0; h < nh; ++h) {
                            uint8_t *head = s + h * p.head_bytes;
                            const float2 y = turned(ld_ch<EB>(head, c1), ld_ch<EB>(head, c2), c);
                            st_ch<EB>(head, c1, y.x);
                            st_ch<EB>(head, c2, y.y);
                        }
                    }
                    __syncwarp();
                    uint8_t *dst = t.dst + rows[r].dst * t.dst_stride + h0 * p.head_bytes;
#pragma unroll
                    for (int f = 0; f < kVecs; ++f)
                        if (f * 32 + lane < nv)
                            st_row(dst + (f * 32 + lane) * 16,
                                   *reinterpret_cast<const uint4 *>(s + (f * 32 + lane) * 16));
                    __syncwarp();
                }
            }
        }
    }
}

// Angle per position of pair k of a segment of width d, scaled as `r` says.
double omega_of(const atlas_rotary &r, int axis, int32_t d, int32_t k) {
    const double factor = axis == 0 ? r.factor_t : (axis == 1 ? r.factor_h : r.factor_w);
    const double original = axis == 0 ? r.original_t : (axis == 1 ? r.original_h : r.original_w);
    double theta = r.theta;
    if (r.scaling == ATLAS_ROTARY_NTK && d > 2)
        theta *= std::pow(factor, static_cast<double>(d) / (d - 2));
    const double omega = std::pow(theta, -2.0 * k / static_cast<double>(d));
    if (r.scaling != ATLAS_ROTARY_BY_PARTS) return omega;
    const double turns = original * omega / (2.0 * M_PI);
    const double keep =
        std::min(1.0, std::max(0.0, (turns - r.beta_slow) / (r.beta_fast - r.beta_slow)));
    return omega * (keep + (1.0 - keep) / factor);
}

template <int EB, bool HALF>
atlas_status launch(const Params &p, const DeviceInfo &dev, cudaStream_t stream) {
    const uint32_t grid = std::min(p.n_tiles, static_cast<uint32_t>(dev.sm_count) * 8u);
    if (log_enabled())
        log_launch(HALF ? "rotary_kernel<half>" : "rotary_kernel", static_cast<int>(grid),
                   kThreads, 0, "elem_bytes %d rows %u tensors %d head_bytes %u pairs %u tile %u order %d",
                   EB, p.total_rows, p.n_tensors, p.head_bytes, p.n_pairs, p.tile_rows, p.order);
    rotary_kernel<EB, HALF><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace

atlas_status launch_rotary(const RotaryArgs &a, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return ATLAS_ERR_DEVICE;
    const atlas_rotary &r = *a.rot;
    Params p{};
    const uint32_t T = static_cast<uint32_t>(a.T), H = static_cast<uint32_t>(a.H),
                   W = static_cast<uint32_t>(a.W);
    // A cube longer than its axis is the whole axis.
    const uint32_t ct = std::min<uint32_t>(a.ct, T), ch = std::min<uint32_t>(a.ch, H),
                   cw = std::min<uint32_t>(a.cw, W);
    p.g = geom::make_geom(T, H, W, ct, ch, cw);
    p.even = T % ct == 0 && H % ch == 0 && W % cw == 0;
    p.order = a.order;
    p.rows = T * H * W;
    p.total_rows = static_cast<uint32_t>(a.batch * p.rows);
    p.by_rows = FastDiv(p.rows);
    p.head_bytes = static_cast<uint32_t>(a.head_dim * a.elem_bytes);
    p.vph = p.head_bytes / 16;
    p.by_vph = FastDiv(p.vph);
    p.positions = a.positions;
    p.n_axes = a.n_axes;
    p.magnitude = static_cast<float>(r.magnitude);
    p.sign = r.transpose ? -1.f : 1.f;
    const int32_t d[3] = {r.d_t, r.d_h, r.d_w};
    const double scale[3] = {r.scale_t, r.scale_h, r.scale_w};
    uint32_t n = 0, channel = 0;
    for (int axis = 0; axis < 3; ++axis) {
        for (int32_t k = 0; k < d[axis] / 2; ++k)
            p.turn[n++] = scale[axis] * omega_of(r, axis, d[axis], k) / M_PI;
        p.seg_first[axis] = channel;
        p.seg_half[axis] = d[axis] / 2;
        channel += d[axis];
        if (axis < 2) p.pair_end[axis] = n;
    }
    p.n_pairs = n;
    p.by_pairs = FastDiv(n);
    p.pitch = (n + 1) / 2 * 2;
    p.step_rows = n > 0 ? kThreads / n : 0;
    p.step_pairs = n > 0 ? kThreads % n : 0;
    p.vph_mask = (p.vph & (p.vph - 1)) == 0 ? static_cast<int32_t>(p.vph) - 1 : -1;
    int n_tensors = 0;
    bool turns = false;
    int64_t widest = 0;
    for (int i = 0; i < a.n_tensors; ++i) {
        const atlas_rotary_tensor &x = a.tensors[i];
        const bool rotate = x.rotate && n > 0;
        // In place without a rotation: every row is already there.
        if (!rotate && x.src == x.dst) continue;
        Tensor &t = p.t[n_tensors++];
        const int64_t width = static_cast<int64_t>(x.heads) * a.head_dim;
        t.src = static_cast<const uint8_t *>(x.src);
        t.dst = static_cast<uint8_t *>(x.dst);
        t.src_stride = (x.src_stride ? x.src_stride : width) * a.elem_bytes;
        t.dst_stride = (x.dst_stride ? x.dst_stride : width) * a.elem_bytes;
        t.heads = x.heads;
        t.rotate = rotate;
        t.row_jobs = (x.heads * p.vph + 31) / 32;
        t.by_jobs = FastDiv(t.row_jobs);
        turns |= rotate;
        widest = std::max(widest, width * a.elem_bytes);
    }
    if (n_tensors == 0) return ATLAS_OK;
    p.n_tensors = n_tensors;
    if (!turns) p.n_pairs = 0;   // nothing rotates: no angles
    // Rows of a tile: as many as their angles fit the buffer, no more than
    // leave every SM two tiles, and vectors of a tile below 2^31.
    uint32_t tile = n > 0 ? kTileAngles / p.pitch : kMaxTileRows;
    tile = std::min<uint32_t>(tile, kMaxTileRows);
    tile = std::min(tile, std::max(1u, p.total_rows / (2u * dev.sm_count)));
    tile = std::min<uint32_t>(tile, std::max<int64_t>(1, (1ll << 30) / (widest / 16)));
    p.tile_rows = tile;
    p.n_tiles = (p.total_rows + tile - 1) / tile;
    const bool half = r.layout == ATLAS_ROTARY_HALF && turns;
    if (a.elem_bytes == 2)
        return half ? launch<2, true>(p, dev, stream)
                    : launch<2, false>(p, dev, stream);
    return half ? launch<4, true>(p, dev, stream)
                : launch<4, false>(p, dev, stream);
}

}  // namespace atlas
