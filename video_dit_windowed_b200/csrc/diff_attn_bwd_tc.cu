// diff_attn_bwd_tc.cu -- backward of the differential attention, bf16, tcgen05 +
// TMA + TMEM.
//
// With P_m = exp(s_m - lse_m), dP = dO V^T and D_m (diff_attn.cu):
//   dS_m = P_m (dP - D_m),  W = P_1 - lambda P_2,
//   dQ_m = c_m scale dS_m K_m,  dK_m = c_m scale dS_m^T Q_m,  dV = W^T dO,
// c_1 = 1, c_2 = -lambda (in the epilogue). dP is one product for both maps, and
// the joint weights W make dV one: five products of width D a pair, as many as an
// ordinary head's backward, with two exponentials.
//
// One kernel template, two forms (every gradient row is owned by one unit, no
// atomics; S and dP are formed in both):
//   DQ    resident: 128 rows of Q and dO, in tensor memory (A operands of S and
//         dP); streamed: 64-row tiles of K and V; accumulates dQ.
//   DKDV  resident: 128 rows of K and V in shared memory; streamed: 48-row tiles
//         of Q and dO with their lse and D; accumulates dV and dK. With few heads
//         the units over global keys are few and long (each streams every query):
//         their queries are cut into parts, whose fp32 sums a second kernel joins
//         in order (diff_attn.cu, diff_split_plan).
// Measured at 720p, one head of 128: dQ 584 us, dK/dV 777 us (their products alone 230
// and 307: S, dP and the accumulations, 6 D and 8 D flops a pair); bound by the compute
// warps' instructions, two exponentials and two gradients a pair (issue slots 58 to
// 60 % busy with two such warps a scheduler; tensor 31 to 33 %).
// Tensor memory holds S_1 | S_2 | dP of one tile, the packed bf16 dS_1 | dS_2 (and
// W) in columns of their own, and the accumulators:
//   DQ    3 x 64 + 64 + 128 (dQ) + 128 (resident Q, dO) = 512,
//   DKDV  3 x 48 (64 apart) + 72 + 128 (dV) + 128 (dK): with 64-row tiles the
//         packed columns would not fit beside both accumulators.
// Because P and dS do not overwrite S, the next tile's S and dP products are
// issued as soon as the compute threads have loaded this tile's, and run while
// those compute; the products that read P and dS follow when they are stored.
//
// D comes from outputs that were rounded to 16 bits, which dlambda = -sum D_2, a
// sum of terms of both signs, would show (0.7% of it at head width 128). The sum of
// a row's dS is what D lacks, so DQ, which runs first, adds it: D is then as exact
// as P and dP. A query with one key has dS = 0 whatever D's rounding: DQ sets it, DKDV
// sets dK of a key that has such a query only (NaN stays).
//
// Warps (352 threads): 0-7 compute (thread = resident row = lane; warpgroup g
// takes half of a tile's columns), 8 TMA producer, 9 / 10 MMA issuers (S and dP;
// the accumulating products).
// Pairs outside the mask: P and dS are set to 0 whatever S and dP hold. 0 * NaN
// would still reach a row through the accumulating products' streamed operand, so
// streamed rows that not every resident row meets are zeroed in shared memory
// before those products where they hold a non-finite value: rows past the unit's
// ranges always; in DKDV the query rows whose D is NaN (diff_attn.cu; W and dS of
// the keys that do see such a query are NaN); in DQ's packed units the K rows with
// a non-finite channel (dQ of the queries that see one is made NaN in the epilogue:
// their dS is 0 where such a key has weight 0). Every wait is bounded, as in the
// forward.
#include <cuda.h>
#include <cuda_bf16.h>

#include "attn_units.cuh"
#include "sm100_diff.cuh"

namespace atlas {
namespace {

using units::Sched;
using units::Shape;
using units::Unit;

constexpr int kRows = units::kRows;
constexpr int kCompute = 256;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kThreads = 352;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

enum Form { kDQ = 0, kDKDV = 1 };

template <int FORM>
struct Tile {
    static constexpr int kStream = FORM == kDQ ? 64 : 48;   // streamed rows of a tile
    static constexpr int kCols = kStream / 2;               // a warpgroup's columns
    static constexpr int kPack = kCols / 2;                 // its packed columns
};

// Tensor-memory columns.
template <int HD, int FORM>
struct Tmem {
    static constexpr uint32_t kS = 0, kDP = 128;            // S_1, S_2 (64 apart); dP
    static constexpr uint32_t kPacked = FORM == kDQ ? 192 : 176;
    static constexpr uint32_t kPackedStride = Tile<FORM>::kStream / 2;
    static constexpr uint32_t kDS = kPacked + (FORM == kDQ ? 0 : kPackedStride);   // after W
    static constexpr uint32_t kDV = 256;                    // DKDV
    static constexpr uint32_t kGrad = FORM == kDQ ? 256 : 384;   // dQ or dK, map m at + 64 m
    static constexpr uint32_t kResX = 384, kResY = kResX + HD / 2;   // DQ: Q, dO
    static_assert(kDS + 2 * kPackedStride <= 256, "packed columns end before the accumulators");
};

template <int HD, int FORM>
struct Smem {
    static constexpr int kStream = Tile<FORM>::kStream;
    static constexpr int kResident = FORM == kDQ ? 1024 : kRows * HD * 2;   // DQ: in TMEM
    static constexpr int kTileBytes = kStream * HD * 2;
    static constexpr int kBudget = FORM == kDQ ? 192 * 1024 : 144 * 1024;
    static constexpr int kStages = kBudget / (2 * kTileBytes) < 8 ? kBudget / (2 * kTileBytes) : 8;
    alignas(1024) uint8_t x[kResident];
    alignas(1024) uint8_t y[kResident];
    alignas(1024) uint8_t xs[kStages][kTileBytes];   // streamed K (DQ) or Q
    alignas(1024) uint8_t ys[kStages][kTileBytes];   // streamed V (DQ) or dO
    alignas(16) float lse[kStages][2][FORM == kDQ ? 4 : kStream];     // DKDV: of the streamed queries
    alignas(16) float delta[kStages][2][FORM == kDQ ? 4 : kStream];
    float row_sum[2][2][FORM == kDQ ? kRows : 1];   // DQ: [unit & 1][map], of warpgroup 1
    uint32_t bad_k[2][8];   // DQ: [tile & 1][K row / 8], bit 4 (row % 8): not finite
    volatile uint32_t any_bad_k;   // set with the first such row
    uint64_t x_full, x_empty;
    uint64_t st_full[kStages], st_empty[kStages];
    uint64_t s_full;     // S_1, S_2, dP of a tile in TMEM           (commit)
    uint64_t s_read;     // ... loaded by the compute threads        (256)
    uint64_t p_full;     // packed P / dS in TMEM                    (256)
    uint64_t acc_done;   // the products that read them are done     (commit)
    uint64_t acc_full, acc_empty;
    uint64_t drain[2];
    uint32_t tmem_base;
    int32_t max_len;
    volatile int abort;
    uint32_t *err_word;
};

struct Params {
    CUtensorMap res_x[2], res_y[2];   // DKDV: K, V with 128-row boxes; [0] detail, [1] global
    CUtensorMap st_x[2], st_y[2];     // streamed, with tile-row boxes
    __nv_bfloat16 *dv[2], *grad[2];   // DKDV: dV; dQ or dK
    const __nv_bfloat16 *row_x[2], *row_y[2];   // DQ: Q and dO rows
    const float *lse, *lambda;
    float *delta;   // DKDV reads it; DQ reads and corrects its own rows'
    int32_t n_lambda;
    uint32_t *err_word;
    float scale_log2, scale;
    int32_t o_v8;
    float *split;   // DKDV: [n_split][batch * heads][G][dV | dK: D each] (n_split > 1)
    Shape shape;
};

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    bool bad = false;
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (u[i] & 0x7f80u) == 0x7f80u || (u[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

template <int FORM>
__device__ __forceinline__ Unit unit_at(const Params &p, const Sched &S, int32_t u) {
    if constexpr (FORM == kDQ) return units::query_unit<Tile<FORM>::kStream>(p.shape, S, u);
    else return units::key_unit<Tile<FORM>::kStream>(p.shape, S, u);
}

// Bounded wait. SLEEP: nanoseconds to sleep between tries, for the producer, which
// runs ahead: its tries otherwise take issue slots from the compute warps of its
// sub-partition.
template <int SLEEP = 0, typename SM>
__device__ __forceinline__ bool wait_phase(SM &sm, uint64_t &bar, uint32_t parity, uint32_t err,
                                           bool honor_abort = true) {
    const uint32_t a = ptx::smem_addr(&bar);
    // The timer is read only once a wait has failed many times: reading it takes
    // about as long as a tile's exponentials.
    uint64_t t0 = 0;
    for (uint32_t spin = 1;; ++spin) {
        if (ptx::mbar_try_wait(a, parity)) return true;
        if (SLEEP > 0) __nanosleep(SLEEP);
        if ((spin & 63u) == 0) {
            if (honor_abort && sm.abort) return false;
            const uint64_t now = global_timer_ns();
            if (t0 == 0) t0 = now;
            if (now - t0 > kWaitLimitNs) {
                atomicOr(sm.err_word, err);
                sm.abort = 1;
                return false;
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Producer warp.
// ---------------------------------------------------------------------------
template <int HD, int FORM>
__device__ void producer(const Params &p, const Sched &S, Smem<HD, FORM> &sm) {
    using SM = Smem<HD, FORM>;
    constexpr int kStages = SM::kStages, kStream = SM::kStream;
    const uint32_t lane = threadIdx.x & 31;
    const int32_t N = p.shape.N, G = p.shape.G;
    uint32_t it = 0, unit_iter = 0, x_armed = 0;
    uint32_t armed[kStages];
#pragma unroll
    for (int s = 0; s < kStages; ++s) armed[s] = 0;
    bool ok = true;
    auto tile = [&](uint8_t *dst, const CUtensorMap *map, uint32_t bar, int32_t head, int32_t row,
                    uint32_t panel) {
#pragma unroll
        for (int db = 0; db < HD / 64; ++db)
            ptx::tma_load_3d(ptx::smem_addr(dst + db * panel), map, bar, db * 64, head, row);
    };
    for (int32_t u = blockIdx.x; u < S.n_units && ok; u += gridDim.x) {
        const Unit U = unit_at<FORM>(p, S, u);
        const int32_t n = U.n_a + U.n_b;
        if (n == 0) continue;
        // Every lane waits and the warp agrees, so the lanes stay together
        // around the warp-wide steps below.
        if (FORM == kDKDV) {
            if (unit_iter > 0 &&
                !(ok = __all_sync(kAll, wait_phase<200>(sm, sm.x_empty, (unit_iter - 1) & 1,
                                                   kErrTimeoutProducer))))
                break;
            if (lane == 0) {
                const int side = U.detail ? 0 : 1;
                const int32_t row = U.b * (U.detail ? N : G) + U.r0;
                const uint32_t bar = ptx::smem_addr(&sm.x_full);
                ptx::mbar_arrive_expect_tx(bar, 2 * SM::kResident);
                tile(sm.x, &p.res_x[side], bar, U.head, row, kRows * 128);
                tile(sm.y, &p.res_y[side], bar, U.head, row, kRows * 128);
            }
            x_armed = unit_iter + 1;
        }
        for (int32_t j = 0; j < n && ok; ++j, ++it) {
            const uint32_t s = it % kStages, round = it / kStages;
            if (round > 0 &&
                !(ok = __all_sync(kAll, wait_phase<200>(sm, sm.st_empty[s], (round - 1) & 1,
                                                   kErrTimeoutProducer))))
                break;
            const bool det = j < U.n_a;
            const int32_t row = units::tile_row<kStream>(U, j), rows = det ? N : G;
            const uint32_t bar = ptx::smem_addr(&sm.st_full[s]);
            if (FORM == kDKDV) {
                // lse and D of the streamed queries, both maps. Rows past the
                // problem copy its last row's: those columns are masked.
                const int64_t per = static_cast<int64_t>(N) + G;
                const int64_t col = (static_cast<int64_t>(U.b) * p.shape.heads + U.head) * 2 * per +
                                    (det ? 0 : N);
#pragma unroll
                for (int i = 0; i < (2 * kStream + 31) / 32; ++i) {
                    const int c = i * 32 + lane, m = c / kStream, k = c - m * kStream;
                    if (c < 2 * kStream) {
                        const int64_t at = col + m * per + min(row + k, rows - 1);
                        ptx::cp_async_4(ptx::smem_addr(&sm.lse[s][m][k]), p.lse + at);
                        ptx::cp_async_4(ptx::smem_addr(&sm.delta[s][m][k]), p.delta + at);
                    }
                }
                ptx::cp_async_mbar_arrive(bar);
                __syncwarp();
            }
            if (lane == 0) {
                const int32_t at = U.b * rows + row, side = det ? 0 : 1;
                ptx::mbar_arrive_expect_tx(bar, 2 * SM::kTileBytes);
                tile(sm.xs[s], &p.st_x[side], bar, U.head, at, kStream * 128);
                tile(sm.ys[s], &p.st_y[side], bar, U.head, at, kStream * 128);
            }
#pragma unroll
            for (int t = 0; t < kStages; ++t)
                if (t == static_cast<int>(s)) armed[t] = round + 1;
        }
        ++unit_iter;
    }
    if (!ok && lane == 0) {
        // Let every copy already issued land before the CTA can exit.
        if (x_armed) wait_phase(sm, sm.x_full, (x_armed - 1) & 1, kErrTimeoutTeardown, false);
        for (int t = 0; t < kStages; ++t)
            if (armed[t])
                wait_phase(sm, sm.st_full[t], (armed[t] - 1) & 1, kErrTimeoutTeardown, false);
    }
}

// ---------------------------------------------------------------------------
// MMA issuers, each one converged warp (sm100_diff.cuh): S and dP of
// tile t as soon as tile t-1 was loaded; the products of P and dS when they are
// stored. They share no accumulator, and each one's waits and issues take the
// time of the other's MMAs. Tensor memory starts at column 0, so its addresses
// are constants.
// ---------------------------------------------------------------------------
template <int HD, int FORM>
__device__ void score_issuer(const Params &p, const Sched &S, Smem<HD, FORM> &sm) {
    using SM = Smem<HD, FORM>;
    using TM = Tmem<HD, FORM>;
    constexpr int kStages = SM::kStages, kStream = SM::kStream;
    constexpr int kMapSteps = HD / 32;
    constexpr uint32_t kTile16 = SM::kTileBytes >> 4;
    constexpr uint32_t kPanel = kStream * 128;              // bytes of a streamed 64-channel panel
    constexpr uint32_t kIdS = ptx::idesc_bf16_f32(kRows, kStream, 0);
    constexpr uint32_t kHi = ptx::desc_sw128_hi(1024);
    const uint32_t x_lo = ptx::desc_sw128_lo(ptx::smem_addr(sm.x), 16);
    const uint32_t y_lo = ptx::desc_sw128_lo(ptx::smem_addr(sm.y), 16);
    const uint32_t xs_lo = ptx::desc_sw128_lo(ptx::smem_addr(sm.xs[0]), 16);
    const uint32_t ys_lo = ptx::desc_sw128_lo(ptx::smem_addr(sm.ys[0]), 16);
    uint32_t ring = 0, ring_phase = 0, unit_iter = 0, c = 0;   // c: tiles
    bool ok = true;
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(kAll, wait_phase(sm, bar, parity, kErrTimeoutMma));
    };
    // D = A B^T over K = 16 steps [k0, k1) of the channels.
    auto product = [&](uint32_t d, uint32_t a_smem, uint32_t a_tmem, uint32_t b_lo, int k0, int k1) {
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) {
            const int ks = k0 + i;
            if (ks >= k1) break;
            const uint32_t a_off = ((ks / 4) * (kRows * 128) + (ks % 4) * 32) >> 4;
            const uint32_t b_off = ((ks / 4) * kPanel + (ks % 4) * 32) >> 4;
            if (FORM == kDQ)
                ptx::mma_ts_elect(d, a_tmem + ks * 8, ptx::desc_join(b_lo + b_off, kHi), kIdS, i > 0);
            else
                ptx::mma_ss_elect(d, ptx::desc_join(a_smem + a_off, kHi),
                                  ptx::desc_join(b_lo + b_off, kHi), kIdS, i > 0);
        }
    };
    for (int32_t u = blockIdx.x; u < S.n_units && ok; u += gridDim.x) {
        const Unit U = unit_at<FORM>(p, S, u);
        const int32_t n = ptx::uniform(U.n_a + U.n_b);
        if (n == 0) continue;
        if (!(ok = wait(sm.x_full, unit_iter & 1))) break;
        for (int32_t j = 0; j < n; ++j, ++c) {
            if (!(ok = wait(sm.st_full[ring], ring_phase))) break;
            // S's columns were read by the previous tile.
            if (c > 0 && !(ok = wait(sm.s_read, (c - 1) & 1))) break;
            ptx::tc_fence_after();
            const uint32_t xb = xs_lo + ring * kTile16, yb = ys_lo + ring * kTile16;
            product(TM::kS, x_lo, TM::kResX, xb, 0, kMapSteps);
            product(TM::kS + 64, x_lo, TM::kResX, xb, kMapSteps, 2 * kMapSteps);
            product(TM::kDP, y_lo, TM::kResY, yb, 0, HD / 16);
            ptx::mma_commit_elect(ptx::smem_addr(&sm.s_full));
            if (++ring == kStages) {
                ring = 0;
                ring_phase ^= 1;
            }
        }
        if (!ok) break;
        // The resident rows are read by S and dP only.
        ptx::mma_commit_elect(ptx::smem_addr(&sm.x_empty));
        ++unit_iter;
    }
    // Drain: every MMA issued must finish before tensor memory is freed.
    ptx::mma_commit_elect(ptx::smem_addr(&sm.drain[0]));
    wait_phase(sm, sm.drain[0], 0, kErrTimeoutTeardown, false);
}

template <int HD, int FORM>
__device__ void grad_issuer(const Params &p, const Sched &S, Smem<HD, FORM> &sm) {
    using SM = Smem<HD, FORM>;
    using TM = Tmem<HD, FORM>;
    constexpr int kStages = SM::kStages, kStream = SM::kStream;
    constexpr uint32_t kTile16 = SM::kTileBytes >> 4;
    constexpr uint32_t kPanel = kStream * 128;
    constexpr uint32_t kIdGrad = ptx::idesc_bf16_f32(kRows, 64, 1);
    constexpr uint32_t kIdV = ptx::idesc_bf16_f32(kRows, HD, 1);
    constexpr uint32_t kHi = ptx::desc_sw128_hi(1024);
    // The streamed tiles as MN-major B operands.
    const uint32_t xs_mn = ptx::desc_sw128_lo(ptx::smem_addr(sm.xs[0]), kPanel);
    const uint32_t ys_mn = ptx::desc_sw128_lo(ptx::smem_addr(sm.ys[0]), kPanel);
    uint32_t ring = 0, unit_iter = 0, c = 0;   // c: tiles
    bool ok = true;
    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        return __all_sync(kAll, wait_phase(sm, bar, parity, kErrTimeoutMma));
    };
    // acc += A (packed, tensor memory) B over the tile's rows.
    auto accumulate = [&](uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, bool first) {
#pragma unroll
        for (int ks = 0; ks < kStream / 16; ++ks)
            ptx::mma_ts_elect(d, a + ks * 8, ptx::desc_join(b_lo + ((ks * 16 * 128) >> 4), kHi),
                              idesc, (first && ks == 0) ? 0u : 1u);
    };
    for (int32_t u = blockIdx.x; u < S.n_units && ok; u += gridDim.x) {
        const Unit U = unit_at<FORM>(p, S, u);
        const int32_t n = ptx::uniform(U.n_a + U.n_b);
        if (n == 0) continue;
        for (int32_t j = 0; j < n; ++j, ++c) {
            // (p_full follows s_full, which follows the tile's loads)
            if (!(ok = wait(sm.p_full, c & 1))) break;
            if (j == 0 && unit_iter > 0 && !(ok = wait(sm.acc_empty, (unit_iter - 1) & 1))) break;
            ptx::tc_fence_after();
            const uint32_t xb = xs_mn + ring * kTile16, yb = ys_mn + ring * kTile16;
            if (FORM == kDKDV) accumulate(TM::kDV, TM::kPacked, yb, kIdV, j == 0);
            // Map m's channels: panel m, or (D = 64) both maps' one panel, of
            // which the epilogue takes map m's half.
#pragma unroll
            for (int m = 0; m < 2; ++m)
                accumulate(TM::kGrad + 64 * m, TM::kDS + m * TM::kPackedStride,
                           xb + (HD == 128 ? m * (kPanel >> 4) : 0), kIdGrad, j == 0);
            ptx::mma_commit_elect(ptx::smem_addr(&sm.st_empty[ring]));
            ptx::mma_commit_elect(ptx::smem_addr(&sm.acc_done));
            if (++ring == kStages) ring = 0;
        }
        if (!ok) break;
        ptx::mma_commit_elect(ptx::smem_addr(&sm.acc_full));
        ++unit_iter;
    }
    ptx::mma_commit_elect(ptx::smem_addr(&sm.drain[1]));
    wait_phase(sm, sm.drain[1], 0, kErrTimeoutTeardown, false);
}

// ---------------------------------------------------------------------------
// Compute warps: thread = resident row = tensor-memory lane.
// ---------------------------------------------------------------------------
template <int HD, int FORM>
__device__ void compute(const Params &p, const Sched &S, Smem<HD, FORM> &sm, uint32_t tmem) {
    using SM = Smem<HD, FORM>;
    using TM = Tmem<HD, FORM>;
    constexpr int kStages = SM::kStages, kStream = SM::kStream;
    constexpr int kCols = Tile<FORM>::kCols, kPack = Tile<FORM>::kPack;
    const uint32_t warp = threadIdx.x / 32, r = threadIdx.x & 127;
    const int part = static_cast<int>(warp / 4);     // warpgroup: half of the columns
    const uint32_t t = tmem + (((warp & 3) * 32u) << 16);
    const int32_t N = p.shape.N, G = p.shape.G;
    const int64_t per = static_cast<int64_t>(N) + G;
    const float c2 = p.scale_log2;
    uint32_t cnt = 0, unit_iter = 0;   // tiles, units

    // DQ: the resident rows of unit V into tensor memory: warpgroup 0 the Q
    // row, warpgroup 1 the dO row (bf16 pairs: the A-operand layout). Rows past
    // the unit are zeros. The previous unit's S and dP must be done (x_empty).
    auto write_resident = [&](const Unit &V) {
        const int32_t vrow = V.r0 + static_cast<int32_t>(r);
        uint32_t rv[HD / 2];
        if (vrow < V.rend) {
            const int64_t abs_row = static_cast<int64_t>(V.b) * (V.detail ? N : G) + vrow;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                (part == 0 ? p.row_x : p.row_y)[V.detail ? 0 : 1] +
                (abs_row * p.shape.heads + V.head) * HD);
#pragma unroll
            for (int i = 0; i < HD / 8; ++i) {
                const uint4 w4 = __ldg(src + i);
                rv[4 * i] = w4.x;
                rv[4 * i + 1] = w4.y;
                rv[4 * i + 2] = w4.z;
                rv[4 * i + 3] = w4.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < HD / 2; ++i) rv[i] = 0u;
        }
        const uint32_t dst = t + (part == 0 ? TM::kResX : TM::kResY);
        if constexpr (HD == 128) ptx::tmem_st64(dst, rv);
        else ptx::tmem_st32(dst, rv);
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&sm.x_full));
    };
    bool resident_ready = false;   // DQ: this unit's rows were written ahead
    // DQ, packed units: whether keys [lo, hi) of the tile at t0, tile count c, hold a
    // bad K row. Read behind the tile's products (acc_done, acc_full), which follow
    // every thread's p_full; written again two tiles on, behind the p_full in between.
    auto sees_bad = [&](int32_t t0, int32_t lo, int32_t hi, uint32_t c) -> bool {
        for (int k = max(lo - t0, 0); k < min(hi - t0, kStream); ++k)
            if ((sm.bad_k[c & 1][k / 8] >> (4 * (k % 8))) & 1u) return true;
        return false;
    };

    for (int32_t u = blockIdx.x; u < S.n_units; u += gridDim.x) {
        const Unit U = unit_at<FORM>(p, S, u);
        const int32_t n = U.n_a + U.n_b;
        const int32_t row = U.r0 + static_cast<int32_t>(r);   // resident row (in problem)
        const bool valid = row < U.rend;
        // A part's sums of this row (warpgroup 0: dV, 1: dK).
        float *sums = nullptr;
        if (FORM == kDKDV && !U.detail && p.shape.n_split > 1 && valid)
            sums = p.split + (((static_cast<int64_t>(U.part) * p.shape.batch + U.b) * p.shape.heads +
                               U.head) * G + row) * (2 * HD) + part * HD;
        if (n == 0) {
            if (sums != nullptr)
                for (int c = 0; c < HD; c += 4)
                    *reinterpret_cast<float4 *>(sums + c) = make_float4(0.f, 0.f, 0.f, 0.f);
            continue;
        }
        const float nlam = -__ldg(p.lambda + (p.n_lambda == 1 ? 0 : U.head));
        int32_t da = 0, db = 0, ga = 0, gb = 0;   // streamed rows this row meets
        float own_l[2] = {__builtin_huge_valf(), __builtin_huge_valf()}, own_d[2] = {0.f, 0.f};
        float sum_d[2] = {0.f, 0.f};              // DQ: of this warpgroup's dS
        float dk_on = 1.f;                        // DKDV: 0 where dK is; DQ: NaN where dQ is
        const bool scan = FORM == kDQ && U.detail && U.win < 0;
        auto check_bad = [&](int32_t j, uint32_t c) {
            if (sees_bad(units::tile_row<kStream>(U, j), j < U.n_a ? da : ga, j < U.n_a ? db : gb, c))
                dk_on = __uint_as_float(0x7fffffffu);
        };
        const int64_t col = (static_cast<int64_t>(U.b) * p.shape.heads + U.head) * 2 * per +
                            (U.detail ? row : static_cast<int64_t>(N) + row);
        if (valid) {
            if (FORM == kDQ) {
                units::query_ranges(p.shape, U, row, da, db, ga, gb);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    own_l[m] = __ldg(p.lse + col + m * per) * kLog2e;
                    own_d[m] = p.delta[col + m * per];
                }
                // The one key of a query has P = 1 and dS = 0 (or NaN).
                if (db - da + gb - ga == 1 && !isnan(own_d[0])) da = db = ga = gb = 0;
            } else {
                units::key_ranges(p.shape, U, row, da, db, ga, gb);
                // The key's one query sees no other key: P = 1 and dS = 0 (or NaN).
                if (U.detail ? db - da == 1 && units::no_global_key(p.shape, U, row)
                             : G == 1 && da == db)
                    dk_on = 0.f;
            }
        }
        if (FORM == kDQ && !resident_ready) {
            if (unit_iter > 0 &&
                !__all_sync(kAll, wait_phase(sm, sm.x_empty, (unit_iter - 1) & 1,
                                             kErrTimeoutSoftmax)))
                return;
            write_resident(U);
        }
        resident_ready = false;
        for (int32_t j = 0; j < n; ++j, ++cnt) {
            const uint32_t stage = cnt % kStages;
            if (FORM == kDKDV &&
                !__all_sync(kAll, wait_phase(sm, sm.st_full[stage], (cnt / kStages) & 1,
                                             kErrTimeoutSoftmax)))
                return;
            if (!__all_sync(kAll, wait_phase(sm, sm.s_full, cnt & 1, kErrTimeoutSoftmax))) return;
            ptx::tc_fence_after();
            uint32_t s1[kCols], s2[kCols], dp[kCols];
            const uint32_t src = t + TM::kS + part * kCols;
            if constexpr (kCols == 32) ptx::tmem_ld3x32(src, src + 64, src + TM::kDP, s1, s2, dp);
            else ptx::tmem_ld3x24(src, src + 64, src + TM::kDP, s1, s2, dp);
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_addr(&sm.s_read));
            const int32_t lo = j < U.n_a ? da : ga, hi = j < U.n_a ? db : gb;
            const int32_t t0 = units::tile_row<kStream>(U, j), c0 = t0 + part * kCols;   // column 0
            const bool partial = c0 < lo || c0 + kCols > hi;
            uint32_t pw[kPack], pd1[kPack], pd2[kPack];
#pragma unroll
            for (int e = 0; e < kPack; ++e) {
                float w[2], d1[2], d2[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int c = 2 * e + k;
                    float l[2], dl[2];
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        if (FORM == kDQ) {
                            l[m] = own_l[m];
                            dl[m] = own_d[m];
                        } else {
                            l[m] = sm.lse[stage][m][part * kCols + c] * kLog2e;
                            dl[m] = sm.delta[stage][m][part * kCols + c];
                        }
                    }
                    const float p1 = ptx::ex2(fmaf(__uint_as_float(s1[c]), c2, -l[0]));
                    const float p2 = ptx::ex2(fmaf(__uint_as_float(s2[c]), c2, -l[1]));
                    const float g = __uint_as_float(dp[c]);
                    // (a query whose D is NaN makes W NaN too)
                    w[k] = FORM == kDQ ? 0.f : fmaf(dl[0], 0.f, fmaf(nlam, p2, p1));
                    d1[k] = p1 * (g - dl[0]);
                    d2[k] = p2 * (g - dl[1]);
                    if (partial && (c0 + c < lo || c0 + c >= hi)) w[k] = d1[k] = d2[k] = 0.f;
                    if (FORM == kDQ) {
                        sum_d[0] += d1[k];
                        sum_d[1] += d2[k];
                    }
                }
                pw[e] = ptx::pack_bf16x2(w[0], w[1]);
                pd1[e] = ptx::pack_bf16x2(d1[0], d1[1]);
                pd2[e] = ptx::pack_bf16x2(d2[0], d2[1]);
            }
            // The products of the previous tile have read the packed columns.
            if (cnt > 0 &&
                !__all_sync(kAll, wait_phase(sm, sm.acc_done, (cnt - 1) & 1, kErrTimeoutSoftmax)))
                return;
            ptx::tc_fence_after();
            const uint32_t any_bad = scan && j > 0 ? sm.any_bad_k : 0;
            const uint32_t dst = t + TM::kDS + part * kPack;
            if constexpr (FORM == kDQ) {
                ptx::tmem_st16_nowait(dst, pd1);
                ptx::tmem_st16_nowait(dst + TM::kPackedStride, pd2);
            } else {
                ptx::tmem_st12_nowait(t + TM::kPacked + part * kPack, pw);
                ptx::tmem_st12_nowait(dst, pd1);
                ptx::tmem_st12_nowait(dst + TM::kPackedStride, pd2);
            }
            ptx::tmem_wait_st();
            if (any_bad != 0) check_bad(j - 1, cnt - 1);
            // Rows to zero (S and dP of this tile are done with them; s_full, which
            // follows the issuer's wait for the loads, orders them before).
            constexpr int kVecs = HD / 64 * 8;   // 16-byte vectors of a row
            auto vec_at = [&](int sr, int v) {
                return (v / 8) * kStream * 128 + sr * 128 + (v % 8) * 16;
            };
            const int32_t seen = units::tile_rows<kStream>(U, j);
            bool wrote = false;
            if (seen < kStream) {
                for (int i = threadIdx.x; i < (kStream - seen) * kVecs; i += kCompute) {
                    const int off = vec_at(seen + i / kVecs, i % kVecs);
                    ptx::st_shared_v4(sm.xs[stage] + off, 0, 0, 0, 0);
                    if (FORM == kDKDV) ptx::st_shared_v4(sm.ys[stage] + off, 0, 0, 0, 0);
                    wrote = true;
                }
            }
            if (FORM == kDKDV) {
                const int sr = threadIdx.x;
                if (sr < kStream && isnan(sm.delta[stage][0][sr])) {
                    for (int v = 0; v < kVecs; ++v) {
                        ptx::st_shared_v4(sm.xs[stage] + vec_at(sr, v), 0, 0, 0, 0);
                        ptx::st_shared_v4(sm.ys[stage] + vec_at(sr, v), 0, 0, 0, 0);
                    }
                    wrote = true;
                }
            } else if (scan) {
                // four threads per K row (8 rows of a warp's LDS: no conflicts)
                const int sr = threadIdx.x / 4, q = threadIdx.x & 3;
                bool bad = false;
                for (int v = q; v < kVecs; v += 4)
                    bad |= not_finite(*reinterpret_cast<const uint4 *>(sm.xs[stage] + vec_at(sr, v)));
                bad |= __shfl_xor_sync(kAll, static_cast<int>(bad), 1) != 0;
                bad |= __shfl_xor_sync(kAll, static_cast<int>(bad), 2) != 0;
                const uint32_t rows = __ballot_sync(kAll, bad && sr < seen);
                if ((threadIdx.x & 31) == 0) {
                    sm.bad_k[cnt & 1][warp] = rows;
                    if (rows != 0) sm.any_bad_k = 1;
                }
                if (bad) {
                    for (int v = q; v < kVecs; v += 4)
                        ptx::st_shared_v4(sm.xs[stage] + vec_at(sr, v), 0, 0, 0, 0);
                    wrote = true;
                }
            }
            if (wrote) ptx::fence_proxy_async_smem();
            // Read by warpgroup 0 after acc_full; it has left the unit before last by
            // the time that this unit's S is there.
            if (FORM == kDQ && part == 1 && j == n - 1) {
                sm.row_sum[unit_iter & 1][0][r] = sum_d[0];
                sm.row_sum[unit_iter & 1][1][r] = sum_d[1];
            }
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_addr(&sm.p_full));
        }
        if (FORM == kDQ) {
            // The next unit's resident rows go in as soon as this unit's
            // S and dP are done, so its first ones run during this epilogue.
            int32_t u2 = u + gridDim.x;
            Unit V;
            for (; u2 < S.n_units; u2 += gridDim.x) {
                V = unit_at<FORM>(p, S, u2);
                if (V.n_a + V.n_b != 0) break;
            }
            if (u2 < S.n_units) {
                if (!__all_sync(kAll, wait_phase(sm, sm.x_empty, unit_iter & 1,
                                                 kErrTimeoutSoftmax)))
                    return;
                write_resident(V);
                resident_ready = true;
            }
        }
        // Epilogue: accumulators -> bf16 rows.
        if (!__all_sync(kAll, wait_phase(sm, sm.acc_full, unit_iter & 1, kErrTimeoutSoftmax)))
            return;
        ptx::tc_fence_after();
        if (scan && sm.any_bad_k != 0) check_bad(n - 1, cnt - 1);
        __syncwarp();   // (a search may end early; tensor-memory loads want the whole warp)
        if (FORM == kDQ && part == 0 && valid) {
            // dS sums to P (dP - D) = <do, P v> - D: what D lacks.
#pragma unroll
            for (int m = 0; m < 2; ++m)
                p.delta[col + m * per] = own_d[m] + (sum_d[m] + sm.row_sum[unit_iter & 1][m][r]);
        }
        const int side = U.detail ? 0 : 1;
        const int64_t out_row = (static_cast<int64_t>(U.b) * (U.detail ? N : G) +
                                 (valid ? row : 0)) * p.shape.heads + U.head;
        // ncol columns of tensor memory from `col`, times f (a part's sums: times
        // on), to channel ch0 on.
        auto store = [&](__nv_bfloat16 *out, uint32_t col, int ch0, int ncol, float f, float on) {
            uint8_t *dst = reinterpret_cast<uint8_t *>(out + out_row * HD + ch0);
#pragma unroll 1
            for (int c = 0; c < ncol / 32; ++c) {
                uint32_t o[32];
                ptx::tmem_ld32(t + col + c * 32, o);
                if (sums != nullptr) {
                    uint4 *at = reinterpret_cast<uint4 *>(sums + ch0 + c * 32);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[e] = __float_as_uint(__uint_as_float(o[e]) * on);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        at[v] = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
                } else if (valid) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        uint32_t w[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            w[e] = ptx::pack_bf16x2(__uint_as_float(o[16 * v + 2 * e]) * f,
                                                    __uint_as_float(o[16 * v + 2 * e + 1]) * f);
                        uint8_t *at = dst + c * 64 + v * 32;
                        if (p.o_v8) {
                            ptx::st_global_v8(at, w);
                        } else {
                            reinterpret_cast<uint4 *>(at)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                            reinterpret_cast<uint4 *>(at)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                        }
                    }
                }
            }
        };
        // Map m's gradient: channels [m D/2, +D/2), columns 64 m on (D = 64: the
        // half of its 64 columns that its channels are).
        auto store_map = [&](int m) {
            store(p.grad[side], TM::kGrad + 64 * m + (HD == 64 ? 32 * m : 0), m * (HD / 2), HD / 2,
                  (m == 0 ? p.scale : p.scale * nlam) * dk_on, dk_on);
        };
        if (FORM == kDQ) {
            store_map(part);
        } else if (part == 0) {
            store(p.dv[side], TM::kDV, 0, HD, 1.f, 1.f);
        } else {
            store_map(0);
            store_map(1);
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&sm.acc_empty));
        ++unit_iter;
    }
}

template <int HD, int FORM>
__global__ void __launch_bounds__(kThreads, 1) diff_bwd_tc_kernel(const __grid_constant__ Params p) {
    using SM = Smem<HD, FORM>;
    extern __shared__ uint8_t smem_raw[];
    SM &sm = *reinterpret_cast<SM *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                     ~static_cast<uintptr_t>(1023));
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_addr(&sm.x_full), FORM == kDQ ? kCompute : 1);
        ptx::mbar_init(ptx::smem_addr(&sm.x_empty), 1);
        for (int s = 0; s < SM::kStages; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sm.st_full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sm.st_empty[s]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&sm.s_full), 1);
        ptx::mbar_init(ptx::smem_addr(&sm.s_read), kCompute);
        ptx::mbar_init(ptx::smem_addr(&sm.p_full), kCompute);
        ptx::mbar_init(ptx::smem_addr(&sm.acc_done), 1);
        ptx::mbar_init(ptx::smem_addr(&sm.acc_full), 1);
        ptx::mbar_init(ptx::smem_addr(&sm.acc_empty), kCompute);
        ptx::mbar_init(ptx::smem_addr(&sm.drain[0]), 1);
        ptx::mbar_init(ptx::smem_addr(&sm.drain[1]), 1);
        sm.abort = 0;
        sm.max_len = 0;
        sm.any_bad_k = 0;
        sm.err_word = p.err_word;
        ptx::fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(&sm.tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            if (FORM == kDKDV) {
                ptx::prefetch_tmap(&p.res_x[i]);
                ptx::prefetch_tmap(&p.res_y[i]);
            }
            ptx::prefetch_tmap(&p.st_x[i]);
            ptx::prefetch_tmap(&p.st_y[i]);
        }
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (p.shape.upw < 0) {
        units::longest_window(p.shape, &sm.max_len);
        __syncthreads();
    }
    const Sched S = units::make_sched(p.shape, sm.max_len);
    const uint32_t tmem = sm.tmem_base;
    const bool tmem_ok = tmem == 0;   // a 512-column allocation starts at column 0
    if (!tmem_ok && threadIdx.x == 0) atomicOr(p.err_word, kErrTmemAlloc);
    if (tmem_ok) {
        if (warp < 8) compute<HD, FORM>(p, S, sm, tmem);
        else if (warp == kProducerWarp) producer<HD, FORM>(p, S, sm);
        else if (warp == kMmaWarp) score_issuer<HD, FORM>(p, S, sm);
        else grad_issuer<HD, FORM>(p, S, sm);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

// ---------------------------------------------------------------------------
// Host side.
// ---------------------------------------------------------------------------
template <int HD, int FORM>
atlas_status launch_form(const DiffBwdArgs &b, const DeviceInfo &dev, cudaStream_t stream) {
    using SM = Smem<HD, FORM>;
    const AttnArgs &a = b.fwd.attn;
    Params p{};
    int64_t n_units = 0;
    if (!units::make_shape(a, dev.sm_count, &p.shape, &n_units)) return ATLAS_ERR_SHAPE;
    const bool dq = FORM == kDQ;
    const void *q[2] = {a.q_d, a.q_g}, *k[2] = {a.k_d, a.k_g}, *v[2] = {a.v_d, a.v_g},
               *go[2] = {b.do_d, b.do_g};
    const int64_t rows[2] = {a.n_detail * a.batch, a.n_global * a.batch};
    for (int side = 0; side < 2; ++side) {
        // Maps of an absent side point at the other side; they are never used.
        const int use = rows[side] > 0 ? side : 1 - side;
        if (!make_rows_map(&p.st_x[side], dq ? k[use] : q[use], rows[use], a.heads, HD, SM::kStream) ||
            !make_rows_map(&p.st_y[side], dq ? v[use] : go[use], rows[use], a.heads, HD, SM::kStream))
            return ATLAS_ERR_CUDA;
        if (!dq && (!make_rows_map(&p.res_x[side], k[use], rows[use], a.heads, HD, kRows) ||
                    !make_rows_map(&p.res_y[side], v[use], rows[use], a.heads, HD, kRows)))
            return ATLAS_ERR_CUDA;
        p.row_x[side] = static_cast<const __nv_bfloat16 *>(q[side]);
        p.row_y[side] = static_cast<const __nv_bfloat16 *>(go[side]);
    }
    p.dv[0] = dq ? nullptr : static_cast<__nv_bfloat16 *>(b.dv_d);
    p.dv[1] = dq ? nullptr : static_cast<__nv_bfloat16 *>(b.dv_g);
    p.grad[0] = static_cast<__nv_bfloat16 *>(dq ? b.dq_d : b.dk_d);
    p.grad[1] = static_cast<__nv_bfloat16 *>(dq ? b.dq_g : b.dk_g);
    uintptr_t bits = 0;
    for (int side = 0; side < 2; ++side)
        bits |= reinterpret_cast<uintptr_t>(p.dv[side]) | reinterpret_cast<uintptr_t>(p.grad[side]);
    p.o_v8 = (bits & 31) == 0;
    p.lse = a.lse;
    p.delta = b.delta;
    p.lambda = b.fwd.lambda;
    p.n_lambda = b.fwd.n_lambda;
    p.err_word = device_error_word();
    if (!p.err_word) return ATLAS_ERR_CUDA;
    p.scale = a.scale;
    p.scale_log2 = a.scale * kLog2e;
    if (!dq) {
        p.shape.n_split = diff_split_plan(a.batch, a.n_detail, a.n_global, a.heads, 2);
        n_units += static_cast<int64_t>(p.shape.n_split - 1) * p.shape.n_long;
        p.split = b.split;
    }
    const size_t smem = sizeof(SM) + 1024;
    if (!set_smem_limit(reinterpret_cast<const void *>(diff_bwd_tc_kernel<HD, FORM>),
                        static_cast<int>(smem)))
        return ATLAS_ERR_CUDA;
    const int grid = static_cast<int>(n_units < dev.sm_count ? n_units : dev.sm_count);
    if (log_enabled())
        log_launch(dq ? "diff_bwd_tc_kernel<dQ>" : "diff_bwd_tc_kernel<dK/dV>", grid, kThreads, smem,
                   "head_dim %d units %lld split %d batch %d heads %d n_detail %d n_global %d", HD,
                   static_cast<long long>(n_units), p.shape.n_split, p.shape.batch, p.shape.heads,
                   p.shape.N, p.shape.G);
    diff_bwd_tc_kernel<HD, FORM><<<grid, kThreads, smem, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return ATLAS_ERR_CUDA;
    return p.shape.n_split > 1 ? launch_diff_split_join(b, p.shape.n_split, stream) : ATLAS_OK;
}

}  // namespace

atlas_status launch_diff_bwd_tc(const DiffBwdArgs &b, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return ATLAS_ERR_DEVICE;
    if (b.fwd.attn.head_dim == 128) {
        const atlas_status st = launch_form<128, kDQ>(b, dev, stream);
        return st != ATLAS_OK ? st : launch_form<128, kDKDV>(b, dev, stream);
    }
    const atlas_status st = launch_form<64, kDQ>(b, dev, stream);
    return st != ATLAS_OK ? st : launch_form<64, kDKDV>(b, dev, stream);
}

}  // namespace atlas
