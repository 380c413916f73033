// diff_attn_tc.cu -- differential attention, bf16, tcgen05 + TMA + TMEM.
//
// o = (softmax(s_1) - lambda softmax(s_2)) v with s_m = scale <q_m, k_m>, the
// maps being the halves of a head's channels. Each map keeps its own running
// maximum, sum and fp32 accumulator O_m = sum exp(s_m - max) v; the epilogue
// joins them: o = O_1 / l_1 - lambda O_2 / l_2.
//
// Why one pass over the keys with two accumulators: the joint weights need both
// sums, so a single accumulator would take a second pass over the logits, and
// the exponentials, not the products, are what bounds the kernel: two per (query,
// key) pair at 16 a clock and SM are 2048 clk per 128 x 128 tile, against 1536
// clk of products (2 D of logits and 4 D with v per pair, D = 128).
//
// A unit is 128 query rows of one head (attn_units.cuh); a Q, K or V tile is
// the same 128 x D tile an ordinary head has, its channel halves being the maps,
// so K and V are read once for both maps. Persistent CTAs walk the units
// head-major. Warps (384 threads):
//   0-3 / 4-7  softmax of map 1 / 2 (thread = query row = TMEM lane); in the
//              epilogue each group joins half of the output's columns,
//   8          TMA producer, 9 / 10  MMA issuer of map 1 / 2, 11  idle.
// Tensor memory: two 64-column regions per map, then O_1 | O_2 (D each). A tile's
// logits come in two halves: keys 0-63 in one region, keys 64-127 in the other;
// P (bf16, 64 columns) overwrites the first half's region. Once the second half has
// been loaded its region is free, so the next tile's first half is computed there
// while this tile's exponentials still run, and its second half follows P V into
// the region of P; regions swap roles every tile. A softmax therefore finds its
// next 64 keys waiting and never sits out its own P V. (With one 128-column S per
// map, whose next tile can only follow P V, a tile took 4020 clk; the exponentials
// are 2048.) Issue order per key tile j, for each map (one
// thread's MMAs run in order):
//   S(j+1) first half, O += P(j) V(j), S(j+1) second half.
// Masked keys: their logits are set to -inf whatever they hold; 0 * NaN
// would still reach a row through P V, so the V rows past the unit's range are
// zeroed in shared memory before the product. In packed units (PACK), whose rows
// see different windows, so are V rows with a non-finite value, and the rows that
// do see such a key become NaN in the epilogue.
// Measured: 720p (80,640 + 5,040 rows, windows of 768), 4 heads, D = 128: 1,580-1,590
// us at 1,965 MHz, 0.96 PFLOP/s (products alone 923 us, exponentials alone 878), and
// 1,740 in a row, when the power cap holds the clock at 1,780-1,800 MHz; 32,760 tokens,
// D = 64: 850-860 us (exponentials 477). No pipe is saturated (MUFU 54 %, tensor and
// issue slots 45 % busy): a scheduler has two softmax warps, whose dependent steps
// (logits from tensor memory, exponentials, conversion, P back, hand-over) do not hide
// one another. Warps of half a tile's columns each, four a scheduler, as the backward
// splits them, have not been tried.
// Every wait is bounded: on expiry a bit is set in the device error word, the
// CTA drains its copies and MMAs, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_bf16.h>

#include <type_traits>

#include "attn_units.cuh"
#include "sm100_diff.cuh"

namespace atlas {
namespace {

using units::Sched;
using units::Shape;
using units::Unit;

constexpr int kBM = units::kRows;   // query rows of a unit
constexpr int kBN = 128;            // keys of a tile
constexpr int kMaps = 2;
constexpr int kProducerWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kThreads = 384;
// Register split: 384 x 168 at launch; 256 x 200 + 128 x 104 after.
constexpr uint32_t kRegsSoftmax = 200;
constexpr uint32_t kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther == kThreads * 168, "register split");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kRescaleThreshold = 8.0f;  // log2 units: P stays <= 2^8
constexpr int kFewKeys = 32;   // softmax_epilogue

template <int HD>
struct Smem {
    static constexpr int kTileBytes = kBM * HD * 2;
    static constexpr int kSlots = (160 * 1024) / kTileBytes < 8 ? (160 * 1024) / kTileBytes : 8;
    alignas(1024) uint8_t q[kTileBytes];
    alignas(1024) uint8_t kv[kSlots][kTileBytes];
    float inv_l[2][kMaps][kBM];  // by unit parity
    uint32_t bad[kMaps][4][4];   // PACK: non-finite V rows of the last four tiles,
    uint32_t mark[kMaps][4][kBM];   // and the tile count of those that a map zeroed
    uint64_t q_full, q_empty;
    uint64_t kv_full[kSlots];
    uint64_t kv_empty[kSlots];   // (and q_empty, o_final: a commit by each map's issuer)
    uint64_t s_lo[kMaps];        // first half of S_m(j) in TMEM            (commit)
    uint64_t s_hi[kMaps];        // second half, and O_m += P_m(j-1) V done (commit)
    uint64_t s_read[kMaps];      // second half loaded                      (128 threads)
    uint64_t p_full[kMaps];      // P_m(j) in TMEM, O_m rescaled            (128 threads)
    uint64_t o_final;            // every MMA of the unit done              (commit)
    uint64_t joined;             // both maps' inv_l written                (256 threads)
    uint64_t o_empty;            // both accumulators read                  (256 threads)
    uint64_t drain[kMaps];
    uint32_t tmem_base;
    int32_t max_len;
    volatile int abort;
    uint32_t *err_word;
};

struct Params {
    CUtensorMap tm_q[2], tm_k[2], tm_v[2];   // [0] detail, [1] global
    __nv_bfloat16 *o[2], *s[2];
    float *lse;
    const float *lambda;
    int32_t n_lambda;
    uint32_t *err_word;
    float scale_log2;
    int32_t stall_unit;   // test hook: this unit's first K tile is never loaded (-1: off)
    int32_t o_v8;         // every output 32-byte aligned: 32-byte stores
    Shape shape;
};

// Bounded wait. SLEEP: nanoseconds to sleep between tries, for the producer, which
// runs ahead: its tries otherwise take issue slots from the two softmax warps of
// its sub-partition, whose tiles then took 600 clk longer than the others'.
template <int SLEEP = 0, int HD>
__device__ __forceinline__ bool wait_phase(Smem<HD> &sm, uint64_t &bar, uint32_t parity,
                                           uint32_t err, bool honor_abort = true) {
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

// Whether one of eight bf16 values is infinite or NaN.
__device__ __forceinline__ bool not_finite(const uint4 &v) {
    bool bad = false;
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        bad |= (u[i] & 0x7f80u) == 0x7f80u || (u[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// K = 16 steps of P V that hold an allowed key of tile j. A tile of at most 64
// keys also skips the second half of S (stale columns, masked).
__device__ __forceinline__ int32_t tile_steps(const Unit &U, int32_t j) {
    return (min(units::tile_rows<kBN>(U, j), kBN) + 15) / 16;
}
// First column of the region of tile c's first half (and of its P); the second
// half has the other region.
__device__ __forceinline__ uint32_t lo_region(uint32_t c) { return (c & 1) * 64; }

// ---------------------------------------------------------------------------
// Producer: Q once per unit, then K(0), V(0), K(1), V(1), ...
// ---------------------------------------------------------------------------
template <int HD>
__device__ void producer(const Params &p, const Sched &S, Smem<HD> &sm) {
    constexpr uint32_t kBytes = Smem<HD>::kTileBytes;
    constexpr int kSlots = Smem<HD>::kSlots;
    uint32_t it = 0, unit_iter = 0, q_armed = 0;
    uint32_t armed[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) armed[s] = 0;
    bool ok = true;
    auto load = [&](const CUtensorMap *map, int32_t head, int32_t row) -> bool {
        const uint32_t slot = it % kSlots, round = it / kSlots;
        if (round > 0 &&
            !wait_phase<200>(sm, sm.kv_empty[slot], (round - 1) & 1, kErrTimeoutProducer))
            return false;
        const uint32_t bar = ptx::smem_addr(&sm.kv_full[slot]);
        ptx::mbar_arrive_expect_tx(bar, kBytes);
#pragma unroll
        for (int db = 0; db < HD / 64; ++db)
            ptx::tma_load_3d(ptx::smem_addr(sm.kv[slot] + db * kBN * 128), map, bar, db * 64,
                             head, row);
#pragma unroll
        for (int s = 0; s < kSlots; ++s)
            if (s == static_cast<int>(slot)) armed[s] = round + 1;
        ++it;
        return true;
    };
    for (int32_t u = blockIdx.x; u < S.n_units && ok; u += gridDim.x) {
        const Unit U = units::query_unit<kBN>(p.shape, S, u);
        const int32_t n = U.n_a + U.n_b;
        if (n == 0) continue;
        if (unit_iter > 0 && !(ok = wait_phase<200>(sm, sm.q_empty, (unit_iter - 1) & 1,
                                               kErrTimeoutProducer)))
            break;
        const int32_t base[2] = {U.b * p.shape.N, U.b * p.shape.G};
        const int side = U.detail ? 0 : 1;
        const uint32_t bar = ptx::smem_addr(&sm.q_full);
        ptx::mbar_arrive_expect_tx(bar, kBytes);
#pragma unroll
        for (int db = 0; db < HD / 64; ++db)
            ptx::tma_load_3d(ptx::smem_addr(sm.q + db * kBM * 128), &p.tm_q[side], bar, db * 64,
                             U.head, base[side] + U.r0);
        q_armed = ++unit_iter;
        for (int32_t j = 0; j < n && ok; ++j) {
            const int kind = j < U.n_a ? 0 : 1;
            const int32_t row = base[kind] + units::tile_row<kBN>(U, j);
            if (j == 0 && u == p.stall_unit) {
                // Failure-path test: this slot stays unarmed, so the waits
                // on it expire.
                ++it;
                ok = load(&p.tm_v[kind], U.head, row);
                continue;
            }
            ok = load(&p.tm_k[kind], U.head, row) && load(&p.tm_v[kind], U.head, row);
        }
    }
    if (!ok) {
        // Let every copy already issued land before the CTA can exit.
        if (q_armed) wait_phase(sm, sm.q_full, (q_armed - 1) & 1, kErrTimeoutTeardown, false);
        for (int s = 0; s < kSlots; ++s)
            if (armed[s])
                wait_phase(sm, sm.kv_full[s], (armed[s] - 1) & 1, kErrTimeoutTeardown, false);
    }
}

// ---------------------------------------------------------------------------
// MMA issuer of map m: one converged warp (sm100_diff.cuh). Each
// map's products depend only on its own, so each map has a warp to issue them; one
// warp for both took 3550 clk of waits and issues per tile (D = 128). Tensor
// memory starts at column 0, so its addresses are constants.
// ---------------------------------------------------------------------------
template <int HD>
__device__ void mma_issuer(const Params &p, const Sched &S, Smem<HD> &sm, int m) {
    constexpr int kSlots = Smem<HD>::kSlots;
    constexpr int kMapSteps = HD / 32;   // K = 16 steps of one map's channels
    constexpr uint32_t kIdescQK = ptx::idesc_bf16_f32(kBM, 64, 0);
    constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, HD, 1);
    constexpr uint32_t kHi = ptx::desc_sw128_hi(1024);
    constexpr uint32_t kTile16 = Smem<HD>::kTileBytes >> 4;
    const uint32_t q_lo = ptx::desc_sw128_lo(ptx::smem_addr(sm.q), 16);
    const uint32_t k_lo0 = ptx::desc_sw128_lo(ptx::smem_addr(sm.kv[0]), 16);
    const uint32_t v_lo0 = ptx::desc_sw128_lo(ptx::smem_addr(sm.kv[0]), kBN * 128);
    uint32_t ring = 0, ring_phase = 0, unit_iter = 0, c = 0;   // c: key tiles
    bool ok = true;

    auto wait = [&](uint64_t &bar, uint32_t parity) -> bool {
        const bool r = __all_sync(kAll, wait_phase(sm, bar, parity, kErrTimeoutMma));
        ptx::tc_fence_after();
        return r;
    };
    auto next_slot = [&](uint32_t &slot) -> bool {
        slot = ring;
        const bool r = wait(sm.kv_full[slot], ring_phase);
        if (++ring == kSlots) {
            ring = 0;
            ring_phase ^= 1;
        }
        return r;
    };
    // Half `hi` of S_m = Q_m K_m^T for tile t: map m's channels are the K = 16
    // steps m * kMapSteps .. of the tile (64-channel panels of 128-byte rows,
    // four steps each), its keys rows 64 hi .. of K.
    auto issue_s = [&](int hi, uint32_t t, uint32_t k_slot) {
        const uint32_t k_lo = k_lo0 + k_slot * kTile16 + ((hi * 64 * 128) >> 4);
        const uint32_t d_s = m * kBN + (hi ? 64 - lo_region(t) : lo_region(t));
#pragma unroll
        for (int i = 0; i < kMapSteps; ++i) {
            const int ks = m * kMapSteps + i;
            const uint32_t off = ((ks / 4) * (kBM * 128) + (ks % 4) * 32) >> 4;
            ptx::mma_ss_elect(d_s, ptx::desc_join(q_lo + off, kHi),
                              ptx::desc_join(k_lo + off, kHi), kIdescQK, i > 0);
        }
    };
    // O_m += P_m V, P_m from tensor memory, over `steps` K = 16 steps.
    auto issue_pv = [&](uint32_t v_slot, bool first, int32_t steps) {
        const uint32_t v_lo = v_lo0 + v_slot * kTile16;
        const uint32_t d_o = kMaps * kBN + m * HD, a_p = m * kBN + lo_region(c);
        if (steps == kBN / 16) {
#pragma unroll
            for (int ks = 0; ks < kBN / 16; ++ks)
                ptx::mma_ts_elect(d_o, a_p + ks * 8,
                                  ptx::desc_join(v_lo + ((ks * 16 * 128) >> 4), kHi), kIdescPV,
                                  (first && ks == 0) ? 0u : 1u);
        } else {
#pragma unroll 1
            for (int ks = 0; ks < steps; ++ks)
                ptx::mma_ts_elect(d_o, a_p + ks * 8,
                                  ptx::desc_join(v_lo + ((ks * 16 * 128) >> 4), kHi), kIdescPV,
                                  (first && ks == 0) ? 0u : 1u);
        }
    };

    for (int32_t u = blockIdx.x; u < S.n_units && ok; u += gridDim.x) {
        Unit U = units::query_unit<kBN>(p.shape, S, u);
        units::make_uniform(U);
        const int32_t n = U.n_a + U.n_b;
        if (n == 0) continue;
        uint32_t k_slot, v_slot;
        if (!(ok = wait(sm.q_full, unit_iter & 1)) || !(ok = next_slot(k_slot))) break;
        int32_t steps = tile_steps(U, 0);
        // Both regions: the previous unit's last S was loaded, and its P V is
        // ahead in the queue.
        if (c > 0 && !(ok = wait(sm.s_read[m], (c - 1) & 1))) break;
        issue_s(0, c, k_slot);
        ptx::mma_commit_elect(ptx::smem_addr(&sm.s_lo[m]));
        if (steps > 4) issue_s(1, c, k_slot);
        ptx::mma_commit_elect(ptx::smem_addr(&sm.s_hi[m]));
        ptx::mma_commit_elect(ptx::smem_addr(&sm.kv_empty[k_slot]));
        // Only the S MMAs read Q: after the unit's last one it is free.
        if (n == 1) ptx::mma_commit_elect(ptx::smem_addr(&sm.q_empty));
        // The accumulators of the previous unit have been read.
        if (unit_iter > 0 && !(ok = wait(sm.o_empty, (unit_iter - 1) & 1))) break;
        for (int32_t j = 0; j < n && ok; ++j) {
            const bool more = j + 1 < n;
            const int32_t next_steps = more ? tile_steps(U, j + 1) : 0;
            // ring order: V(j) was loaded before K(j+1)
            if (!(ok = next_slot(v_slot))) break;
            if (more) {
                if (!(ok = next_slot(k_slot)) || !(ok = wait(sm.s_read[m], c & 1))) break;
                issue_s(0, c + 1, k_slot);
                ptx::mma_commit_elect(ptx::smem_addr(&sm.s_lo[m]));
            }
            if (!(ok = wait(sm.p_full[m], c & 1))) break;
            issue_pv(v_slot, j == 0, steps);
            if (more) {
                if (next_steps > 4) issue_s(1, c + 1, k_slot);
                ptx::mma_commit_elect(ptx::smem_addr(&sm.s_hi[m]));
            }
            ptx::mma_commit_elect(ptx::smem_addr(&sm.kv_empty[v_slot]));
            if (more) {
                ptx::mma_commit_elect(ptx::smem_addr(&sm.kv_empty[k_slot]));
                if (j + 2 == n) ptx::mma_commit_elect(ptx::smem_addr(&sm.q_empty));
            }
            steps = next_steps;
            ++c;
        }
        if (!ok) break;
        ptx::mma_commit_elect(ptx::smem_addr(&sm.o_final));
        ++unit_iter;
    }
    // Drain: every MMA issued must finish before tensor memory is freed.
    ptx::mma_commit_elect(ptx::smem_addr(&sm.drain[m]));
    wait_phase(sm, sm.drain[m], 0, kErrTimeoutTeardown, false);
}

// ---------------------------------------------------------------------------
// Softmax of map `map`, and the epilogue; 128 threads, thread = row = lane.
// ---------------------------------------------------------------------------
template <int HD, bool PACK>
__device__ void softmax_epilogue(const Params &p, const Sched &S, Smem<HD> &sm, uint32_t tmem,
                                 int map) {
    constexpr int kSlots = Smem<HD>::kSlots;
    const uint32_t r = threadIdx.x & 127;
    const uint32_t lane_sel = ((threadIdx.x / 32) & 3) * (32u << 16);
    const uint32_t t_s = tmem + map * kBN + lane_sel;
    const uint32_t t_o = tmem + kMaps * kBN + map * HD + lane_sel;
    const uint32_t err = kErrTimeoutSoftmax;
    const float sc = p.scale_log2;

    // Columns [B, B + N) of 64 keys' S: P = exp2(S*scale*log2e - m) as bf16 pairs
    // into pk (rounding P halves the product's operand and is 2^-8 of each weight;
    // the row sum adds the fp32 P). FAST: the maximum of the raw S joins mx, NaN
    // kept, and one pair of eight takes its exponentials on the FMA pipe (720p, D =
    // 128 / 32,760 global tokens, D = 64: none 1628 / 906-975 us, one 1612 / 889, two
    // 1597 / 920, three 1640 / 970, four 1703 / 1015: beyond one the issue slots cost
    // what the MUFU saves).
    auto exps = [&](auto fast, auto from, auto count, const uint32_t (&sr)[64], float m,
                    ptx::F2 &sum, float (&mx)[2], uint32_t (&pk)[16]) {
        constexpr bool kFast = decltype(fast)::value;
        constexpr int B = decltype(from)::value, N = decltype(count)::value;
        const ptx::F2 scale2 = ptx::f2(sc, sc), negm2 = ptx::f2(-m, -m);
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            const int c = B + 2 * e;
            const float s0 = __uint_as_float(sr[c]), s1 = __uint_as_float(sr[c + 1]);
            if constexpr (kFast) mx[e & 1] = ptx::max3_nan(mx[e & 1], s0, s1);
            const ptx::F2 x = ptx::fma2(ptx::f2(s0, s1), scale2, negm2);
            float p0, p1;
            if (kFast && e % 8 == 3) {
                ptx::exp2_pair(x, p0, p1);
            } else {
                ptx::unpack(x, p0, p1);
                p0 = ptx::ex2(p0);
                p1 = ptx::ex2(p1);
            }
            sum = ptx::add2(sum, ptx::f2(p0, p1));
            pk[(c % 32) / 2] = ptx::pack_bf16x2(p0, p1);
        }
    };
    constexpr std::integral_constant<int, 0> c0{};
    constexpr std::integral_constant<int, 32> c32{};
    // All 64 with ex2, stored (masked tiles).
    auto exps_all = [&](const uint32_t (&sr)[64], float m, uint32_t dst, ptx::F2 &sum) {
        float unused[2];
        uint32_t pk[16];
        exps(std::false_type{}, c0, c32, sr, m, sum, unused, pk);
        ptx::tmem_st16_nowait(dst, pk);
        exps(std::false_type{}, c32, c32, sr, m, sum, unused, pk);
        ptx::tmem_st16_nowait(dst + 16, pk);
    };
    auto row_max = [&](const uint32_t (&sr)[64]) -> float {
        float m4[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = __uint_as_float(sr[k]);
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                m4[k] = ptx::max3(m4[k], __uint_as_float(sr[c + k]), __uint_as_float(sr[c + 4 + k]));
#pragma unroll
        for (int k = 0; k < 4; ++k) m4[k] = fmaxf(m4[k], __uint_as_float(sr[60 + k]));
        return fmaxf(ptx::max3(m4[0], m4[1], m4[2]), m4[3]);
    };
    // O *= alpha, in warps where some row moved its reference. The P V of the
    // previous tile is done: the commit that signalled s_hi covers it.
    auto rescale_o = [&](bool need, float alpha) {
        if (!__any_sync(kAll, need)) return;
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
            uint32_t o[32];
            ptx::tmem_ld32(t_o + c * 32, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            ptx::tmem_st32(t_o + c * 32, o);
        }
    };

    // The sum of a tile's 128 weights as stored.
    auto rounded_sum = [&](uint32_t src) -> float {
        ptx::tmem_wait_st();
        ptx::F2 sum = ptx::f2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
            uint32_t w[32];
            ptx::tmem_ld32(src + c * 32, w);
#pragma unroll
            for (int e = 0; e < 32; ++e)
                sum = ptx::add2(sum, ptx::f2(__uint_as_float(w[e] << 16),
                                             __uint_as_float(w[e] & 0xffff0000u)));
        }
        float s0, s1;
        ptx::unpack(sum, s0, s1);
        return s0 + s1;
    };

    // PACK: tiles whose keys not every row of the unit sees.
    auto scanned = [&](const Unit &U, int32_t j) {
        return PACK && U.detail && U.win < 0 && (j < U.n_a || p.shape.gwin_off != nullptr);
    };
    // Whether keys [klo, khi) of the tile at k0, tile count c, hold a bad V row.
    auto sees_bad = [&](int32_t k0, int32_t klo, int32_t khi, uint32_t c) {
        uint32_t hit = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int32_t a = max(klo - k0 - 32 * w, 0), b = min(khi - k0 - 32 * w, 32);
            if (a < b) hit |= sm.bad[map][c & 3][w] & (kAll >> (32 - b)) & (kAll << a);
        }
        return hit != 0;
    };

    uint32_t cnt = 0, unit_iter = 0;   // key tiles, units
    for (int32_t u = blockIdx.x; u < S.n_units; u += gridDim.x) {
        const Unit U = units::query_unit<kBN>(p.shape, S, u);
        const int32_t n = U.n_a + U.n_b;
        if (n == 0) continue;
        const int32_t row = U.r0 + static_cast<int32_t>(r);
        const bool valid = row < U.rend;
        int32_t da, db, ga, gb;   // keys of this row
        units::query_ranges(p.shape, U, row, da, db, ga, gb);
        const float lam = __ldg(p.lambda + (p.n_lambda == 1 ? 0 : U.head));
        // The reference m_run (log2 units) is whole, so that moving it scales by a
        // power of two, exactly.
        // l_fix: what the sum of the weights changes by their rounding, in warps with a
        // row of at most kFewKeys keys (which only masked tiles hold). O is divided by
        // the sum of the weights as its products had them, so that a row with one key
        // gets its V exactly and a row with few keys no common error, which o_1 -
        // lambda o_2 would enlarge. Over many keys it averages out (and two
        // instructions more for every weight cost 2%).
        const bool few = __any_sync(kAll, valid && db - da + gb - ga <= kFewKeys);
        float m_run = kNegInf, l_run = 0.f, l_fix = 0.f;
        bool bad = false;
        // The bad rows of tile j (tile count c), which this map's threads wrote
        // before its product was issued; s_hi of the next tile and o_final follow.
        auto check_bad = [&](int32_t j, uint32_t c) {
            if (scanned(U, j))
                bad |= sees_bad(units::tile_row<kBN>(U, j), j < U.n_a ? da : ga,
                                j < U.n_a ? db : gb, c);
        };
        uint32_t lo[64], hi[64];
        // Move the reference of rows whose maximum mx2 exceeds it by more than the
        // threshold; returns the factor of everything summed so far. O: the P V of
        // the previous tile is done once s_hi is.
        auto move = [&](float mx2, bool o_empty) -> float {
            const bool need = m_run == kNegInf ? mx2 != kNegInf : mx2 > m_run + kRescaleThreshold;
            float alpha = 1.f;
            if (need) {
                const float m_new = ceilf(mx2);
                alpha = m_run == kNegInf ? 0.f : ptx::ex2(m_run - m_new);
                m_run = m_new;
            }
            l_run *= alpha;
            l_fix *= alpha;
            if (!o_empty) rescale_o(need, alpha);
            return alpha;
        };
        for (int32_t j = 0; j < n; ++j, ++cnt) {
            const int32_t k0 = units::tile_row<kBN>(U, j);
            const int32_t klo = j < U.n_a ? da : ga, khi = j < U.n_a ? db : gb;
            const bool masked = k0 < klo || k0 + kBN > khi;
            const uint32_t t_lo = t_s + lo_region(cnt), t_hi = t_s + 64 - lo_region(cnt);
            if (!__all_sync(kAll, wait_phase(sm, sm.s_lo[map], cnt & 1, err))) return;
            ptx::tc_fence_after();
            ptx::tmem_ld64(t_lo, lo);
            ptx::F2 sum = ptx::f2(0.f, 0.f);
            // (which form a tile takes follows from the layout alone, not from what
            // the keys hold)
            if (__any_sync(kAll, j == 0 || masked)) {
                if (!__all_sync(kAll, wait_phase(sm, sm.s_hi[map], cnt & 1, err))) return;
                ptx::tc_fence_after();
                ptx::tmem_ld64(t_hi, hi);
                ptx::tc_fence_before();
                ptx::mbar_arrive(ptx::smem_addr(&sm.s_read[map]));
                if (PACK && j > 0) check_bad(j - 1, cnt - 1);
                if (masked) {
#pragma unroll
                    for (int e = 0; e < 64; ++e) {
                        if (k0 + e < klo || k0 + e >= khi) lo[e] = __float_as_uint(kNegInf);
                        if (k0 + 64 + e < klo || k0 + 64 + e >= khi)
                            hi[e] = __float_as_uint(kNegInf);
                    }
                }
                move(fmaxf(row_max(lo), row_max(hi)) * sc, j == 0);
                const float m = m_run == kNegInf ? 0.f : m_run;
                exps_all(lo, m, t_lo, sum);
                exps_all(hi, m, t_lo + 32, sum);
                if (few) {
                    float s0, s1;
                    ptx::unpack(sum, s0, s1);
                    l_fix += rounded_sum(t_lo) - (s0 + s1);
                }
            } else {
                // Exponentials against the running reference right away. Where a row's
                // maximum turns out past the threshold its warp repeats the half: the
                // rows whose reference stays get the same bits again, so that no row's
                // weights depend on its neighbours' keys.
                float mx[2], mx2;
                uint32_t pk[16];
                for (;;) {
                    const float m = m_run == kNegInf ? 0.f : m_run;
                    mx[0] = mx[1] = kNegInf;
                    sum = ptx::f2(0.f, 0.f);
                    exps(std::true_type{}, c0, c32, lo, m, sum, mx, pk);
                    ptx::tmem_st16_nowait(t_lo, pk);
                    exps(std::true_type{}, c32, c32, lo, m, sum, mx, pk);
                    ptx::tmem_st16_nowait(t_lo + 16, pk);
                    if (!__all_sync(kAll, wait_phase(sm, sm.s_hi[map], cnt & 1, err))) return;
                    ptx::tc_fence_after();
                    mx2 = ptx::max_nan(mx[0], mx[1]) * sc;
                    if (!__any_sync(kAll, mx2 > m_run + kRescaleThreshold)) break;
                    ptx::tmem_wait_st();
                    move(mx2, false);
                }
                ptx::tmem_ld64(t_hi, hi);
                ptx::tc_fence_before();
                ptx::mbar_arrive(ptx::smem_addr(&sm.s_read[map]));
                if (PACK && j > 0) check_bad(j - 1, cnt - 1);
                const ptx::F2 sum_lo = sum;
                const float mx_lo = mx2;
                float f = 1.f;
                for (;;) {
                    const float m = m_run == kNegInf ? 0.f : m_run;
                    mx[0] = mx[1] = kNegInf;
                    sum = ptx::f2(0.f, 0.f);
                    exps(std::true_type{}, c0, c32, hi, m, sum, mx, pk);
                    ptx::tmem_st16_nowait(t_lo + 32, pk);
                    exps(std::true_type{}, c32, c32, hi, m, sum, mx, pk);
                    ptx::tmem_st16_nowait(t_lo + 48, pk);
                    mx2 = ptx::max_nan(mx[0], mx[1]) * sc;
                    if (!__any_sync(kAll, mx2 > m_run + kRescaleThreshold)) break;
                    ptx::tmem_wait_st();
                    f = move(mx2, false);
                    uint32_t plo[32];
                    ptx::tmem_ld32(t_lo, plo);
                    const __nv_bfloat162 f2 = __float2bfloat162_rn(f);
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const __nv_bfloat162 v =
                            __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&plo[e]), f2);
                        plo[e] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    ptx::tmem_st32_nowait(t_lo, plo);
                }
                // +inf and NaN make the row NaN (exp2_pair need not).
                if (!(ptx::max_nan(mx_lo, mx2) < __builtin_huge_valf()))
                    l_run = __uint_as_float(0x7fffffffu);
                sum = ptx::fma2(sum_lo, ptx::f2(f, f), sum);
            }
            ptx::tmem_wait_st();
            // V rows to zero, by both maps' threads (thread = V row), each before
            // its own product. V(j) is load 2 cnt + 1 of the ring, and stays until
            // both products ran. Nothing orders the maps within a tile, so a thread
            // that scans a non-finite row (PACK) may find the zeros of the other
            // map's thread: each leaves its mark before its zeros, and looks for the
            // other's after its scan. (Four tiles' marks are enough: with at most
            // eight slots, V(j + 4) is not loaded before both maps are done with V(j).)
            const int32_t seen = units::tile_rows<kBN>(U, j);
            if (seen < kBN || scanned(U, j)) {
                const uint32_t it = 2 * cnt + 1, slot = it % kSlots;
                if (!__all_sync(kAll, wait_phase(sm, sm.kv_full[slot], (it / kSlots) & 1, err)))
                    return;
                constexpr int kVecs = HD / 64 * 8;
                auto vec = [&](int i) {   // rotated by row: no bank conflicts
                    return sm.kv[slot] + (i / 8) * kBN * 128 + r * 128 + ((i + r) % 8) * 16;
                };
                const int32_t vr = static_cast<int32_t>(r);
                bool zero = vr >= seen && vr < 16 * tile_steps(U, j);
                if (scanned(U, j)) {
                    bool b = false;
                    if (vr < seen) {
#pragma unroll
                        for (int i = 0; i < kVecs; ++i)
                            b |= not_finite(ptx::ld_shared_v4(vec(i)));
                        volatile uint32_t &own = sm.mark[map][cnt & 3][r];
                        volatile uint32_t &other = sm.mark[1 - map][cnt & 3][r];
                        if (b) own = cnt + 1;
                        __threadfence_block();
                        b |= other == cnt + 1;
                    }
                    const uint32_t rows = __ballot_sync(kAll, b);
                    if ((r & 31) == 0) sm.bad[map][cnt & 3][r / 32] = rows;
                    zero |= b;
                }
                if (zero) {
#pragma unroll
                    for (int i = 0; i < kVecs; ++i) ptx::st_shared_v4(vec(i), 0, 0, 0, 0);
                    ptx::fence_proxy_async_smem();
                }
            }
            float sum0, sum1;
            ptx::unpack(sum, sum0, sum1);
            l_run += sum0 + sum1;
            ptx::tc_fence_before();
            ptx::mbar_arrive(ptx::smem_addr(&sm.p_full[map]));
        }
        // Epilogue: both maps' 1/l through shared memory; this group joins
        // columns [map * D/2, +D/2) of O_1 and O_2.
        const uint32_t par = unit_iter & 1;
        // (no reference: every logit is -inf, and 0 / 0 is NaN; rows past the unit have
        // none to store)
        const float l_o = l_run + l_fix, nan = __uint_as_float(0x7fffffffu);
        sm.inv_l[par][map][r] = l_o > 0.f && m_run != kNegInf ? 1.f / l_o : nan;
        ptx::mbar_arrive(ptx::smem_addr(&sm.joined));
        if (p.lse != nullptr && valid) {
            const int64_t rows = static_cast<int64_t>(p.shape.N) + p.shape.G;
            p.lse[((static_cast<int64_t>(U.b) * p.shape.heads + U.head) * 2 + map) * rows +
                  (U.detail ? row : static_cast<int64_t>(p.shape.N) + row)] =
                (m_run + __log2f(l_run)) * 0.69314718055994531f;
        }
        if (!__all_sync(kAll, wait_phase(sm, sm.joined, par, err) &&
                                  wait_phase(sm, sm.o_final, par, err)))
            return;
        ptx::tc_fence_after();
        if (PACK) check_bad(n - 1, cnt - 1);
        const float f1 = bad ? nan : sm.inv_l[par][0][r], f2 = bad ? nan : sm.inv_l[par][1][r];
        constexpr int kHalf = HD / 2;
        uint32_t o1[kHalf], o2[kHalf];
        const uint32_t t_o1 = tmem + kMaps * kBN + lane_sel + map * kHalf, t_o2 = t_o1 + HD;
        if constexpr (kHalf == 64) {
            ptx::tmem_ld64(t_o1, o1);
            ptx::tmem_ld64(t_o2, o2);
        } else {
            ptx::tmem_ld32(t_o1, o1);
            ptx::tmem_ld32(t_o2, o2);
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(ptx::smem_addr(&sm.o_empty));
        ++unit_iter;
        if (!valid) continue;
        const int side = U.detail ? 0 : 1;
        const int64_t at = ((static_cast<int64_t>(U.b) * (U.detail ? p.shape.N : p.shape.G) + row) *
                                p.shape.heads + U.head) * HD + map * kHalf;
#pragma unroll
        for (int e = 0; e < kHalf; ++e) {
            const float b = __uint_as_float(o2[e]) * f2;
            o1[e] = __float_as_uint(fmaf(-lam, b, __uint_as_float(o1[e]) * f1));
            o2[e] = __float_as_uint(b);
        }
        auto store = [&](__nv_bfloat16 *out, const uint32_t (&v)[kHalf]) {
            uint8_t *dst = reinterpret_cast<uint8_t *>(out + at);
#pragma unroll
            for (int i = 0; i < kHalf / 16; ++i) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    w[e] = ptx::pack_bf16x2(__uint_as_float(v[16 * i + 2 * e]),
                                            __uint_as_float(v[16 * i + 2 * e + 1]));
                if (p.o_v8) {
                    ptx::st_global_v8(dst + i * 32, w);
                } else {
                    reinterpret_cast<uint4 *>(dst)[2 * i] = make_uint4(w[0], w[1], w[2], w[3]);
                    reinterpret_cast<uint4 *>(dst)[2 * i + 1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        };
        store(p.o[side], o1);
        if (p.s[side] != nullptr) store(p.s[side], o2);
    }
}

template <int HD, bool PACK>
__global__ void __launch_bounds__(kThreads, 1) diff_tc_kernel(const __grid_constant__ Params p) {
    extern __shared__ uint8_t smem_raw[];
    Smem<HD> &sm = *reinterpret_cast<Smem<HD> *>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        ptx::mbar_init(ptx::smem_addr(&sm.q_full), 1);
        ptx::mbar_init(ptx::smem_addr(&sm.q_empty), kMaps);
        for (int s = 0; s < Smem<HD>::kSlots; ++s) {
            ptx::mbar_init(ptx::smem_addr(&sm.kv_full[s]), 1);
            ptx::mbar_init(ptx::smem_addr(&sm.kv_empty[s]), kMaps);
        }
        for (int m = 0; m < kMaps; ++m) {
            ptx::mbar_init(ptx::smem_addr(&sm.s_lo[m]), 1);
            ptx::mbar_init(ptx::smem_addr(&sm.s_hi[m]), 1);
            ptx::mbar_init(ptx::smem_addr(&sm.s_read[m]), kBM);
            ptx::mbar_init(ptx::smem_addr(&sm.p_full[m]), kBM);
            ptx::mbar_init(ptx::smem_addr(&sm.drain[m]), 1);
        }
        ptx::mbar_init(ptx::smem_addr(&sm.o_final), kMaps);
        ptx::mbar_init(ptx::smem_addr(&sm.joined), kMaps * kBM);
        ptx::mbar_init(ptx::smem_addr(&sm.o_empty), kMaps * kBM);
        sm.abort = 0;
        sm.max_len = 0;
        sm.err_word = p.err_word;
        ptx::fence_mbar_init();
    }
    if (PACK)
        for (int i = threadIdx.x; i < kMaps * 4 * kBM; i += kThreads)
            sm.mark[i / (4 * kBM)][i / kBM % 4][i % kBM] = 0;
    if (warp == kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(&sm.tmem_base), kTmemCols);
        ptx::tmem_relinquish();
    }
    if (warp == kProducerWarp && lane == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::prefetch_tmap(&p.tm_q[i]);
            ptx::prefetch_tmap(&p.tm_k[i]);
            ptx::prefetch_tmap(&p.tm_v[i]);
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
    if (warp < 8) {
        ptx::setmaxnreg_inc<kRegsSoftmax>();
        if (tmem_ok) softmax_epilogue<HD, PACK>(p, S, sm, tmem, warp / 4);
    } else {
        ptx::setmaxnreg_dec<kRegsOther>();
        if (tmem_ok && warp == kProducerWarp && lane == 0) producer<HD>(p, S, sm);
        if (tmem_ok && (warp == kMmaWarp || warp == kMmaWarp + 1))
            mma_issuer<HD>(p, S, sm, static_cast<int>(warp) - kMmaWarp);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (warp == kMmaWarp) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int HD>
atlas_status launch_hd(const DiffArgs &d, const DeviceInfo &dev, cudaStream_t stream) {
    const AttnArgs &a = d.attn;
    Params p{};
    int64_t n_units = 0;
    if (!units::make_shape(a, dev.sm_count, &p.shape, &n_units)) return ATLAS_ERR_SHAPE;
    const void *src[2][3] = {{a.q_d, a.k_d, a.v_d}, {a.q_g, a.k_g, a.v_g}};
    const int64_t rows[2] = {a.n_detail * a.batch, a.n_global * a.batch};
    CUtensorMap *maps[3] = {p.tm_q, p.tm_k, p.tm_v};
    for (int side = 0; side < 2; ++side) {
        // Maps of an absent side point at the other side; they are never used.
        const int use = rows[side] > 0 ? side : 1 - side;
        for (int t = 0; t < 3; ++t)
            if (!make_rows_map(&maps[t][side], src[use][t], rows[use], a.heads, HD))
                return ATLAS_ERR_CUDA;
    }
    p.o[0] = static_cast<__nv_bfloat16 *>(a.o_d);
    p.o[1] = static_cast<__nv_bfloat16 *>(a.o_g);
    p.s[0] = static_cast<__nv_bfloat16 *>(d.s_d);
    p.s[1] = static_cast<__nv_bfloat16 *>(d.s_g);
    uintptr_t bits = 0;
    for (int side = 0; side < 2; ++side)
        bits |= reinterpret_cast<uintptr_t>(p.o[side]) | reinterpret_cast<uintptr_t>(p.s[side]);
    p.o_v8 = (bits & 31) == 0;
    p.lse = a.lse;
    p.lambda = d.lambda;
    p.n_lambda = d.n_lambda;
    p.err_word = device_error_word();
    if (!p.err_word) return ATLAS_ERR_CUDA;
    p.scale_log2 = a.scale * 1.4426950408889634f;
    p.stall_unit = take_stall_request() ? 0 : -1;
    // Packed units may occur: windows below 128 rows, or unknown ones.
    const bool pack = p.shape.upw < 0 || (p.shape.upw == 0 && p.shape.N > 0);
    const size_t smem = sizeof(Smem<HD>) + 1024;
    auto kernel = pack ? diff_tc_kernel<HD, true> : diff_tc_kernel<HD, false>;
    if (!set_smem_limit(reinterpret_cast<const void *>(kernel), static_cast<int>(smem)))
        return ATLAS_ERR_CUDA;
    const int grid = static_cast<int>(n_units < dev.sm_count ? n_units : dev.sm_count);
    if (log_enabled())
        log_launch(pack ? "diff_tc_kernel<PACK>" : "diff_tc_kernel", grid, kThreads, smem,
                   "head_dim %d units %lld batch %d heads %d n_detail %d window %d n_global %d", HD,
                   static_cast<long long>(n_units), p.shape.batch, p.shape.heads, p.shape.N,
                   p.shape.L, p.shape.G);
    kernel<<<grid, kThreads, smem, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ATLAS_OK : ATLAS_ERR_CUDA;
}

}  // namespace

atlas_status launch_diff_attn_tc(const DiffArgs &d, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return ATLAS_ERR_DEVICE;
    return d.attn.head_dim == 128 ? launch_hd<128>(d, dev, stream)
                                  : launch_hd<64>(d, dev, stream);
}

}  // namespace atlas
