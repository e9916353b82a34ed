// Which kernel a grouped product takes: a function of the sizes and the type
// alone, on the host.
#pragma once

#include <algorithm>
#include <cmath>

#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNT = 0, kNN = 1, kTN = 2;
constexpr int kXcds = 8;
constexpr int kGroupM = 8;  // row tiles per group of the tile order

// Whether a weight gradient's queues (or parts of them) go to the XCDs whole.
__host__ __device__ __forceinline__ bool whole_queues(int64_t queues) { return queues >= 32 || queues % kXcds == 0; }

// Row tiles of bm rows that any queues of `rows` rows can have: each queue
// that is not empty ends in at most one partial tile.
int64_t row_tiles(const moe_grouped_t& g, int bm) {
    return (g.rows + (bm - 1) * std::min<int64_t>(g.E, g.rows)) / bm;
}

// The kernels and their tiles (rows x columns).
enum Variant { kSplit32, kSplit64, kTile64, kTile64x128, kTile128, kTile256, kVariants };
constexpr int kTileM[kVariants] = {32, 64, 64, 64, 128, 256};
constexpr int kTileN[kVariants] = {32, 64, 64, 128, 128, 256};

// What a round of one tile per CU takes, in 10 ns: for every slice, and once
// (start, epilogue), and no less than its stores.  Fitted to sweeps of rows,
// queues and widths (E 1 to 128, rows per queue 1 to 1024, widths 768 to 4096);
// on 361 random products the choice is 2.1 % slower than the best variant in the
// mean, at worst 1.9x (a weight gradient with one queue of nine times the mean,
// whose tiles of 256 last longest: the host does not know the queues' lengths).
// A tile of a quarter the size takes more than a quarter of the time, so the
// choice is between filling the last round and the rate within a round.  Both
// sides, bf16: 8 queues of 512 rows, 4096 x 2048, tiles of 128 in 5 rounds 78 us,
// tiles of 256 in 2 rounds 89 us; 64 queues of 512, 1408 x 2048, 13 rounds of
// 128 239 us, 4 rounds of 256 208 us; one queue of 128 rows, 4096 x 4096, split
// tiles of 32 in 2 rounds 17 us, tiles of 128 in one round 33 us.
struct Cost {
    int slice, once;
};
constexpr Cost kCost16[kVariants] = {{9, 100}, {25, 300}, {0, 0}, {30, 200}, {48, 170}, {148, 400}};
// float32 is bound by its matrix instructions: 64 x 64 tiles are as fast per
// output as larger ones.
constexpr Cost kCost32[kVariants] = {{17, 130}, {0, 0}, {50, 20}, {0, 0}, {0, 0}, {0, 0}};
// Weight gradients of short queues are bound by their stores and starts (128
// queues of 32 rows, 768 x 2048: float32 tiles of 64 378 us, of 128 287 us, of
// 256 225 us; bf16 tiles of 128 143 us, of 256 80 us).
constexpr Cost kCostW16[kVariants] = {{0, 0}, {0, 0}, {0, 0}, {0, 0}, {53, 350}, {150, 500}};
constexpr Cost kCostW32[kVariants] = {{0, 0}, {0, 0}, {50, 150}, {0, 0}, {195, 330}, {800, 600}};
constexpr int kCus = 256;
constexpr int kMaxParts = 32;

// What each mode and type has.
bool has(Variant v, int mode, bool f32) {
    if (mode == kTN) return v == kTile128 || v == kTile256 || (f32 && v == kTile64);
    return f32 ? v == kSplit32 || v == kTile64 : v != kTile64;
}

struct Plan {
    Variant v;
    int parts;      // kTN: ranges each queue is cut into
    int64_t tiles;  // at most
};

// The cheapest variant for mode `mode` of problem g.  The host knows the queues'
// number and sum only: a queue is taken to end in half a tile.
Plan plan_for(const moe_grouped_t& g, int mode, bool int8) {
    const bool f32 = g.dtype == MOE_DTYPE_F32 && !int8;
    const Cost* const cost = mode == kTN ? (f32 ? kCostW32 : kCostW16) : (f32 ? kCost32 : kCost16);
    const int64_t M = g.N, P = mode == kNT ? g.N : g.K;
    const int64_t qs = int8 ? 128 : (f32 ? 32 : 64);
    const int64_t live = std::max<int64_t>(std::min<int64_t>(g.E, g.rows), 1);
    Plan best{kTile128, 1, 0};
    double least = 0;
    // a round's stores at 5.5 TB/s
    auto round_time = [&](int v, int64_t n, int bytes) {
        const double stores = 100.0 * kCus * kTileM[v] * kTileN[v] * bytes / 5.5e6;
        return std::max(static_cast<double>(cost[v].once + cost[v].slice * n), stores);
    };
    const int out_bytes = g.dtype == MOE_DTYPE_BF16 ? 2 : 4;
    for (int i = 0; i < kVariants; ++i) {
        const Variant v = static_cast<Variant>(i);
        if (!has(v, mode, f32)) continue;
        const int64_t pt = ceil_div(P, kTileN[v]);
        if (mode == kTN) {
            const int64_t whole = g.E * ceil_div(M, kTileM[v]) * pt;
            const int64_t n = std::max<int64_t>(ceil_div(ceil_div(g.rows, live), qs), 1);
            for (int parts = 1; parts <= kMaxParts && (parts == 1 || (n >= 4 * parts && whole * parts <= 16 * kCus)); ++parts) {
                const int64_t rounds = ceil_div(whole * parts, kCus);
                double t = static_cast<double>(rounds) * round_time(v, ceil_div(n, parts), parts > 1 ? 4 : out_bytes);
                // the operands into the XCDs' L2s at 8 TB/s: each into one when whole
                // (parts of) queues are dealt, else into every XCD whose eighth
                // of the tiles needs it
                const int64_t mtn = ceil_div(M, kTileM[v]), per_x = ceil_div(mtn * pt, kXcds);
                const int64_t m_x = std::min(mtn, kGroupM * ceil_div(per_x, kGroupM * pt));
                const int64_t p_x = std::min(pt, ceil_div(per_x, kGroupM));
                const bool dealt = whole_queues(g.E * parts);
                const double reads = static_cast<double>(g.rows) * (f32 ? 4 : 2) *
                                     (g.N * (dealt ? 1.0 : static_cast<double>(kXcds * m_x) / mtn) +
                                      g.K * (dealt ? 1.0 : static_cast<double>(kXcds * p_x) / pt));
                t = std::max(t, 100.0 * reads / 8e6);
                // (a launch of the largest tiles takes longer to start)
                if (v == kTile256) t += 500;
                // the parts' sums written, read and added (4 TB/s), and a launch
                if (parts > 1)
                    t += 300 + 100.0 * (parts * 8.0 + 4.0) * static_cast<double>(g.E) * g.N * g.K / 4e6;
                if (least == 0 || t < least) {
                    least = t;
                    best = Plan{v, parts, whole * parts};
                }
            }
        } else {
            const int64_t n = ceil_div(mode == kNT ? g.K : g.N, qs);
            // row tiles: a queue's last one is half full in the mean, and their
            // number varies by sqrt(live / 12); rounds: the mean over that spread
            const double mt = static_cast<double>(g.rows) / kTileM[v] + 0.5 * live;
            const double spread = std::sqrt(live / 12.0);
            const double low = std::max<double>(live, mt - spread), high = std::max<double>(live, mt + spread);
            const double rounds = 0.5 * (std::ceil(low * pt / kCus) + std::ceil(high * pt / kCus));
            const double t = rounds * round_time(v, n, out_bytes);
            if (least == 0 || t < least) {
                least = t;
                best = Plan{v, 1, row_tiles(g, kTileM[v]) * pt};
            }
        }
    }
    return best;
}

size_t parts_bytes(const moe_grouped_t& g, const Plan& p) {
    return p.parts > 1 ? static_cast<size_t>(p.parts) * g.E * g.N * g.K * 4 : 0;
}

// Workgroups that plan p takes, one per tile: a multiple of 8.
int64_t workgroups(const moe_grouped_t& g, int mode, const Plan& p) {
    if (mode != kTN) return static_cast<int64_t>(align_up(p.tiles, kXcds));
    // (every XCD's list is sized for the most tiles one XCD receives)
    const int64_t queues = static_cast<int64_t>(g.E) * p.parts, whole = p.tiles / queues;
    return kXcds * (whole_queues(queues) ? ceil_div(queues, kXcds) * whole : g.E * ceil_div(whole * p.parts, kXcds));
}

// Whether both gradients go into one launch.  Not with the largest tiles nor the
// split kernel's 64 x 64 ones, which leave no room for a second workgroup in a
// CU's LDS, and not float32's 64 x 64 tiles with 128 x 128: of the former 4
// workgroups fit a CU, of the pair 2 (16 queues of 256 rows, 512 x 1024: 113 us
// together, 101 us one after the other).  Otherwise, together and one after the
// other: bf16, 8 queues of 250 rows, 1000 x 520, 14.2 and 20.6 us; 17 of 289,
// 648 x 304, 17.5 and 23.6 us; 8 of 1070, 552 x 1608, 61.8 and 60.7 us; one of 2
// rows, 72 x 248, 5.8 and 9.4 us.
bool pairs(const moe_grouped_t& g, const Plan& pa, const Plan& pw) {
    return pa.v != kTile256 && pa.v != kSplit64 && pw.v != kTile256 && !(pa.v == kTile64 && pw.v == kTile128) &&
           workgroups(g, kNN, pa) + workgroups(g, kTN, pw) < (1 << 24);
}

}  // namespace

}  // namespace moe
