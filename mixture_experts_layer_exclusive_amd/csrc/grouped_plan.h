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
// kHalves..: tiles whose slices two halves of the workgroup take in turn.
enum Variant { kSplit32, kSplit64, kTile64, kTile64x128, kTile128, kTile256, kHalves64x128, kHalves128, kTile128x256, kVariants };
constexpr int kTileM[kVariants] = {32, 64, 64, 64, 128, 256, 64, 128, 128};
constexpr int kTileN[kVariants] = {32, 64, 64, 128, 128, 256, 128, 128, 256};

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
    int alone;  // for every slice, where a CU has one tile and nothing beside it to do (4-bit values)
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
bool has(Variant v, int mode, bool f32, bool mx4) {
    if (v >= kHalves64x128) return mx4;
    if (mode == kTN) return v == kTile128 || v == kTile256 || (f32 && v == kTile64);
    return f32 ? v == kSplit32 || v == kTile64 : v != kTile64;
}

struct Plan {
    Variant v;
    int parts;      // kTN: ranges each queue is cut into
    int64_t tiles;  // at most
};

// The cheapest variant for mode `mode` of problem g.  The host knows the queues'
// number and sum only: a queue is taken to end in half a tile (with `mx4`, 4-bit
// values, not a single queue, whose rows it knows).
Plan plan_of(const moe_grouped_t& g, int mode, bool f32, const Cost* cost, int64_t qs, bool mx4 = false) {
    const int64_t M = g.N, P = mode == kNT ? g.N : g.K;
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
        if (!has(v, mode, f32, mx4)) continue;
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
            const bool known = mx4 && g.E == 1;
            const double mt = known ? ceil_div(g.rows, kTileM[v]) : static_cast<double>(g.rows) / kTileM[v] + 0.5 * live;
            const double spread = known ? 0.0 : std::sqrt(live / 12.0);
            const double low = std::max<double>(live, mt - spread), high = std::max<double>(live, mt + spread);
            const double rounds = 0.5 * (std::ceil(low * pt / kCus) + std::ceil(high * pt / kCus));
            const double alone = rounds < 2 ? (2 - rounds) * cost[v].alone * static_cast<double>(n) : 0.0;
            const double t = rounds * round_time(v, n, out_bytes) + alone;
            if (least == 0 || t < least) {
                least = t;
                best = Plan{v, 1, row_tiles(g, kTileM[v]) * pt};
            }
        }
    }
    return best;
}

Plan plan_for(const moe_grouped_t& g, int mode, bool int8) {
    const bool f32 = g.dtype == MOE_DTYPE_F32 && !int8;
    const Cost* const cost = mode == kTN ? (f32 ? kCostW32 : kCostW16) : (f32 ? kCost32 : kCost16);
    return plan_of(g, mode, f32, cost, int8 ? 128 : (f32 ? 32 : 64));
}

// The forward of 4-bit floats.  Fitted to 61000 random products (E 1 to 256, rows per
// queue 1 to 60000, N 64 to 14400, K 128 to 9600), of which the choice is 0.5 % slower than
// the best variant in the mean, 11 to 17 % in one of 100 (with bf16's costs 2.7 %).  Both
// sides: 512 rows, 4096 x 4096, tiles of 64 x 128 12.5 us, of 128 15.2 us; 2048 rows, of 128
// 22.8, of 256 29.6; 16384 rows, 14336 x 4096, in 8 queues, of 128 622, of 256 506; 128 rows,
// split tiles of 32 9.1, tiles of 64 x 128 11.7.  (A single queue with half a tile more, as
// many: 2048 rows, 4096 x 2048, in 3 rounds of 128 or one of 256, 20.7 us; known to be 2
// rounds, 16.6.)
// A tile alone on its CU takes longer than its loads or its products: the 4 waves wait for
// each other at every step (a ring of 3, 4 or 5 stages changes nothing).  Two halves, each
// with its own slices and stages, fill the waits: 599 rows, 4456 x 8512, tiles of 128 25 us
// for 31; 375, 7744 x 4096, 14.4 and 17.5; 113, 8656 x 2496, tiles of 64 x 128 9.9 and 11.1.
// Short reductions keep the whole tiles, two of which share a CU: 113 rows, 11312 x 1472, 9.2
// us either way.
// Tiles of 128 x 256, walked as a stream like the largest: between these and those of 128
// (LDS reads 0.55 of the products' time, those of 128 1.0), and where short reductions of many
// queues end: 498 rows in 92 queues, 3896 x 352, 14.3 us, the best other 19.3; 3756 in 95,
// 6632 x 288, 41 and 55; over products whose floor is 5 to 50 us 3 % in the mean.
constexpr Cost kCostMx4[kVariants] = {{4, 163, 0},  {13, 401, 0}, {0, 0, 0},    {28, 126, 11}, {28, 190, 13},
                                      {58, 538, 4}, {27, 170, 4}, {26, 275, 4}, {39, 257, 19}};
// float32 outputs: the same, with twice the stores at a tile's end (7000 such products: the
// choice 0.9 % slower than the best in the mean, with the costs above 2.1 %).
constexpr Cost kCostMx4Out32[kVariants] = {{6, 157, 0},  {10, 472, 0}, {0, 0, 0},    {29, 158, 9}, {29, 248, 10},
                                           {60, 660, 0}, {27, 276, 2}, {26, 338, 8}, {42, 320, 20}};
Plan plan_mxfp4(const moe_grouped_t& g) {
    return plan_of(g, kNT, false, g.dtype == MOE_DTYPE_F32 ? kCostMx4Out32 : kCostMx4, 256, true);
}

// Whether it goes to the kernel for reductions of one slice: where the queues are short,
// too, and a tile of 64 rows or more is mostly start and end.  Both sides: 75 queues of 2
// rows, 10816 x 64, 11 us, the best other kernel 61; 255 of 12 rows, 12000 x 96, 63 and 200;
// 200 of 60 rows, 12000 x 128, 197 and 213; 16 of 50 rows, 5600 x 256, 12.9 and 12.2; 200 of
// 100 rows, 1600 x 256, 47 and 40.
bool short_mxfp4(const moe_grouped_t& g) {
    return g.K <= 256 && g.rows <= 64 * std::min<int64_t>(g.E, g.rows);
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
