// Matrix products grouped by expert: the forward, its two gradients, and the
// 8-bit integer product.
//
//   kNT  C[r, n]   = sum_k A[r, k] W_e[n, k]       rows r of queue e
//   kNN  dA[r, k]  = sum_n dC[r, n] W_e[n, k]
//   kTN  dW_e[n, k] = sum_{r in queue e} dC[r, n] A[r, k]
//
// In every mode the output tile is C[m, p] = sum_q X[m, q] Y[p, q] over a
// reduction index q.  An operand is "row-major" (q is contiguous: A and W in
// kNT, dC in kNN) or "column-major" (a memory row holds one q for all m or p:
// W in kNN, both operands in kTN).  One pipeline serves all of them; only how
// a slice is laid out in LDS and read into fragments differs.
#include <algorithm>
#include <type_traits>

#include "grouped_common.h"
#include "grouped_plan.h"

namespace moe {

namespace {

// ---- the tile kernel ------------------------------------------------------------
//
// 4 waves in 2 x 2; a wave owns MB x NB blocks of 32 x 32 outputs.  A slice is
// 128 bytes of q of every tile row (64 bf16, 32 f32 or 128 int8 values), in
// two LDS stages.  The MFMA takes Y's fragment first and X's second, so a lane
// holds one output row (lane & 31) and runs of 4 consecutive columns.
//
// A workgroup of the largest tiles walks its XCD's tiles in rounds of blocks /
// 8, and the slices of all its tiles are one stream: while a tile's last slices
// are multiplied and its outputs stored, the first slices of the next are
// landing.  (Weight gradients, whose tiles fall in cost: every other round is
// dealt backwards.  16 uneven queues, 4096 rows in the mean, 1408 x 2048: 388
// us, dealt one way 404; 24, 2048 in the mean, 2048 x 1024: 262 and 277; even
// queues, and those dealt by load, the same either way.)
//
// Each slice has 4 steps of 32 bytes of q (16 bytes per half wave).  Step 0
// multiplies fragments read during the slice before; the fragments of steps 1
// and 2 are read during step 0, those of step 3 early in step 1 (all of them
// in step 0 would take longer than its MFMAs: 24 KB per wave at 128 bytes a
// clock).  Then the stage is free, and the loads of the next-but-one slice go
// out spread over the other MFMAs (an LDS-bound load holds up the MFMAs
// behind it, so a burst of them stalls; the stream spreads them on over step 0
// of the next slice: bf16, 8 x 2048 rows, 14336 x 4096, over 20 MFMAs 1643 us,
// 28 1541, 36 1498, 52 1463).  Before step 3 the next slice has landed, and
// step 3 reads its first fragments.
//
// The largest tiles at a long reduction are bound by power first: products of
// normal values from registers alone hold 1.8 GHz (16384 rows, 14336 x 4096:
// 1045 us), of zeros 2.4 GHz (786 us), and this kernel 1.5 GHz.  One queue of
// those rows takes 1358 us; 1334 over operands from the caches only, 1332
// without half of the fragment reads.  8 queues of 2048: 1428, 1328, 1406.
template <int MB, int NB, int NS, typename O>
struct TileLds {
    static constexpr int STAGE = 64 * (MB + NB) * 128;
    static constexpr int NP = sizeof(O) == 2 && NB >= 2 ? 2 : 1;  // column blocks the epilogue stages at a time
    static constexpr int EROW = NP * 32 * sizeof(O);  // bytes of a staged row: a 128-byte line (bf16, NB = 1: 64)
    static constexpr int EPI = 32 * EROW;             // staged bytes per wave
    // the largest tiles walk the tile order as one stream and stage their
    // outputs beside the stages; the others take one tile and stage over them
    static constexpr bool STREAM = MB * NB > 4;
    static constexpr int EPI_AT = STREAM ? NS * STAGE : 0;
    static constexpr int Q_AT = NS * STAGE + (STREAM ? 4 * EPI : 0);
    static_assert(4 * EPI <= NS * STAGE, "the staged outputs must fit the stages");
    static constexpr int RING_AT = Q_AT + sizeof(Queues);
    static constexpr int DEAL_AT = RING_AT + 512;
    static constexpr int BYTES = DEAL_AT + (STREAM ? sizeof(Deal) : 0);
    static_assert(BYTES <= 160 * 1024, "LDS");
};

// smem: TileLds::BYTES, 1024-byte aligned; workgroup `block` of `blocks`
template <int TY, int MODE, int MB, int NB, int NS, typename O>
__device__ __forceinline__ void grouped_tile(char* __restrict__ smem, int block, int blocks, const void* __restrict__ Xp,
                                             const void* __restrict__ Yp, const int32_t* __restrict__ offsets, int E,
                                             int rows, int N, int K, O* __restrict__ C, const float* __restrict__ sx,
                                             const float* __restrict__ sy, int parts) {
    using Lds = TileLds<MB, NB, NS, O>;
    constexpr bool XC = MODE == kTN;             // X column-major
    constexpr bool YC = MODE != kNT;             // Y column-major
    static_assert(TY != kI8 || MODE == kNT, "int8: forward only");
    constexpr int TM = 64 * MB, TN = 64 * NB;    // output tile
    using XS = Slice<TY, XC, TM>;
    using YS = Slice<TY, YC, TN>;
    constexpr int EB = XS::EB;
    constexpr int QS = 128 / EB;                 // q per slice
    constexpr int XL = XS::LOADS / 4, YL = YS::LOADS / 4;  // loads per wave and slice
    constexpr int NL = XL + YL;
    constexpr int X_BYTES = TM * 128;
    constexpr int STAGE = Lds::STAGE;
    constexpr int NM = MB * NB;
    constexpr int NR = MB + NB;
    constexpr bool BF_OUT = sizeof(O) == 2;
    constexpr int NP = Lds::NP, EROW = Lds::EROW, EPI = Lds::EPI;
    constexpr int CPR = EROW / 16;               // 16-byte chunks per staged row
    constexpr int RPS = 64 / CPR;                // rows per store
    constexpr bool STREAM = Lds::STREAM;
    constexpr int EPI_AT = Lds::EPI_AT, Q_AT = Lds::Q_AT;
    Queues& queues = *reinterpret_cast<Queues*>(smem + Q_AT);

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int P = MODE == kNT ? N : K;           // output columns
    const int64_t xrow = static_cast<int64_t>(MODE == kNT ? K : N) * EB;  // bytes of an operand's memory row
    const int64_t yrow = static_cast<int64_t>(K) * EB;

    load_queues<MODE == kTN>(offsets, E, rows, TM, queues);
    const int xcd = block % kXcds;
    const int stride = blocks / kXcds;
    // weight gradients: how their tiles are dealt.  A stream's queues are uneven
    // if the longest is over 1.25 times the mean.  Few of them (below 32) then
    // go over all XCDs (8 queues of 4096 rows in the mean, 4096 x 2048: 427 us,
    // by load 557 us; with smaller tiles, whose problems are small, it changes
    // nothing); more are dealt by load where the work is worth it: from half a
    // slice per workgroup and expert (128 queues, 768 x 2048, of 512 rows, 96
    // slices: 258 us, in snake order 273; of 256 rows, 48 slices, 151 either way).
    bool dealt = MODE == kTN && whole_queues(static_cast<int64_t>(E) * parts), uneven = false;
    Deal& deal = *reinterpret_cast<Deal*>(smem + (STREAM ? Lds::DEAL_AT : 0));
    const int tiles_of_queue = ((N + TM - 1) / TM) * ((K + TN - 1) / TN);
    if constexpr (MODE == kTN && STREAM) {
        const int e = queues.order[0];
        const int64_t longest = __builtin_amdgcn_readfirstlane(queues.hi[e] - queues.lo[e]);
        if (parts == 1 && dealt && longest * 4 * E > static_cast<int64_t>(rows) * 5) {
            dealt = E >= 32;
            uneven = dealt && stride <= 32 &&
                     2 * static_cast<int64_t>(rows) * tiles_of_queue >= static_cast<int64_t>(E) * QS * blocks;
            if (uneven) deal_queues(queues, E, QS, tiles_of_queue, xcd, block / kXcds, stride, deal);
        }
    }
    int dealt_queue = 0, dealt_tile = 0;         // uneven: the next tile
    auto tile_at = [&](int place, Tile& t) -> Found {
        if constexpr (MODE == kTN) {
            if (STREAM && uneven) {
                const int full = quick_div(tiles_of_queue, stride), rest = tiles_of_queue - full * stride;
                for (; dealt_queue < __builtin_amdgcn_readfirstlane(deal.queues); ++dealt_queue, dealt_tile = 0) {
                    const int last = __builtin_amdgcn_readfirstlane(static_cast<int>(deal.place[dealt_queue]));
                    if (dealt_tile >= full + (last < rest ? 1 : 0)) continue;
                    const int local = dealt_tile * stride + (dealt_tile < full ? block / kXcds : last);
                    ++dealt_tile;
                    weight_tile_of(queues, __builtin_amdgcn_readfirstlane(static_cast<int>(deal.expert[dealt_queue])), 0,
                                   local, E, N, K, TM, TN, QS, 1, t);
                    return kTile;
                }
                return kEnd;
            }
            return weight_tile(queues, E, N, K, TM, TN, QS, parts, dealt, xcd, place, t);
        } else {
            t.q0 = 0;
            t.q1 = MODE == kNT ? K : N;
            return row_tile(queues, E, TM, TN, P, xcd, place, t);
        }
    };

    // (an empty queue's weight gradient is one slice that is out of range
    // altogether: zeros)
    auto slices_of = [&](const Tile& t) { return max((t.q1 - t.q0 + QS - 1) / QS, 1); };

    // ---- the load side: the tile being loaded, and how much of it is left
    constexpr int64_t kLineStep = 128;
    const int64_t xstep = XC ? QS * xrow : kLineStep, ystep = YC ? QS * yrow : kLineStep;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const uint32_t lds_x = lds0 + wave * (XL * 1024);
    const uint32_t lds_y = lds0 + X_BYTES + wave * (YL * 1024);
    int lround = 0;
    int left = 0;                                // slices still to load
    uint64_t xbase = 0, ybase = 0;
    // This wave's loads j fill the KB at (wave * L + j) * 1024 of the operand's
    // part of the stage.  Bit j of the tail masks: the lane's part of load j is
    // out of range in the tile's last slice.
    uint32_t xoff[XL], yoff[YL], xtail = 0, ytail = 0;
    bool tailed = false;                         // the last slice is not a whole one
    auto aim = [&](const Tile& t) {
        left = slices_of(t);
        const int qtail = t.q1 - t.q0 - (left - 1) * QS;  // q in the last slice
        int ln = lane;
        asm volatile("" : "+v"(ln));  // (keeps the lane's part from being computed ahead and held in registers)
        xtail = ytail = 0;
        tailed = qtail < QS;
        xbase = reinterpret_cast<uint64_t>(Xp) +
                static_cast<uint64_t>(XC ? t.q0 * xrow + static_cast<int64_t>(t.m0) * EB : t.m0 * xrow);
        ybase = reinterpret_cast<uint64_t>(Yp) +
                static_cast<uint64_t>(MODE == kTN   ? t.q0 * yrow + static_cast<int64_t>(t.p0) * EB
                                      : MODE == kNN ? static_cast<int64_t>(t.e) * N * yrow + static_cast<int64_t>(t.p0) * EB
                                                    : (static_cast<int64_t>(t.e) * N + t.p0) * yrow);
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            xoff[j] = XS::offset(wave * XL + j, ln, static_cast<uint32_t>(xrow), t.m1 - t.m0);
            xtail |= (XS::beyond(wave * XL + j, ln, qtail) ? 1u : 0u) << j;
        }
#pragma unroll
        for (int j = 0; j < YL; ++j) {
            yoff[j] = YS::offset(wave * YL + j, ln, static_cast<uint32_t>(yrow), P - t.p0);
            ytail |= (YS::beyond(wave * YL + j, ln, qtail) ? 1u : 0u) << j;
        }
        xbase = uniform64(xbase);
        ybase = uniform64(ybase);
    };
    auto nothing = [&]() {
        left = 0x7fffffff;
        tailed = false;
#pragma unroll
        for (int j = 0; j < XL; ++j) xoff[j] = kOutOfRange;
#pragma unroll
        for (int j = 0; j < YL; ++j) yoff[j] = kOutOfRange;
    };
    // the tiles between the load side and the multiplying side (at most two, of
    // one slice each, and the one being multiplied), kept by each wave for itself
    int* const ring = reinterpret_cast<int*>(smem + Lds::RING_AT) + wave * 32;
    int loading = 0;                             // tiles the load side has begun
    // the next tile; after the last, every load is out of range
    auto next_load = [&]() {
        for (;;) {
            Tile t;
            const int at = block / kXcds;
            const Found f = tile_at(lround * stride + (MODE == kTN && (lround & 1) ? stride - 1 - at : at), t);
            ++lround;
            if (f == kTile) {
                aim(t);
                int* const r = ring + (loading & 3) * 8;
                *reinterpret_cast<i32x4_t*>(r) = i32x4_t{t.e, t.m0, t.m1, t.p0};
                r[4] = left;
                ++loading;
                return;
            }
            if (f == kEnd) {
                nothing();
                return;
            }
        }
    };
    // load l (< NL) of the next slice to load, into stage `so`
    auto dma = [&](int l, uint32_t so) {
        const bool y = l < YL;
        const int j = y ? l : l - YL;
        lds_dma16_b(y ? ybase : xbase, y ? yoff[j < YL ? j : 0] : xoff[j < XL ? j : 0],
                    (y ? lds_y : lds_x) + so + j * 1024);
    };
    // before a tile's last slice is loaded (its offsets are not needed again)
    auto cut_tail = [&]() {
        if (left == 1 && tailed) {
#pragma unroll
            for (int j = 0; j < XL; ++j) xoff[j] |= (xtail << (31 - j)) & kOutOfRange;
#pragma unroll
            for (int j = 0; j < YL; ++j) yoff[j] |= (ytail << (31 - j)) & kOutOfRange;
        }
    };
    auto loaded = [&]() {
        xbase += xstep;
        ybase += ystep;
        if (--left == 0) {
            if (STREAM) next_load();
            else nothing();
        }
    };

    // ---- fragments and products
    const Fragments<TY, XC, TM, MB> xfrag(lane, wm * MB);
    const Fragments<TY, YC, TN, NB> yfrag(lane, wn * NB);
    i32x4_t f[4][NR];                            // f[step][X blocks, then Y blocks]
    auto read_frag = [&](int kk, int i, uint32_t so) {
        f[kk][i] = i < MB ? xfrag.read(smem, so, i, kk) : yfrag.read(smem + X_BYTES, so, i - MB, kk);
    };
    Acc<TY> acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = zero_acc<TY>();
    // (there and back over X, so that two products in a row share a fragment: 1 %)
    auto mul = [&](int kk, int q) {
        const int mb = q / MB % 2 ? MB - 1 - q % MB : q % MB;
        multiply<TY>(f[kk][MB + q / MB], f[kk][mb], acc[q / MB][mb]);
    };

    // the refilling loads go out over SLOTS MFMAs: those of step 1 after FREE,
    // steps 2 and 3, and LATE of the next slice's step 0
    constexpr int FREE = NM >= 4 ? NM * 3 / 4 : NM;
    constexpr int LATE = STREAM ? NM : 0;
    constexpr int SLOTS = NM - FREE + 2 * NM + LATE;
    constexpr int BEFORE3 = (2 * NM - FREE) * NL / SLOTS;  // of them before step 3
    constexpr int BEFORE0 = (SLOTS - LATE) * NL / SLOTS;   // before step 0
    static_assert(LATE == 0 || NS == 2, "the late loads go into the other stage");
    constexpr int RD3 = NM >= 2 ? NM / 2 : 1;    // MFMAs of step 1 that read step 3's fragments
    // loads younger than the next slice's at the wait for it
    constexpr int YOUNGER = (NS - 2) * NL + BEFORE3;
    static_assert((NS - 1) * NL < 64, "vmcnt");
    uint32_t so = 0;                             // the stage being multiplied
    auto slice = [&]() {
        const uint32_t nso = so + STAGE == NS * STAGE ? 0 : so + STAGE;
        auto refill = [&](int p, uint32_t stage) {
#pragma unroll
            for (int l = p * NL / SLOTS; l < (p + 1) * NL / SLOTS; ++l) dma(l, stage);
        };
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mul(0, q);
#pragma unroll
            for (int i = q * 2 * NR / NM; i < (q + 1) * 2 * NR / NM; ++i) read_frag(1 + i / NR, i % NR, so);
            if (q < LATE) refill(SLOTS - LATE + q, nso);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (LATE > 0) loaded();
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mul(1, q);
            if (q < RD3) {
#pragma unroll
                for (int i = q * NR / RD3; i < (q + 1) * NR / RD3; ++i) read_frag(3, i, so);
            }
            if (q >= FREE) refill(q - FREE, so);
            __builtin_amdgcn_sched_barrier(0);
            if (q == FREE - 1) {
                wait_vmcnt_lgkm0<63>();
                barrier_lds();
                cut_tail();
            }
        }
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mul(2, q);
            refill(NM - FREE + q, so);
            __builtin_amdgcn_sched_barrier(0);
        }
        wait_vmcnt<YOUNGER>();
        barrier_lds();
        // (after the last slice of all this reads zeros that are never used)
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mul(3, q);
            refill(2 * NM - FREE + q, so);
#pragma unroll
            for (int i = q * NR / NM; i < (q + 1) * NR / NM; ++i) read_frag(0, i, nso);
            __builtin_amdgcn_sched_barrier(0);
        }
        if (LATE == 0) loaded();
        so = nso;
    };

    // ---- epilogue
    // lane: output row m0 + (wm * MB + mb) * 32 + l32, columns p0 + (wn * NB +
    // nb) * 32 + 8 g + 4 half + 0..3 in registers 4 g .. 4 g + 3
    auto epilogue = [&](const Tile& t) {
        int lane = tid & 63;
        asm volatile("" : "+v"(lane));  // (as in aim)
        const int half = lane >> 5, l32 = lane & 31;
        if (!STREAM) {
            wait_vmcnt_lgkm0<0>();
            barrier_lds();
        }
        const int mrow = t.m0 + wm * MB * 32, pcol = t.p0 + wn * NB * 32;
        float rs[MB];
        if constexpr (TY == kI8) {
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) rs[mb] = sx[min(mrow + mb * 32 + l32, t.m1 - 1)];
        }
        O* const out = C + (MODE == kTN ? static_cast<int64_t>(t.e) * N * K : 0) + static_cast<int64_t>(mrow) * P + pcol;
        f32x4_t cs[TY == kI8 ? NB : 1][4];
        if constexpr (TY == kI8) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = min(pcol + nb * 32 + 8 * g + 4 * half, P - 4);
                    cs[nb][g] = *reinterpret_cast<const f32x4_t*>(sy + static_cast<int64_t>(t.e) * N + col);
                }
        }
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
            for (int n0 = 0; n0 < NB; n0 += NP) {
                // (the accumulators leave their registers here, block by block:
                // without this the compiler copies all of them at once)
                if constexpr (STREAM) {
#pragma unroll
                    for (int nb = 0; nb < NP; ++nb) asm volatile("" : "+a"(acc[n0 + nb][mb]));
                }
#pragma unroll
                for (int nb = 0; nb < NP; ++nb)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        f32x4_t v;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[i] = static_cast<float>(acc[n0 + nb][mb][4 * g + i]);
                            if constexpr (TY == kI8) v[i] = v[i] * rs[mb] * cs[TY == kI8 ? n0 + nb : 0][g][i];
                        }
                        // staged in LDS by the wave for itself, 16-byte chunk ch of
                        // row r at ch ^ (r mod CPR)
                        char* const row = smem + EPI_AT + wave * EPI + l32 * EROW;
                        if constexpr (BF_OUT)
                            *reinterpret_cast<uint2*>(row + (((nb * 4 + g) ^ (l32 & (CPR - 1))) * 16) + half * 8) =
                                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                        else
                            *reinterpret_cast<f32x4_t*>(row + (((2 * g + half) ^ (l32 & (CPR - 1))) * 16)) = v;
                    }
                // zero for the next tile (while the staged values settle)
                if constexpr (STREAM) {
#pragma unroll
                    for (int nb = 0; nb < NP; ++nb) {
                        acc[n0 + nb][mb] = zero_acc<TY>();
                        asm volatile("" : "+a"(acc[n0 + nb][mb]));
                    }
                }
                // whole chunks, consecutive lanes on consecutive chunks of a row
                u32x4_t v[32 / RPS];
                uint32_t off[32 / RPS];
#pragma unroll
                for (int i = 0; i < 32 / RPS; ++i) {
                    const int r = i * RPS + lane / CPR;
                    v[i] = *reinterpret_cast<const u32x4_t*>(smem + EPI_AT + wave * EPI + r * EROW +
                                                             (((lane % CPR) ^ (r & (CPR - 1))) * 16));
                }
                const uint64_t base =
                    uniform64(reinterpret_cast<uint64_t>(out) +
                              static_cast<uint64_t>((static_cast<int64_t>(mb) * 32 * P + n0 * 32) * sizeof(O)));
                const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
                    reinterpret_cast<void*>(base), 0, static_cast<int>(kOutOfRange), static_cast<int>(kRsrcWord3));
#pragma unroll
                for (int i = 0; i < 32 / RPS; ++i) {
                    const int r = i * RPS + lane / CPR;
                    const int c = (lane % CPR) * (16 / static_cast<int>(sizeof(O)));
                    off[i] = mrow + mb * 32 + r < t.m1 && pcol + n0 * 32 + c < P
                                 ? (static_cast<uint32_t>(r) * static_cast<uint32_t>(P) + c) * static_cast<uint32_t>(sizeof(O))
                                 : kOutOfRange;
                }
                // rows of whole 128-byte lines past the L2's lifetime (bf16, 65536 x
                // 2048 x 256: 90 us, 97 through it; 16384 x 4864 x 128 and the large
                // products the same to 1 %); other rows' stores share lines, which
                // the L2 has to put together (16384 x 4904 x 128: 100 us past it, 42
                // through it)
                if (P % (128 / static_cast<int>(sizeof(O))) == 0) {
#pragma unroll
                    for (int i = 0; i < 32 / RPS; ++i)
                        __builtin_amdgcn_raw_buffer_store_b128(v[i], rsrc, off[i], 0, kNonTemporal);
                } else {
#pragma unroll
                    for (int i = 0; i < 32 / RPS; ++i) __builtin_amdgcn_raw_buffer_store_b128(v[i], rsrc, off[i], 0, 0);
                }
                if constexpr (STREAM) __builtin_amdgcn_sched_barrier(0);
            }
        }
    };

    // ---- the stream
    next_load();
#pragma unroll
    for (int st = 0; st < NS; ++st) {
        cut_tail();
#pragma unroll
        for (int l = 0; l < (st < NS - 1 ? NL : BEFORE0); ++l) dma(l, st * STAGE);
        if (LATE == 0 || st < NS - 1) loaded();
    }
    wait_vmcnt<(NS - 2) * NL + BEFORE0>();
    barrier_lds();
#pragma unroll
    for (int i = 0; i < NR; ++i) read_frag(0, i, 0);
    __builtin_amdgcn_sched_barrier(0);
    // (one flat loop over slices, with the tile's end inside: nested loops make
    // the compiler move the accumulators between registers at every tile)
    Tile t;
    int tiles = 0, n;
    auto next_tile = [&]() {
        if (tiles == loading) return false;
        const int* const r = ring + (tiles & 3) * 8;
        const i32x4_t v = *reinterpret_cast<const i32x4_t*>(r);
        n = __builtin_amdgcn_readfirstlane(r[4]);
        t.e = __builtin_amdgcn_readfirstlane(v[0]);
        t.m0 = __builtin_amdgcn_readfirstlane(v[1]);
        t.m1 = __builtin_amdgcn_readfirstlane(v[2]);
        t.p0 = __builtin_amdgcn_readfirstlane(v[3]);
        ++tiles;
        return true;
    };
    bool more = next_tile();
    while (more) {
        slice();
        if (--n == 0) {
            epilogue(t);
            more = next_tile();
        }
    }
    wait_vmcnt<0>();  // (the last loads still write LDS)
}

template <int TY, int MODE, int MB, int NB, int NS, typename O>
__global__ __launch_bounds__(256, (MB * NB > 4 ? 1 : 2)) void grouped_tile_kernel(
    const void* __restrict__ Xp, const void* __restrict__ Yp, const int32_t* __restrict__ offsets, int E, int rows,
    int N, int K, O* __restrict__ C, const float* __restrict__ sx, const float* __restrict__ sy, int parts) {
    __shared__ __attribute__((aligned(1024))) char smem[TileLds<MB, NB, NS, O>::BYTES];
    grouped_tile<TY, MODE, MB, NB, NS, O>(smem, blockIdx.x, gridDim.x, Xp, Yp, offsets, E, rows, N, K, C, sx, sy, parts);
}

// ---- the split kernel ---------------------------------------------------------------
//
// For problems of too few tiles to fill the card: a 32 MB x 32 NB output tile per
// workgroup, its slices dealt to the 4 waves in turn.  Each wave multiplies its
// own slices into a whole tile of its own, from a private ring of 2 LDS stages,
// without a barrier: a tile kernel's wave of this size would wait at two
// barriers for every slice of a few MFMAs.  At the end the 4 partial tiles are
// added in the order of the waves.
//
// The fragments of a slice are read while those of the slice before are
// multiplied, then its stage takes the loads of the slice after next.  Slices
// past the end are loaded out of range (zeros, no traffic), so that the number
// of loads in flight, and with it the waits, is constant.
constexpr int split_lds(int MB, int NB) { return 4 * 2 * (32 * MB + 32 * NB) * 128; }

// smem: split_lds bytes, 1024-byte aligned
template <int TY, int MODE, int MB, int NB, typename O>
__device__ __forceinline__ void grouped_split(char* __restrict__ smem, int block, const void* __restrict__ Xp,
                                              const void* __restrict__ Yp, const int32_t* __restrict__ offsets, int E,
                                              int rows, int N, int K, O* __restrict__ C, const float* __restrict__ sx,
                                              const float* __restrict__ sy) {
    static_assert(MODE != kTN && (TY != kI8 || MODE == kNT), "no weight gradients; int8: forward only");
    constexpr bool YC = MODE != kNT;
    constexpr int TM = 32 * MB, TN = 32 * NB;
    using XS = Slice<TY, false, TM>;
    using YS = Slice<TY, YC, TN>;
    constexpr int EB = XS::EB;
    constexpr int QS = 128 / EB;
    constexpr int X_BYTES = TM * 128;
    constexpr int STAGE = (TM + TN) * 128;
    constexpr int RING = 2 * STAGE;              // per wave
    constexpr int PADC = TN + 4;                 // row length of a partial tile in LDS
    static_assert(TM * PADC * 4 <= RING && sizeof(Queues) <= 4 * RING, "LDS");
    using Val = std::conditional_t<TY == kI8, int, float>;
    typedef Val val4_t __attribute__((ext_vector_type(4)));
    static_assert(4 * RING == split_lds(MB, NB), "LDS");
    Queues& queues = *reinterpret_cast<Queues*>(smem);

    const int P = MODE == kNT ? N : K;
    Tile t;
    load_queues<false>(offsets, E, rows, TM, queues);
    t.q0 = 0;
    t.q1 = MODE == kNT ? K : N;
    if (row_tile(queues, E, TM, TN, P, block % kXcds, block / kXcds, t) != kTile) return;
    __syncthreads();  // every lookup is done before the loads overwrite the table

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t xrow = static_cast<int64_t>(MODE == kNT ? K : N) * EB;
    const int64_t yrow = static_cast<int64_t>(K) * EB;
    const int64_t xstep = 128, ystep = YC ? QS * yrow : 128;
    const int nk = (t.q1 - t.q0 + QS - 1) / QS;
    const int qtail = t.q1 - t.q0 - (nk - 1) * QS;
    const uint64_t xbase = uniform64(reinterpret_cast<uint64_t>(Xp) + static_cast<uint64_t>(t.m0 * xrow));
    const uint64_t ybase = uniform64(
        reinterpret_cast<uint64_t>(Yp) +
        static_cast<uint64_t>(MODE == kNN ? static_cast<int64_t>(t.e) * N * yrow + static_cast<int64_t>(t.p0) * EB
                                          : (static_cast<int64_t>(t.e) * N + t.p0) * yrow));
    const uint32_t lds_w = __builtin_amdgcn_readfirstlane(lds_addr(smem)) + wave * RING;
    char* const mine = smem + wave * RING;
    uint32_t xoff[XS::LOADS], yoff[YS::LOADS], xtail = 0, ytail = 0;
#pragma unroll
    for (int j = 0; j < XS::LOADS; ++j) {
        xoff[j] = XS::offset(j, lane, static_cast<uint32_t>(xrow), t.m1 - t.m0);
        xtail |= (XS::beyond(j, lane, qtail) ? 1u : 0u) << j;
    }
#pragma unroll
    for (int j = 0; j < YS::LOADS; ++j) {
        yoff[j] = YS::offset(j, lane, static_cast<uint32_t>(yrow), P - t.p0);
        ytail |= (YS::beyond(j, lane, qtail) ? 1u : 0u) << j;
    }
    const Fragments<TY, false, TM, MB> xfrag(lane, 0);
    const Fragments<TY, YC, TN, NB> yfrag(lane, 0);
    Acc<TY> acc[NB][MB];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) acc[nb][mb] = zero_acc<TY>();

    // NX: the loads of X that have a row in range (the others' LDS rows keep
    // what was there, and only rows of C that are not stored see it)
    auto stream = [&](auto nx_c) {
        constexpr int NX = decltype(nx_c)::value;
        constexpr int NL = YS::LOADS + NX;
        auto dma = [&](int kt, uint32_t st) {
            // all lanes out of range past the end, in the last slice those beyond it
            const uint32_t xo = kt >= nk ? ~0u : (kt == nk - 1 ? xtail : 0u);
            const uint32_t yo = kt >= nk ? ~0u : (kt == nk - 1 ? ytail : 0u);
#pragma unroll
            for (int j = 0; j < YS::LOADS; ++j)
                lds_dma16_b(ybase + kt * ystep, yoff[j] | ((yo << (31 - j)) & kOutOfRange), lds_w + st + X_BYTES + j * 1024);
#pragma unroll
            for (int j = 0; j < NX; ++j)
                lds_dma16_b(xbase + kt * xstep, xoff[j] | ((xo << (31 - j)) & kOutOfRange), lds_w + st + j * 1024);
        };
        i32x4_t f[2][4][MB + NB];
        auto read = [&](int b, uint32_t st) {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
                for (int i = 0; i < MB; ++i) f[b][kk][i] = xfrag.read(mine, st, i, kk);
#pragma unroll
                for (int i = 0; i < NB; ++i) f[b][kk][MB + i] = yfrag.read(mine + X_BYTES, st, i, kk);
            }
        };
        dma(wave, 0);
        dma(wave + 4, STAGE);
        // (the compiler does not know what the loads write: it keeps LDS accesses
        // behind each wait because of the empty statement)
        wait_vmcnt<NL>();
        asm volatile("" ::: "memory");
        read(0, 0);
        wait_vmcnt_lgkm0<63>();
        __builtin_amdgcn_sched_barrier(0);
        dma(wave + 8, 0);
        // two slices a round (the second possibly past the end: zeros)
        for (int kt = wave; kt < nk; kt += 8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t st = u == 0 ? STAGE : 0;  // the stage of the slice after this one
                wait_vmcnt<NL>();
                asm volatile("" ::: "memory");
                read(1 - u, st);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
#pragma unroll
                    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) multiply<TY>(f[u][kk][MB + nb], f[u][kk][mb], acc[nb][mb]);
                wait_vmcnt_lgkm0<63>();
                __builtin_amdgcn_sched_barrier(0);
                dma(kt + 4 * u + 12, st);
            }
        }
        wait_vmcnt<0>();
        asm volatile("" ::: "memory");
    };
    if constexpr (MB == 1) {
        const int nx = (t.m1 - t.m0 + 7) / 8;
        if (nx == 1) stream(std::integral_constant<int, 1>{});
        else if (nx == 2) stream(std::integral_constant<int, 2>{});
        else stream(std::integral_constant<int, 4>{});
    } else {
        stream(std::integral_constant<int, XS::LOADS>{});
    }

    // the waves' partial tiles side by side, each in its wave's ring
    {
        const int half = lane >> 5, l32 = lane & 31;
        Val* const part = reinterpret_cast<Val*>(mine);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *reinterpret_cast<val4_t*>(part + (mb * 32 + l32) * PADC + nb * 32 + 8 * g + 4 * half) =
                        val4_t{acc[nb][mb][4 * g], acc[nb][mb][4 * g + 1], acc[nb][mb][4 * g + 2], acc[nb][mb][4 * g + 3]};
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < TM * TN / 1024; ++it) {
        const int idx = it * 256 + tid;
        const int r = idx / (TN / 4), c = idx % (TN / 4) * 4;
        const int m = t.m0 + r, col = t.p0 + c;
        if (m >= t.m1 || col >= P) continue;
        const char* const src = smem + (r * PADC + c) * 4;
        val4_t v = *reinterpret_cast<const val4_t*>(src);
#pragma unroll
        for (int w = 1; w < 4; ++w) v += *reinterpret_cast<const val4_t*>(src + w * RING);
        f32x4_t o;
        if constexpr (TY == kI8) {
            const float rs = sx[m];
            const f32x4_t cs = *reinterpret_cast<const f32x4_t*>(sy + static_cast<int64_t>(t.e) * N + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = static_cast<float>(v[i]) * rs * cs[i];
        } else {
            o = v;
        }
        O* const dst = C + static_cast<int64_t>(m) * P + col;
        if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4_t*>(dst) = o;
        else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
}

template <int TY, int MODE, int MB, int NB, typename O>
__global__ __launch_bounds__(256) void grouped_split_kernel(
    const void* __restrict__ Xp, const void* __restrict__ Yp, const int32_t* __restrict__ offsets, int E, int rows,
    int N, int K, O* __restrict__ C, const float* __restrict__ sx, const float* __restrict__ sy) {
    __shared__ __attribute__((aligned(1024))) char smem[split_lds(MB, NB)];
    grouped_split<TY, MODE, MB, NB, O>(smem, blockIdx.x, Xp, Yp, offsets, E, rows, N, K, C, sx, sy);
}

// ---- both gradients in one launch -----------------------------------------------
//
// The input gradient's workgroups, then the weight gradient's: for problems of
// a few rounds most of a kernel is its start and its last round, and the two
// products fill each other's.
// DMB = 0: the input gradient by the split kernel's 32 x 32 tiles.
template <int TY, int DMB, int DNB, int DNS, int WMB, typename DO, typename WO>
__global__ __launch_bounds__(256, 2) void grouped_gradients_kernel(
    const void* __restrict__ dc, const void* __restrict__ w, const void* __restrict__ a,
    const int32_t* __restrict__ offsets, int E, int rows, int N, int K, DO* __restrict__ da, WO* __restrict__ dw,
    int da_blocks, int parts) {
    constexpr int DA_LDS = DMB == 0 ? split_lds(1, 1) : TileLds<DMB == 0 ? 1 : DMB, DMB == 0 ? 1 : DNB, DNS, DO>::BYTES;
    constexpr int DW_LDS = TileLds<WMB, WMB, 2, WO>::BYTES;
    __shared__ __attribute__((aligned(1024))) char smem[DA_LDS > DW_LDS ? DA_LDS : DW_LDS];
    const int block = blockIdx.x;
    if (block < da_blocks) {
        if constexpr (DMB == 0)
            grouped_split<TY, kNN, 1, 1, DO>(smem, block, dc, w, offsets, E, rows, N, K, da, nullptr, nullptr);
        else
            grouped_tile<TY, kNN, DMB, DNB, DNS, DO>(smem, block, da_blocks, dc, w, offsets, E, rows, N, K, da, nullptr,
                                                     nullptr, 1);
    } else {
        grouped_tile<TY, kTN, WMB, WMB, 2, WO>(smem, block - da_blocks, gridDim.x - da_blocks, dc, a, offsets, E, rows,
                                               N, K, dw, nullptr, nullptr, parts);
    }
}

// Sums of a cut weight gradient: dst[i] = sum of the parts, in their order.
template <typename O>
__global__ __launch_bounds__(256) void grouped_parts_kernel(const float* __restrict__ src, int64_t n, int parts,
                                                            O* __restrict__ dst) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
    if (i >= n) return;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(src + i);
    for (int p = 1; p < parts; ++p) v += *reinterpret_cast<const f32x4_t*>(src + p * n + i);
    if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4_t*>(dst + i) = v;
    else *reinterpret_cast<uint2*>(dst + i) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

// ---- the launches ---------------------------------------------------------------------

// CUs of the device of stream s.
int compute_units(hipStream_t s) {
    hipDevice_t dev = 0;
    int cus = 0;
    if (hipStreamGetDevice(s, &dev) != hipSuccess ||
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
        return kCus;
    return cus;
}

struct Args {
    const moe_grouped_t& g;
    const void* X;
    const void* Y;
    const int32_t* offsets;
    const float* sx;
    const float* sy;
    hipStream_t s;
};

template <int TY, int MODE, int MB, int NB, int NS, typename O>
void start_tile(const Args& a, const Plan& p, unsigned grid, O* C) {
    grouped_tile_kernel<TY, MODE, MB, NB, NS, O><<<grid, 256, 0, a.s>>>(
        a.X, a.Y, a.offsets, a.g.E, static_cast<int>(a.g.rows), a.g.N, a.g.K, C, a.sx, a.sy, p.parts);
}
template <int TY, int MODE, int MB, int NB, typename O>
void start_split(const Args& a, unsigned grid, O* C) {
    grouped_split_kernel<TY, MODE, MB, NB, O><<<grid, 256, 0, a.s>>>(
        a.X, a.Y, a.offsets, a.g.E, static_cast<int>(a.g.rows), a.g.N, a.g.K, C, a.sx, a.sy);
}

template <int TY, int MODE, typename O>
hipError_t start(const Args& a, const Plan& p, void* out) {
    O* const C = static_cast<O*>(out);
    int64_t n = workgroups(a.g, MODE, p);
    // the largest tiles leave room for one workgroup per CU: that many walk
    // all tiles
    if (p.v == kTile256) n = std::min<int64_t>(n, align_up(compute_units(a.s), kXcds));
    const unsigned grid = static_cast<unsigned>(n);
    if constexpr (MODE == kTN) {
        if (p.v == kTile256) {
            start_tile<TY, MODE, 4, 4, 2>(a, p, grid, C);
        } else if (p.v == kTile64) {
            if constexpr (TY == kF32) start_tile<TY, MODE, 1, 1, 2>(a, p, grid, C);
        } else {
            start_tile<TY, MODE, 2, 2, 2>(a, p, grid, C);
        }
    } else if constexpr (TY == kF32) {
        if (p.v == kSplit32) start_split<TY, MODE, 1, 1>(a, grid, C);
        else start_tile<TY, MODE, 1, 1, 2>(a, p, grid, C);
    } else {
        switch (p.v) {
            case kSplit32: start_split<TY, MODE, 1, 1>(a, grid, C); break;
            case kSplit64: start_split<TY, MODE, 2, 2>(a, grid, C); break;
            case kTile64x128: start_tile<TY, MODE, 1, 2, 3>(a, p, grid, C); break;
            case kTile256: start_tile<TY, MODE, 4, 4, 2>(a, p, grid, C); break;
            default: start_tile<TY, MODE, 2, 2, 2>(a, p, grid, C); break;
        }
    }
    return hipGetLastError();
}

template <int TY, int DMB, int DNB, int DNS, int WMB, typename DO, typename WO>
void start_gradients_of(const moe_grouped_t& g, const Plan& pa, const Plan& pw, const void* dc, const void* w,
                        const void* a, const int32_t* offsets, void* da, void* dw, hipStream_t s) {
    const int64_t na = workgroups(g, kNN, pa), nw = workgroups(g, kTN, pw);
    grouped_gradients_kernel<TY, DMB, DNB, DNS, WMB, DO, WO><<<static_cast<unsigned>(na + nw), 256, 0, s>>>(
        dc, w, a, offsets, g.E, static_cast<int>(g.rows), g.N, g.K, static_cast<DO*>(da), static_cast<WO*>(dw),
        static_cast<int>(na), pw.parts);
}

template <int TY, typename DO, typename WO>
void start_gradients(const moe_grouped_t& g, const Plan& pa, const Plan& pw, const void* dc, const void* w,
                     const void* a, const int32_t* offsets, void* da, void* dw, hipStream_t s) {
    auto go = [&](auto wmb) {
        constexpr int WMB = decltype(wmb)::value;
        if (pa.v == kSplit32) {
            start_gradients_of<TY, 0, 0, 2, WMB, DO, WO>(g, pa, pw, dc, w, a, offsets, da, dw, s);
        } else if constexpr (TY == kF32) {
            if constexpr (WMB == 1) start_gradients_of<TY, 1, 1, 2, 1, DO, WO>(g, pa, pw, dc, w, a, offsets, da, dw, s);
        } else if (pa.v == kTile64x128) {
            start_gradients_of<TY, 1, 2, 3, WMB, DO, WO>(g, pa, pw, dc, w, a, offsets, da, dw, s);
        } else {
            start_gradients_of<TY, 2, 2, 2, WMB, DO, WO>(g, pa, pw, dc, w, a, offsets, da, dw, s);
        }
    };
    if constexpr (TY == kF32) {
        if (pw.v == kTile64) {
            go(std::integral_constant<int, 1>{});
            return;
        }
    }
    go(std::integral_constant<int, 2>{});
}

}  // namespace

// (of the smallest tile each mode has; parts of queues are made only below 16
// rounds)
int64_t grouped_tiles(const moe_grouped_t& g) {
    const int64_t widest = std::max(g.N, g.K);
    return std::max(row_tiles(g, kTileM[kSplit32]) * ceil_div(widest, kTileN[kSplit32]),
                    g.E * ceil_div(g.N, kTileM[kTile64]) * ceil_div(g.K, kTileN[kTile64]));
}

size_t grouped_ws_bytes(const moe_grouped_t& g, int op) {
    return op == MOE_GROUPED_OP_BACKWARD ? parts_bytes(g, plan_for(g, kTN, false)) : 0;
}

hipError_t launch_grouped_matmul(const moe_grouped_t& g, const void* a, const void* w, const int32_t* offsets, void* c,
                                 hipStream_t s) {
    const Args args{g, a, w, offsets, nullptr, nullptr, s};
    const Plan p = plan_for(g, kNT, false);
    return g.dtype == MOE_DTYPE_BF16 ? start<kBf16, kNT, bf16_t>(args, p, c) : start<kF32, kNT, float>(args, p, c);
}

hipError_t launch_grouped_gradients(const moe_grouped_t& g, const void* a, const void* w, const int32_t* offsets,
                                    const void* dc, void* da, void* dw, void* ws, hipStream_t s) {
    const bool bf16 = g.dtype == MOE_DTYPE_BF16;
    if (g.rows == 0) da = nullptr;
    const Plan pa = plan_for(g, kNN, false), pw = plan_for(g, kTN, false);
    void* const sums = pw.parts > 1 ? ws : dw;  // float32 if in parts
    hipError_t e = hipSuccess;
    if (da != nullptr && dw != nullptr && pairs(g, pa, pw)) {
        if (!bf16) start_gradients<kF32, float, float>(g, pa, pw, dc, w, a, offsets, da, sums, s);
        else if (pw.parts > 1) start_gradients<kBf16, bf16_t, float>(g, pa, pw, dc, w, a, offsets, da, sums, s);
        else start_gradients<kBf16, bf16_t, bf16_t>(g, pa, pw, dc, w, a, offsets, da, sums, s);
        e = hipGetLastError();
    } else {
        if (da != nullptr) {
            const Args args{g, dc, w, offsets, nullptr, nullptr, s};
            e = bf16 ? start<kBf16, kNN, bf16_t>(args, pa, da) : start<kF32, kNN, float>(args, pa, da);
        }
        if (e == hipSuccess && dw != nullptr) {
            const Args args{g, dc, a, offsets, nullptr, nullptr, s};
            if (!bf16) e = start<kF32, kTN, float>(args, pw, sums);
            else if (pw.parts > 1) e = start<kBf16, kTN, float>(args, pw, sums);
            else e = start<kBf16, kTN, bf16_t>(args, pw, sums);
        }
    }
    if (e != hipSuccess || dw == nullptr || pw.parts == 1) return e;
    const int64_t n = static_cast<int64_t>(g.E) * g.N * g.K;  // (a multiple of 16)
    const unsigned grid = static_cast<unsigned>(ceil_div(n, 1024));
    const float* const src = static_cast<const float*>(ws);
    if (bf16) grouped_parts_kernel<<<grid, 256, 0, s>>>(src, n, pw.parts, static_cast<bf16_t*>(dw));
    else grouped_parts_kernel<<<grid, 256, 0, s>>>(src, n, pw.parts, static_cast<float*>(dw));
    return hipGetLastError();
}

hipError_t launch_grouped_int8(const moe_grouped_t& g, const void* a, const float* sa, const void* w, const float* sw,
                               const int32_t* offsets, void* c, hipStream_t s) {
    const Args args{g, a, w, offsets, sa, sw, s};
    const Plan p = plan_for(g, kNT, true);
    return g.dtype == MOE_DTYPE_BF16 ? start<kI8, kNT, bf16_t>(args, p, c) : start<kI8, kNT, float>(args, p, c);
}

}  // namespace moe
