// What the grouped products' kernels share: the queues and the order of the
// tiles, loads into LDS, and how a slice of an operand lies there.
#pragma once

#include <type_traits>

#include "device_util.h"
#include "grouped_plan.h"
#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kBf16 = 0, kF32 = 1, kI8 = 2;

// ---- queues and the tile order ---------------------------------------------

// The queues, clamped to the matrix, so that no offsets, whatever they hold,
// lead outside it: 0 <= lo <= hi <= rows.
struct Queues {
    int end[MOE_MAX_EXPERTS];              // row tiles of the experts up to and with e
    int lo[MOE_MAX_EXPERTS];
    int hi[MOE_MAX_EXPERTS];
    uint32_t key[MOE_MAX_EXPERTS];         // kTN
    unsigned char order[MOE_MAX_EXPERTS];  // kTN: experts by descending length
};

// Filled by the first wave (lane l: experts 4 l .. 4 l + 3, all loads
// together), then a barrier.  offsets = NULL: one queue of all rows.  ORDER:
// the experts' order by length too.
template <bool ORDER>
__device__ __forceinline__ void load_queues(const int32_t* __restrict__ offsets, int E, int rows, int bm, Queues& q) {
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x;
        int o[5];
        if (offsets != nullptr) {
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = offsets[min(lane * 4 + i, E)];
        } else {
#pragma unroll
            for (int i = 0; i < 5; ++i) o[i] = lane * 4 + i == 0 ? 0 : rows;
        }
        i32x4_t lo, hi, end;
        int local = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min(max(o[i], 0), rows);
            hi[i] = max(min(o[i + 1], rows), lo[i]);
            local += lane * 4 + i < E ? (hi[i] - lo[i] + bm - 1) / bm : 0;
            end[i] = local;
        }
        int incl = local;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if (lane >= off) incl += v;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) end[i] += incl - local;
        *reinterpret_cast<i32x4_t*>(q.end + lane * 4) = end;
        *reinterpret_cast<i32x4_t*>(q.lo + lane * 4) = lo;
        *reinterpret_cast<i32x4_t*>(q.hi + lane * 4) = hi;
    }
    __syncthreads();
    if constexpr (ORDER) {
        // rank of expert e: the experts that are longer, or as long and before it
        // (in units of 64 rows, so that one 32-bit key holds both)
        static_assert(MOE_MAX_EXPERTS <= 256, "one thread per expert, one byte of the key");
        const int e = threadIdx.x;
        const uint32_t len = e < E ? min((q.hi[e] - q.lo[e] + 63) >> 6, (1 << 23) - 1) : 0;
        const uint32_t key = e < E ? (len << 8) + (255u - e) : 0u;
        q.key[e] = key;
        __syncthreads();
        int rank = 0;
        for (int i = 0; i < E; i += 8) {
            const u32x4_t a = *reinterpret_cast<const u32x4_t*>(q.key + i);
            const u32x4_t b = *reinterpret_cast<const u32x4_t*>(q.key + i + 4);
#pragma unroll
            for (int j = 0; j < 4; ++j) rank += (a[j] > key ? 1 : 0) + (b[j] > key ? 1 : 0);
        }
        if (e < E) q.order[rank] = static_cast<unsigned char>(e);
        __syncthreads();
    }
}

// An output tile: rows [m0, m1) and columns from p0, of expert e, summed over
// [q0, q1) (kTN: queue rows; otherwise the whole reduction).
struct Tile {
    int e, m0, m1, p0, q0, q1;
};
enum Found { kEnd, kSkip, kTile };

// a / b for 0 <= a < 2^24, 0 < b < 2^24.  The float32 quotient is off by a few
// at most; dividing what it leaves the same way brings that to one.
__device__ __forceinline__ int quick_div(int a, int b) {
    const float inv = __builtin_amdgcn_rcpf(static_cast<float>(b));
    int q = static_cast<int>(static_cast<float>(a) * inv);
    q += static_cast<int>(static_cast<float>(a - q * b) * inv);
    const int r = a - q * b;
    if (r < 0) --q;
    else if (r >= b) ++q;
    return __builtin_amdgcn_readfirstlane(q);
}

// kNT, kNN.  Workgroups are dealt to the 8 XCDs round-robin; each XCD walks one
// contiguous range of the tile order, `place` counting within it.  The order
// groups row tiles per column tile, so that the tiles running on one XCD at a
// time share operand rows in its L2: kGroupM of them, or half as many for tiles
// of 256 in at most 8 columns, so that the 32 workgroups of an XCD span whole
// rows of C and read them once (bf16, 128 queues of 2048 rows, 2048 x 768: 788
// us, in groups of 8 844; 8 queues, 14336 x 4096, 56 columns: in groups of 4
// 1455 us, of 8 1434).
__device__ __forceinline__ Found row_tile(const Queues& q, int E, int bm, int bn, int P, int xcd, int place,
                                          Tile& t) {
    const int total_m = __builtin_amdgcn_readfirstlane(q.end[E - 1]);
    const int ptiles = (P + bn - 1) / bn;
    // (queues that keep the rules have fewer than 2^24 tiles)
    const int64_t total64 = static_cast<int64_t>(total_m) * ptiles;
    if (total64 <= 0 || total64 >= (1 << 24)) return kEnd;
    const int total = static_cast<int>(total64);
    const int per_xcd = (total + kXcds - 1) / kXcds;
    const int id = xcd * per_xcd + place;
    if (place >= per_xcd || id >= total) return kEnd;
    const int height = bm == 256 && ptiles <= 8 ? kGroupM / 2 : kGroupM;
    const int group = quick_div(id, height * ptiles);
    const int first = group * height;
    const int gsz = min(height, total_m - first);
    const int local = id - group * height * ptiles;
    const int pt = quick_div(local, gsz);
    const int mt = first + local - pt * gsz;
    // the expert: how many experts' tiles end at or before mt
    const i32x4_t ends = *reinterpret_cast<const i32x4_t*>(q.end + (threadIdx.x & 63) * 4);
    int e = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) e += __builtin_popcountll(__ballot(ends[i] <= mt));
    if (e >= E) return kSkip;  // (only if broken offsets overflowed the sums)
    const int before = e == 0 ? 0 : __builtin_amdgcn_readfirstlane(q.end[e - 1]);
    t.e = e;
    const int lo = __builtin_amdgcn_readfirstlane(q.lo[e]), hi = __builtin_amdgcn_readfirstlane(q.hi[e]);
    t.m0 = lo + (mt - before) * bm;
    t.m1 = min(t.m0 + bm, hi);
    t.p0 = pt * bn;
    return t.m0 >= lo && t.m0 < t.m1 ? kTile : kSkip;
}

// kTN: tile `local` of (part `part` of) expert e's weight gradient.  Within it,
// groups of kGroupM row tiles walk the column tiles.
__device__ __forceinline__ void weight_tile_of(const Queues& q, int e, int part, int local, int E, int M, int P, int bm,
                                               int bn, int qs, int parts, Tile& t) {
    const int mtn = (M + bm - 1) / bm, ptn = (P + bn - 1) / bn;
    const int group = quick_div(local, kGroupM * ptn);
    const int first = group * kGroupM;
    const int gsz = min(kGroupM, mtn - first);
    const int l2 = local - group * kGroupM * ptn;
    const int pt = quick_div(l2, gsz);
    t.e = part * E + e;
    t.m0 = (first + l2 - pt * gsz) * bm;
    t.m1 = min(t.m0 + bm, M);
    t.p0 = pt * bn;
    t.q0 = __builtin_amdgcn_readfirstlane(q.lo[e]);
    t.q1 = __builtin_amdgcn_readfirstlane(q.hi[e]);
    if (parts > 1) {
        const int slices = (t.q1 - t.q0 + qs - 1) / qs;
        const int per = (slices + parts - 1) / parts * qs;
        t.q0 = min(t.q0 + part * per, t.q1);
        t.q1 = min(t.q0 + per, t.q1);
    }
}

// kTN.  With parts > 1 each queue is cut into that many ranges of rows
// (multiples of qs), each with tiles of its own whose sums go to matrix part *
// E + e.  A tile's cost is its queue's length, so the experts are dealt longest
// first.  Each XCD takes whole (parts of) queues, in a snake order, XCD 0 to 7
// and back: their tiles read the same two operand blocks and share its L2
// (dealing every expert's tiles over all XCDs: 128 queues of 2048 rows, 768 x
// 2048, 747 us against 694).  With too few of them to keep the XCDs even
// (whole_queues), every XCD takes an eighth of each expert's tiles instead.
__device__ __forceinline__ Found weight_tile(const Queues& q, int E, int M, int P, int bm, int bn, int qs, int parts,
                                             bool dealt, int xcd, int place, Tile& t) {
    const int whole = ((M + bm - 1) / bm) * ((P + bn - 1) / bn);
    int rank, part, local;
    if (dealt) {
        const int j = quick_div(place, whole);
        if (j * kXcds >= E * parts) return kEnd;
        const int i = j * kXcds + (j & 1 ? kXcds - 1 - xcd : xcd);
        if (i >= E * parts) return kSkip;
        rank = quick_div(i, parts);
        part = i - rank * parts;
        local = place - j * whole;
    } else {
        const int per_e = whole * parts;
        const int per_x = (per_e + kXcds - 1) / kXcds;
        rank = quick_div(place, per_x);
        if (rank >= E) return kEnd;
        local = ((xcd + rank) & (kXcds - 1)) * per_x + place - rank * per_x;
        if (local >= per_e) return kSkip;
        part = quick_div(local, whole);
        local -= part * whole;
    }
    weight_tile_of(q, __builtin_amdgcn_readfirstlane(static_cast<int>(q.order[rank])), part, local, E, M, P, bm, bn, qs,
                   parts, t);
    return kTile;
}

// kTN, many uneven queues and workgroups that each walk several tiles: the
// experts, longest first, each to the XCD that has the least so far; and of
// an expert's `whole` tiles, one more to those of the XCD's `stride` (at most
// 32) workgroups that have the least.  128 queues of 2048 rows in the mean, the
// longest of 19000, 768 x 2048: 763 us, 829 us in the snake order; 64 queues of
// 2560, the longest of 17000, 1408 x 2048: 896 and 1044 us.  Filled by the first wave, the same in every
// workgroup, in 0.05 to 0.1 us per expert; costs are counted in slices, a tile's
// start as two.  (Sums that overflow would only deal badly: the places stay a
// permutation.)
struct Deal {
    int queues;                                // of this XCD
    unsigned char expert[MOE_MAX_EXPERTS];
    unsigned char place[MOE_MAX_EXPERTS];      // this workgroup's place for the queue's last, partial round
};

__device__ __forceinline__ uint32_t min_of_8(uint32_t v) {
    // within each 8 lanes: neighbours, pairs, fours
    v = min(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xf, 0xf, true)));
    v = min(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x4E, 0xf, 0xf, true)));
    return min(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x141, 0xf, 0xf, true)));
}

__device__ __forceinline__ void deal_queues(const Queues& q, int E, int qs, int whole, int xcd, int at, int stride,
                                            Deal& d) {
    if (threadIdx.x < 64) {
        const uint32_t lane = threadIdx.x;
        const int full = whole / stride, rest = whole - full * stride;
        uint32_t on_xcd = 0, on_cu = 0;        // lane i: what XCD i, and workgroup i of this XCD, have so far
        int n = 0;
        for (int i0 = 0; i0 < E; i0 += 64) {
            const int e = i0 + static_cast<int>(lane) < E ? q.order[i0 + lane] : 0;
            const int cost = max((q.hi[e] - q.lo[e] + qs - 1) / qs, 1) + 2;
            for (int i = 0; i < min(64, E - i0); ++i) {
                const uint32_t c = __builtin_amdgcn_readlane(cost, i);
                const uint32_t to = __builtin_amdgcn_readfirstlane(min_of_8((on_xcd << 3) | (lane & 7))) & 7;
                on_xcd += (lane & 7) == to ? c : 0;
                if (static_cast<int>(to) != xcd) continue;
                const uint32_t key = static_cast<int>(lane) < stride ? (on_cu << 6) | lane : ~0u;
                int rank = 0;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    rank += static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(key), j)) < key ? 1 : 0;
                on_cu += c * (full + (rank < rest ? 1 : 0));
                const int mine = __builtin_amdgcn_readlane(rank, at);
                const int expert = __builtin_amdgcn_readlane(e, i);
                if (lane == 0) {
                    d.expert[n] = static_cast<unsigned char>(expert);
                    d.place[n] = static_cast<unsigned char>(mine);
                }
                ++n;
            }
        }
        if (lane == 0) d.queues = n;
    }
    __syncthreads();
}

// ---- global -> LDS -----------------------------------------------------------

// A buffer descriptor over the 2^31 bytes from base: a lane whose offset is
// 2^31 or more is out of range, reads nothing and puts zeros into LDS.  That
// is how rows past a queue, columns past a matrix and the end of the reduction
// become zeros in both operands (a zero in one alone would not do: zero times
// the infinity or NaN of whatever lies there is NaN).
constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw buffer, 32-bit data format
constexpr int kNonTemporal = 2;               // cache policy of a buffer access

// 16 bytes per lane from base + voff into LDS at lds_base + 16 * lane.  Inline
// assembly so that the compiler does not take every later LDS read for
// dependent on it; ordered by wait_vmcnt and the workgroup barrier.  The
// compiler's hazard checks do not look inside: s_nop 4 stands for the 5 wait
// states between a vector instruction's write of a scalar register (a
// readfirstlane, or a readlane where the compiler keeps scalars in vector
// lanes) and a load that reads it, and for the one after a write of M0.
__device__ __forceinline__ void lds_dma16_b(uint64_t base, uint32_t voff, uint32_t lds_base) {
    i32x4_t rsrc;
    rsrc[0] = static_cast<int>(static_cast<uint32_t>(base));
    rsrc[1] = static_cast<int>(static_cast<uint32_t>(base >> 32) & 0xffffu);
    rsrc[2] = static_cast<int>(kOutOfRange);
    rsrc[3] = static_cast<int>(kRsrcWord3);
    asm volatile(
        "s_nop 4\n\t"
        "buffer_load_dwordx4 %0, %1, 0 offen lds"
        :
        : "v"(voff), "s"(rsrc), "{m0}"(lds_base)
        : "memory");
}

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return (static_cast<uint64_t>(hi) << 32) | lo;
}

// ---- a slice of an operand in LDS ------------------------------------------------
//
// A slice is 128 bytes of q (64 bf16, 32 f32 or 128 int8 values) of TX tile
// rows, TX * 128 bytes in all.
//   row-major     an LDS row is one tile row's 128 bytes of q: 8 words of 16
//                 bytes, word c at place c ^ ((row >> 1) & 7), which spreads the
//                 32 rows of a fragment read over the banks
//   column-major  an LDS row is one q of all TX tile rows.  bf16: word c at
//                 place c ^ ((row & 3) << 2): the transposing reads of one
//                 instruction touch 4 neighbouring LDS rows, and this puts them
//                 on different banks
// A load moves 1 KB: lane l fills place l % CH of LDS row i * RPL + l / CH.
template <int TY, bool COL, int TX>
struct Slice {
    static constexpr int EB = TY == kBf16 ? 2 : (TY == kF32 ? 4 : 1);
    static constexpr int WORD = 16 / EB;               // values per word
    static constexpr int CH = COL ? TX * EB / 16 : 8;  // words per LDS row
    static constexpr int RPL = 64 / CH;                // LDS rows per load
    static constexpr int LOADS = TX / 8;
    static_assert(CH >= 1 && CH <= 64, "an LDS row is at most one load");

    static __device__ __forceinline__ int word(int row, int place) {
        if constexpr (!COL) return place ^ ((row >> 1) & 7);
        if constexpr (TY == kBf16) return place ^ (((row & 3) << 2) & (CH - 1));
        return place;
    }
    // The lane's byte offset in load i, out of range beyond `valid` tile rows.
    static __device__ __forceinline__ uint32_t offset(int i, int lane, uint32_t row_bytes, int valid) {
        const int r = i * RPL + lane / CH, c = word(r, lane % CH);
        return (COL ? c * WORD : r) < valid ? static_cast<uint32_t>(r) * row_bytes + c * 16 : kOutOfRange;
    }
    // Whether the lane's part of load i lies beyond `q` values of q.
    static __device__ __forceinline__ bool beyond(int i, int lane, int q) {
        const int r = i * RPL + lane / CH, c = word(r, lane % CH);
        return (COL ? r : c * WORD) >= q;
    }
};

// A lane's fragments of `NBLK` blocks of 32 tile rows, from block `block0`, of a
// slice: 16 bytes of q per step and half wave (step kk: bytes 32 kk + 16 half of
// a row).  Both operands of a product are read by the same rule, so every
// product pairs equal q.
template <int TY, bool COL, int TX, int NBLK>
struct Fragments {
    static constexpr bool TRANSPOSE = COL && TY == kBf16;
    static constexpr int ROWB = COL ? Slice<TY, COL, TX>::CH * 16 : 128;  // bytes per LDS row
    uint32_t at[TRANSPOSE ? NBLK : 1];

    __device__ __forceinline__ Fragments(int lane, int block0) {
        const int half = lane >> 5, l32 = lane & 31;
        if constexpr (TRANSPOSE) {
            // two transposing reads: in each 16-lane group g (lanes 16 g + i), lane
            // i addresses q row (g >> 1) * 8 + (i >> 2) (+ 4 in the second read) and
            // columns (g & 1) * 16 + 4 (i & 3) .. + 4, and receives column (g & 1) *
            // 16 + i at 4 rows
            const int g = lane >> 4, i = lane & 15;
            const int r = (g >> 1) * 8 + (i >> 2);
            const int low = (g & 1) * 2 + ((i & 3) >> 1);
#pragma unroll
            for (int b = 0; b < NBLK; ++b)
                at[b] = r * ROWB + Slice<TY, COL, TX>::word(r, (block0 + b) * 4 + low) * 16 + 8 * (i & 1);
        } else if constexpr (COL) {
            at[0] = 4 * half * ROWB + block0 * 128 + l32 * 4;
        } else {
            // (word 2 kk + half of a row is at place (2 kk) ^ that of word `half`)
            at[0] = block0 * 4096 + l32 * 128 + Slice<TY, COL, TX>::word(l32, half) * 16;
        }
    }
    // block b, step kk of the slice at smem + base
    __device__ __forceinline__ i32x4_t read(const char* smem, uint32_t base, int b, int kk) const {
        if constexpr (TRANSPOSE) {
            typedef short s4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4_t* lds_s4_t;
            const uint32_t a = lds_addr(smem) + base + at[b] + kk * 16 * ROWB;
            const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4_t>(a));
            const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4_t>(a + 4 * ROWB));
            return __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else if constexpr (COL) {
            i32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = *reinterpret_cast<const int*>(smem + base + at[0] + b * 128 + (8 * kk + i) * ROWB);
            return v;
        } else {
            // (base is a multiple of 128: the steps differ by an exclusive or)
            return *reinterpret_cast<const i32x4_t*>(smem + ((at[0] + base) ^ (kk * 32)) + b * 4096);
        }
    }
};

// ---- products -------------------------------------------------------------------

template <int TY>
using Acc = std::conditional_t<TY == kI8, i32x16_t, f32x16_t>;

template <int TY>
__device__ __forceinline__ Acc<TY> zero_acc() {
    Acc<TY> v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0;
    return v;
}

// acc += Y's fragment times X's, a 32 x 32 block: lane l holds output row l & 31
// (X's) and columns 8 g + 4 (l >> 5) + 0..3 (Y's) in registers 4 g .. 4 g + 3.
template <int TY>
__device__ __forceinline__ void multiply(const i32x4_t& y, const i32x4_t& x, Acc<TY>& acc) {
    if constexpr (TY == kBf16) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, y), __builtin_bit_cast(bf16x8_t, x),
                                                      acc, 0, 0, 0);
    } else if constexpr (TY == kI8) {
        acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(y, x, acc, 0, 0, 0);
    } else {
        const f32x4_t yf = __builtin_bit_cast(f32x4_t, y), xf = __builtin_bit_cast(f32x4_t, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(yf[i], xf[i], acc, 0, 0, 0);
    }
}

}  // namespace

}  // namespace moe
