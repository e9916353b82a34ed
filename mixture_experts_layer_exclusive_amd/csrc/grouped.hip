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

#include "device_util.h"
#include "lds_dma.h"
#include "moe_internal.h"

namespace moe {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x16_t __attribute__((ext_vector_type(16)));

constexpr int kNT = 0, kNN = 1, kTN = 2;
constexpr int kBf16 = 0, kF32 = 1, kI8 = 2;
constexpr int kXcds = 8;
constexpr int kGroupM = 8;  // row tiles per group of the tile order

// ---- queues and the tile order ---------------------------------------------

// The queues in LDS: clamped to the matrix, so that no offsets, whatever they
// hold, lead outside it (0 <= lo <= hi <= rows), and the prefix sums of their
// row tiles.
struct Queues {
    int prefix[MOE_MAX_EXPERTS + 1];
    int lo[MOE_MAX_EXPERTS];
    int hi[MOE_MAX_EXPERTS];
};

// Filled by the first wave (lane l: experts 4l .. 4l + 3, all loads together),
// then a barrier.  offsets = NULL: one queue of all rows.
__device__ __forceinline__ void build_queues(const int32_t* __restrict__ offsets, int E, int rows, int bm, Queues& q) {
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
        int lo[4], hi[4], c[4], local = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = min(max(o[i], 0), rows);
            hi[i] = max(min(o[i + 1], rows), lo[i]);
            c[i] = lane * 4 + i < E ? (hi[i] - lo[i] + bm - 1) / bm : 0;
            local += c[i];
        }
        int incl = local;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int v = __shfl_up(incl, off, 64);
            if (lane >= off) incl += v;
        }
        int run = incl - local;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = lane * 4 + i;
            if (e < E) {
                q.prefix[e] = run;
                q.lo[e] = lo[i];
                q.hi[e] = hi[i];
            }
            run += c[i];
        }
        if (lane == 63) q.prefix[E] = incl;
    }
    __syncthreads();
}

// An output tile: rows [m0, m1) and columns from p0, of expert e, summed over
// q0 .. q1 (kTN: queue rows; otherwise 0 .. the reduction length).
struct Tile {
    int e, m0, m1, p0, q0, q1;
};

// kNT, kNN: workgroups are dealt to the 8 XCDs round-robin; the id is remapped
// so that each XCD walks one contiguous range of the tile order, which groups
// kGroupM row tiles per column tile: the tiles running on one XCD at a time
// share operand rows in its L2.
__device__ __forceinline__ bool find_row_tile(const Queues& q, int E, int bm, int bn, int P, Tile& t) {
    const int ptiles = (P + bn - 1) / bn;
    const int total_m = q.prefix[E];
    // (the launch holds total_m * ptiles below 2^24 workgroups for every
    // offsets that keeps the rules; others may ask for more, and then only
    // the tiles of this grid are computed)
    const int64_t total = static_cast<int64_t>(total_m) * ptiles;
    const int64_t per_xcd = (total + kXcds - 1) / kXcds;
    const int64_t place = blockIdx.x / kXcds;
    const int64_t pid64 = (blockIdx.x % kXcds) * per_xcd + place;
    if (place >= per_xcd || pid64 >= total || pid64 > 0x7fffffff) return false;
    const int pid = static_cast<int>(pid64);
    const int group = pid / (kGroupM * ptiles);
    const int first = group * kGroupM;
    const int gsz = min(kGroupM, total_m - first);
    const int local = pid - group * kGroupM * ptiles;
    const int mt = first + local % gsz;
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.prefix[mid] <= mt) lo = mid; else hi = mid;
    }
    t.e = lo;
    t.m0 = q.lo[lo] + (mt - q.prefix[lo]) * bm;
    t.m1 = min(t.m0 + bm, q.hi[lo]);
    t.p0 = (local / gsz) * bn;
    // (always so unless broken offsets overflowed the prefix sums)
    return t.m0 >= q.lo[lo] && t.m0 < t.m1;
}

// ---- global -> LDS -----------------------------------------------------------

// A buffer descriptor over the 2^31 bytes from base: a lane whose offset is
// 2^31 or more is out of range, reads nothing and puts zeros into LDS.  That
// is how rows past a queue, columns past a matrix and the end of the reduction
// become zeros in both operands (a zero in one alone would not do: zero times
// the infinity or NaN of whatever lies there is NaN).
constexpr uint32_t kOutOfRange = 0x80000000u;
constexpr uint32_t kRsrcWord3 = 0x00020000u;  // raw buffer, 32-bit data format

// 16 bytes per lane from base + voff into LDS at lds_base + 16 * lane.  Inline
// assembly so that the compiler does not take every later LDS read for
// dependent on it; ordered by wait_vmcnt and the workgroup barrier.  The
// descriptor comes from scalar instructions, and s_nop covers the wait state
// between a scalar write of M0 and its use.
__device__ __forceinline__ void lds_dma16_b(uint64_t base, uint32_t voff, uint32_t lds_base) {
    i32x4_t rsrc;
    rsrc[0] = static_cast<int>(static_cast<uint32_t>(base));
    rsrc[1] = static_cast<int>(static_cast<uint32_t>(base >> 32) & 0xffffu);
    rsrc[2] = static_cast<int>(kOutOfRange);
    rsrc[3] = static_cast<int>(kRsrcWord3);
    asm volatile(
        "s_nop 0\n\t"
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

// LDS slot of 16-byte chunk c of row r in a row-major slice (128-byte rows):
// c ^ row_swizzle(r), which spreads a fragment read's 32 rows over the banks.
__device__ __forceinline__ int row_swizzle(int r) { return (r >> 1) & 7; }

// The same in a column-major bf16 slice of CH chunks per row: the transposing
// reads of one instruction touch 4 neighbouring rows; flipping chunk bits 2-3
// by r & 3 puts them on different banks.
template <int CH>
__device__ __forceinline__ int col_swizzle(int r) {
    return ((r & 3) << 2) & (CH - 1);
}

__device__ __forceinline__ f32x16_t zero16(f32x16_t) {
    f32x16_t v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    return v;
}
__device__ __forceinline__ i32x16_t zero16(i32x16_t) {
    i32x16_t v;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0;
    return v;
}

// ---- the tile kernel ------------------------------------------------------------
//
// 4 waves in 2 x 2; a wave owns MB x NB blocks of 32 x 32 outputs.  A slice is
// 128 bytes of q of every tile row (64 bf16, 32 f32 or 128 int8 values), in
// two LDS stages.  The MFMA takes Y's fragment first and X's second, so a lane
// holds one output row (lane & 31) and runs of 4 consecutive columns.
//
// Each slice has 4 steps of 32 bytes of q (16 bytes per half wave).  Step 0
// multiplies fragments read during the slice before, while the fragments of
// steps 1-3 are read; then the stage is free, and the loads of the
// next-but-one slice go out spread over steps 1-3 (an LDS-bound load holds up
// the MFMAs behind it, so a burst of them stalls); before step 3 the next
// slice has landed, and step 3 reads its first fragments.
template <int TY, int MODE, int MB, int NB, typename O>
__global__ __launch_bounds__(256, (MB * NB > 4 ? 1 : 2)) void grouped_tile_kernel(
    const void* __restrict__ Xp, const void* __restrict__ Yp, const int32_t* __restrict__ offsets, int E, int rows,
    int N, int K, O* __restrict__ C, const float* __restrict__ sx, const float* __restrict__ sy) {
    constexpr int EB = TY == kBf16 ? 2 : (TY == kF32 ? 4 : 1);
    constexpr bool XC = MODE == kTN;             // X column-major
    constexpr bool YC = MODE != kNT;             // Y column-major
    static_assert(TY != kI8 || MODE == kNT, "int8: forward only");
    constexpr int TM = 64 * MB, TN = 64 * NB;    // output tile
    constexpr int QS = 128 / EB;                 // q per slice
    constexpr int XL = TM / 32, YL = TN / 32;    // loads per wave and slice (1 KB each)
    constexpr int NL = XL + YL;
    constexpr int X_BYTES = TM * 128;
    constexpr int STAGE = (TM + TN) * 128;
    constexpr int XCH = TM * EB / 16, YCH = TN * EB / 16;  // chunks per column-major row
    constexpr int NM = MB * NB;
    constexpr int NR = MB + NB;
    using Acc = std::conditional_t<TY == kI8, i32x16_t, f32x16_t>;
    __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
    static_assert(sizeof(Queues) <= 2 * STAGE, "the queues' table lives in the stages until the first load");
    Queues& queues = *reinterpret_cast<Queues*>(smem);

    Tile t;
    t.q0 = 0;
    t.q1 = MODE == kNT ? K : N;
    build_queues(offsets, E, rows, TM, queues);
    if constexpr (MODE == kTN) {
        const int mt = (N + TM - 1) / TM, pt = (K + TN - 1) / TN;
        const int per_e = mt * pt;
        t.e = blockIdx.x / per_e;
        const int l = blockIdx.x % per_e;
        t.m0 = (l % mt) * TM;
        t.m1 = min(t.m0 + TM, N);
        t.p0 = (l / mt) * TN;
        t.q0 = queues.lo[t.e];
        t.q1 = queues.hi[t.e];
    } else {
        if (!find_row_tile(queues, E, TM, TN, MODE == kNT ? N : K, t)) return;
    }
    const int e = __builtin_amdgcn_readfirstlane(t.e);
    const int m0 = __builtin_amdgcn_readfirstlane(t.m0), m1 = __builtin_amdgcn_readfirstlane(t.m1);
    const int p0 = __builtin_amdgcn_readfirstlane(t.p0);
    const int q0 = __builtin_amdgcn_readfirstlane(t.q0), q1 = __builtin_amdgcn_readfirstlane(t.q1);
    __syncthreads();  // every lookup is done before the loads overwrite the table

    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int half = lane >> 5, l32 = lane & 31;
    const int P = MODE == kNT ? N : K;           // output columns
    const int64_t xrow = static_cast<int64_t>(MODE == kNT ? K : N) * EB;  // bytes of an operand's memory row
    const int64_t yrow = static_cast<int64_t>(K) * EB;

    // ---- loads: load j of this wave fills 1 KB at (wave * L + j) * 1024 of the
    // operand's part of the stage
    const int nk = (q1 - q0 + QS - 1) / QS;
    const int qtail = q1 - q0 - (nk - 1) * QS;   // q in the last slice
    uint32_t xoff[XL], yoff[YL];
    uint32_t xtail = 0, ytail = 0;               // bit j: out of range in the last slice
    uint64_t xbase, ybase;
    int64_t xstep = 128, ystep = 128;
    if constexpr (XC) {
        xstep = QS * xrow;
        xbase = reinterpret_cast<uint64_t>(Xp) + static_cast<uint64_t>(q0 * xrow + static_cast<int64_t>(m0) * EB);
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int r = (wave * XL + j) * (64 / XCH) + lane / XCH;
            const int c = (lane % XCH) ^ (TY == kBf16 ? col_swizzle<XCH>(r) : 0);
            xoff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(xrow) + c * 16;
            if (m0 + c * (16 / EB) >= N) xoff[j] = kOutOfRange;
            xtail |= (r >= qtail ? 1u : 0u) << j;
        }
    } else {
        xbase = reinterpret_cast<uint64_t>(Xp) + static_cast<uint64_t>(m0 * xrow);
#pragma unroll
        for (int j = 0; j < XL; ++j) {
            const int r = (wave * XL + j) * 8 + (lane >> 3);
            const int c = (lane & 7) ^ row_swizzle(r);
            xoff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(xrow) + c * 16;
            if (m0 + r >= m1) xoff[j] = kOutOfRange;
            xtail |= (c * (16 / EB) >= qtail ? 1u : 0u) << j;
        }
    }
    if constexpr (YC) {
        ystep = QS * yrow;
        ybase = reinterpret_cast<uint64_t>(Yp) +
                static_cast<uint64_t>((MODE == kTN ? q0 : static_cast<int64_t>(e) * N) * yrow + static_cast<int64_t>(p0) * EB);
#pragma unroll
        for (int j = 0; j < YL; ++j) {
            const int r = (wave * YL + j) * (64 / YCH) + lane / YCH;
            const int c = (lane % YCH) ^ (TY == kBf16 ? col_swizzle<YCH>(r) : 0);
            yoff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(yrow) + c * 16;
            if (p0 + c * (16 / EB) >= P) yoff[j] = kOutOfRange;
            ytail |= (r >= qtail ? 1u : 0u) << j;
        }
    } else {
        ybase = reinterpret_cast<uint64_t>(Yp) + static_cast<uint64_t>((static_cast<int64_t>(e) * N + p0) * yrow);
#pragma unroll
        for (int j = 0; j < YL; ++j) {
            const int r = (wave * YL + j) * 8 + (lane >> 3);
            const int c = (lane & 7) ^ row_swizzle(r);
            yoff[j] = static_cast<uint32_t>(r) * static_cast<uint32_t>(yrow) + c * 16;
            if (p0 + r >= P) yoff[j] = kOutOfRange;
            ytail |= (c * (16 / EB) >= qtail ? 1u : 0u) << j;
        }
    }
    xbase = uniform64(xbase);
    ybase = uniform64(ybase);
    // (a scalar register that a vector instruction has written, as
    // readfirstlane does, may be read by a load 5 wait states later)
    asm volatile("s_nop 4" : "+s"(xbase), "+s"(ybase));
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const uint32_t lds_x = lds0 + wave * (XL * 1024);
    const uint32_t lds_y = lds0 + X_BYTES + wave * (YL * 1024);
    // load l (< NL) of slice kt
    auto dma = [&](int l, int kt) {
        const uint32_t so = (kt & 1) * STAGE;
        const bool last = kt == nk - 1;
        if (l < YL) {
            const uint32_t tm = last ? ytail : 0u;
            lds_dma16_b(ybase + kt * ystep, yoff[l < YL ? l : 0] | ((tm << (31 - l)) & kOutOfRange), lds_y + so + l * 1024);
        } else {
            const int j = l - YL;
            const uint32_t tm = last ? xtail : 0u;
            lds_dma16_b(xbase + kt * xstep, xoff[j < XL && j >= 0 ? j : 0] | ((tm << (31 - j)) & kOutOfRange),
                        lds_x + so + j * 1024);
        }
    };

    // ---- fragment reads
    uint32_t foff[4];                            // row-major: per step
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) foff[kk] = l32 * 128 + (((2 * kk + half) ^ row_swizzle(l32)) * 16);
    // column-major bf16: a fragment (32 columns x 16 q) is two transposing
    // reads: in each 16-lane group g (lanes 16 g + i), lane i addresses q row
    // (g >> 1) * 8 + (i >> 2) (+ 4 in the second read) and columns (g & 1) * 16
    // + 4 (i & 3) .. + 4, and receives column (g & 1) * 16 + i at 4 rows.
    uint32_t xcof[XC && TY == kBf16 ? MB : 1], ycof[YC && TY == kBf16 ? NB : 1];
    {
        const int g = lane >> 4, i = lane & 15;
        const int r = (g >> 1) * 8 + (i >> 2);
        const int low = (g & 1) * 2 + ((i & 3) >> 1);
        if constexpr (XC && TY == kBf16) {
#pragma unroll
            for (int b = 0; b < MB; ++b)
                xcof[b] = r * (TM * EB) + ((((wm * MB + b) * 4 + low) ^ col_swizzle<XCH>(r)) << 4) + 8 * (i & 1);
        }
        if constexpr (YC && TY == kBf16) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
                ycof[b] = X_BYTES + r * (TN * EB) + ((((wn * NB + b) * 4 + low) ^ col_swizzle<YCH>(r)) << 4) + 8 * (i & 1);
        }
    }
    i32x4_t f[4][NR];  // f[step][X blocks, then Y blocks]
    auto read_frag = [&](int kk, int i, uint32_t so) {
        const bool is_x = i < MB;
        const int b = is_x ? i : i - MB;
        if ((is_x && !XC) || (!is_x && !YC)) {
            const char* base = smem + so + (is_x ? (wm * MB + b) * 32 * 128 : X_BYTES + (wn * NB + b) * 32 * 128);
            f[kk][i] = *reinterpret_cast<const i32x4_t*>(base + foff[kk]);
        } else if constexpr (TY == kBf16) {
            typedef short s4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s4_t* lds_s4_t;
            constexpr int XB = TM * EB, YB = TN * EB;
            const int rb = is_x ? XB : YB;
            const uint32_t a = lds_addr(smem) + so + (is_x ? xcof[is_x && XC ? b : 0] : ycof[!is_x && YC ? b : 0]) + kk * 16 * rb;
            const s4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4_t>(a));
            const s4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s4_t>(a + 4 * rb));
            f[kk][i] = __builtin_bit_cast(i32x4_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            const int rb = (is_x ? TM : TN) * EB;
            const char* base = smem + so + (is_x ? (wm * MB + b) * 128 : X_BYTES + (wn * NB + b) * 128) + l32 * 4;
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4)
                f[kk][i][i4] = *reinterpret_cast<const int*>(base + (8 * kk + 4 * half + i4) * rb);
        }
    };

    Acc acc[NB][MB];
#pragma unroll
    for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = 0; b < MB; ++b) acc[a][b] = zero16(Acc{});
    auto mul = [&](int kk, int q) {
        const int nb = q / MB, mb = q % MB;
        if constexpr (TY == kBf16) {
            acc[nb][mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, f[kk][MB + nb]),
                                                                  __builtin_bit_cast(bf16x8_t, f[kk][mb]), acc[nb][mb], 0, 0, 0);
        } else if constexpr (TY == kI8) {
            acc[nb][mb] = __builtin_amdgcn_mfma_i32_32x32x32_i8(f[kk][MB + nb], f[kk][mb], acc[nb][mb], 0, 0, 0);
        } else {
            const f32x4_t y = __builtin_bit_cast(f32x4_t, f[kk][MB + nb]), x = __builtin_bit_cast(f32x4_t, f[kk][mb]);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                acc[nb][mb] = __builtin_amdgcn_mfma_f32_32x32x2f32(y[i], x[i], acc[nb][mb], 0, 0, 0);
        }
    };

    // loads issued by the end of slot p of the 3 NM slots of steps 1..3
    auto refill = [&](int p, int kt) {
#pragma unroll
        for (int l = p * NL / (3 * NM); l < (p + 1) * NL / (3 * NM); ++l) dma(l, kt + 2);
    };
    constexpr int BEFORE3 = 2 * NM * NL / (3 * NM);

    if (nk > 0) {
#pragma unroll
        for (int l = 0; l < NL; ++l) dma(l, 0);
        if (nk > 1) {
#pragma unroll
            for (int l = 0; l < NL; ++l) dma(l, 1);
            wait_vmcnt<NL>();
        } else {
            wait_vmcnt<0>();
        }
        barrier_lds();
#pragma unroll
        for (int i = 0; i < NR; ++i) read_frag(0, i, 0);
        __builtin_amdgcn_sched_barrier(0);
    }
    auto slice = [&](int kt, auto more_c) {
        constexpr bool MORE = decltype(more_c)::value;
        const uint32_t so = (kt & 1) * STAGE, nso = ((kt + 1) & 1) * STAGE;
#pragma unroll
        for (int kk = 1; kk < 4; ++kk)
#pragma unroll
            for (int i = 0; i < NR; ++i) read_frag(kk, i, so);
#pragma unroll
        for (int q = 0; q < NM; ++q) mul(0, q);
        __builtin_amdgcn_sched_barrier(0);
        wait_vmcnt_lgkm0<63>();
        barrier_lds();
#pragma unroll
        for (int step = 1; step <= 2; ++step) {
#pragma unroll
            for (int q = 0; q < NM; ++q) {
                mul(step, q);
                if (MORE) {
                    refill((step - 1) * NM + q, kt);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (MORE) {
            wait_vmcnt<BEFORE3>();
            barrier_lds();
        } else if (kt + 1 < nk) {
            wait_vmcnt<0>();
            barrier_lds();
        }
        // (after the last slice this reads a stale stage whose values are
        // never used)
#pragma unroll
        for (int q = 0; q < NM; ++q) {
            mul(3, q);
            if (MORE) {
                refill(2 * NM + q, kt);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = q * NR / NM; i < (q + 1) * NR / NM; ++i) read_frag(0, i, nso);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    int kt = 0;
    for (; kt + 2 < nk; ++kt) slice(kt, std::true_type{});
    for (; kt < nk; ++kt) slice(kt, std::false_type{});

    // ---- epilogue
    // lane: output row m0 + (wm * MB + mb) * 32 + l32, columns p0 + (wn * NB +
    // nb) * 32 + 8 g + 4 half + 0..3 in registers 4 g .. 4 g + 3
    float rs[MB];
    if constexpr (TY == kI8) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int m = m0 + (wm * MB + mb) * 32 + l32;
            rs[mb] = m < m1 ? sx[m] : 0.f;
        }
    }
    auto values = [&](int nb, int mb, int g, float* v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(acc[nb][mb][4 * g + i]);
        if constexpr (TY == kI8) {
            const int col = p0 + (wn * NB + nb) * 32 + 8 * g + 4 * half;
            f32x4_t s = {0.f, 0.f, 0.f, 0.f};
            if (col < P) s = *reinterpret_cast<const f32x4_t*>(sy + static_cast<int64_t>(e) * N + col);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = v[i] * rs[mb] * s[i];
        }
    };
    O* const out = C + (MODE == kTN ? static_cast<int64_t>(e) * N * K : 0);
    if constexpr (sizeof(O) == 4) {
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int m = m0 + (wm * MB + mb) * 32 + l32;
            float* const row = reinterpret_cast<float*>(out) + static_cast<int64_t>(m) * P;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = p0 + (wn * NB + nb) * 32 + 8 * g + 4 * half;
                    float v[4];
                    values(nb, mb, g, v);
                    if (m < m1 && col < P) *reinterpret_cast<f32x4_t*>(row + col) = f32x4_t{v[0], v[1], v[2], v[3]};
                }
        }
    } else {
        // bf16: each wave stages its own part of the tile in LDS (16-byte chunk
        // ch of row r at ch ^ (r mod CPR)) and writes whole chunks, consecutive
        // lanes on consecutive chunks of a row: full 128-byte lines
        constexpr int CPR = NB * 4;
        constexpr int ROWO = NB * 64;
        static_assert(4 * MB * 32 * ROWO <= 2 * STAGE, "the staged tile must fit the stages");
        wait_vmcnt_lgkm0<0>();
        barrier_lds();
        char* const st = smem + wave * (MB * 32 * ROWO);
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
            const int r = mb * 32 + l32;
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    float v[4];
                    values(nb, mb, g, v);
                    *reinterpret_cast<uint2*>(st + r * ROWO + (((nb * 4 + g) ^ (r & (CPR - 1))) * 16) + half * 8) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                }
        }
#pragma unroll 4
        for (int idx = lane; idx < MB * 32 * CPR; idx += 64) {
            const int r = idx / CPR, ch = idx % CPR;
            const int m = m0 + wm * MB * 32 + r;
            const int col = p0 + wn * NB * 32 + ch * 8;
            if (m >= m1 || col >= P) continue;
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(st + r * ROWO + ((ch ^ (r & (CPR - 1))) * 16));
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(reinterpret_cast<bf16_t*>(out) + static_cast<int64_t>(m) * P + col));
        }
    }
}

template <int TY, int MODE, int MB, int NB, typename O>
hipError_t launch_tile(const moe_grouped_t& g, const void* X, const void* Y, const int32_t* offsets, void* C,
                       const float* sx, const float* sy, hipStream_t s) {
    const int tm = 64 * MB, tn = 64 * NB;
    int64_t grid;
    if (MODE == kTN)
        grid = g.E * ceil_div(g.N, tm) * ceil_div(g.K, tn);
    else
        grid = static_cast<int64_t>(align_up(max_m_tiles(g.rows, g.E, tm) * ceil_div(MODE == kNT ? g.N : g.K, tn), kXcds));
    grouped_tile_kernel<TY, MODE, MB, NB, O><<<static_cast<unsigned>(grid), 256, 0, s>>>(
        X, Y, offsets, g.E, static_cast<int>(g.rows), g.N, g.K, static_cast<O*>(C), sx, sy);
    return hipGetLastError();
}

template <int TY, int MODE, typename O>
hipError_t launch(const moe_grouped_t& g, const void* X, const void* Y, const int32_t* offsets, void* C,
                  const float* sx, const float* sy, hipStream_t s) {
    const int64_t P = MODE == kNT ? g.N : g.K;
    if constexpr (TY != kF32) {
        const int64_t tiles = MODE == kTN ? g.E * ceil_div(g.N, 256) * ceil_div(P, 256)
                                          : ceil_div(g.rows, 256) * ceil_div(P, 256);
        if (tiles >= 256 && (MODE == kTN || g.rows >= 128 * static_cast<int64_t>(g.E)))
            return launch_tile<TY, MODE, 4, 4, O>(g, X, Y, offsets, C, sx, sy, s);
    }
    if (MODE != kTN && g.rows < 64 * static_cast<int64_t>(g.E))
        return launch_tile<TY, MODE, 1, 2, O>(g, X, Y, offsets, C, sx, sy, s);
    return launch_tile<TY, MODE, 2, 2, O>(g, X, Y, offsets, C, sx, sy, s);
}

}  // namespace

int64_t grouped_grid_bound(const moe_grouped_t& g) {
    const int64_t n = ceil_div(g.N, 128), k = ceil_div(g.K, 128);
    return std::max(max_m_tiles(g.rows, g.E, 64) * std::max(n, k) + kXcds, g.E * n * k);
}

size_t grouped_ws_bytes(const moe_grouped_t&, int) { return 0; }

hipError_t launch_grouped_matmul(const moe_grouped_t& g, const void* a, const void* w, const int32_t* offsets, void* c,
                                 void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch<kBf16, kNT, bf16_t>(g, a, w, offsets, c, nullptr, nullptr, s);
    return launch<kF32, kNT, float>(g, a, w, offsets, c, nullptr, nullptr, s);
}

hipError_t launch_grouped_da(const moe_grouped_t& g, const void* dc, const void* w, const int32_t* offsets, void* da,
                             void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch<kBf16, kNN, bf16_t>(g, dc, w, offsets, da, nullptr, nullptr, s);
    return launch<kF32, kNN, float>(g, dc, w, offsets, da, nullptr, nullptr, s);
}

hipError_t launch_grouped_dw(const moe_grouped_t& g, const void* dc, const void* a, const int32_t* offsets, void* dw,
                             void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch<kBf16, kTN, bf16_t>(g, dc, a, offsets, dw, nullptr, nullptr, s);
    return launch<kF32, kTN, float>(g, dc, a, offsets, dw, nullptr, nullptr, s);
}

hipError_t launch_grouped_int8(const moe_grouped_t& g, const void* a, const float* sa, const void* w, const float* sw,
                               const int32_t* offsets, void* c, void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch<kI8, kNT, bf16_t>(g, a, w, offsets, c, sa, sw, s);
    return launch<kI8, kNT, float>(g, a, w, offsets, c, sa, sw, s);
}

}  // namespace moe
