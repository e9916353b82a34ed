// Matrix product by expert of 4-bit microscaled floats:
//   C[r, n] = sum_k A[r, k] W_e[n, k]       rows r of queue e
// by the kernels of the other grouped products, on v_mfma_scale_f32_32x32x64_f8f6f4,
// whose lane holds one block of 32 values of one row (16 bytes) and that block's
// scale.  Products are exact; sums are float32.
//
// To the pipeline a slice is 128 bytes of codes per row, as any type's (256 values here),
// with 8 scale bytes per row beside it.  Small products are bound by the weights' bytes
// (64 queues of 6 rows, 2048 x 1408: 98 MB, 23 us) or by a launch's start and end, large ones
// by matrix products and the card's power: 16384 rows, 14336 x 4096, one queue, 460 us (4180
// TFLOP/s), K = 14336 1424 us (4730); products alone, from registers, reach 5800 on random
// codes, 8960 on zeros (unscaled 6470, 9600: a scale costs the instruction 2 cycles in 32).
// The bf16 kernel takes 414 us for as many tiles, bytes and instructions, int8 443.
#include "grouped_tile.h"

namespace moe {

namespace {

// ---- short reductions --------------------------------------------------------------
//
// K <= 256, one slice: the other kernels spend their time on a tile's start and end (first
// loads into LDS, waits, staged stores). Here each wave takes 32 rows and 128 columns straight
// from memory, all its loads in flight together; a workgroup's 4 waves are neighbours in a
// strip of 512 columns.
constexpr int kShortN = 512;

template <int KS, typename O>
__global__ __launch_bounds__(256) void grouped_mxfp4_short_kernel(
    const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA, const uint8_t* __restrict__ W,
    const uint8_t* __restrict__ SW, const int32_t* __restrict__ offsets, int E, int rows, int N, int K,
    O* __restrict__ C) {
    __shared__ Queues queues;
    load_queues<false>(offsets, E, rows, 32, queues);
    Tile t;
    if (row_tile(queues, E, 32, kShortN, N, blockIdx.x % kXcds, blockIdx.x / kXcds, t) != kTile) return;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, half = lane >> 5, l32 = lane & 31;
    const int p0 = t.p0 + wave * 128;
    if (p0 >= N) return;
    const int blocks = K / 32;
    // (rows past the queue and columns past the matrix: the last one's, not stored)
    const int64_t row = min(t.m0 + l32, t.m1 - 1);
    i32x4_t x[KS], y[4][KS];
    uint2 sx, sy[4];
    // block 2 kk + half of a row; past its end the row's last (no branch: all loads go out
    // together)
    auto load = [&](const uint8_t* at, i32x4_t (&v)[KS]) {
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
            v[kk] = *reinterpret_cast<const i32x4_t*>(at + min(2 * kk + half, blocks - 1) * 16);
    };
    load(A + row * (K / 2), x);
    sx = *reinterpret_cast<const uint2*>(SA + row * 8);
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
        const int64_t col = static_cast<int64_t>(t.e) * N + min(p0 + nb * 32 + l32, N - 1);
        load(W + col * (K / 2), y[nb]);
        sy[nb] = *reinterpret_cast<const uint2*>(SW + col * 8);
    }
    // (past the row's end zeros in X; both scales are finite there)
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[kk][i] = 2 * kk + half < blocks ? x[kk][i] : 0;
    const uint32_t sel = scale_select(half, blocks);
    const int scx = pick_scales(sx, sel);
    f32x16_t acc[4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
        acc[nb] = zero_acc<kMx4>();
        const int scy = pick_scales(sy[nb], sel);
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) multiply_mx4(kk, y[nb][kk], x[kk], scy, scx, acc[nb]);
        // (a product needs every lane's operands, whichever rows are stored: it stays above
        // the branch)
        asm volatile("" : "+v"(acc[nb]));
    }
    if (t.m0 + l32 >= t.m1) return;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int c = p0 + nb * 32 + 8 * g + 4 * half;
            if (c >= N) continue;
            O* const dst = C + row * N + c;
            const f32x4_t v = {acc[nb][4 * g], acc[nb][4 * g + 1], acc[nb][4 * g + 2], acc[nb][4 * g + 3]};
            if constexpr (sizeof(O) == 4) *reinterpret_cast<f32x4_t*>(dst) = v;
            else *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        }
    }
}

template <typename O>
hipError_t start_short(const moe_grouped_t& g, const void* a, const void* sa, const void* w, const void* sw,
                       const int32_t* offsets, O* C, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(align_up(row_tiles(g, 32) * ceil_div(g.N, kShortN), kXcds));
    const uint8_t *A = static_cast<const uint8_t*>(a), *SA = static_cast<const uint8_t*>(sa);
    const uint8_t *W = static_cast<const uint8_t*>(w), *SW = static_cast<const uint8_t*>(sw);
    const int rows = static_cast<int>(g.rows);
    auto go = [&](auto ks) {
        grouped_mxfp4_short_kernel<decltype(ks)::value, O>
            <<<grid, 256, 0, s>>>(A, SA, W, SW, offsets, g.E, rows, g.N, g.K, C);
    };
    switch (ceil_div(g.K, 64)) {
        case 1: go(std::integral_constant<int, 1>{}); break;
        case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: go(std::integral_constant<int, 3>{}); break;
        default: go(std::integral_constant<int, 4>{}); break;
    }
    return hipGetLastError();
}

template <typename O>
hipError_t start(const moe_grouped_t& g, const void* a, const void* sa, const void* w, const void* sw,
                 const int32_t* offsets, O* C, hipStream_t s) {
    if (short_mxfp4(g)) return start_short(g, a, sa, w, sw, offsets, C, s);
    const Plan p = plan_mxfp4(g);
    int64_t n = workgroups(g, kNT, p);
    if (p.v == kTile256 || p.v == kTile128x256) n = std::min<int64_t>(n, align_up(compute_units(s), kXcds));
    const unsigned grid = static_cast<unsigned>(n);
    const int rows = static_cast<int>(g.rows), K = g.K / 2;
    switch (p.v) {
        case kSplit32:
            grouped_split_kernel<kMx4, kNT, 1, 1, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw);
            break;
        case kSplit64:
            grouped_split_kernel<kMx4, kNT, 2, 2, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw);
            break;
        case kTile64x128:
            grouped_tile_kernel<kMx4, kNT, 1, 2, 2, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
        case kHalves64x128:
            grouped_tile_kernel<kMx4, kNT, 1, 2, 2, O, 2><<<grid, 512, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
        case kHalves128:
            grouped_tile_kernel<kMx4, kNT, 2, 2, 2, O, 2><<<grid, 512, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
        case kTile128x256:
            grouped_tile_kernel<kMx4, kNT, 2, 4, 2, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
        case kTile256:
            grouped_tile_kernel<kMx4, kNT, 4, 4, 2, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
        default:
            grouped_tile_kernel<kMx4, kNT, 2, 2, 2, O><<<grid, 256, 0, s>>>(a, w, offsets, g.E, rows, g.N, K, C, sa, sw, 1);
            break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_mxfp4(const moe_grouped_t& g, const void* a, const void* sa, const void* w, const void* sw,
                                const int32_t* offsets, void* c, hipStream_t s) {
    return g.dtype == MOE_DTYPE_BF16 ? start(g, a, sa, w, sw, offsets, static_cast<bf16_t*>(c), s)
                                     : start(g, a, sa, w, sw, offsets, static_cast<float*>(c), s);
}

}  // namespace moe
