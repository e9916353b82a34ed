// Matrix product by expert of 4-bit microscaled floats:
//   C[r, n] = sum_k A[r, k] W_e[n, k]       rows r of queue e
// by the kernels of the other grouped products, on v_mfma_scale_f32_32x32x64_f8f6f4,
// whose lane holds one block of 32 values of one row (16 bytes) and that block's
// scale.
#include "grouped_tile.h"

namespace moe {

namespace {

template <typename O>
hipError_t start(const moe_grouped_t& g, const void* a, const void* sa, const void* w, const void* sw,
                 const int32_t* offsets, O* C, hipStream_t s) {
    const Plan p = plan_mxfp4(g);
    int64_t n = workgroups(g, kNT, p);
    if (p.v == kTile256) n = std::min<int64_t>(n, align_up(compute_units(s), kXcds));
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
