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
#include "grouped_tile.h"

namespace moe {

namespace {

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
