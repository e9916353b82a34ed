// Matrix product by expert of 4-bit microscaled floats:
//   C[r, n] = sum_k A[r, k] W_e[n, k]       rows r of queue e
// on v_mfma_scale_f32_32x32x64_f8f6f4, whose lane holds one block of 32 values of
// one row (16 bytes) and that block's scale.
#include "grouped_common.h"

namespace moe {

namespace {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// A 32 x 32 output tile per wave, its operands straight from memory.
template <typename O>
__global__ __launch_bounds__(64) void grouped_mxfp4_kernel(const uint8_t* __restrict__ A, const uint8_t* __restrict__ SA,
                                                          const uint8_t* __restrict__ W, const uint8_t* __restrict__ SW,
                                                          const int32_t* __restrict__ offsets, int E, int rows, int N,
                                                          int K, O* __restrict__ C) {
    __shared__ Queues queues;
    load_queues<false>(offsets, E, rows, 32, queues);
    Tile t;
    if (row_tile(queues, E, 32, 32, N, blockIdx.x % kXcds, blockIdx.x / kXcds, t) != kTile) return;
    const int half = threadIdx.x >> 5, l32 = threadIdx.x & 31;
    const int blocks = K / 32;
    // (rows past the queue and columns past the matrix: the last one's, not stored)
    const int64_t row = min(t.m0 + l32, t.m1 - 1);
    const int64_t col = static_cast<int64_t>(t.e) * N + min(t.p0 + l32, N - 1);
    const int64_t cols = static_cast<int64_t>(E) * N;
    f32x16_t acc = zero_acc<kBf16>();
    for (int b0 = 0; b0 < blocks; b0 += 2) {
        const int b = b0 + half;
        i32x4_t x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
        int sx = 0, sy = 0;
        if (b < blocks) {
            x = *reinterpret_cast<const i32x4_t*>(A + row * (K / 2) + b * 16);
            y = *reinterpret_cast<const i32x4_t*>(W + col * (K / 2) + b * 16);
            sx = SA[((b / 8) * static_cast<int64_t>(rows) + row) * 8 + (b & 7)];
            sy = SW[((b / 8) * cols + col) * 8 + (b & 7)];
        }
        const i32x8_t xv = __builtin_shufflevector(x, x, 0, 1, 2, 3, -1, -1, -1, -1);
        const i32x8_t yv = __builtin_shufflevector(y, y, 0, 1, 2, 3, -1, -1, -1, -1);
        acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(yv, xv, acc, 4, 4, 0, sy, 0, sx);
    }
    if (t.m0 + l32 >= t.m1) return;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const int c = t.p0 + 8 * g + 4 * half;
        if (c >= N) continue;
        O* const dst = C + row * N + c;
        if constexpr (sizeof(O) == 4)
            *reinterpret_cast<f32x4_t*>(dst) = f32x4_t{acc[4 * g], acc[4 * g + 1], acc[4 * g + 2], acc[4 * g + 3]};
        else
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_bf16x2(acc[4 * g], acc[4 * g + 1]), pack_bf16x2(acc[4 * g + 2], acc[4 * g + 3]));
    }
}

}  // namespace

hipError_t launch_grouped_mxfp4(const moe_grouped_t& g, const void* a, const void* sa, const void* w, const void* sw,
                                const int32_t* offsets, void* c, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(align_up(row_tiles(g, 32) * ceil_div(g.N, 32), kXcds));
    const uint8_t *A = static_cast<const uint8_t*>(a), *SA = static_cast<const uint8_t*>(sa);
    const uint8_t *W = static_cast<const uint8_t*>(w), *SW = static_cast<const uint8_t*>(sw);
    const int rows = static_cast<int>(g.rows);
    if (g.dtype == MOE_DTYPE_BF16)
        grouped_mxfp4_kernel<<<grid, 64, 0, s>>>(A, SA, W, SW, offsets, g.E, rows, g.N, g.K, static_cast<bf16_t*>(c));
    else
        grouped_mxfp4_kernel<<<grid, 64, 0, s>>>(A, SA, W, SW, offsets, g.E, rows, g.N, g.K, static_cast<float*>(c));
    return hipGetLastError();
}

}  // namespace moe
