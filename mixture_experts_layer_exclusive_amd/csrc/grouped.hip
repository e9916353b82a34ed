// Matrix products grouped by expert: forward, its two gradients, and the
// 8-bit integer product.
//
//   kNT  C[r, n] = sum_k A[r, k] W_e[n, k]        rows r of queue e
//   kNN  dA[r, k] = sum_n dC[r, n] W_e[n, k]
//   kTN  dW_e[n, k] = sum_{r in queue e} dC[r, n] A[r, k]
#include <algorithm>

#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNT = 0, kNN = 1, kTN = 2;

// A queue's rows, clamped to the matrix: whatever offsets holds, 0 <= lo <=
// hi <= rows.
__device__ __forceinline__ void queue_rows(const int32_t* __restrict__ offsets, int e, int rows, int& lo, int& hi) {
    lo = min(max(offsets[e], 0), rows);
    hi = max(min(offsets[e + 1], rows), lo);
}

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16_t v) { return bf16_to_f32(v); }
__device__ __forceinline__ int widen(int8_t v) { return v; }

__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(bf16_t* p, float v) { *p = static_cast<bf16_t>(pack_bf16x2(v, 0.f)); }

constexpr int TS = 64;  // output tile
constexpr int RS = 16;  // reduction step

template <int MODE, typename T, typename O>
__global__ __launch_bounds__(256) void grouped_simple_kernel(const T* __restrict__ A, const T* __restrict__ B,
                                                             const int32_t* __restrict__ offsets, int E, int rows,
                                                             int N, int K, O* __restrict__ C,
                                                             const float* __restrict__ sa,
                                                             const float* __restrict__ sw) {
    using W = decltype(widen(T{}));
    __shared__ W s_a[RS][TS + 1];
    __shared__ W s_b[RS][TS + 1];
    const int tid = threadIdx.x;
    // output [M rows of the tile's matrix] x [P columns], reduction length R
    const int P = MODE == kNT ? N : K;
    const int ptiles = (P + TS - 1) / TS;
    int e = 0, lo = 0, hi = rows, m0, mend;
    const int p0 = (blockIdx.x % ptiles) * TS;
    int mt = blockIdx.x / ptiles;
    if (MODE == kTN) {
        const int mtiles = (N + TS - 1) / TS;
        e = mt / mtiles;
        m0 = (mt % mtiles) * TS;
        mend = min(m0 + TS, N);
        queue_rows(offsets, e, rows, lo, hi);
    } else {
        for (;; ++e) {
            if (e >= E) return;
            if (offsets != nullptr) queue_rows(offsets, e, rows, lo, hi);
            const int tiles = (hi - lo + TS - 1) / TS;
            if (mt < tiles) break;
            mt -= tiles;
        }
        m0 = lo + mt * TS;
        mend = min(m0 + TS, hi);
    }
    const int R = MODE == kNT ? K : (MODE == kNN ? N : hi - lo);
    const T* const Be = MODE == kTN ? B : B + static_cast<int64_t>(e) * N * K;
    const int tx = tid & 15, ty = tid >> 4;
    W acc[4][4] = {};
    for (int r0 = 0; r0 < R; r0 += RS) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int idx = tid + 256 * i;
            const int c = MODE == kTN ? idx / TS : idx % RS;  // reduction index of A's element
            const int m = MODE == kTN ? idx % TS : idx / RS;
            W v = 0;
            if (r0 + c < R && m0 + m < mend)
                v = widen(MODE == kTN ? A[static_cast<int64_t>(lo + r0 + c) * N + m0 + m]
                                      : A[static_cast<int64_t>(m0 + m) * (MODE == kNT ? K : N) + r0 + c]);
            s_a[c][m] = v;
            const int cb = MODE == kNT ? idx % RS : idx / TS;
            const int p = MODE == kNT ? idx / RS : idx % TS;
            v = 0;
            if (r0 + cb < R && p0 + p < P)
                v = widen(MODE == kNT ? Be[static_cast<int64_t>(p0 + p) * K + r0 + cb]
                                      : Be[static_cast<int64_t>((MODE == kTN ? lo : 0) + r0 + cb) * K + p0 + p]);
            s_b[cb][p] = v;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < RS; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += s_a[c][ty * 4 + i] * s_b[c][tx * 4 + j];
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (m >= mend) continue;
        const int64_t row = MODE == kTN ? static_cast<int64_t>(e) * N + m : m;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = p0 + tx * 4 + j;
            if (p >= P) continue;
            float v = static_cast<float>(acc[i][j]);
            if (sa != nullptr) v = v * sa[m] * sw[static_cast<int64_t>(e) * N + p];
            store(C + row * P + p, v);
        }
    }
}

template <int MODE, typename T, typename O>
hipError_t launch_simple(const moe_grouped_t& g, const void* A, const void* B, const int32_t* offsets, void* C,
                         const float* sa, const float* sw, hipStream_t s) {
    const int64_t mt = MODE == kTN ? g.E * ceil_div(g.N, TS) : max_m_tiles(g.rows, g.E, TS);
    const int64_t grid = mt * ceil_div(MODE == kNT ? g.N : g.K, TS);
    grouped_simple_kernel<MODE, T, O><<<static_cast<unsigned>(grid), 256, 0, s>>>(
        static_cast<const T*>(A), static_cast<const T*>(B), offsets, g.E, static_cast<int>(g.rows), g.N, g.K,
        static_cast<O*>(C), sa, sw);
    return hipGetLastError();
}

}  // namespace

int64_t grouped_grid_bound(const moe_grouped_t& g) {
    const int64_t n = ceil_div(g.N, TS), k = ceil_div(g.K, TS);
    return std::max(max_m_tiles(g.rows, g.E, TS) * std::max(n, k), g.E * n * k);
}

size_t grouped_ws_bytes(const moe_grouped_t&, int) { return 0; }

hipError_t launch_grouped_matmul(const moe_grouped_t& g, const void* a, const void* w, const int32_t* offsets, void* c,
                                 void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch_simple<kNT, bf16_t, bf16_t>(g, a, w, offsets, c, nullptr, nullptr, s);
    return launch_simple<kNT, float, float>(g, a, w, offsets, c, nullptr, nullptr, s);
}

hipError_t launch_grouped_da(const moe_grouped_t& g, const void* dc, const void* w, const int32_t* offsets, void* da,
                             void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch_simple<kNN, bf16_t, bf16_t>(g, dc, w, offsets, da, nullptr, nullptr, s);
    return launch_simple<kNN, float, float>(g, dc, w, offsets, da, nullptr, nullptr, s);
}

hipError_t launch_grouped_dw(const moe_grouped_t& g, const void* dc, const void* a, const int32_t* offsets, void* dw,
                             void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch_simple<kTN, bf16_t, bf16_t>(g, dc, a, offsets, dw, nullptr, nullptr, s);
    return launch_simple<kTN, float, float>(g, dc, a, offsets, dw, nullptr, nullptr, s);
}

hipError_t launch_grouped_int8(const moe_grouped_t& g, const void* a, const float* sa, const void* w, const float* sw,
                               const int32_t* offsets, void* c, void*, hipStream_t s) {
    if (g.dtype == MOE_DTYPE_BF16) return launch_simple<kNT, int8_t, bf16_t>(g, a, w, offsets, c, sa, sw, s);
    return launch_simple<kNT, int8_t, float>(g, a, w, offsets, c, sa, sw, s);
}

}  // namespace moe
