// Gate-weighted combine (reverse dispatch; MoEBlaze summary, Methodology 2):
//   y[t, :] = sum_j gates[t, j] * y_perm[assign_pos[t*k + j], :]
// One workgroup per token; each thread owns 16-byte column chunks, reads the
// k expert rows of its token and accumulates in fp32 in ascending j, then
// rounds once.  Every y row is written exactly once, so the result does not
// depend on scheduling.
//
// And its gradient:
//   dy_perm[assign_pos[t*k + j], :] = gates[t, j] * dy[t, :]
//   dgates[t, j] = sum_c dy[t, c] * y_perm[assign_pos[t*k + j], c]
#include <type_traits>

#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

// KM > 0: k <= KM, the k row loads of a chunk issued together (the token's
// positions and gates read once, into LDS); KM = 0: any k, one row at a time.
template <int KM>
__global__ __launch_bounds__(256) void combine_bf16_kernel(const uint4* __restrict__ y_perm,
                                                          const int32_t* __restrict__ assign_pos,
                                                          const float* __restrict__ gates, int k,
                                                          int chunks_per_row,
                                                          uint4* __restrict__ y) {
    const int64_t t = blockIdx.x;
    if constexpr (KM > 0) {
        __shared__ int s_pos[KM];
        __shared__ float s_g[KM];
        if (threadIdx.x < KM) {
            const int j = threadIdx.x;
            s_pos[j] = j < k ? assign_pos[t * k + j] : -1;
            s_g[j] = j < k ? gates[t * k + j] : 0.f;
        }
        __syncthreads();
        int pos[KM];
        float g[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            pos[j] = s_pos[j];
            g[j] = s_g[j];
        }
        for (int c = threadIdx.x; c < chunks_per_row; c += 256) {
            uint4 v[KM];
#pragma unroll
            for (int j = 0; j < KM; ++j)
                v[j] = pos[j] >= 0 ? load_nt(y_perm + static_cast<int64_t>(pos[j]) * chunks_per_row + c)
                                   : make_uint4(0u, 0u, 0u, 0u);
            float acc[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = 0.f;
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (pos[j] < 0) continue;
                const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    acc[2 * i] = fmaf(g[j], lo_bf16(w[i]), acc[2 * i]);
                    acc[2 * i + 1] = fmaf(g[j], hi_bf16(w[i]), acc[2 * i + 1]);
                }
            }
            uint4 o;
            o.x = pack_bf16x2(acc[0], acc[1]);
            o.y = pack_bf16x2(acc[2], acc[3]);
            o.z = pack_bf16x2(acc[4], acc[5]);
            o.w = pack_bf16x2(acc[6], acc[7]);
            y[t * chunks_per_row + c] = o;
        }
        return;
    }
    for (int c = threadIdx.x; c < chunks_per_row; c += 256) {
        float acc[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
        for (int j = 0; j < k; ++j) {
            const int pos = assign_pos[t * k + j];
            if (pos < 0) continue;
            const float g = gates[t * k + j];
            const uint4 v = load_nt(y_perm + static_cast<int64_t>(pos) * chunks_per_row + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                acc[2 * i] = fmaf(g, lo_bf16(w[i]), acc[2 * i]);
                acc[2 * i + 1] = fmaf(g, hi_bf16(w[i]), acc[2 * i + 1]);
            }
        }
        uint4 o;
        o.x = pack_bf16x2(acc[0], acc[1]);
        o.y = pack_bf16x2(acc[2], acc[3]);
        o.z = pack_bf16x2(acc[4], acc[5]);
        o.w = pack_bf16x2(acc[6], acc[7]);
        y[t * chunks_per_row + c] = o;
    }
}

__global__ __launch_bounds__(256) void combine_f32_kernel(const float* __restrict__ y_perm,
                                                         const int32_t* __restrict__ assign_pos,
                                                         const float* __restrict__ gates, int k,
                                                         int d, float* __restrict__ y) {
    const int64_t t = blockIdx.x;
    for (int c = threadIdx.x; c < d; c += 256) {
        float acc = 0.f;
        for (int j = 0; j < k; ++j) {
            const int pos = assign_pos[t * k + j];
            if (pos < 0) continue;
            acc = fmaf(gates[t * k + j], y_perm[static_cast<int64_t>(pos) * d + c], acc);
        }
        y[t * d + c] = acc;
    }
}

// ---- the gradient --------------------------------------------------------------
//
// L lanes per token, 256 / L tokens per workgroup (1024 lanes: one): a thread keeps its columns of dy, and of
// KM slots at a time reads y_perm's rows, adds to the slots' products and writes dy_perm's
// rows.  The products' sums over the lanes are taken at the end, in a fixed order.
// A float32 row starts at any multiple of 4 bytes and is moved 16 bytes at a time all the
// same; its last chunk starts 4 values before its end and leaves those that the chunk
// before it has out of the sums (and writes the same values to them again).
// Rows of more than 64 lanes are read and written past the caches, short ones (whose ends
// share cache lines) are read through them, those of 16 lanes also written (30000 tokens,
// 8 slots of 33 floats: 19 us for 27; 512 floats and more gain nothing).
// Bound by memory: 32768 tokens, 8 slots of 2048 bf16, 2.28 GB in 413 to 421 us (5.4 to 5.5
// TB/s, a copy 6.0), 449 with 4 slots at a time through the caches; 30000 tokens of 128 bf16
// 23 us, at a copy's rate 22.6; 1023 floats, whose rows begin inside cache lines, 10000
// tokens 149, at a copy's rate 118.
typedef float f32x4_any_t __attribute__((ext_vector_type(4), aligned(4)));  // at any float

// Rows read and written once go past the caches.
__device__ __forceinline__ void store_nt(uint4* p, const uint4& v) {
    const u32x4_t w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
}
__device__ __forceinline__ void store_nt(f32x4_any_t* p, const f32x4_any_t& v) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void store_nt(float* p, float v) { __builtin_nontemporal_store(v, p); }

template <typename T, int V>
struct Chunk;  // V values
template <>
struct Chunk<bf16_t, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ uint4 load(const uint4* p) { return load_nt(p); }
    static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = lo_bf16(u[i]);
            v[2 * i + 1] = hi_bf16(u[i]);
        }
    }
    static __device__ __forceinline__ uint4 scaled(const float (&v)[8], float g) {
        return make_uint4(pack_bf16x2(g * v[0], g * v[1]), pack_bf16x2(g * v[2], g * v[3]),
                          pack_bf16x2(g * v[4], g * v[5]), pack_bf16x2(g * v[6], g * v[7]));
    }
};
template <>
struct Chunk<float, 4> {
    using Raw = f32x4_any_t;
    static __device__ __forceinline__ f32x4_any_t load(const f32x4_any_t* p) { return __builtin_nontemporal_load(p); }
    static __device__ __forceinline__ void unpack(const f32x4_any_t& w, float (&v)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = w[i];
    }
    static __device__ __forceinline__ f32x4_any_t scaled(const float (&v)[4], float g) {
        return f32x4_any_t{g * v[0], g * v[1], g * v[2], g * v[3]};
    }
};
template <>
struct Chunk<float, 1> {
    using Raw = float;
    static __device__ __forceinline__ float load(const float* p) { return load_nt(p); }
    static __device__ __forceinline__ void unpack(const float& w, float (&v)[1]) { v[0] = w; }
    static __device__ __forceinline__ float scaled(const float (&v)[1], float g) { return g * v[0]; }
};

template <typename T, int V, int KM, int L>
__global__ __launch_bounds__(L > 256 ? L : 256) void combine_backward_kernel(
    const T* __restrict__ dy, const T* __restrict__ y_perm, const int32_t* __restrict__ assign_pos,
    const float* __restrict__ gates, int64_t T_, int k, int n, int d, T* __restrict__ dy_perm,
    float* __restrict__ dgates) {
    using C = Chunk<T, V>;
    using Raw = typename C::Raw;
    const int lane = threadIdx.x & (L - 1), wave = threadIdx.x >> 6;
    int64_t t = blockIdx.x;
    if constexpr (L == 64) t = t * 4 + __builtin_amdgcn_readfirstlane(wave);
    if constexpr (L < 64) t = t * (256 / L) + threadIdx.x / L;
    if (L < 256 && t >= T_) return;  // (a token's lanes leave together, and meet no barrier)
    const int chunks = (d + V - 1) / V;
    for (int j0 = 0; j0 < k; j0 += KM) {
        int pos[KM];
        float g[KM], dot[KM];
#pragma unroll
        for (int j = 0; j < KM; ++j) {
            pos[j] = j0 + j < k ? assign_pos[t * k + j0 + j] : -1;
            if (pos[j] >= n) pos[j] = -1;
            g[j] = j0 + j < k ? gates[t * k + j0 + j] : 0.f;
            dot[j] = 0.f;
        }
        for (int c = lane; c < chunks; c += L) {
            const int at = min(c * V, d - V);
            float a[V];
            Raw y[KM];
            if (dgates != nullptr) {
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    if (pos[j] >= 0) {
                        const Raw* const from = reinterpret_cast<const Raw*>(y_perm + static_cast<int64_t>(pos[j]) * d + at);
                        if constexpr (L >= 256) y[j] = C::load(from);
                        else y[j] = *from;
                    }
            }
            C::unpack(*reinterpret_cast<const Raw*>(dy + t * d + at), a);
#pragma unroll
            for (int j = 0; j < KM; ++j) {
                if (pos[j] < 0) continue;
                if (dgates != nullptr) {
                    float b[V];
                    C::unpack(y[j], b);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const float sum = fmaf(a[i], b[i], dot[j]);
                        dot[j] = std::is_same<T, float>::value && i < c * V - at ? dot[j] : sum;
                    }
                }
                if (dy_perm != nullptr) {
                    Raw* const to = reinterpret_cast<Raw*>(dy_perm + static_cast<int64_t>(pos[j]) * d + at);
                    if constexpr (L >= 64) store_nt(to, C::scaled(a, g[j]));
                    else *to = C::scaled(a, g[j]);
                }
            }
        }
        if (dgates == nullptr) continue;
#pragma unroll
        for (int j = 0; j < KM; ++j)
#pragma unroll
            for (int off = (L < 64 ? L : 64) / 2; off > 0; off >>= 1) dot[j] += __shfl_xor(dot[j], off, 64);
        if constexpr (L >= 256) {
            __shared__ float s_dot[L / 64][KM];
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if ((threadIdx.x & 63) == 0) s_dot[wave][j] = dot[j];
            __syncthreads();
            if (threadIdx.x < KM && j0 + threadIdx.x < k) {
                float total = 0.f;
#pragma unroll
                for (int w = 0; w < L / 64; ++w) total += s_dot[w][threadIdx.x];
                dgates[t * k + j0 + threadIdx.x] = total;
            }
            __syncthreads();
        } else {
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (lane == j && j0 + j < k) dgates[t * k + j0 + j] = dot[j];
        }
    }
}

template <typename T, int V>
hipError_t start_combine_backward(const moe_problem_t& p, const void* dy, const void* y_perm,
                                  const int32_t* assign_pos, const float* gates, void* dy_perm, float* dgates,
                                  hipStream_t s) {
    const int n = static_cast<int>(p.T * p.k);
    auto start = [&](auto km, auto lanes) {
        constexpr int kLanes = decltype(lanes)::value;
        constexpr int kThreads = kLanes > 256 ? kLanes : 256, kTokens = kThreads / kLanes;
        const unsigned grid = static_cast<unsigned>((p.T + kTokens - 1) / kTokens);
        combine_backward_kernel<T, V, decltype(km)::value, kLanes><<<grid, kThreads, 0, s>>>(
            static_cast<const T*>(dy), static_cast<const T*>(y_perm), assign_pos, gates, p.T, p.k, n, p.d,
            static_cast<T*>(dy_perm), dgates);
    };
    auto with_lanes = [&](auto lanes) {
        if (p.k <= 2) start(std::integral_constant<int, 2>{}, lanes);
        else if (p.k <= 4) start(std::integral_constant<int, 4>{}, lanes);
        else start(std::integral_constant<int, 8>{}, lanes);
    };
    // As many lanes as the row can use.  30000 tokens, 8 slots, with 16, 64 and 256 lanes:
    // 64 bf16 (8 chunks) 16, 27 and 66 us, 128 27, 31 and 66, 192 40, 40 and 66, 256 52, 50
    // and 68, 512 (64 chunks) 101, 96 and 89; 33 floats 27, 40 and 84, 130 120, 74 and 96;
    // 100 tokens of 512 bf16 7.7, 4.9 and 4.7 (all past the caches).  (With one slot 204
    // floats, 51 chunks, keep 51 of 256 lanes busy: 21135 tokens 26 us, at a copy's rate
    // 8.8.)  And a token per
    // compute unit with 256 and 1024 lanes: 38 tokens, 8 slots of 7168 floats 18 and 10 us,
    // 200 of 4096 floats 17 and 12, of 2048 9.6 and 7.9; 500 of 2048 14 and 16.
    const int chunks = (p.d + V - 1) / V;
    if constexpr (V == 1) {  // (fewer than 4 floats)
        with_lanes(std::integral_constant<int, 16>{});
    } else {
        if (chunks <= 16) with_lanes(std::integral_constant<int, 16>{});
        else if (chunks <= 48) with_lanes(std::integral_constant<int, 64>{});
        else if (chunks <= 256 || p.T > 256) with_lanes(std::integral_constant<int, 256>{});
        else with_lanes(std::integral_constant<int, 1024>{});
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_combine_backward(const moe_problem_t& p, const void* dy, const void* y_perm,
                                   const int32_t* assign_pos, const float* gates, void* dy_perm, float* dgates,
                                   hipStream_t s) {
    if (p.dtype == MOE_DTYPE_BF16)
        return start_combine_backward<bf16_t, 8>(p, dy, y_perm, assign_pos, gates, dy_perm, dgates, s);
    if (p.d >= 4) return start_combine_backward<float, 4>(p, dy, y_perm, assign_pos, gates, dy_perm, dgates, s);
    return start_combine_backward<float, 1>(p, dy, y_perm, assign_pos, gates, dy_perm, dgates, s);
}

hipError_t launch_combine(const moe_problem_t& p, const void* y_perm, const int32_t* assign_pos,
                          const float* gates, void* y, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.T);
    const uint4* yp = static_cast<const uint4*>(y_perm);
    uint4* yo = static_cast<uint4*>(y);
    if (p.dtype == MOE_DTYPE_BF16 && p.k <= 2)
        combine_bf16_kernel<2><<<grid, 256, 0, s>>>(yp, assign_pos, gates, p.k, p.d / 8, yo);
    else if (p.dtype == MOE_DTYPE_BF16 && p.k <= 4)
        combine_bf16_kernel<4><<<grid, 256, 0, s>>>(yp, assign_pos, gates, p.k, p.d / 8, yo);
    else if (p.dtype == MOE_DTYPE_BF16 && p.k <= 8)
        combine_bf16_kernel<8><<<grid, 256, 0, s>>>(yp, assign_pos, gates, p.k, p.d / 8, yo);
    else if (p.dtype == MOE_DTYPE_BF16)
        combine_bf16_kernel<0><<<grid, 256, 0, s>>>(yp, assign_pos, gates, p.k, p.d / 8, yo);
    else
        combine_f32_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(y_perm), assign_pos, gates,
                                                p.k, p.d, static_cast<float*>(y));
    return hipGetLastError();
}

}  // namespace moe
