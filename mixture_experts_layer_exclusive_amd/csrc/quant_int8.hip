// 8-bit integer codes of a matrix's rows, one float32 scale per row:
//   scale = max(amax / 127, 2^-126), code = rint(x / scale)
// (1 for an all-zero row; NaN and codes 0 for a row with a NaN or infinity).
// The scale floor keeps a row of subnormal values from a scale of zero.
// Both quotients are IEEE divisions, so the codes are a function of the row
// alone that any float32 host reproduces bit for bit.
//
// The division itself would take about as long as the row's memory traffic.
// Instead q = x * (1 / scale), which is within 2^-16 of the quotient (|q| <=
// 127.01: half an ulp from the reciprocal, at most one ulp of q = 2^-17, and
// half an ulp from the product): wherever q is further than 2^-15 from the
// middle between two integers, both round to the same one.  A lane that meets
// a q nearer than that (about 6 in 100000 of smooth data) divides its values
// properly.
#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

// The values of one 16-byte word: 8 bf16 or 4 f32.
template <typename T>
struct Word;
template <>
struct Word<bf16_t> {
    static constexpr int N = 8;
    using Codes = uint2;
    static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = lo_bf16(u[i]);
            v[2 * i + 1] = hi_bf16(u[i]);
        }
    }
    // largest |x| as the bits of a float: integer order is the values' order,
    // with infinities and NaNs above every finite value
    static __device__ __forceinline__ uint32_t amax(const uint4& w, uint32_t m) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(u[i] & 0x7fff0000u, (u[i] << 16) & 0x7fff0000u));
        return m;
    }
};
template <>
struct Word<float> {
    static constexpr int N = 4;
    using Codes = uint32_t;
    static __device__ __forceinline__ void unpack(const uint4& w, float* v) {
        v[0] = __uint_as_float(w.x);
        v[1] = __uint_as_float(w.y);
        v[2] = __uint_as_float(w.z);
        v[3] = __uint_as_float(w.w);
    }
    static __device__ __forceinline__ uint32_t amax(const uint4& w, uint32_t m) {
        return max(max(m, max(w.x & 0x7fffffffu, w.y & 0x7fffffffu)), max(w.z & 0x7fffffffu, w.w & 0x7fffffffu));
    }
};

__device__ __forceinline__ float scale_of(uint32_t m) {
    if (m >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    return m == 0 ? 1.f : fmaxf(__uint_as_float(m) / 127.f, 0x1p-126f);
}

// Low bytes of a, b, c, d in one word.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    const uint32_t ab = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
    const uint32_t cd = __builtin_amdgcn_perm(d, c, 0x04000c0cu);
    return ab | cd;
}

// The codes of a word.  1.5 * 2^23 added to |q| < 2^22 leaves rint(q) (ties to
// even) in the low bits of the sum.
template <typename T>
__device__ __forceinline__ typename Word<T>::Codes codes_of(const uint4& w, float scale, float inv, bool finite) {
    constexpr int N = Word<T>::N;
    constexpr float kMagic = 12582912.f;
    float v[N];
    Word<T>::unpack(w, v);
    uint32_t t[N];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float q = v[i] * inv;
        const float r = q + kMagic;
        t[i] = __float_as_uint(r);
        off = fmaxf(off, fabsf(q - (r - kMagic)));
    }
    if (off > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = __float_as_uint(v[i] / scale + kMagic);
    }
    if (!finite) {
#pragma unroll
        for (int i = 0; i < N; ++i) t[i] = 0u;
    }
    if constexpr (N == 8)
        return make_uint2(low_bytes(t[0], t[1], t[2], t[3]), low_bytes(t[4], t[5], t[6], t[7]));
    else
        return low_bytes(t[0], t[1], t[2], t[3]);
}

// Short rows: G lanes (a power of two up to the wave) per row, RW words per
// lane, all in registers; the maximum by wave shuffles alone.
template <typename T, int G, int RW>
__global__ __launch_bounds__(256) void quant_rows_int8_wave_kernel(const uint4* __restrict__ src, int64_t rows,
                                                                  int words, typename Word<T>::Codes* __restrict__ dst,
                                                                  float* __restrict__ scales) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * (256 / G) + threadIdx.x / G;
    const int lane = threadIdx.x & (G - 1);
    const bool has = r < rows;
    const uint4* row = src + (has ? r : 0) * words;
    uint4 keep[RW];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int c = lane + G * i;
        keep[i] = has && c < words ? load_nt(row + c) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) m = Word<T>::amax(keep[i], m);
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off, 64)));
    if (!has) return;
    const float scale = scale_of(m);
    const float inv = 1.f / scale;
    if (lane == 0) scales[r] = scale;
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int c = lane + G * i;
        if (c < words) dst[r * words + c] = codes_of<T>(keep[i], scale, inv, m < 0x7f800000u);
    }
}

// Longer rows: one workgroup per row, RC words per thread in registers; the
// longest (RC = 0) are read twice, the second time from the caches.
template <typename T, int RC>
__global__ __launch_bounds__(256) void quant_rows_int8_kernel(const uint4* __restrict__ src, int words,
                                                             typename Word<T>::Codes* __restrict__ dst,
                                                             float* __restrict__ scales) {
    __shared__ uint32_t s_max[4];
    const int64_t r = blockIdx.x;
    const uint4* row = src + r * words;
    uint4 keep[RC > 0 ? RC : 1];
    uint32_t m = 0;
    if constexpr (RC > 0) {
#pragma unroll
        for (int i = 0; i < RC; ++i) {
            const int c = threadIdx.x + 256 * i;
            keep[i] = c < words ? load_nt(row + c) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < RC; ++i) m = Word<T>::amax(keep[i], m);
    } else {
        for (int c = threadIdx.x; c < words; c += 256) m = Word<T>::amax(row[c], m);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off, 64)));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
    const float scale = scale_of(m);
    const float inv = 1.f / scale;
    if (threadIdx.x == 0) scales[r] = scale;
    const bool finite = m < 0x7f800000u;
    if constexpr (RC > 0) {
#pragma unroll
        for (int i = 0; i < RC; ++i) {
            const int c = threadIdx.x + 256 * i;
            if (c < words) dst[r * words + c] = codes_of<T>(keep[i], scale, inv, finite);
        }
    } else {
        for (int c = threadIdx.x; c < words; c += 256) dst[r * words + c] = codes_of<T>(row[c], scale, inv, finite);
    }
}

template <typename T>
hipError_t launch_rows(const void* src, int64_t rows, int cols, void* codes, float* scales, hipStream_t s) {
    const int words = cols / Word<T>::N;
    const uint4* in = static_cast<const uint4*>(src);
    auto* out = static_cast<typename Word<T>::Codes*>(codes);
    const unsigned g = static_cast<unsigned>(rows);
    auto wgs = [&](int per) { return static_cast<unsigned>(ceil_div(rows, per)); };
    if (words <= 8) quant_rows_int8_wave_kernel<T, 8, 1><<<wgs(32), 256, 0, s>>>(in, rows, words, out, scales);
    else if (words <= 32) quant_rows_int8_wave_kernel<T, 32, 1><<<wgs(8), 256, 0, s>>>(in, rows, words, out, scales);
    else if (words <= 128) quant_rows_int8_wave_kernel<T, 64, 2><<<wgs(4), 256, 0, s>>>(in, rows, words, out, scales);
    else if (words <= 256) quant_rows_int8_wave_kernel<T, 64, 4><<<wgs(4), 256, 0, s>>>(in, rows, words, out, scales);
    else if (words <= 256 * 2) quant_rows_int8_kernel<T, 2><<<g, 256, 0, s>>>(in, words, out, scales);
    else if (words <= 256 * 8) quant_rows_int8_kernel<T, 8><<<g, 256, 0, s>>>(in, words, out, scales);
    else quant_rows_int8_kernel<T, 0><<<g, 256, 0, s>>>(in, words, out, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_rows_int8(const void* src, int64_t rows, int cols, int dtype, void* codes, float* scales,
                                  hipStream_t s) {
    if (dtype == MOE_DTYPE_BF16) return launch_rows<bf16_t>(src, rows, cols, codes, scales, s);
    return launch_rows<float>(src, rows, cols, codes, scales, s);
}

}  // namespace moe
