// 4-bit microscaled floats (OCP MX, MXFP4): a row's blocks of 32 values, each with
// a power of two as its scale,
//   scale = 2^(floor(log2 amax) - 2), at least 2^-127    (one byte, exponent + 127)
//   code  = sign, and |x| / scale rounded to 0, .5, 1, 1.5, 2, 3, 4 or 6, ties to
//           the even code, larger ones to 6
// An all-zero block has the scale 1; a block with a NaN or an infinity has the
// scale byte 255 (NaN) and codes 0.  Dividing by a power of two is exact, so the
// conversion is the only rounding.
//
// Codes are two to a byte, the even column in the low half.  Scale bytes lie as
// [ceil(cols / 256)][rows][8], so that what a tile of the product needs of a 128-byte
// slice of codes is contiguous.
#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

// 8 values per lane, 4 lanes per block; consecutive lanes hold consecutive values of
// the matrix, a workgroup 2048 of them.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float (&v)[8]) {
    const uint4 w = load_nt(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = lo_bf16(u[i]);
        v[2 * i + 1] = hi_bf16(u[i]);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
    const uint4 a = load_nt(reinterpret_cast<const uint4*>(p)), b = load_nt(reinterpret_cast<const uint4*>(p) + 1);
    const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(u[i]);
}

template <typename T>
__global__ __launch_bounds__(256) void quant_rows_mxfp4_kernel(const T* __restrict__ src, int64_t rows, int cols,
                                                              uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // words of 8 values
    const int words = cols / 8;
    if (at >= rows * words) return;  // (whole blocks leave together)
    const int64_t r = at / words;
    const int c = static_cast<int>(at - r * words);
    float v[8];
    load8(src + at * 8, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 1, 64)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 2, 64)));
    const bool finite = m < 0x7f800000u;
    const int byte = finite ? (m == 0 ? 127 : max(static_cast<int>(m >> 23) - 2, 0)) : 255;
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = fminf(fmaxf(__builtin_amdgcn_ldexpf(v[i], 127 - byte), -6.f), 6.f);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[0], v[1], 1.f, 0);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[2], v[3], 1.f, 1);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[4], v[5], 1.f, 2);
    out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, v[6], v[7], 1.f, 3);
    codes[at] = finite ? out : 0u;
    if ((c & 3) == 0) {
        const int b = c / 4, blocks = cols / 32;
        uint8_t* const dst = scales + static_cast<int64_t>(b / 8) * rows * 8 + r * 8;
        dst[b & 7] = static_cast<uint8_t>(byte);
        // the last slice's bytes past the row
        if (b == blocks - 1)
            for (int i = (b & 7) + 1; i < 8; ++i) dst[i] = 127;
    }
}

template <typename O>
__global__ __launch_bounds__(256) void dequant_rows_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int cols, O* __restrict__ dst) {
    const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int words = cols / 8;
    if (at >= rows * words) return;
    const int64_t r = at / words;
    const int b = static_cast<int>(at - r * words) / 4;
    const int byte = scales[static_cast<int64_t>(b / 8) * rows * 8 + r * 8 + (b & 7)];
    const uint32_t w = codes[at];
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t code = w >> (4 * i) & 15u, e = code >> 1 & 3u, odd = code & 1u;
        // 0 or 0.5 below exponent 1, else (1 + odd / 2) 2^(e - 1)
        const float f = e == 0 ? 0.5f * odd : __builtin_amdgcn_ldexpf(1.f + 0.5f * odd, static_cast<int>(e) - 1);
        const float x = __builtin_amdgcn_ldexpf(code & 8u ? -f : f, byte - 127);
        v[i] = byte == 255 ? __uint_as_float(0x7fc00000u) : x;
    }
    if constexpr (sizeof(O) == 4) {
        float4* const out = reinterpret_cast<float4*>(dst + at * 8);
        out[0] = make_float4(v[0], v[1], v[2], v[3]);
        out[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4*>(dst + at * 8) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    }
}

}  // namespace

hipError_t launch_quant_rows_mxfp4(const void* src, int64_t rows, int cols, int dtype, void* codes, void* scales,
                                   hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(rows * (cols / 8), 256));
    uint32_t* const c = static_cast<uint32_t*>(codes);
    uint8_t* const sc = static_cast<uint8_t*>(scales);
    if (dtype == MOE_DTYPE_BF16)
        quant_rows_mxfp4_kernel<<<grid, 256, 0, s>>>(static_cast<const bf16_t*>(src), rows, cols, c, sc);
    else
        quant_rows_mxfp4_kernel<<<grid, 256, 0, s>>>(static_cast<const float*>(src), rows, cols, c, sc);
    return hipGetLastError();
}

hipError_t launch_dequant_rows_mxfp4(const void* codes, const void* scales, int64_t rows, int cols, int dtype,
                                     void* dst, hipStream_t s) {
    const unsigned grid = static_cast<unsigned>(ceil_div(rows * (cols / 8), 256));
    const uint32_t* const c = static_cast<const uint32_t*>(codes);
    const uint8_t* const sc = static_cast<const uint8_t*>(scales);
    if (dtype == MOE_DTYPE_BF16)
        dequant_rows_mxfp4_kernel<<<grid, 256, 0, s>>>(c, sc, rows, cols, static_cast<bf16_t*>(dst));
    else
        dequant_rows_mxfp4_kernel<<<grid, 256, 0, s>>>(c, sc, rows, cols, static_cast<float*>(dst));
    return hipGetLastError();
}

}  // namespace moe
