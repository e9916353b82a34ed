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
//
// Both ways are bound by memory: 32768 x 2048 bf16, 174 MB each, quantised in 30.7 us (5.7
// TB/s; a copy runs at 6.0) and taken back in 27.6 us (6.3 TB/s, some of it from the caches).
#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

// 8 values (a word of codes) per lane, 4 lanes per block, NW words in flight per lane.
// TILED: a workgroup has one slice (256 columns) of 8 NW rows, whose scale bytes are whole
// lines (otherwise each line of them is put together from 16 workgroups on several XCDs).
// Otherwise it has NW * 256 consecutive words of the matrix: rows that are short or end
// within a slice leave no lanes idle.
struct At {
    int64_t word, row;
    int col;  // of words
    bool has;
};
template <bool TILED, int NW>
struct Places {
    int64_t first, row0, all;
    int col0, words;
    float inv;
    __device__ __forceinline__ Places(int64_t rows, int words_) : all(rows * words_), words(words_) {
        if constexpr (TILED) {
            const unsigned slices = (words + 31) / 32;
            row0 = static_cast<int64_t>(blockIdx.x / slices) * (8 * NW);
            col0 = static_cast<int>(blockIdx.x % slices) * 32;
        } else {
            first = static_cast<int64_t>(blockIdx.x) * (NW * 256);
            row0 = first / words;
            col0 = static_cast<int>(first - row0 * words);
            inv = 1.f / static_cast<float>(words);
        }
    }
    __device__ __forceinline__ At operator()(int n) const {
        if constexpr (TILED) {
            const int64_t row = row0 + n * 8 + threadIdx.x / 32;
            const int col = col0 + threadIdx.x % 32;
            const int64_t word = row * words + col;
            return At{word, row, col, col < words && word < all};
        } else {
            // words per row below 2^17 + 1: the quotient in floats is off by one at most
            const int i = n * 256 + threadIdx.x;
            const int x = col0 + i;
            int q = static_cast<int>(static_cast<float>(x) * inv);
            int r = x - q * words;
            if (r < 0) {
                --q;
                r += words;
            } else if (r >= words) {
                ++q;
                r -= words;
            }
            return At{first + i, row0 + q, r, first + i < all};
        }
    }
};

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

template <typename T, bool TILED, int NW>
__global__ __launch_bounds__(256) void quant_rows_mxfp4_kernel(const T* __restrict__ src, int64_t rows, int cols,
                                                              uint32_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
    const int words = cols / 8, blocks = cols / 32;
    const Places<TILED, NW> places(rows, words);
    float v[NW][8];
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const At at = places(n);
        if (at.has) {  // (whole blocks are in or out)
            load8(src + at.word * 8, v[n]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[n][i] = 0.f;
        }
    }
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const At at = places(n);
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[n][i]) & 0x7fffffffu);
        m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0xB1, 0xf, 0xf, true)));
        m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x4E, 0xf, 0xf, true)));
        const bool finite = m < 0x7f800000u;
        const int byte = finite ? (m == 0 ? 127 : max(static_cast<int>(m >> 23) - 2, 0)) : 255;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = __builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[n][i], 127 - byte), -6.f, 6.f);
        uint32_t out = 0;
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, q[0], q[1], 1.f, 0);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, q[2], q[3], 1.f, 1);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, q[4], q[5], 1.f, 2);
        out = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(out, q[6], q[7], 1.f, 3);
        if (!at.has) continue;
        __builtin_nontemporal_store(finite ? out : 0u, codes + at.word);
        const int b = at.col / 4;
        uint8_t* const dst = scales + (static_cast<int64_t>(b / 8) * rows + at.row) * 8;
        if ((at.col & 3) == 0) {
            dst[b & 7] = static_cast<uint8_t>(byte);
            // the last slice's bytes past the row
            if (b == blocks - 1)
                for (int i = (b & 7) + 1; i < 8; ++i) dst[i] = 127;
        }
    }
}

template <typename O, bool TILED, int NW>
__global__ __launch_bounds__(256) void dequant_rows_mxfp4_kernel(const uint32_t* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t rows,
                                                                int cols, O* __restrict__ dst) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    const int words = cols / 8;
    const Places<TILED, NW> places(rows, words);
    uint32_t w[NW];
    int byte[NW];
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const At at = places(n);
        w[n] = 0;
        byte[n] = 127;
        if (at.has) {
            const int b = at.col / 4;
            w[n] = load_nt(codes + at.word);
            byte[n] = scales[(static_cast<int64_t>(b / 8) * rows + at.row) * 8 + (b & 7)];
        }
    }
#pragma unroll
    for (int n = 0; n < NW; ++n) {
        const At at = places(n);
        if (!at.has) continue;
        const f32x2_t p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[n], 1.f, 0),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[n], 1.f, 1),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[n], 1.f, 2),
                              __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[n], 1.f, 3)};
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = byte[n] == 255 ? __uint_as_float(0x7fc00000u) : __builtin_amdgcn_ldexpf(p[i / 2][i % 2], byte[n] - 127);
        if constexpr (sizeof(O) == 4) {
            float4* const out = reinterpret_cast<float4*>(dst + at.word * 8);
            out[0] = make_float4(v[0], v[1], v[2], v[3]);
            out[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(dst + at.word * 8) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                 pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
}

// Tiles for enough work (a fourth of the lanes idle at most), else one word per lane and
// consecutive words.
bool tiled(int64_t rows, int cols) {
    return rows * cols >= 8 * 1024 * 1024 && static_cast<int64_t>(align_up(cols, 256)) * 3 <= static_cast<int64_t>(cols) * 4;
}

template <int NW>
unsigned tiled_grid(int64_t rows, int cols) {
    return static_cast<unsigned>(ceil_div(rows, 8 * NW) * ceil_div(cols, 256));
}

}  // namespace

hipError_t launch_quant_rows_mxfp4(const void* src, int64_t rows, int cols, int dtype, void* codes, void* scales,
                                   hipStream_t s) {
    const int64_t words = rows * (cols / 8);
    uint32_t* const c = static_cast<uint32_t*>(codes);
    uint8_t* const sc = static_cast<uint8_t*>(scales);
    auto start = [&](auto from) {
        using T = decltype(from);
        const T* const in = static_cast<const T*>(src);
        if (tiled(rows, cols))
            quant_rows_mxfp4_kernel<T, true, 2><<<tiled_grid<2>(rows, cols), 256, 0, s>>>(in, rows, cols, c, sc);
        else
            quant_rows_mxfp4_kernel<T, false, 1><<<static_cast<unsigned>(ceil_div(words, 256)), 256, 0, s>>>(in, rows, cols, c, sc);
    };
    if (dtype == MOE_DTYPE_BF16) start(bf16_t{});
    else start(float{});
    return hipGetLastError();
}

hipError_t launch_dequant_rows_mxfp4(const void* codes, const void* scales, int64_t rows, int cols, int dtype,
                                     void* dst, hipStream_t s) {
    const int64_t words = rows * (cols / 8);
    const uint32_t* const c = static_cast<const uint32_t*>(codes);
    const uint8_t* const sc = static_cast<const uint8_t*>(scales);
    auto start = [&](auto to) {
        using O = decltype(to);
        O* const out = static_cast<O*>(dst);
        if (tiled(rows, cols))
            dequant_rows_mxfp4_kernel<O, true, 2><<<tiled_grid<2>(rows, cols), 256, 0, s>>>(c, sc, rows, cols, out);
        else
            dequant_rows_mxfp4_kernel<O, false, 1><<<static_cast<unsigned>(ceil_div(words, 256)), 256, 0, s>>>(c, sc, rows, cols, out);
    };
    if (dtype == MOE_DTYPE_BF16) start(bf16_t{});
    else start(float{});
    return hipGetLastError();
}

}  // namespace moe
