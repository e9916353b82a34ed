// 8-bit integer codes of a matrix's rows, one float32 scale per row:
//   scale = max(amax / 127, 2^-126), code = rint(x / scale)
// (1 for an all-zero row; NaN and codes 0 for a row with a NaN or infinity).
// The scale floor keeps a row of subnormal values from a scale of zero.
// Both quotients are IEEE divisions, so the codes are a function of the row
// alone that any float32 host reproduces bit for bit; |x| / scale is at most
// 127 (1 + 2^-23), which rounds to 127.
#include "device_util.h"
#include "moe_internal.h"

namespace moe {

namespace {

// One workgroup per row, the row read twice.
template <typename T>
__global__ __launch_bounds__(256) void quant_rows_int8_kernel(const T* __restrict__ src, int cols,
                                                             int8_t* __restrict__ codes, float* __restrict__ scales) {
    __shared__ uint32_t s_max[4];
    const int64_t r = blockIdx.x;
    const T* row = src + r * cols;
    auto at = [&](int c) -> float {
        if constexpr (sizeof(T) == 2) return bf16_to_f32(row[c]);
        else return row[c];
    };
    // |x| as its bit pattern: integer order is the values' order, with
    // infinities and NaNs above every finite value
    uint32_t m = 0;
    for (int c = threadIdx.x; c < cols; c += 256) m = max(m, __float_as_uint(at(c)) & 0x7fffffffu);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), off, 64)));
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
    const bool finite = m < 0x7f800000u;
    const float scale = !finite ? __uint_as_float(0x7fc00000u)
                                : (m == 0 ? 1.f : fmaxf(__uint_as_float(m) / 127.f, 0x1p-126f));
    if (threadIdx.x == 0) scales[r] = scale;
    for (int c = threadIdx.x; c < cols; c += 256)
        codes[r * cols + c] = finite ? static_cast<int8_t>(static_cast<int>(rintf(at(c) / scale))) : int8_t{0};
}

}  // namespace

hipError_t launch_quant_rows_int8(const void* src, int64_t rows, int cols, int dtype, void* codes, float* scales,
                                  hipStream_t s) {
    const unsigned g = static_cast<unsigned>(rows);
    if (dtype == MOE_DTYPE_BF16)
        quant_rows_int8_kernel<<<g, 256, 0, s>>>(static_cast<const bf16_t*>(src), cols, static_cast<int8_t*>(codes),
                                                 scales);
    else
        quant_rows_int8_kernel<<<g, 256, 0, s>>>(static_cast<const float*>(src), cols, static_cast<int8_t*>(codes),
                                                 scales);
    return hipGetLastError();
}

}  // namespace moe
