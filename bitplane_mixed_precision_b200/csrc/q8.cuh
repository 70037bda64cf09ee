// q8 rows: e4m3 codes with one power-of-two scale (a byte, exponent + 127) per 32 columns.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace pmoe {
namespace q8 {

// Scale byte of a block whose largest magnitude has the float bits `top` (sign cleared; compared as
// integers, so that a NaN or an infinity is the largest): the least e >= -127 with
// amax <= 448 * 2^e. 448 = 1.75 * 2^8, so e = exponent - 8, one more above 1.75 * 2^exponent.
__host__ __device__ __forceinline__ uint32_t scale_byte(uint32_t top)
{
    const int ex = (int)(top >> 23);
    if (ex == 255)
        return 255u;
    const int e = ex - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    return e > 0 ? (uint32_t)e : 0u;
}

// 2^-e for a scale byte of a finite block (0..247): exact, never subnormal.
__device__ __forceinline__ float inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Four values of one block to codes (rounded to nearest even: e4m3 has 3 mantissa bits, an error of at
// most 2^-4 of the value). NaN blocks get the code of NaN throughout.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, uint32_t byte)
{
    if (byte == 255u)
        return 0x7f7f7f7fu;
    const float m = inverse(byte);
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * m, b * m), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * m, d * m), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t top4(float a, float b, float c, float d)
{
    return max(max(magnitude(a), magnitude(b)), max(magnitude(c), magnitude(d)));
}

// The largest over the 8 lanes (4 columns each) that hold one block.
__device__ __forceinline__ uint32_t top_of_8_lanes(uint32_t top)
{
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 4));
}

} // namespace q8
} // namespace pmoe
