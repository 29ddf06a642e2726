// mx8.cuh -- 8-bit data in blocks: 32 e4m3 values along the contracted axis
// share one power-of-two scale 2^(byte - 127) (byte 255: NaN), the operand form
// of the tensor cores' block-scaled MMA.
//
// The scale of a block is the least 2^e with max|v| <= 448 * 2^e, 448 = 1.75 *
// 2^8 the largest e4m3 value: no element saturates, and e follows from the
// maximum's own exponent and mantissa bits, without a logarithm.  A block of
// zeros has byte 0.  A block that holds an infinity or a NaN has no such scale:
// its byte is 255 and its elements are e4m3 NaN, so that the fault stays
// visible instead of turning into a finite number.
#pragma once
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

constexpr int kMxBlock = 32;

// Scale byte of a block whose largest |v| has these fp32 bits (NaN and infinity
// compare above every finite value as integers).
MOE_DEVICE uint32_t mx_scale_byte(uint32_t amax_bits)
{
    const uint32_t ex = amax_bits >> 23;
    if (ex == 255u) return 255u;
    const int b = (int)ex - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b > 0 ? (uint32_t)b : 0u;
}

// 2^(127 - byte), the factor onto the e4m3 grid (byte <= 247 from mx_scale_byte:
// exact and normal); NaN for byte 255.
MOE_DEVICE float mx_inv_scale(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); 2^-127 is below the normal range.
MOE_DEVICE float mx_scale(uint32_t byte)
{
    if (byte == 255u) return __uint_as_float(0x7fc00000u);
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// Four values onto the grid, round to nearest even (first value in the low byte).
// Each rounding is at most half an e4m3 step, 2^-4 of the value.
MOE_DEVICE uint32_t mx_pack4(float a, float b, float c, float d, float inv)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

MOE_DEVICE float e4m3_to_f32(uint32_t byte)
{
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
}

MOE_DEVICE uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

}  // namespace moe
