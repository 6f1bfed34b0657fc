// fp8.cuh -- block-scaled e4m3 values: the scale of a block and the
// conversion, shared by the quantisation kernels and the expert GEMM's
// epilogue.
//
// A block holds q = e4m3(x / s) with s the smallest power of two for which
// max |x| <= 448 s (448 is e4m3's largest value), at least 2^-126.  With a
// power of two x / s is exact, so the only rounding is e4m3's own (half a
// step is 2^-4 of a value), and a scale that lands one step higher because
// max |x| was computed with another rounding changes no value above the
// subnormal range.  A block that holds a NaN or an infinity gets a NaN scale
// and NaN values throughout.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moe {

constexpr int kFp8Block = 128;

__host__ __device__ __forceinline__ int fp8_blocks(int64_t n) { return static_cast<int>((n + kFp8Block - 1) / kFp8Block); }

// |x| as an integer that orders like the value; NaN lies above infinity.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The scale for a block whose largest |x| has these bits, and 1 / scale
// (both NaN for a block that is not finite).  448 = 1.75 * 2^8: adding
// 0x1FFFFF to the bits carries into the exponent exactly when the mantissa
// is above 1.75, and the exponent less 8 is the scale's.
__device__ __forceinline__ float2 fp8_scale(uint32_t amax)
{
    if (amax >= 0x7F800000u) return make_float2(__uint_as_float(0x7FC00000u), __uint_as_float(0x7FC00000u));
    const uint32_t ex = max((amax + 0x1FFFFFu) >> 23, 9u) - 8u;
    return make_float2(__uint_as_float(ex << 23), __uint_as_float((254u - ex) << 23));
}

// Two values to e4m3, round to nearest even; `lo` in the low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t cvt_e4m3x4(float a, float b, float c, float d)
{
    return cvt_e4m3x2(a, b) | (cvt_e4m3x2(c, d) << 16);
}

}  // namespace moe
