// epx_rows8.h -- values in 8 bits, as the conversions and the experts'
// products use them (internal).
//
// MXINT8: 32 neighbouring values share a scale byte b; a value is its int8
// code times the step 2^(b - 127 - 6). Codes have 7 bits and a sign, so every
// value is exactly a bf16 number.
#pragma once

#include "epx_device.h"
#include "epx_operators.h"

namespace epx {

// v rounded to the nearest integer, ties to even, in the low 8 bits of the
// result (|v| <= 127): adding 1.5 * 2^23 leaves the integer in the last bits
// of the float32.
__device__ __forceinline__ uint32_t int_bits(float v) { return __float_as_uint(v + 12582912.0f); }

// The low bytes of four words, the first one's lowest.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u), hi = __builtin_amdgcn_perm(d, c, 0x04000C0Cu);
    return lo | hi;
}

// Byte `i` of w as a signed number.
__device__ __forceinline__ float signed_byte(uint32_t w, int i) { return (float)(int8_t)(w >> (8 * i)); }

// The step of scale byte b: 2^(b - 133), subnormal below b = 7; NaN for 255.
__device__ __forceinline__ float mxint8_step(uint32_t b)
{
    const float s = __builtin_amdgcn_ldexpf(1.0f, (int)b - 133);
    return b == 255 ? __uint_as_float(0x7FC00000u) : s;
}

// The codes of 8 values of a block whose scale byte is b (the exponent field
// of its largest magnitude; 255, an infinity or NaN: codes 0). The division by
// a power of two is exact, and below 2^-126 what ldexp rounds is far below
// half a step. (One fma in place of ldexp and the addition needs a second way
// for b below 7, whose registers cost the forward product more than it saves:
// 1600 against 1577 us.)
__device__ __forceinline__ u32x2 mxint8_codes(const float (&v)[8], uint32_t b)
{
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        c[i] = int_bits(__builtin_amdgcn_fmed3f(__builtin_amdgcn_ldexpf(v[i], 133 - (int)b), -127.0f, 127.0f));
    const u32x2 o = {pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7])};
    return b == 255 ? u32x2{0, 0} : o;
}

// 4 codes times their step, as bf16: the products are bf16 numbers, so their
// upper halves are all there is.
__device__ __forceinline__ u32x2 mxint8_bf16(uint32_t c, float step)
{
    u32x2 w;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __builtin_amdgcn_perm(__float_as_uint(signed_byte(c, 2 * i + 1) * step),
                                     __float_as_uint(signed_byte(c, 2 * i) * step), 0x07060302u);
    return w;
}

}  // namespace epx
