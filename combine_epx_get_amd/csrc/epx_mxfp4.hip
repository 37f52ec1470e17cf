// epx_mxfp4.hip -- rows of bf16 to MXFP4 and back (OCP Microscaling Formats:
// E2M1 codes, one power-of-two scale byte per 32 values).
//
// A block's scale is 2^(floor(log2(amax)) - 2): the exponent field of the
// largest magnitude, so it is found with integer maxima on the bf16 bits
// (magnitudes order as their bits do). Codes come from the packed hardware
// conversion, which divides by the (power of two) scale exactly, rounds to
// nearest even and saturates at 6; checked on every bf16 pattern.
// HBM bound: 2 + 17/32 bytes an element in either direction.
#include "epx_device.h"

namespace epx {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ bf16x2 bf16_pair(uint32_t w) { return __builtin_bit_cast(bf16x2, w); }

__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w)
{
    return max(m, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
}

// 2^(b - 127) as a float32, for b in 0 .. 254 (b = 0 is subnormal); NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t b)
{
    return b == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float(b == 0 ? 0x00400000u : b << 23);
}

// A lane takes 8 values (16 bytes in, 4 bytes of codes out), four lanes a
// block: reads and writes are contiguous over the wave.
__global__ __launch_bounds__(256) void quantize_kernel(const u32x4 *__restrict__ x, int64_t nvec,
                                                       uint32_t *__restrict__ codes,
                                                       uint8_t *__restrict__ scales)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < nvec; i += stride) {
        const u32x4 v = x[i];
        uint32_t m = max_magnitude(max_magnitude(max_magnitude(max_magnitude(0, v.x), v.y), v.z), v.w);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1, 4));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2, 4));
        // bf16's exponent field is biased by 127 like the scale byte; values
        // below 2^-125 take the smallest scale
        const uint32_t ex = m >> 7;
        const uint32_t b = ex == 255 ? 255 : ex > 2 ? ex - 2 : 0;
        uint32_t c = 0;
        if (b >= 8) {
            const float s = e8m0(b == 255 ? 127 : b);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(v.x), s, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(v.y), s, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(v.z), s, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, bf16_pair(v.w), s, 3);
        } else {
            const float s = e8m0(b + 100), up = 0x1p100f;
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v.x) * up, bf16_hi(v.x) * up, s, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v.y) * up, bf16_hi(v.y) * up, s, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v.z) * up, bf16_hi(v.z) * up, s, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, bf16_lo(v.w) * up, bf16_hi(v.w) * up, s, 3);
        }
        codes[i] = b == 255 ? 0u : c;
        if ((i & 3) == 0)
            scales[i >> 2] = (uint8_t)b;
    }
}

// bf16 bits of a code's magnitude times 2: codes 0..7 stand for 0, 1, 2, 3,
// 4, 6, 8, 12 halves.
__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t ex = (c >> 1) & 3, man = c & 1;
    const float mag = ex == 0 ? 0.5f * (float)man
                              : __uint_as_float(((ex + 126) << 23) | (man << 22));
    return (c & 8) ? -mag : mag;
}

__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t *__restrict__ codes,
                                                         const uint8_t *__restrict__ scales,
                                                         int64_t nvec, u32x4 *__restrict__ out)
{
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < nvec; i += stride) {
        const uint32_t c = codes[i];
        const float s = e8m0(scales[i >> 2]);
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            o[q] = f32_to_bf16(e2m1(c >> (8 * q)) * s) | (f32_to_bf16(e2m1(c >> (8 * q + 4)) * s) << 16);
        out[i] = o;
    }
}

inline dim3 flat_grid(int64_t nvec)
{
    const int64_t want = (nvec + 255) / 256;
    return dim3((unsigned)(want < 16384 ? want : 16384));
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void *x, int64_t num_rows, int32_t inner, uint8_t *codes,
                                 uint8_t *scales, hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    launch(quantize_kernel, flat_grid(nvec), dim3(256), 0, stream, (const u32x4 *)x, nvec,
           (uint32_t *)codes, scales);
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t num_rows,
                                   int32_t inner, void *out, hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    launch(dequantize_kernel, flat_grid(nvec), dim3(256), 0, stream, (const uint32_t *)codes,
           scales, nvec, (u32x4 *)out);
    return hipGetLastError();
}

}  // namespace epx
