// epx_mxfp4.hip -- rows of bf16 to MXFP4 and back (OCP Microscaling Formats:
// E2M1 codes, one power-of-two scale byte per 32 values).
//
// A block's scale is 2^(floor(log2(amax)) - 2): the exponent field of the
// largest magnitude, so it is found with integer maxima on the bf16 bits
// (magnitudes order as their bits do). Codes come from the packed hardware
// conversion, which divides by the (power of two) scale exactly, rounds to
// nearest even and saturates at 6; checked on every bf16 pattern.
// HBM bound: 2 + 17/32 bytes an element in either direction (65536 x 7168,
// both directions: 343-368 us, 6.5 to 6.9 TB/s; 2048 x 7168: 13.5 us).
#include "epx_device.h"
#include "epx_operators.h"

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

// A lane takes 8 values (16 bytes of bf16, 4 bytes of codes), four lanes a
// block: reads and writes are contiguous over the wave. kUnroll such pieces
// of a lane are loaded before the first is converted.
constexpr int kUnroll = 4, kThreads = 256;

__global__ __launch_bounds__(kThreads) void quantize_kernel(const u32x4 *__restrict__ x, int64_t nvec,
                                                            uint32_t *__restrict__ codes,
                                                            uint8_t *__restrict__ scales)
{
    const int64_t base = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x;
    u32x4 in[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (base + u * kThreads < nvec)
            in[u] = __builtin_nontemporal_load(x + base + u * kThreads);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        if (i >= nvec)
            return;   // whole blocks of four lanes: nvec is a multiple of 4
        const u32x4 v = in[u];
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

// A code's value: 0, 0.5, 1, 1.5, 2, 3, 4, 6, and negative from 8 on.
__device__ __forceinline__ float e2m1(uint32_t c)
{
    const uint32_t ex = (c >> 1) & 3, man = c & 1;
    const float mag = ex == 0 ? 0.5f * (float)man
                              : __uint_as_float(((ex + 126) << 23) | (man << 22));
    return (c & 8) ? -mag : mag;
}

__global__ __launch_bounds__(kThreads) void dequantize_kernel(const uint32_t *__restrict__ codes,
                                                              const uint8_t *__restrict__ scales,
                                                              int64_t nvec, u32x4 *__restrict__ out)
{
    const int64_t base = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x;
    uint32_t cs[kUnroll], bs[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        cs[u] = i < nvec ? codes[i] : 0u;
        bs[u] = i < nvec ? scales[i >> 2] : 127u;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        if (i >= nvec)
            return;
        const uint32_t c = cs[u], b = bs[u];
        u32x4 o;
        if (b >= 8 && b < 253) {
            // the packed hardware conversion, where no result is subnormal
            // or infinite
            const float s = __uint_as_float(b << 23);
            o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 0));
            o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 1));
            o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 2));
            o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, s, 3));
        } else {
            const float s = e8m0(b);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = f32_to_bf16(e2m1(c >> (8 * q)) * s) | (f32_to_bf16(e2m1(c >> (8 * q + 4)) * s) << 16);
        }
        __builtin_nontemporal_store(o, out + i);
    }
}

// Pieces a launch can take: grid x up to 2^31 - 1 workgroups, and fewer than
// 2^32 threads (2^24 workgroups of 256).
constexpr int64_t kMostPieces = ((int64_t)1 << 24) * kThreads * kUnroll - kThreads * kUnroll;

}  // namespace

hipError_t launch_mxfp4_quantize(const void *x, int64_t num_rows, int32_t inner, uint8_t *codes,
                                 uint8_t *scales, hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    for (int64_t at = 0; at < nvec; at += kMostPieces) {
        const int64_t n = nvec - at < kMostPieces ? nvec - at : kMostPieces;
        launch(quantize_kernel, dim3((unsigned)((n + kThreads * kUnroll - 1) / (kThreads * kUnroll))), dim3(kThreads),
               0, stream, (const u32x4 *)x + at, n, (uint32_t *)codes + at, scales + at / 4);
    }
    return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t num_rows,
                                   int32_t inner, void *out, hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    for (int64_t at = 0; at < nvec; at += kMostPieces) {
        const int64_t n = nvec - at < kMostPieces ? nvec - at : kMostPieces;
        launch(dequantize_kernel, dim3((unsigned)((n + kThreads * kUnroll - 1) / (kThreads * kUnroll))),
               dim3(kThreads), 0, stream, (const uint32_t *)codes + at, scales + at / 4, n, (u32x4 *)out + at);
    }
    return hipGetLastError();
}

}  // namespace epx
