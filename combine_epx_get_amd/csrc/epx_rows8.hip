// epx_rows8.hip -- rows of bf16 in 8 bits and back: int8 with a float32 scale
// per row, and blocks of 32 int8 under a power of two (OCP Microscaling
// Formats: MXINT8).
//
// HBM bound: 3 bytes an element in either direction, and the scales (32768 x
// 7168, both directions: int8 217 us, MXINT8 213, 6.5 and 6.7 TB/s; a large copy
// has 5.2). A row of int8 stays in its lanes' registers between the maximum and
// the conversion, up to 32768 values; a longer one is read again. Small batches
// are as long as their two calls (128 x 7168: 3.6 and 4.0 us of kernels, 8.7 with
// both calls from Python).
#include "epx_device.h"
#include "epx_rows8.h"
#include "epx_operators.h"

namespace epx {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t w)
{
    return max(m, max(w & 0x7FFFu, (w >> 16) & 0x7FFFu));
}

// ---------------------------------------------------------------- int8 rows
// s = max(fl32(amax / 127), 2^-125), codes the nearest integers of the exact
// quotients x / s, ties to even. The product q with the rounded reciprocal can
// land on the wrong side of a tie between two integers, so its floor f only
// names the tie f + 1/2, and the sign of x - (f + 1/2) s, which one fma gives
// exactly, decides: a quarter is added to the tie or taken off it (nothing at
// a tie), and the sum rounded. (f itself may be off by one where q is near an
// integer; the tie it names then still has x / s on the right side.)
struct RowScale {
    float s, inv;
    __device__ __forceinline__ explicit RowScale(float amax)
    {
        s = amax > 0.0f ? fmaxf(amax / 127.0f, 0x1p-125f) : 0.0f;
        inv = s > 0.0f ? 1.0f / s : 0.0f;
    }
    // The integer in the low 8 bits.
    __device__ __forceinline__ uint32_t code(float x) const
    {
        const float tie = floorf(x * inv) + 0.5f;
        const float d = __builtin_fmaf(-tie, s, x);
        // d is 0 or at least half a step of the float32 scale: 2^-25 s, and a
        // float32 number (2^-149 at least) because s is 2^-125 at least
        const float side = __builtin_amdgcn_fmed3f(d * inv * 0x1p24f, -0.25f, 0.25f);
        return int_bits(tie + side);
    }
};

// Rows of nvec pieces of 8 values (16 bytes), LANES lanes a row, kHold pieces
// of a lane kept in registers between the maximum and the conversion; longer
// rows are read again. A row's lanes are neighbours in a wave, or the whole
// workgroup.
constexpr int kHold = 4;

template <int LANES>
__global__ __launch_bounds__(LANES > kThreads ? LANES : kThreads)
void int8_quantize_kernel(const u32x4 *__restrict__ x, int64_t rows, int32_t nvec, u32x2 *__restrict__ codes,
                          float *__restrict__ scales)
{
    constexpr int kBlock = LANES > kThreads ? LANES : kThreads, kRows = kBlock / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t row = item_index() * kRows + threadIdx.x / LANES;
    const bool live = row < rows;   // the same for a row's lanes
    if (LANES >= kThreads && !live)
        return;
    const u32x4 *in = x + row * nvec;
    u32x4 v[kHold];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
        const int i = u * LANES + lane;
        if (live && i < nvec)
            v[u] = __builtin_nontemporal_load(in + i);
        else
            v[u] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kHold; ++u)
        m = max_magnitude(max_magnitude(max_magnitude(max_magnitude(m, v[u].x), v[u].y), v[u].z), v[u].w);
    if (live)
        for (int i = kHold * LANES + lane; i < nvec; i += LANES) {
            const u32x4 w = in[i];
            m = max_magnitude(max_magnitude(max_magnitude(max_magnitude(m, w.x), w.y), w.z), w.w);
        }
#pragma unroll
    for (int d = 1; d < (LANES < kWave ? LANES : kWave); d *= 2)
        m = max(m, (uint32_t)__shfl_xor((int)m, d, kWave));
    if constexpr (LANES > kWave) {
        __shared__ uint32_t part[LANES / kWave];
        if (threadIdx.x % kWave == 0)
            part[threadIdx.x / kWave] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < LANES / kWave; ++i)
            m = max(m, part[i]);
    }
    if (!live)
        return;
    // an infinity or NaN: the row's scale is NaN, its codes 0
    const bool odd = m >= 0x7F80u;
    const RowScale q(odd ? 0.0f : __uint_as_float(m << 16));
    u32x2 *out = codes + row * nvec;
    auto convert = [&](u32x4 w) {
        u32x2 c;
        c.x = pack4(q.code(bf16_lo(w.x)), q.code(bf16_hi(w.x)), q.code(bf16_lo(w.y)), q.code(bf16_hi(w.y)));
        c.y = pack4(q.code(bf16_lo(w.z)), q.code(bf16_hi(w.z)), q.code(bf16_lo(w.w)), q.code(bf16_hi(w.w)));
        return odd || m == 0 ? u32x2{0, 0} : c;
    };
#pragma unroll
    for (int u = 0; u < kHold; ++u) {
        const int i = u * LANES + lane;
        if (i < nvec)
            out[i] = convert(v[u]);
    }
    for (int i = kHold * LANES + lane; i < nvec; i += LANES)
        out[i] = convert(in[i]);
    if (lane == 0)
        scales[row] = odd ? __uint_as_float(0x7FC00000u) : q.s;
}

// bf16(code * scale), rounded once.
template <int LANES>
__global__ __launch_bounds__(LANES > kThreads ? LANES : kThreads)
void int8_dequantize_kernel(const u32x2 *__restrict__ codes, const float *__restrict__ scales, int64_t rows,
                            int32_t nvec, u32x4 *__restrict__ out)
{
    constexpr int kBlock = LANES > kThreads ? LANES : kThreads, kRows = kBlock / LANES;
    const int lane = threadIdx.x % LANES;
    const int64_t row = item_index() * kRows + threadIdx.x / LANES;
    if (row >= rows)
        return;
    const u32x2 *in = codes + row * nvec;
    u32x4 *to = out + row * nvec;
    const float s = scales[row];
    auto convert = [&](u32x2 c) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t half = i < 2 ? c.x : c.y;
            w[i] = f32_to_bf16(signed_byte(half, i % 2 * 2) * s) | (f32_to_bf16(signed_byte(half, i % 2 * 2 + 1) * s) << 16);
        }
        return w;
    };
    u32x2 v[kHold];
#pragma unroll
    for (int u = 0; u < kHold; ++u)
        v[u] = u * LANES + lane < nvec ? in[u * LANES + lane] : u32x2{0, 0};
#pragma unroll
    for (int u = 0; u < kHold; ++u)
        if (u * LANES + lane < nvec)
            __builtin_nontemporal_store(convert(v[u]), to + u * LANES + lane);
    for (int i = kHold * LANES + lane; i < nvec; i += LANES)
        __builtin_nontemporal_store(convert(in[i]), to + i);
}

// Lanes a row: the fewest that hold it in registers, so that a row is read
// once and short rows leave no lanes idle.
template <typename F> hipError_t by_row_length(int32_t nvec, int64_t rows, F start)
{
    auto go = [&](auto lanes) {
        constexpr int L = decltype(lanes)::value, kRows = L > kThreads ? 1 : kThreads / L;
        start(lanes, item_grid((rows + kRows - 1) / kRows, 1), dim3(L > kThreads ? L : kThreads));
        return hipGetLastError();
    };
    if (nvec <= 4 * kHold)
        return go(std::integral_constant<int, 4>{});
    if (nvec <= 16 * kHold)
        return go(std::integral_constant<int, 16>{});
    if (nvec <= 64 * kHold)
        return go(std::integral_constant<int, 64>{});
    if (nvec <= 256 * kHold)
        return go(std::integral_constant<int, 256>{});
    return go(std::integral_constant<int, 1024>{});
}

// ---------------------------------------------------------------- MXINT8
// As the MXFP4 conversion: a lane takes 8 values, four lanes a block, kUnroll
// pieces of a lane are loaded before the first is converted.
constexpr int kUnroll = 4;

__global__ __launch_bounds__(kThreads) void mxint8_quantize_kernel(const u32x4 *__restrict__ x, int64_t nvec,
                                                                   u32x2 *__restrict__ codes,
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
        const uint32_t b = m >> 7;   // bf16's exponent field is biased like the scale byte
        const float f[8] = {bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y),
                            bf16_lo(v.z), bf16_hi(v.z), bf16_lo(v.w), bf16_hi(v.w)};
        codes[i] = mxint8_codes(f, b);
        if ((i & 3) == 0)
            scales[i >> 2] = (uint8_t)b;
    }
}

__global__ __launch_bounds__(kThreads) void mxint8_dequantize_kernel(const u32x2 *__restrict__ codes,
                                                                     const uint8_t *__restrict__ scales,
                                                                     int64_t nvec, u32x4 *__restrict__ out)
{
    const int64_t base = (int64_t)blockIdx.x * kThreads * kUnroll + threadIdx.x;
    u32x2 cs[kUnroll];
    uint32_t bs[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        cs[u] = i < nvec ? codes[i] : u32x2{0, 0};
        bs[u] = i < nvec ? scales[i >> 2] : 127u;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const int64_t i = base + u * kThreads;
        if (i >= nvec)
            return;
        const float step = mxint8_step(bs[u]);
        const u32x2 lo = mxint8_bf16(cs[u].x, step), hi = mxint8_bf16(cs[u].y, step);
        __builtin_nontemporal_store(u32x4{lo.x, lo.y, hi.x, hi.y}, out + i);
    }
}

// Pieces a launch can take: fewer than 2^32 threads.
constexpr int64_t kMostPieces = ((int64_t)1 << 24) * kThreads * kUnroll - kThreads * kUnroll;

dim3 piece_grid(int64_t n) { return dim3((unsigned)((n + kThreads * kUnroll - 1) / (kThreads * kUnroll))); }

}  // namespace

hipError_t launch_int8_quantize(const void *x, int64_t num_rows, int32_t inner, int8_t *codes, float *scales,
                                hipStream_t stream)
{
    return by_row_length(inner / 8, num_rows, [&](auto lanes, dim3 grid, dim3 block) {
        launch(int8_quantize_kernel<decltype(lanes)::value>, grid, block, 0, stream, (const u32x4 *)x, num_rows,
               inner / 8, (u32x2 *)codes, scales);
    });
}

hipError_t launch_int8_dequantize(const int8_t *codes, const float *scales, int64_t num_rows, int32_t inner,
                                  void *out, hipStream_t stream)
{
    return by_row_length(inner / 8, num_rows, [&](auto lanes, dim3 grid, dim3 block) {
        launch(int8_dequantize_kernel<decltype(lanes)::value>, grid, block, 0, stream, (const u32x2 *)codes, scales,
               num_rows, inner / 8, (u32x4 *)out);
    });
}

hipError_t launch_mxint8_quantize(const void *x, int64_t num_rows, int32_t inner, int8_t *codes, uint8_t *scales,
                                  hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    for (int64_t at = 0; at < nvec; at += kMostPieces) {
        const int64_t n = nvec - at < kMostPieces ? nvec - at : kMostPieces;
        launch(mxint8_quantize_kernel, piece_grid(n), dim3(kThreads), 0, stream, (const u32x4 *)x + at, n,
               (u32x2 *)codes + at, scales + at / 4);
    }
    return hipGetLastError();
}

hipError_t launch_mxint8_dequantize(const int8_t *codes, const uint8_t *scales, int64_t num_rows, int32_t inner,
                                    void *out, hipStream_t stream)
{
    const int64_t nvec = num_rows * (inner / 8);
    for (int64_t at = 0; at < nvec; at += kMostPieces) {
        const int64_t n = nvec - at < kMostPieces ? nvec - at : kMostPieces;
        launch(mxint8_dequantize_kernel, piece_grid(n), dim3(kThreads), 0, stream, (const u32x2 *)codes + at,
               scales + at / 4, n, (u32x4 *)out + at);
    }
    return hipGetLastError();
}

}  // namespace epx
