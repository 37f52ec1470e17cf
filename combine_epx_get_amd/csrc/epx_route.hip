// epx_route.hip -- the router's choice on gfx950: scores -> topk_idx and
// topk_weights, and the gradient of the weights.
//
// L lanes (half a wave up to 256 experts, else a wave) work on one token. Lane
// l of them holds the PER consecutive logits from l * PER on, so that expert
// order is (lane, place in the lane) order: the lowest lane whose best key
// equals the token's best key holds the lowest id, and a tie needs no
// comparison of ids. Keys are the order-preserving integers of the logits (32
// bits), or of score + bias in double precision (64 bits: two biased scores
// can be nearer to each other than float32 tells). Up to 8 places a lane are
// sorted once; each of the k rounds is then a maximum over the lanes' first
// keys (DPP), a ballot, and in the winning lane a move up. Key 0 marks a taken
// or absent place and key 1 a masked expert (-infinity or NaN); every other
// key is larger.
//
// Bound by instruction issue from a few thousand tokens on (16384 tokens, 256
// experts, top-8, float32: 9.8 us, 1.7 TB/s; the gradient about as long, 3.4
// TB/s), by launch latency below (128 tokens: 6.9 us a call).
#include "epx_device.h"

namespace epx {
namespace {

constexpr uint32_t kTaken = 0, kMasked = 1;

// Order-preserving integer of a number that is neither NaN nor -infinity
// (those have smaller values than any of these); -0 counts as +0.
__device__ __forceinline__ uint32_t sortable(float f)
{
    const uint32_t u = __float_as_uint(f + 0.0f);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t sortable(double f)
{
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

__device__ __forceinline__ float wave_sum(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ float wave_maxf(float v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor(v, d, kWave));
    return v;
}
__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1)
        v += __shfl_xor(v, d, kWave);
    return v;
}

__device__ __forceinline__ bool masked(float l) { return !(l > -__builtin_inff()); }

template <typename TIn> struct Row;
template <> struct Row<float> {
    static __device__ __forceinline__ float get(const float *p) { return *p; }
};
template <> struct Row<uint16_t> {
    static __device__ __forceinline__ float get(const uint16_t *p)
    {
        return __uint_as_float((uint32_t)*p << 16);
    }
};

// The lane's logits (-infinity behind the last expert). `whole`: E is a
// multiple of PER, so a lane's places are all in or all out and its loads
// are aligned to their size.
template <typename TIn, int PER>
__device__ __forceinline__ void load_row(const TIn *row, int lane, int E, bool whole, float (&l)[PER])
{
    const int at = lane * PER;
    if (whole) {
        struct alignas(PER * sizeof(TIn) < 16 ? PER * sizeof(TIn) : 16) Pack { TIn v[PER]; };
        Pack p;
        if (at < E)
            p = *(const Pack *)(row + at);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            l[i] = at < E ? Row<TIn>::get(&p.v[i]) : -__builtin_inff();
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            l[i] = at + i < E ? Row<TIn>::get(row + at + i) : -__builtin_inff();
    }
}

// 1 / (1 + exp(-l)) in double: only the chosen experts' scores, and the keys
// of a biased choice, are computed this way.
__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }

// exp(l - m) with m the row's maximum; a row of +infinities counts them alike.
__device__ __forceinline__ float exp_to(float l, float m)
{
    return masked(l) ? 0.0f : l == m ? 1.0f : expf(l - m);
}

// Maximum over the L lanes of a token.
template <int L> __device__ __forceinline__ uint32_t token_max(uint32_t v)
{
    v = max(v, (uint32_t)dpp<kDppRowShr + 1>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 2>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 4>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 8>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowBcast15, 0xa, false>((int)v));
    if (L == 32) {
        const int low = __builtin_amdgcn_readlane((int)v, 31), high = __builtin_amdgcn_readlane((int)v, 63);
        return (uint32_t)(lane_id() < 32 ? low : high);
    }
    v = max(v, (uint32_t)dpp<kDppRowBcast31, 0xc, false>((int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}

template <int L, typename T> __device__ __forceinline__ T token_sum(T v)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1)
        v += __shfl_xor(v, d, L);
    return v;
}
template <int L> __device__ __forceinline__ float token_maxf(float v)
{
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1)
        v = fmaxf(v, __shfl_xor(v, d, L));
    return v;
}

template <typename TIn, int PER, int L, bool BIASED>
__global__ __launch_bounds__(256) void route_kernel(const TIn *__restrict__ logits, int64_t T, int E,
                                                    int k, bool softmax,
                                                    const float *__restrict__ bias,
                                                    bool renormalize, float scale,
                                                    int32_t *__restrict__ idx,
                                                    float *__restrict__ weights)
{
    constexpr int kTokens = 256 / L;   // of a workgroup
    constexpr bool kSorted = PER <= 8;
    __shared__ int32_t s_pick[kTokens][kMaxTopk];
    const int tok = threadIdx.x / L, lane = threadIdx.x % L, at = lane * PER;
    const int64_t t_own = (int64_t)blockIdx.x * kTokens + tok, t = t_own < T ? t_own : T - 1;
    const TIn *row = logits + t * E;
    float l[PER];
    load_row<TIn, PER>(row, lane, E, E % PER == 0, l);
    uint32_t hi[PER], lo[BIASED ? PER : 1];
    int id[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = at + i < E;
        id[i] = at + i;
        if (BIASED) {
            const double key = in ? sigmoid64(l[i]) + (double)bias[at + i] : 0.0;
            // a NaN or -infinity bias masks like such a logit
            const bool none = masked(l[i]) || !(key > -__builtin_inf());
            const uint64_t s = sortable(key);
            hi[i] = !in ? kTaken : none ? kMasked : (uint32_t)(s >> 32);
            lo[i] = !in || none ? 0u : (uint32_t)s;
        } else {
            hi[i] = !in ? kTaken : masked(l[i]) ? kMasked : sortable(l[i]);
        }
    }
    if (kSorted) {
        // exchanges of neighbours only: equal keys keep the order of ids
#pragma unroll
        for (int end = PER - 1; end > 0; --end)
#pragma unroll
            for (int i = 0; i < end; ++i) {
                const bool up = BIASED ? hi[i + 1] > hi[i] || (hi[i + 1] == hi[i] && lo[i + 1] > lo[i])
                                       : hi[i + 1] > hi[i];
                const uint32_t h = hi[i];
                const int n = id[i];
                hi[i] = up ? hi[i + 1] : h;
                hi[i + 1] = up ? h : hi[i + 1];
                id[i] = up ? id[i + 1] : n;
                id[i + 1] = up ? n : id[i + 1];
                if (BIASED) {
                    const uint32_t w = lo[i];
                    lo[i] = up ? lo[i + 1] : w;
                    lo[i + 1] = up ? w : lo[i + 1];
                }
            }
    }

    for (int j = 0; j < k; ++j) {
        uint32_t bh = hi[0], bl = BIASED ? lo[0] : 0u;
        int bi = 0;
        if (!kSorted) {
#pragma unroll
            for (int i = 1; i < PER; ++i) {
                const bool better = BIASED ? hi[i] > bh || (hi[i] == bh && lo[i] > bl) : hi[i] > bh;
                bh = better ? hi[i] : bh;
                if (BIASED)
                    bl = better ? lo[i] : bl;
                bi = better ? i : bi;
            }
        }
        bool best = bh == token_max<L>(bh);
        if (BIASED) {
            const uint32_t wl = token_max<L>(best ? bl : 0u);
            best = best && bl == wl;
        }
        // the lowest lane of each token
        uint64_t win = __ballot(best);
        if (L == 32)
            win = ((uint32_t)win & -(uint32_t)win) | ((uint64_t)((uint32_t)(win >> 32) & -(uint32_t)(win >> 32)) << 32);
        else
            win &= -win;
        if ((win >> lane_id()) & 1) {
            if (kSorted) {
                s_pick[tok][j] = id[0];
#pragma unroll
                for (int i = 0; i + 1 < PER; ++i) {
                    hi[i] = hi[i + 1];
                    id[i] = id[i + 1];
                    if (BIASED)
                        lo[i] = lo[i + 1];
                }
                hi[PER - 1] = kTaken;
            } else {
                s_pick[tok][j] = at + bi;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    if (i == bi)
                        hi[i] = kTaken;
            }
        }
    }
    __syncthreads();

    // weights: lane q of a token takes choices q, q + L
    float m = -__builtin_inff(), sum = 0.0f;
    if (softmax && !renormalize) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            m = fmaxf(m, l[i]);
        m = token_maxf<L>(m);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += exp_to(l[i], m);
        sum = token_sum<L>(sum);
    }
    constexpr int kMine = kMaxTopk / L;
    float c[kMine];
    double p[kMine], all = 0.0;
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
        const int j = lane + x * L;
        c[x] = j < k ? Row<TIn>::get(row + s_pick[tok][j]) : -__builtin_inff();
    }
    if (softmax && renormalize) {
#pragma unroll
        for (int x = 0; x < kMine; ++x)
            m = fmaxf(m, c[x]);
        m = token_maxf<L>(m);
#pragma unroll
        for (int x = 0; x < kMine; ++x)
            sum += exp_to(c[x], m);
        sum = token_sum<L>(sum);
    }
    if (!softmax) {
#pragma unroll
        for (int x = 0; x < kMine; ++x) {
            p[x] = lane + x * L < k && !masked(c[x]) ? sigmoid64(c[x]) : 0.0;
            all += p[x];
        }
        all = renormalize ? token_sum<L>(all) : 1.0;
    }
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
        const int j = lane + x * L;
        if (j < k && t_own < T) {
            idx[t * k + j] = s_pick[tok][j];
            weights[t * k + j] = softmax ? (sum > 0.0f ? scale * (exp_to(c[x], m) / sum) : 0.0f)
                                         : (all > 0.0 ? scale * (float)(p[x] / all) : 0.0f);
        }
    }
}

// dlogits of one token; lane j < k holds (id, score, dweight) of choice j.
template <typename TIn, int PER>
__global__ __launch_bounds__(256) void route_backward_kernel(
    const TIn *__restrict__ logits, int64_t T, int E, int k, bool softmax, bool renormalize,
    float scale, const int32_t *__restrict__ idx, const float *__restrict__ dweights,
    TIn *__restrict__ dlogits)
{
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T)
        return;
    const int lane = lane_id(), at = lane * PER;
    const TIn *row = logits + t * E;
    int e = -1;
    float g = 0.0f, le = -__builtin_inff();
    if (lane < k) {
        e = idx[t * k + lane];
        if (e < 0 || e >= E)
            e = -1;
        else {
            le = Row<TIn>::get(row + e);
            g = scale * dweights[t * k + lane];
        }
    }
    float d[PER];   // every expert's gradient before the chosen ones' part
#pragma unroll
    for (int i = 0; i < PER; ++i)
        d[i] = 0.0f;
    float c;        // the chosen expert's part
    if (softmax && !renormalize) {
        float l[PER];
        load_row<TIn, PER>(row, lane, E, E % PER == 0, l);
        float m = -__builtin_inff(), sum = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            m = fmaxf(m, l[i]);
        m = wave_maxf(m);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += exp_to(l[i], m);
        sum = wave_sum(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float p = exp_to(le, m) * inv;
        c = e >= 0 ? g * p : 0.0f;
        const float all = wave_sum(c);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] = -(exp_to(l[i], m) * inv) * all;
    } else if (softmax) {
        const float m = wave_maxf(le);
        const float x = e >= 0 ? exp_to(le, m) : 0.0f;
        const float sum = wave_sum(x);
        const float p = sum > 0.0f ? x / sum : 0.0f;
        const float mean = wave_sum(e >= 0 ? g * p : 0.0f);
        c = e >= 0 ? p * (g - mean) : 0.0f;
    } else {
        // 1 - p is formed as 1 / (1 + exp(l)): p alone loses it near 1
        const bool on = e >= 0 && !masked(le);
        const double p = on ? sigmoid64(le) : 0.0, q = on ? 1.0 / (1.0 + exp((double)le)) : 0.0;
        if (renormalize) {
            const double sum = wave_sum(p);
            const double r = sum > 0.0 ? p / sum : 0.0;
            const double mean = wave_sum(on ? (double)g * r : 0.0);
            c = on ? (float)(r * ((double)g - mean) * q) : 0.0f;
        } else {
            c = on ? (float)((double)g * p * q) : 0.0f;
        }
    }
    for (int j = 0; j < k; ++j) {   // in order: an id given twice counts twice
        const int ej = __builtin_amdgcn_readlane(e, j);
        const float cj = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(c), j));
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at + i == ej)
                d[i] += cj;
    }
    TIn *out = dlogits + t * E;
    struct alignas(PER * sizeof(TIn) < 16 ? PER * sizeof(TIn) : 16) Pack { TIn v[PER]; };
    Pack o;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if constexpr (sizeof(TIn) == 4)
            o.v[i] = d[i];
        else
            o.v[i] = (uint16_t)f32_to_bf16(d[i]);
    }
    if (E % PER == 0) {
        if (at < E)
            *(Pack *)(out + at) = o;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at + i < E)
                out[at + i] = o.v[i];
    }
}

// Places per lane for E experts: the smallest power of two with 64 lanes.
template <typename F> void with_per(int E, F f)
{
    if (E <= 64)
        f(std::integral_constant<int, 1>());
    else if (E <= 128)
        f(std::integral_constant<int, 2>());
    else if (E <= 256)
        f(std::integral_constant<int, 4>());
    else if (E <= 512)
        f(std::integral_constant<int, 8>());
    else if (E <= 1024)
        f(std::integral_constant<int, 16>());
    else
        f(std::integral_constant<int, 32>());
}

}  // namespace

hipError_t launch_route(const Geometry &g, const void *logits, bool bf16, bool softmax,
                        const float *bias, bool renormalize, float scale, int32_t *idx,
                        float *weights, hipStream_t stream)
{
    auto with_shape = [&](auto per, auto lanes) {
        constexpr int P = decltype(per)::value, L = decltype(lanes)::value;
        const dim3 grid((unsigned)((g.T + 256 / L - 1) / (256 / L)));
        auto go = [&](auto *row, auto biased) {
            using TIn = std::remove_pointer_t<decltype(row)>;
            launch(route_kernel<TIn, P, L, decltype(biased)::value>, grid, dim3(256), 0, stream,
                   (const TIn *)logits, (int64_t)g.T, g.E, g.k, softmax, bias, renormalize, scale,
                   idx, weights);
        };
        if (bf16 && bias)
            go((uint16_t *)nullptr, std::true_type());
        else if (bf16)
            go((uint16_t *)nullptr, std::false_type());
        else if (bias)
            go((float *)nullptr, std::true_type());
        else
            go((float *)nullptr, std::false_type());
    };
    // Half a wave a token up to 256 experts: a round's maximum and ballot then
    // serve two tokens (16384 tokens, 256 experts, top-8: 9.8 us, against
    // 13.3 with a wave each).
    using H = std::integral_constant<int, 32>;
    using W = std::integral_constant<int, 64>;
    if (g.E <= 32)
        with_shape(std::integral_constant<int, 1>(), H());
    else if (g.E <= 64)
        with_shape(std::integral_constant<int, 2>(), H());
    else if (g.E <= 128)
        with_shape(std::integral_constant<int, 4>(), H());
    else if (g.E <= 256)
        with_shape(std::integral_constant<int, 8>(), H());
    else if (g.E <= 512)
        with_shape(std::integral_constant<int, 8>(), W());
    else if (g.E <= 1024)
        with_shape(std::integral_constant<int, 16>(), W());
    else
        with_shape(std::integral_constant<int, 32>(), W());
    return hipGetLastError();
}

hipError_t launch_route_backward(const Geometry &g, const void *logits, bool bf16, bool softmax,
                                 bool renormalize, float scale, const int32_t *idx,
                                 const float *dweights, void *dlogits, hipStream_t stream)
{
    const dim3 grid((unsigned)((g.T + 3) / 4));
    with_per(g.E, [&](auto per) {
        constexpr int P = decltype(per)::value;
        if (bf16)
            launch(route_backward_kernel<uint16_t, P>, grid, dim3(256), 0, stream,
                   (const uint16_t *)logits, (int64_t)g.T, g.E, g.k, softmax, renormalize, scale,
                   idx, dweights, (uint16_t *)dlogits);
        else
            launch(route_backward_kernel<float, P>, grid, dim3(256), 0, stream,
                   (const float *)logits, (int64_t)g.T, g.E, g.k, softmax, renormalize, scale, idx,
                   dweights, (float *)dlogits);
    });
    return hipGetLastError();
}

}  // namespace epx
