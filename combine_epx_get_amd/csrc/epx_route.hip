// epx_route.hip -- the router's choice on gfx950: scores -> topk_idx and
// topk_weights, and the gradient of the weights.
//
// One wave per token. Lane l holds the PER consecutive logits from l * PER
// on, so that expert order is (lane, place in the lane) order: the lowest
// lane whose best key equals the wave's best key holds the lowest id, and a
// tie needs no comparison of ids. Keys are the order-preserving integers of
// the logits (32 bits), or of score + bias in double precision (64 bits: two
// biased scores can be nearer to each other than float32 tells). The k
// rounds are a wave maximum (DPP), a ballot and an update in one lane each.
// Key 0 marks a taken or absent place and key 1 a masked expert (-infinity
// or NaN); every other key is larger.
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

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v)
{
    v = max(v, (uint32_t)dpp<kDppRowShr + 1>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 2>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 4>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowShr + 8>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowBcast15, 0xa, false>((int)v));
    v = max(v, (uint32_t)dpp<kDppRowBcast31, 0xc, false>((int)v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
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
__device__ __forceinline__ void load_row(const TIn *row, int E, bool whole, float (&l)[PER])
{
    const int at = lane_id() * PER;
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

template <typename TIn, int PER, bool BIASED>
__global__ __launch_bounds__(256) void route_kernel(const TIn *__restrict__ logits, int64_t T, int E,
                                                    int k, bool softmax,
                                                    const float *__restrict__ bias,
                                                    bool renormalize, float scale,
                                                    int32_t *__restrict__ idx,
                                                    float *__restrict__ weights)
{
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= T)
        return;
    const int lane = lane_id(), at = lane * PER;
    float l[PER];
    load_row<TIn, PER>(logits + t * E, E, E % PER == 0, l);
    uint32_t hi[PER], lo[BIASED ? PER : 1];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool in = at + i < E;
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

    // k rounds; lane j keeps round j's expert and logit
    int mine = 0;
    float my_logit = -__builtin_inff();
    for (int j = 0; j < k; ++j) {
        uint32_t bh = 0, bl = 0;
        int bi = 0;
        float bv = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool better = BIASED ? hi[i] > bh || (hi[i] == bh && lo[i] > bl) : hi[i] > bh;
            bh = better ? hi[i] : bh;
            if (BIASED)
                bl = better ? lo[i] : bl;
            bi = better ? i : bi;
            bv = better ? l[i] : bv;
        }
        const uint32_t wh = wave_max_u32(bh);
        bool cand = bh == wh;
        if (BIASED) {
            const uint32_t wl = wave_max_u32(cand ? bl : 0u);
            cand = cand && bl == wl;
        }
        const int win = __builtin_ctzll(__ballot(cand));
        const int e = __builtin_amdgcn_readlane(at + bi, win);
        const float v = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(bv), win));
        if (lane == j) {
            mine = e;
            my_logit = v;
        }
        if (lane == win) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (i == bi) {
                    hi[i] = kTaken;
                    if (BIASED)
                        lo[i] = 0;
                }
        }
    }

    float w;
    if (softmax) {
        float m = -__builtin_inff(), sum = 0.0f;
        if (!renormalize) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                m = fmaxf(m, l[i]);
            m = wave_maxf(m);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                sum += exp_to(l[i], m);
            sum = wave_sum(sum);
        } else {
            m = wave_maxf(lane < k ? my_logit : -__builtin_inff());
            sum = wave_sum(lane < k ? exp_to(my_logit, m) : 0.0f);
        }
        w = sum > 0.0f ? scale * (exp_to(my_logit, m) / sum) : 0.0f;
    } else {
        const double p = lane < k && !masked(my_logit) ? sigmoid64(my_logit) : 0.0;
        const double sum = renormalize ? wave_sum(p) : 1.0;
        w = sum > 0.0 ? scale * (float)(p / sum) : 0.0f;
    }
    if (lane < k) {
        idx[t * k + lane] = mine;
        weights[t * k + lane] = w;
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
        load_row<TIn, PER>(row, E, E % PER == 0, l);
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
    const dim3 grid((unsigned)((g.T + 3) / 4));
    with_per(g.E, [&](auto per) {
        constexpr int P = decltype(per)::value;
        auto go = [&](auto *row, auto biased) {
            using TIn = std::remove_pointer_t<decltype(row)>;
            launch(route_kernel<TIn, P, decltype(biased)::value>, grid, dim3(256), 0, stream,
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
    });
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
