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
// Measured in a graph of such calls, 256 experts, top-8: 128 tokens 3.9 us, 6.4
// with a bias (8 double precision exponentials and quotients a lane, one after
// another, on 16 workgroups), the gradient 3.2; a call from Python takes the
// host 6 us beside that. 16384 tokens, float32: 8.9 us, biased 20.5, the
// gradient 7.9. These are bound by their instructions (a lane's sort, then k
// rounds of a maximum over the lanes, a ballot and moves), not by their 17 and
// 34 MB, which a copy of that size would move in 3.5 and 7 us.
#include "epx_device.h"
#include "epx_operators.h"

namespace epx {
namespace {

constexpr uint32_t kTaken = 0, kMasked = 1;
constexpr int kDppRowRor = 0x120;   // row_ror:n rotates each row's values by n lanes

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

// All lanes of a token (L of them, L / 16 rows) combined by `op`, the same
// bits in every lane: rotations within a row, then swaps of rows (no LDS).
template <int N> __device__ __forceinline__ uint32_t row_ror(uint32_t v)
{
    return (uint32_t)dpp<kDppRowRor + N>((int)v);
}
template <int N> __device__ __forceinline__ float row_ror(float v)
{
    return __uint_as_float(row_ror<N>(__float_as_uint(v)));
}
template <int N> __device__ __forceinline__ double row_ror(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v);
    return __longlong_as_double(
        (long long)(((uint64_t)row_ror<N>((uint32_t)(b >> 32)) << 32) | row_ror<N>((uint32_t)b)));
}
// The other row of a pair of rows (N = 16) or half of the wave (N = 32): the
// pair (x of the lower, x of the higher) in both.
template <int N> __device__ __forceinline__ void both(uint32_t v, uint32_t &lo, uint32_t &hi)
{
    typedef uint32_t u32p __attribute__((ext_vector_type(2)));
    u32p p;
    if constexpr (N == 16)
        p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    else
        p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    lo = p.x;
    hi = p.y;
}
template <int N> __device__ __forceinline__ void both(float v, float &lo, float &hi)
{
    uint32_t a, b;
    both<N>(__float_as_uint(v), a, b);
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
template <int N> __device__ __forceinline__ void both(double v, double &lo, double &hi)
{
    const uint64_t bits = (uint64_t)__double_as_longlong(v);
    uint32_t a, b, c, d;
    both<N>((uint32_t)(bits >> 32), a, b);
    both<N>((uint32_t)bits, c, d);
    lo = __longlong_as_double((long long)(((uint64_t)a << 32) | c));
    hi = __longlong_as_double((long long)(((uint64_t)b << 32) | d));
}
template <int L, typename T, typename F> __device__ __forceinline__ T over_token(T v, F op)
{
    v = op(v, row_ror<8>(v));
    v = op(v, row_ror<4>(v));
    v = op(v, row_ror<2>(v));
    v = op(v, row_ror<1>(v));
    if constexpr (L >= 32) {
        T lo, hi;
        both<16>(v, lo, hi);
        v = op(lo, hi);
    }
    if constexpr (L == 64) {
        T lo, hi;
        both<32>(v, lo, hi);
        v = op(lo, hi);
    }
    return v;
}
template <int L> __device__ __forceinline__ uint32_t token_max(uint32_t v)
{
    return over_token<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L> __device__ __forceinline__ float token_maxf(float v)
{
    return over_token<L>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int L, typename T> __device__ __forceinline__ T token_sum(T v)
{
    return over_token<L>(v, [](T a, T b) { return a + b; });
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
            // a NaN or -infinity bias ranks like such a logit (the weight is
            // the score's all the same)
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

    const uint64_t below = (1ull << lane) - 1;   // the token's lower lanes
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
        const uint64_t all = __ballot(best);
        if (best && ((L == 64 ? all : all >> (lane_id() & -L)) & below) == 0) {
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

// dlogits; lane j < k of the L lanes of a token holds (id, score, dweight) of
// choice j, and every lane the gradients of PER consecutive experts.
template <typename TIn, int PER, int L>
__global__ __launch_bounds__(256) void route_backward_kernel(
    const TIn *__restrict__ logits, int64_t T, int E, int k, bool softmax, bool renormalize,
    float scale, const int32_t *__restrict__ idx, const float *__restrict__ dweights,
    TIn *__restrict__ dlogits)
{
    constexpr int kTokens = 256 / L;   // of a workgroup
    struct Choice { int32_t id; float part; };
    __shared__ Choice s_choice[kTokens][L];
    const int tok = threadIdx.x / L, lane = threadIdx.x % L, at = lane * PER;
    const int64_t t_own = (int64_t)blockIdx.x * kTokens + tok, t = t_own < T ? t_own : T - 1;
    const TIn *row = logits + t * E;
    int e = -1;
    float g = 0.0f, le = -__builtin_inff();
    if (lane < k) {
        e = idx[t * k + lane];
        if (e < 0 || e >= E)
            e = -1;
        else {
            le = Row<TIn>::get(row + e);
            // a masked choice's weight is 0 whatever the logits: its gradient
            // (which may be infinite or NaN) reaches nothing
            if (!masked(le))
                g = scale * dweights[t * k + lane];
        }
    }
    const bool on = !masked(le);
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
        m = token_maxf<L>(m);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sum += exp_to(l[i], m);
        sum = token_sum<L>(sum);
        const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
        const float p = exp_to(le, m) * inv;
        c = on ? g * p : 0.0f;
        const float all = token_sum<L>(c);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            d[i] = masked(l[i]) ? 0.0f : -(exp_to(l[i], m) * inv) * all;
    } else if (softmax) {
        const float m = token_maxf<L>(le);
        const float x = on ? exp_to(le, m) : 0.0f;
        const float sum = token_sum<L>(x);
        const float p = sum > 0.0f ? x / sum : 0.0f;
        const float mean = token_sum<L>(on ? g * p : 0.0f);
        c = on ? p * (g - mean) : 0.0f;
    } else {
        // 1 - p is formed as 1 / (1 + exp(l)): p alone loses it near 1
        const double p = on ? sigmoid64(le) : 0.0, q = on ? 1.0 / (1.0 + exp((double)le)) : 0.0;
        if (renormalize) {
            const double sum = token_sum<L>(p);
            const double r = sum > 0.0 ? p / sum : 0.0;
            const double mean = token_sum<L>(on ? (double)g * r : 0.0);
            c = on ? (float)(r * ((double)g - mean) * q) : 0.0f;
        } else {
            c = on ? (float)((double)g * p * q) : 0.0f;
        }
    }
    s_choice[tok][lane] = Choice{e, c};
    __syncthreads();
    for (int j = 0; j < k; ++j) {   // in order: an id given twice counts twice
        const Choice own = s_choice[tok][j];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (at + i == own.id)
                d[i] += own.part;
    }
    if (t_own >= T)
        return;
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

// Lanes for a token's gradient, and places per lane, the smallest power of two
// for E experts with them. Half a wave up to 256 experts where it holds the
// choices too (16384 tokens of 256 experts, top-8, softmax of the chosen / of
// all / sigmoid: 7.9 / 11.9 / 8.5 us; 9.6 / 13.2 / 9.8 with 16 lanes; a wave,
// with sums through LDS, 9.7 / 12.9 / 11.5).
template <typename F> void with_shape(int E, int k, F f)
{
    const std::integral_constant<int, 64> wave;
    const std::integral_constant<int, 32> part;
    if (k > 32 || E > 256) {
        if (E <= 64)
            f(std::integral_constant<int, 1>(), wave);
        else if (E <= 128)
            f(std::integral_constant<int, 2>(), wave);
        else if (E <= 256)
            f(std::integral_constant<int, 4>(), wave);
        else if (E <= 512)
            f(std::integral_constant<int, 8>(), wave);
        else if (E <= 1024)
            f(std::integral_constant<int, 16>(), wave);
        else
            f(std::integral_constant<int, 32>(), wave);
    } else if (E <= 32) {
        f(std::integral_constant<int, 1>(), part);
    } else if (E <= 2 * 32) {
        f(std::integral_constant<int, 2>(), part);
    } else if (E <= 4 * 32) {
        f(std::integral_constant<int, 4>(), part);
    } else {
        f(std::integral_constant<int, 8>(), part);
    }
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
    // serve two tokens (16384 tokens, 256 experts, top-8: 9.4 us, against
    // 13.3 with a wave each; 16 lanes 9.2, but 11.8 against 7.2 for 128 biased
    // tokens).
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
    with_shape(g.E, g.k, [&](auto per, auto lanes) {
        constexpr int P = decltype(per)::value, L = decltype(lanes)::value;
        const dim3 grid((unsigned)((g.T + 256 / L - 1) / (256 / L)));
        if (bf16)
            launch(route_backward_kernel<uint16_t, P, L>, grid, dim3(256), 0, stream,
                   (const uint16_t *)logits, (int64_t)g.T, g.E, g.k, softmax, renormalize, scale,
                   idx, dweights, (uint16_t *)dlogits);
        else
            launch(route_backward_kernel<float, P, L>, grid, dim3(256), 0, stream,
                   (const float *)logits, (int64_t)g.T, g.E, g.k, softmax, renormalize, scale, idx,
                   dweights, (float *)dlogits);
    });
    return hipGetLastError();
}

}  // namespace epx
