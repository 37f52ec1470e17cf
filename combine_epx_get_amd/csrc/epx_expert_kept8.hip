// epx_expert_kept8.hip -- the experts' products that write or read activations
// kept in 8 bits (MXINT8: int8 codes, a power of two per 32 neighbours).
//
// The forward product and the input gradient are the bf16 ones with other
// epilogues: pre-activations are quantised from the float32 sums (the four
// lanes of a row hold a block of 32), and read back for the activation's
// gradient, which can hand out the activation itself too, so that it need not
// be kept.
//
// The weight gradient multiplies rows kept in 8 bits. A value is code * 2^s
// with 7 bits of code, exactly a bf16 number: it is converted on the way to
// LDS, through registers, once a workgroup, and multiplied by the bf16
// instruction without another rounding. What comes to LDS is laid out as in
// the bf16 weight gradient (rows of columns, 16-byte chunks permuted), so
// fragments are read the same way.
#include "epx_expert_tiles.h"

namespace epx {
namespace {

struct KeptArgs : Args {
    const uint8_t *scales;   // of P, a byte per 32 columns
};

// P = x (codes), Q = dy. WP x WQ waves compute a tile, WK groups of them take
// every WK-th step each. A lane stages kPieces pieces of 8 columns a step, all
// of the same columns.
template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK> struct KeptKernel {
    using Base = Kernel<F32 ? kWgradF32 : kWgrad, TP, TQ, BK, 2, WP, WQ, WK>;
    static constexpr int kWaves = WP * WQ, kLanes = kWaves * kWave;
    static constexpr int NI = Base::NI, NJ = Base::NJ;
    static constexpr int kPBytes = Base::kPBytes, kQBytes = Base::kQBytes, kQCopies = Base::kQCopies;
    static constexpr int kBuf = kPBytes + kQBytes, kRing = 2 * kBuf, kLds = WK * kRing;
    static constexpr int kRowPieces = TP / 8, kStride = kLanes / kRowPieces;   // rows between a lane's pieces
    static constexpr int kPieces = BK / kStride;
    // waves a SIMD: as LDS allows, but at least two and at most four (with more
    // a 128 x 128 tile's sums and pieces do not fit the registers)
    static constexpr int kByLds = 160 * 1024 / kLds * kWaves * WK / 4;
    static constexpr int kPerSimd = kByLds < 2 ? 2 : kByLds > 4 ? 4 : kByLds;
    static_assert(kLanes % kRowPieces == 0 && BK % kStride == 0, "");

    static __device__ __forceinline__ void run(const KeptArgs &a, const Tile &t, char *smem)
    {
        const int of_all = uniform(threadIdx.x >> 6), group = of_all / kWaves;
        const int wave = of_all % kWaves, wp = wave % WP, wq = wave / WP;
        const int own_lane = wave * kWave + lane_id();
        const int steps = (t.sum + BK - 1) / BK, own_steps = (steps + WK - 1) / WK;
        const int col0 = t.p * TP, np32 = a.np / 32;
        const char *pb = uniform_ptr(a.p + (int64_t)t.row0 * a.np + col0);
        const char *sb = uniform_ptr(a.scales + (int64_t)t.row0 * np32 + col0 / 32);
        const char *qb = uniform_ptr(a.q + ((int64_t)t.row0 * a.nq + t.q * TQ) * 2);
        uint32_t q_off[kQCopies];
        Base::template copy_offsets<true, TQ, kQCopies, 2, false>(wave, 0, a.nq, 0, q_off);
        const uint32_t lds = lds_offset(smem) + (uint32_t)group * kRing;

        const int piece_row = own_lane / kRowPieces, piece_col = own_lane % kRowPieces;
        u32x2 codes[kPieces];
        uint32_t scale[kPieces];
        // a group's step comes: dy to LDS, codes to registers (zeros past the last)
        auto fetch = [&](int own, uint32_t at) {
            const int step = own * WK + group, k0 = step * BK;
            const uint32_t rows = step < steps ? (uint32_t)min(BK, t.sum - k0) : 0u;
            const i32x4 rq = buffer_of(qb + (int64_t)k0 * a.nq * 2,
                                       rows ? rows * (uint32_t)a.nq * 2u - (uint32_t)t.q * TQ * 2u : 0u);
#pragma unroll
            for (int c = 0; c < kQCopies; ++c)
                copy16_to_lds(at + kPBytes + (wave * kQCopies + c) * 1024, rq, q_off[c]);
            const auto rp = read_buffer(pb + (int64_t)k0 * a.np, rows ? rows * (uint32_t)a.np - (uint32_t)col0 : 0u);
            const auto rs = read_buffer(sb + (int64_t)k0 * np32, rows ? rows * (uint32_t)np32 - (uint32_t)col0 / 32u : 0u);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const uint32_t row = piece_row + i * kStride;
                codes[i] = __builtin_amdgcn_raw_buffer_load_b64(rp, (int)(row * (uint32_t)a.np + piece_col * 8), 0, 0);
                scale[i] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(row * (uint32_t)np32 + piece_col / 4), 0, 0);
            }
        };
        auto convert = [&](uint32_t at) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int k = piece_row + i * kStride;
                *(__attribute__((address_space(3))) u32x4 *)(uintptr_t)(at + k * (TP * 2) + (piece_col ^ col_key<TP>(k)) * 16) =
                    mxint8_bf16(codes[i], mxint8_step(scale[i]));
            }
        };

        f32x4 acc[NI][NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        fetch(0, lds);
        convert(lds);
        uint32_t at = lds, next = lds + kBuf;
        for (int step = 0; step < own_steps; ++step) {
            // this step's dy has arrived and everyone's codes are converted
            if constexpr (WK > 1 && kWaves == 1)
                wait_own_copies<0>();
            else
                wait_copies<0>();
            fetch(step + 1, next);
#pragma unroll
            for (int s = 0; s < BK / 32; ++s) {
                bf16x8 pf[NI], qf[NJ];
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    pf[i] = Base::template read_cols<TP>(at, wp * (TP / WP) + i * 16, s);
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    qf[j] = Base::template read_cols<TQ>(at + kPBytes, wq * (TQ / WQ) + j * 16, s);
#pragma unroll
                for (int i = 0; i < NI; ++i)
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        acc[i][j] = Base::product(acc[i][j], pf[i], qf[j]);
            }
            convert(next);
            const uint32_t free = at;
            at = next;
            next = free;
        }
        drain_copies();
        if constexpr (WK == 1) {
            Base::template write<NJ>(a, t, wp, wq, 0, acc);
        } else {
            constexpr int NE = (NJ + WK - 1) / WK;
            f32x4 all[NI][NE];
            join_groups<WK, kRing, kWaves>(lds_offset(smem), group, wave, acc, all);
            if (group * NE < NJ)
                Base::template write<NE>(a, t, wp, wq, group * NE, all);
        }
    }
};

template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK>
__global__ __launch_bounds__(WP *WQ *WK *kWave, (KeptKernel<F32, TP, TQ, BK, WP, WQ, WK>::kPerSimd))
void wgrad_kept_kernel(KeptArgs a)
{
    using K = KeptKernel<F32, TP, TQ, BK, WP, WQ, WK>;
    __shared__ __attribute__((aligned(1024))) char smem[K::kLds];
    Tile t;
    if (weight_tile<TQ>(a, t))
        K::run(a, t, smem);
}

template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK = 1>
hipError_t start_kept(KeptArgs a, hipStream_t stream)
{
    a.pt = (a.np + TP - 1) / TP;
    a.qt = (a.nq + TQ - 1) / TQ;
    const int64_t blocks = tile_blocks((int64_t)a.r.n * a.pt * a.qt);
    constexpr int kThreads = WP * WQ * WK * kWave;
    if (blocks * kThreads > (int64_t)0xFFFFFFFF)
        return hipErrorInvalidConfiguration;
    launch(wgrad_kept_kernel<F32, TP, TQ, BK, WP, WQ, WK>, dim3((unsigned)blocks), dim3(kThreads), 0, stream, a);
    return hipGetLastError();
}

template <bool F32> hipError_t start_wgrad_kept(const KeptArgs &a, hipStream_t stream)
{
    return start_kept<F32, 128, 128, 32, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_expert_gemm_keep8(const ExpertRows &r, const void *x, const void *w,
                                    int32_t width, int32_t inner, int8_t *kept,
                                    uint8_t *kept_scales, void *out, hipStream_t stream)
{
    Args8 a = {};
    a.r = r;
    a.p = (const char *)w;
    a.q = (const char *)x;
    a.np = width;
    a.sum = inner;
    a.out = out;
    a.kept = kept;
    a.kept_scales = kept_scales;
    return start_forward<kForwardKeep>(a, stream);
}

hipError_t launch_expert_dgrad_kept8(const ExpertRows &r, const void *dy, const void *w,
                                     int32_t width, int32_t inner, const int8_t *kept,
                                     const uint8_t *kept_scales, void *act, void *dx,
                                     hipStream_t stream)
{
    Args8 a = {};
    a.r = r;
    a.p = (const char *)w;
    a.q = (const char *)dy;
    a.np = inner;
    a.sum = width;
    a.kept = const_cast<int8_t *>(kept);
    a.kept_scales = const_cast<uint8_t *>(kept_scales);
    a.act = (uint16_t *)act;
    a.out = dx;
    return start_dgrad<kDgradKept>(a, stream);
}

hipError_t launch_expert_wgrad_kept8(const ExpertRows &r, const void *dy, const int8_t *x,
                                     const uint8_t *x_scales, int32_t width, int32_t inner,
                                     bool f32, bool accumulate, void *dw, hipStream_t stream)
{
    KeptArgs a = {};
    a.r = r;
    a.p = (const char *)x;
    a.q = (const char *)dy;
    a.np = inner;
    a.nq = width;
    a.out = dw;
    a.accumulate = accumulate;
    a.scales = x_scales;
    return f32 ? start_wgrad_kept<true>(a, stream) : start_wgrad_kept<false>(a, stream);
}

}  // namespace epx
