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
//
// 32768 ragged rows on 16 experts: forward of 2 x 2048 x 7168 1430-1550 us, as
// with bf16 pre-activations or a little less (half of their bytes are written);
// input gradient of 7168 x 2048 850-920 us with the activation handed out (35 of
// them for it), of which writing takes about 100 and the epilogue's arithmetic as
// much; weight gradient of 4096 x 7168 1650-1810 us, 1605-1650 from bf16 rows.
// Converting all rows by a call before takes 101 us and 470 MB: what the weight
// gradient from kept rows saves is that memory, and no time (side by side 1746
// and 1741 us; float32 results 1990 and 1849, added to what is there 2350).
#include "epx_expert_tiles.h"

namespace epx {
namespace {

// A step of x on its way to LDS: BK rows of TP columns, spread over LANES lanes.
// A lane has kUnits units of 16 columns, each a load of codes and one of their
// scale byte; all of its units have the same columns.
template <int TP, int BK, int LANES> struct Stage {
    static constexpr int kUnits = BK * TP / 16 / LANES, kRowUnits = TP / 16, kStride = LANES / kRowUnits;
    static constexpr int kLoads = 2 * kUnits;
    static_assert(kUnits * LANES * 16 == BK * TP && LANES % kRowUnits == 0, "");
    u32x4 codes[kUnits], chunk;
    uint32_t scale[kUnits];
    uint32_t c_off, s_off, np, np32;
    int row, col;
    float step;
    __amdgpu_buffer_rsrc_t rp, rs;

    __device__ __forceinline__ Stage(int lane, uint32_t columns)
        : np(columns), np32(columns / 32), row(lane / kRowUnits), col(lane % kRowUnits)
    {
        c_off = row * np + col * 16;
        s_off = row * np32 + col / 2;
    }
    // Descriptors of `rows` rows from these places on, `before` columns into a row.
    __device__ __forceinline__ void aim(const char *p, const char *s, uint32_t rows, uint32_t before)
    {
        rp = read_buffer(p, rows ? rows * np - before : 0u);
        rs = read_buffer(s, rows ? rows * np32 - before / 32 : 0u);
    }
    __device__ __forceinline__ void load(int u)
    {
        codes[u] = __builtin_amdgcn_raw_buffer_load_b128(rp, (int)(c_off + u * kStride * np), 0, 0);
        scale[u] = __builtin_amdgcn_raw_buffer_load_b8(rs, (int)(s_off + u * kStride * np32), 0, 0);
    }
    // Quarter q of a unit: 4 codes, and with every other one a write of 16
    // bytes. (Neighbouring lanes write 32 bytes apart, which takes each bank
    // twice; choosing the half that a lane writes first by its place, so that
    // all banks are used, takes more instructions than it saves: 1865 against
    // 1795 us, 32768 rows on 16 experts of 4096 x 7168.)
    __device__ __forceinline__ void convert(uint32_t at, int u, int q)
    {
        const int k = row + u * kStride;
        if (q == 0)
            step = mxint8_step(scale[u]);
        const u32x2 o = mxint8_bf16(codes[u][q], step);
        chunk[q % 2 * 2] = o.x;
        chunk[q % 2 * 2 + 1] = o.y;
        if (q % 2)
            *(__attribute__((address_space(3))) u32x4 *)(uintptr_t)(at + k * (TP * 2) +
                                                                    ((col * 2 + q / 2) ^ col_key<TP>(k)) * 16) = chunk;
    }
};

// P = x (codes), Q = dy. WP x WQ waves compute a tile, WK groups of them take
// every WK-th step each, a step ahead of what they multiply. (Tiles of 64 x 64
// and more are bound by the instructions of the conversion: copies of codes and
// scale bytes to LDS, three steps ahead, and from there through registers took
// longer at every size of theirs. Those of 32 columns are bound by the memory's
// latency: a step has 4 or 8 matrix instructions, and a wave one step under way.
// 1 expert of 328 x 608, 14922 rows: 58 steps a wave in 48 us, of which waves
// wait 65 %; 1 of 128 x 128, 40000 rows, 16 tiles on 256 CUs: 89 us, 58 %. More
// steps under way are not tried for them.)
template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK> struct KeptKernel {
    using Base = Kernel<F32 ? kWgradKeptF32 : kWgradKept, TP, TQ, BK, 2, WP, WQ, WK>;
    static constexpr int kWaves = WP * WQ, kLanes = kWaves * kWave;
    static constexpr int NI = Base::NI, NJ = Base::NJ;
    static constexpr int kPBytes = Base::kPBytes, kQBytes = Base::kQBytes, kQCopies = Base::kQCopies;
    static constexpr int kBuf = kPBytes + kQBytes;
    // two buffers, or what a group's sums take when they are joined
    static constexpr int kSums = WK > 1 ? kWaves * NI * NJ * kWave * 16 : 0;
    static constexpr int kRing = 2 * kBuf > kSums ? 2 * kBuf : kSums, kLds = WK * kRing;
    // waves a SIMD: as LDS allows, but at least two and at most four (with more
    // a 128 x 128 tile's sums and codes do not fit the registers)
    static constexpr int kByLds = 160 * 1024 / kLds * kWaves * WK / 4;
    static constexpr int kPerSimd = kByLds < 2 ? 2 : kByLds > 4 ? 4 : kByLds;
    static_assert(kLds <= 160 * 1024, "");

    static __device__ __forceinline__ void run(const Args8 &a, const Tile &t, char *smem)
    {
        const int of_all = uniform(threadIdx.x >> 6), group = of_all / kWaves;
        const int wave = of_all % kWaves, wp = wave % WP, wq = wave / WP;
        const int steps = (t.sum + BK - 1) / BK, own_steps = (steps + WK - 1) / WK;
        const int col0 = t.p * TP, np32 = a.np / 32;
        const char *pb = uniform_ptr(a.p + (int64_t)t.row0 * a.np + col0);
        const char *sb = uniform_ptr(a.kept_scales + (int64_t)t.row0 * np32 + col0 / 32);
        const char *qb = uniform_ptr(a.q + ((int64_t)t.row0 * a.nq + t.q * TQ) * 2);
        uint32_t q_off[kQCopies];
        Base::template copy_offsets<true, TQ, kQCopies, 2, false>(wave, 0, a.nq, 0, q_off);
        const uint32_t lds = lds_offset(smem) + (uint32_t)group * kRing;

        Stage<TP, BK, kLanes> x(wave * kWave + lane_id(), (uint32_t)a.np);
        // a group's step comes: dy to LDS, codes to registers (zeros past the last)
        auto fetch = [&](int own, uint32_t at) {
            const int step = own * WK + group, k0 = step * BK;
            const uint32_t rows = step < steps ? (uint32_t)min(BK, t.sum - k0) : 0u;
            const i32x4 rq = buffer_of(qb + (int64_t)k0 * a.nq * 2,
                                       rows ? rows * (uint32_t)a.nq * 2u - (uint32_t)t.q * TQ * 2u : 0u);
#pragma unroll
            for (int c = 0; c < kQCopies; ++c)
                copy16_to_lds(at + kPBytes + (wave * kQCopies + c) * 1024, rq, q_off[c]);
            x.aim(pb + (int64_t)k0 * a.np, sb + (int64_t)k0 * np32, rows, (uint32_t)col0);
#pragma unroll
            for (int u = 0; u < x.kUnits; ++u)
                x.load(u);
        };
        auto convert = [&](uint32_t to) {
#pragma unroll
            for (int u = 0; u < x.kUnits; ++u)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    x.convert(to, u, q);
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
            if constexpr (kWaves == 1)
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
            // a group's own sums take the place of what it reads no more: the
            // last steps' codes are written before
            __builtin_amdgcn_s_waitcnt(0xC07F);
            join_groups<WK, kRing, kWaves>(lds_offset(smem), group, wave, acc, all);
            if (group * NE < NJ)
                Base::template write<NE>(a, t, wp, wq, group * NE, all);
        }
    }
};

// The large tile: 256 x 256, one workgroup of 8 waves a CU, steps of 64.
//
// A step is two halves of 32 of the sum, a half eight rounds: a round reads
// dy's fragment of the round after next and multiplies one by the half's four
// fragments of x, while the next half's come. In a step's first half the codes
// of the next step, loaded a step ago, are converted into the other of P's two
// buffers and the loads of the step after go out; in the second half dy's
// copies do, into the third of Q's buffers. One meeting of the waves, between
// the halves, orders all of it: what was read before it is free after it, what
// was written or copied before it is there. (Whole sets of dy's fragments, as
// the bf16 kernel holds them, would leave no registers for the codes.)
//
// The third buffer is there because this step's dy and the next one's are both
// read in the second half; it does not keep dy's copies under way for a step.
// The waits that the compiler puts before the conversions count its own loads
// alone, so they take in the copies, which went out after those: a step's dy has
// arrived half a step later, before the meeting's own wait for it.
template <bool F32> struct KeptDeep {
    static constexpr int TP = 256, TQ = 256, BK = 64, WP = 4, WQ = 2;
    using Base = Kernel<F32 ? kWgradKeptF32 : kWgradKept, TP, TQ, BK, 2, WP, WQ>;
    static constexpr int NI = Base::NI, NJ = Base::NJ;
    static constexpr int kPBytes = Base::kPBytes, kQBytes = Base::kQBytes, kQCopies = Base::kQCopies;
    static constexpr int kLds = 2 * kPBytes + 3 * kQBytes;
    using X = Stage<TP, BK, WP * WQ * kWave>;
    static constexpr int kLoads = X::kLoads;   // of codes and scales a step
    // Arithmetic may move between the rounds (1700 us against 1750 where nothing
    // may, 32768 rows on 16 experts of 4096 x 7168).
    static constexpr int kMayCross = 0x6;
    static_assert(NI == 4 && NJ == 8 && X::kUnits == 2 && kQCopies == 4, "");

    static __device__ __forceinline__ void run(const Args8 &a, const Tile &t, char *smem)
    {
        const int wave = uniform(threadIdx.x >> 6), wp = wave % WP, wq = wave / WP;
        const int steps = (t.sum + BK - 1) / BK;
        const int col0 = t.p * TP, np32 = a.np / 32;
        const char *pb = uniform_ptr(a.p + (int64_t)t.row0 * a.np + col0);
        const char *sb = uniform_ptr(a.kept_scales + (int64_t)t.row0 * np32 + col0 / 32);
        const char *qb = uniform_ptr(a.q + ((int64_t)t.row0 * a.nq + t.q * TQ) * 2);
        uint32_t q_off[kQCopies];
        Base::template copy_offsets<true, TQ, kQCopies, 2, false>(wave, 0, a.nq, 0, q_off);
        const uint32_t lds = lds_offset(smem);

        X x((int)threadIdx.x, (uint32_t)a.np);
        i32x4 rq;
        auto rows_in = [&](int step) { return step < steps ? (uint32_t)min(BK, t.sum - step * BK) : 0u; };
        auto aim_p = [&](int step) {
            x.aim(pb + (int64_t)step * BK * a.np, sb + (int64_t)step * BK * np32, rows_in(step), (uint32_t)col0);
        };
        auto aim_q = [&](int step) {
            const uint32_t rows = rows_in(step);
            rq = buffer_of(qb + (int64_t)step * BK * a.nq * 2,
                           rows ? rows * (uint32_t)a.nq * 2u - (uint32_t)t.q * TQ * 2u : 0u);
            // a copy may not follow closely on what wrote its descriptor
            asm volatile("s_nop 4" ::"s"(rq));
        };
        auto copy_q = [&](int c, uint32_t at) { copy16_to_lds(at + (wave * kQCopies + c) * 1024, rq, q_off[c]); };
        auto read_p = [&](uint32_t at, int i, int s) { return Base::template read_cols<TP>(at, wp * (TP / WP) + i * 16, s); };
        auto read_q = [&](uint32_t at, int j, int s) { return Base::template read_cols<TQ>(at, wq * (TQ / WQ) + j * 16, s); };

        f32x4 acc[NI][NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

        const uint32_t lq = lds + 2 * kPBytes;
        uint32_t p0 = lds, p1 = lds + kPBytes;                             // this step's, the next
        uint32_t q0 = lq, q1 = lq + kQBytes, q2 = lq + 2 * kQBytes;        // and the one after
        aim_p(0);
        x.load(0);
        x.load(1);
        aim_q(0);
#pragma unroll
        for (int c = 0; c < kQCopies; ++c)
            copy_q(c, q0);
        aim_q(1);
#pragma unroll
        for (int c = 0; c < kQCopies; ++c)
            copy_q(c, q1);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            x.convert(p0, q / 4, q % 4);
        aim_p(1);
        x.load(0);
        x.load(1);
        wait_copies<kLoads>();   // (both steps of dy)
        bf16x8 pf[2][NI], qf[4];
#pragma unroll
        for (int i = 0; i < NI; ++i)
            pf[0][i] = read_p(p0, i, 0);
        qf[0] = read_q(q0, 0, 0);
        qf[1] = read_q(q0, 1, 0);
        for (int step = 0; step < steps; ++step) {
            aim_p(step + 2);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                qf[(j + 2) % 4] = j + 2 < NJ ? read_q(q0, j + 2, 0) : read_q(q0, j + 2 - NJ, 1);
                if (j % 2 == 0)
                    pf[1][j / 2] = read_p(p0, j / 2, 1);
                if (j % 2) {
                    x.convert(p1, j / 4, j % 4 - 1);
                    x.convert(p1, j / 4, j % 4);
                }
                if (j % 4 == 3)
                    x.load(j / 4);
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    mfma_in_place(acc[i][j], pf[0][i], qf[j % 4]);
                __builtin_amdgcn_sched_barrier(kMayCross);
            }
            wait_copies<kLoads>();   // all but the loads just made
            aim_q(step + 2);
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                qf[(j + 2) % 4] = j + 2 < NJ ? read_q(q0, j + 2, 1) : read_q(q1, j + 2 - NJ, 0);
                if (j % 2 == 0)
                    pf[0][j / 2] = read_p(p1, j / 2, 0);
                if (j < kQCopies)
                    copy_q(j, q2);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    if (i == NI - 1 && j == NJ - 1)
                        mfma_in_place_last(acc[i][j], pf[1][i], qf[j % 4], uniform(steps - 1 - step));
                    else
                        mfma_in_place(acc[i][j], pf[1][i], qf[j % 4]);
                }
                __builtin_amdgcn_sched_barrier(kMayCross);
            }
            const uint32_t free_p = p0, free_q = q0;
            p0 = p1;
            p1 = free_p;
            q0 = q1;
            q1 = q2;
            q2 = free_q;
        }
        drain_copies();
        Base::template write<NJ>(a, t, wp, wq, 0, acc);
    }
};

template <bool F32> __global__ __launch_bounds__(512, 2) void wgrad_kept_deep_kernel(Args8 a)
{
    using K = KeptDeep<F32>;
    __shared__ __attribute__((aligned(1024))) char smem[K::kLds];
    Tile t;
    if (weight_tile<K::TQ>(a, t))
        K::run(a, t, smem);
}

template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK>
__global__ __launch_bounds__(WP *WQ *WK *kWave, (KeptKernel<F32, TP, TQ, BK, WP, WQ, WK>::kPerSimd))
void wgrad_kept_kernel(Args8 a)
{
    using K = KeptKernel<F32, TP, TQ, BK, WP, WQ, WK>;
    __shared__ __attribute__((aligned(1024))) char smem[K::kLds];
    Tile t;
    if (weight_tile<TQ>(a, t))
        K::run(a, t, smem);
}

template <bool F32, int TP, int TQ, int BK, int WP, int WQ, int WK = 1>
hipError_t start_kept(Args8 a, hipStream_t stream)
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

template <bool F32> hipError_t start_kept_deep(Args8 a, hipStream_t stream)
{
    a.pt = (a.np + 255) / 256;
    a.qt = (a.nq + 255) / 256;
    const int64_t blocks = tile_blocks((int64_t)a.r.n * a.pt * a.qt);
    if (blocks * 512 > (int64_t)0xFFFFFFFF)
        return hipErrorInvalidConfiguration;
    launch(wgrad_kept_deep_kernel<F32>, dim3((unsigned)blocks), dim3(512), 0, stream, a);
    return hipGetLastError();
}

// Tiles (columns x by columns dy) by measured times, us (of bf16 results, but for
// 1 of 256 x 2048 and 8 of 256 x 256, float32): 64 x 64 with eight
// waves that divide the sum / 64 x 128 with four pairs that do / 128 x 128 with
// two groups that do / 128 x 128, four a CU / 256 x 256. Few tiles, and for
// those of 64 a step of the sum at least for each wave: 2 experts of 376 x 640, 5200 rows each 25 /
// 51 / 63 / 104 / 121 (with four waves in place of eight 37); 1 of 1024 x 1024,
// 20000 rows 81 / 165 / 220 / 375 / 431; 4 of 512 x 512, 512 rows 7.7 / 8.2 / 10.7
// / 11.9 / 22; smaller still where that gives more workgroups, 32 x 32 / 32 x 64 /
// 64 x 64: 1 of 328 x 608, 14922 rows (209 tiles of 32 x 32) 49 / 58 / 59; 1 of 512 x
// 512, 1000 rows (256) 5.8 / 6.1 / 8.0; 1 of 128 x 128, 40000 rows (16) 94 / 103 /
// 138; 1 of 256 x 2048, 8192 rows (256 of 32 x 64) 48 / 30 / 40; 1 of 512 x 512, 32 rows 4.2 / 4.6 / 5.8; 2 of 376 x 640, 5200
// rows (240) 34 / 23.4 / 24.7; 4 of 512 x 1024, 256 rows 12.0 / 7.6 / 8.8 / 9.1 / 16.7, 4096 rows
// 39 / 40 / 51 / 81 / 96; but 8 of 256 x 256, 32 rows 6.1 / 5.9 / 7.3 / 5.0 / 12.8.
// Else the last three, by the rounds of workgroups and a round's time, about
// linear in the rows of an expert: 2 of 4624 x 352, 11246 rows 137 / 218 / 249; 8
// of 512 x 1024, 1024 rows 17.1 / 19.6 / 32; 16 of 512 x 1024, 128 rows 15.7 /
// 11.0 / 15.7; 2 of 1408 x 2912, 647 rows 30 / 24 / 28; 16 of 2048 x 7168, 64 rows
// 362 / 159 / 174, 256 rows 464 / 265 / 258, 1024 rows 973 / 648 / 526; 64 of 1024 x
// 2048, 64 rows 202 / 77 / 100; 1 of 4096 x 4096, 2048 rows 117 / 85 / 66.
// Float32 results take the same rule, though they write twice the bytes: over 62
// drawn sizes it takes 2 % longer than the best of the seven tiles for bf16, 3 %
// for float32 and 4 % for float32 added. It is furthest off where a large tile
// has a short sum: 30 experts of 371 rows, 1768 x 320, 256 x 256 / 128 x 128, bf16
// 38 / 30, float32 47 / 33, added 60 / 44.
template <bool F32> hipError_t start_wgrad_kept(const Args8 &a, hipStream_t stream)
{
    const auto tiles = [&](int p, int q) {
        return (int64_t)((a.np + p - 1) / p) * ((a.nq + q - 1) / q) * a.r.n;
    };
    const int64_t sum = a.r.num_rows / a.r.n, squares = tiles(128, 128);
    if (tiles(32, 32) <= 256)
        return start_kept<F32, 32, 32, 32, 1, 1, 8>(a, stream);
    if (tiles(32, 64) <= 256)
        return start_kept<F32, 32, 64, 32, 1, 1, 8>(a, stream);
    if (sum >= 256 && tiles(64, 64) <= 256)
        return start_kept<F32, 64, 64, 32, 1, 1, 8>(a, stream);
    if (sum >= 256 && tiles(64, 128) <= 256)
        return start_kept<F32, 64, 128, 32, 1, 2, 4>(a, stream);
    const auto rounds = [](int64_t t, int64_t slots) { return (t + slots - 1) / slots; };
    // ns
    const int64_t large = rounds(tiles(256, 256), 256) * (8500 + sum * 27);
    const int64_t pairs = rounds(squares, 256) * (6000 + sum * 23 / 2);
    const int64_t small = squares <= 256   ? 3000 + sum * 37 / 2
                          : squares <= 512 ? 3000 + sum * 26
                                           : rounds(squares, 1024) * (7500 + sum * 35);
    if (pairs < small && pairs < large)
        return start_kept<F32, 128, 128, 64, 2, 2, 2>(a, stream);
    return large < small ? start_kept_deep<F32>(a, stream) : start_kept<F32, 128, 128, 32, 2, 2>(a, stream);
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
    Args8 a = {};
    a.r = r;
    a.p = (const char *)x;
    a.q = (const char *)dy;
    a.np = inner;
    a.nq = width;
    a.out = dw;
    a.accumulate = accumulate;
    a.kept_scales = const_cast<uint8_t *>(x_scales);
    return f32 ? start_wgrad_kept<true>(a, stream) : start_wgrad_kept<false>(a, stream);
}

}  // namespace epx
