// epx_expert_tiles.h -- the tile loop of the experts' products, shared by their
// forms (internal; every source instantiates the operations of its own).
// epx_expert_gemm.hip says how the loop works and what it measured.
#pragma once

#include "epx_gemm.h"
#include "epx_rows8.h"

namespace epx {
namespace {

// Keep: the pre-activations are written in 8 bits (MXINT8). Int8: operands in
// int8 with a scale per row of x and of w. Kept: the input's activation is
// taken from pre-activations kept in 8 bits; for the weight gradient, the rows
// summed over are.
enum Op {
    kForward, kForwardGlu, kDgrad, kDgradGlu, kWgrad, kWgradF32,
    kForwardKeep, kInt8, kInt8Glu, kInt8Keep, kDgradKept, kWgradKept, kWgradKeptF32
};
constexpr bool is_int8(int op) { return op == kInt8 || op == kInt8Glu || op == kInt8Keep; }
constexpr bool is_keep(int op) { return op == kForwardKeep || op == kInt8Keep; }
constexpr bool is_glu(int op) { return op == kForwardGlu || op == kInt8Glu || is_keep(op); }
constexpr bool is_f32(int op) { return op == kWgradF32 || op == kWgradKeptF32; }
constexpr bool is_weights(int op) { return op == kWgrad || op == kWgradKept || is_f32(op); }
constexpr bool is_gradient(int op) { return op == kDgrad || op == kDgradGlu || op == kDgradKept || is_weights(op); }

struct Args {
    ExpertRows r;
    const char *p, *q;      // operands
    int32_t np, nq;         // P's extent (columns of a P row in memory for the gradients); Q's for wgrad
    int32_t sum;            // length of the sum (forward, dgrad)
    int32_t pt, qt;         // tiles along P; along Q (wgrad)
    const uint16_t *preact_in;
    uint16_t *preact_out;
    void *out;
    int32_t accumulate;
};

// Arguments of the forms in 8 bits. With int8 operands `sum` counts pairs of
// values: a pair has the bytes of a bf16, so copies and buffers are the same.
struct Args8 : Args {
    const float *q_scales, *p_scales;   // of a row of x; of a row of w
    int8_t *kept;                       // pre-activations in 8 bits, written or read
    uint8_t *kept_scales;
    uint16_t *act;                      // gradient: null, or the input's activation again
};

// Which 16-byte chunk of a row a chunk is kept at: exclusive or with these.
// Rows of BK: the rows of a fragment differ in their low two bits and in bit
// `high`. Rows of columns: see read_cols.
template <int HIGH> __device__ __forceinline__ int row_key(int r) { return (r & 3) | (((r >> HIGH) & 1) << 2); }
template <int T> __device__ __forceinline__ int col_key(int k)
{
    // rows of 64 (32) columns: two (four) of them fill the banks once, so the
    // row's lowest bits separate them already
    const int key = (k & 3) | (((k >> 3) & 1) << 2);
    return T == 32 ? (key & 4) >> 1 : T == 64 ? key & 6 : key << 1;
}

__host__ __device__ constexpr int log2i(int v) { return v <= 1 ? 0 : 1 + log2i(v / 2); }

// WP x WQ waves compute a tile; WK groups of them take every WK-th step each,
// with buffers of their own, and add up their sums at the end.
template <int OP, int TP, int TQ, int BK, int S, int WP, int WQ, int WK = 1> struct Kernel {
    using A = std::conditional_t<(OP >= kForwardKeep), Args8, Args>;
    static constexpr bool kI8 = is_int8(OP), kKeep = is_keep(OP);
    using Sum = std::conditional_t<kI8, i32x4, f32x4>;   // four results of a lane
    static constexpr bool kGlu = is_glu(OP);
    static constexpr bool kPCols = is_gradient(OP);     // P's sum index is the row in memory
    static constexpr bool kWeights = is_weights(OP);
    static constexpr bool kQCols = kWeights;
    static constexpr int kWaves = WP * WQ;   // of a group
    static constexpr int NI = TP / WP / 16, NJ = TQ / WQ / 16;
    // P fragments whose rows are read such that a lane has 4 * GI consecutive
    // columns of them
    static constexpr int kHalf = kGlu ? NI / 2 : NI;
    static constexpr int GI = kPCols || kHalf % 2 != 0 ? 1 : 2;
    static constexpr int kPBytes = TP * BK * 2, kQBytes = TQ * BK * 2;
    static constexpr int kPCopies = kPBytes / 1024 / kWaves, kQCopies = kQBytes / 1024 / kWaves;
    static constexpr bool kDeep = TP == 256;
    static constexpr int kRing = kDeep ? 3 * kPBytes + 2 * kQBytes : S * (kPBytes + kQBytes);
    static constexpr int kLds = WK * kRing;
    static_assert(WK == 1 || !kDeep, "");
    // A wave a SIMD: sums stay in the accumulation registers.
    static constexpr bool kInPlace = !kDeep && kWaves * WK == 4 && kLds > 80 * 1024 && NI * NJ >= 16;
    // Waves a SIMD: as LDS allows, but at least two: with all 512 registers to
    // itself a wave's sums go to the accumulation registers and are moved to and
    // fro in the loop (128 x 128 weight gradient: 88 moves for 16 instructions).
    static constexpr int kPerSimd = 160 * 1024 / kLds * kWaves * WK / 4 > 2 ? 160 * 1024 / kLds * kWaves * WK / 4 : 2;
    static_assert(kPBytes % (1024 * kWaves) == 0 && kQBytes % (1024 * kWaves) == 0, "copies divide over the waves");
    static_assert(!kGlu || NI % 2 == 0, "gate and up fragments pair up in a wave");
    static_assert(!kKeep || GI == 2, "four lanes hold a block of 32");

    // Row of the tile that lane row m (0..15) of P fragment i reads.
    static __device__ __forceinline__ int p_row(int wp, int i, int m)
    {
        if constexpr (kGlu) {
            const int h = i / kHalf, ii = i % kHalf;
            return h * (TP / 2) + wp * (TP / 2 / WP) + ii / GI * 16 * GI + 4 * GI * (m >> 2) + ii % GI * 4 + (m & 3);
        } else {
            return wp * (TP / WP) + i / GI * 16 * GI + 4 * GI * (m >> 2) + i % GI * 4 + (m & 3);
        }
    }

    // Source offsets of a wave's copies of one operand. `extent` rows are
    // loaded from row0 on (COLS: columns from col0 on); ld is in elements.
    template <bool COLS, int T, int N, int KEY, bool SPLIT>
    static __device__ __forceinline__ void copy_offsets(int wave, int row0, int ld, int up, uint32_t (&off)[N])
    {
#pragma unroll
        for (int c = 0; c < N; ++c) {
            const int inst = wave * N + c;
            if constexpr (COLS) {
                constexpr int lanes = T / 8;   // lanes per row of the tile
                const int k = inst * (64 / lanes) + lane_id() / lanes;
                const int chunk = (lane_id() % lanes) ^ col_key<T>(k);
                off[c] = (uint32_t)(k * ld + chunk * 8) * 2u;
            } else {
                constexpr int lanes = BK / 8;
                const int r = inst * (64 / lanes) + lane_id() / lanes;
                const int chunk = (lane_id() % lanes) ^ row_key<KEY>(r);
                const int src = SPLIT && r >= T / 2 ? up + row0 + r - T / 2 : row0 + r;
                off[c] = ((uint32_t)src * (uint32_t)ld + chunk * 8) * 2u;
            }
        }
    }

    // One fragment (16 rows or columns by 32 of the sum) of an operand kept
    // as rows of columns: two transposing reads. Lane (g, 4 j + s) of a read
    // names 4 columns of sum row g * 8 + j (+ 4); it gets column 4 j + s of
    // the four rows.
    template <int T>
    static __device__ __forceinline__ bf16x8 read_cols(uint32_t buf, int col, int s)
    {
        const int l = lane_id(), g = l >> 4, j = (l >> 2) & 3;
        const int k = s * 32 + g * 8 + j;
        const int chunk = (col / 8 + ((l & 3) >> 1)) ^ col_key<T>(k);
        const uint32_t at = buf + k * (T * 2) + chunk * 16 + (l & 1) * 8;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)at);
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(uintptr_t)(at + 4 * T * 2));
        return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }

    template <int KEY>
    static __device__ __forceinline__ bf16x8 read_rows(uint32_t buf, int row, int s)
    {
        const int chunk = (s * 4 + (lane_id() >> 4)) ^ row_key<KEY>(row);
        return lds_read<bf16x8>(buf + row * (BK * 2) + chunk * 16);
    }

    static __device__ __forceinline__ Sum product(Sum c, bf16x8 p, bf16x8 q)
    {
        if constexpr (kI8)
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, p), __builtin_bit_cast(i32x4, q), c,
                                                         0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, q, c, 0, 0, 0);
    }

    static __device__ __forceinline__ void run(const A &a, const Tile &t, char *smem)
    {
        const int of_all = uniform(threadIdx.x >> 6), group = of_all / kWaves;
        const int wave = of_all % kWaves, wp = wave % WP, wq = wave / WP, m = lane_id() & 15;
        constexpr int PK = 2 + log2i(GI), QK = 2;   // row_key bits

        const int sum = kWeights ? t.sum : a.sum;
        const int steps = (sum + BK - 1) / BK;
        constexpr int PC = kGlu ? TP / 2 : TP;   // output columns of a tile
        const int col0 = t.p * PC;

        // operand bases and, for operands whose sum index is the memory row, their last byte
        const char *pb, *qb;
        uint32_t p_bytes = 0, q_bytes = 0;
        if constexpr (kWeights) {
            pb = a.p + ((int64_t)t.row0 * a.np + col0) * 2;
            qb = a.q + ((int64_t)t.row0 * a.nq + t.q * TQ) * 2;
        } else if constexpr (kPCols) {
            pb = a.p + ((int64_t)t.expert * sum * a.np + col0) * 2;
            qb = a.q + (int64_t)t.row0 * sum * 2;
            q_bytes = (uint32_t)min(t.rows, TQ) * (uint32_t)sum * 2u;
        } else {
            const int rows = kGlu ? 2 * a.np : a.np;
            pb = a.p + (int64_t)t.expert * rows * sum * 2;
            p_bytes = (uint32_t)rows * (uint32_t)sum * 2u;
            qb = a.q + (int64_t)t.row0 * sum * 2;
            q_bytes = (uint32_t)min(t.rows, TQ) * (uint32_t)sum * 2u;
        }
        pb = uniform_ptr(pb);
        qb = uniform_ptr(qb);
        uint32_t p_off[kPCopies], q_off[kQCopies];
        copy_offsets<kPCols, TP, kPCopies, PK, kGlu>(wave, kPCols ? 0 : col0, kPCols ? a.np : sum, a.np, p_off);
        copy_offsets<kQCols, TQ, kQCopies, QK, false>(wave, 0, kQCols ? a.nq : sum, 0, q_off);
        const uint32_t lds = lds_offset(smem) + (uint32_t)group * kRing;

        // descriptors of the operands' parts in a group's step (empty past the last)
        i32x4 rp, rq;
        auto aim = [&](int own) {
            const int step = own * WK + group, k0 = step * BK;
            const bool live = step < steps;
            if constexpr (kPCols)
                rp = buffer_of(pb + (int64_t)k0 * a.np * 2,
                               live ? (uint32_t)min(BK, sum - k0) * (uint32_t)a.np * 2u - (uint32_t)col0 * 2u : 0u);
            else
                rp = buffer_of(pb + (int64_t)k0 * 2, live ? p_bytes - (uint32_t)k0 * 2u : 0u);
            if constexpr (kQCols)
                rq = buffer_of(qb + (int64_t)k0 * a.nq * 2,
                               live ? (uint32_t)min(BK, sum - k0) * (uint32_t)a.nq * 2u - (uint32_t)t.q * TQ * 2u : 0u);
            else
                rq = buffer_of(qb + (int64_t)k0 * 2, live ? q_bytes - (uint32_t)k0 * 2u : 0u);
            // a last step that ends inside BK: chunks past the sum's end
            // would be the next row's first (no live step follows it)
            if (!(kPCols && kQCols) && live && k0 + BK > sum) {
#pragma unroll
                for (int c = 0; c < kPCopies && !kPCols; ++c) {
                    const int r = (wave * kPCopies + c) * (512 / BK) + lane_id() / (BK / 8);
                    if (k0 + ((lane_id() % (BK / 8)) ^ row_key<PK>(r)) * 8 >= sum)
                        p_off[c] = kOutside;
                }
#pragma unroll
                for (int c = 0; c < kQCopies && !kQCols; ++c) {
                    const int r = (wave * kQCopies + c) * (512 / BK) + lane_id() / (BK / 8);
                    if (k0 + ((lane_id() % (BK / 8)) ^ row_key<QK>(r)) * 8 >= sum)
                        q_off[c] = kOutside;
                }
            }
        };
        auto copy_p = [&](int c, uint32_t at) { copy16_to_lds(at + (wave * kPCopies + c) * 1024, rp, p_off[c]); };
        auto copy_q = [&](int c, uint32_t at) { copy16_to_lds(at + (wave * kQCopies + c) * 1024, rq, q_off[c]); };
        auto read_p = [&](uint32_t at, int i, int s) {
            if constexpr (kPCols)
                return read_cols<TP>(at, wp * (TP / WP) + i * 16, s);
            else
                return read_rows<PK>(at, p_row(wp, i, m), s);
        };
        auto read_q = [&](uint32_t at, int j, int s) {
            if constexpr (kQCols)
                return read_cols<TQ>(at, wq * (TQ / WQ) + j * 16, s);
            else
                return read_rows<QK>(at, wq * (TQ / WQ) + j * 16 + m, s);
        };

        Sum acc[NI][NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = Sum{0, 0, 0, 0};

        if constexpr (kDeep) {
            // Two sets of fragments in registers: while one half of a step (32
            // of the sum) is multiplied, the next half's fragments are read.
            // The buffers of a step are free as soon as its second half is
            // read; one meeting of the waves per step, between the halves,
            // orders that and the arrival of the next step. P has three
            // buffers and Q two (160 KB together), so that P's copies for the
            // step after next go out in the first half and Q's in the second:
            // all in one half would ask for more than a CU's 64 bytes a cycle
            // (32768 ragged rows, 16 experts, 2 x 2048 x 7168: 1502 us, and
            // 1662 with two buffers of each and all copies in one half; five
            // buffers of 32 of the sum 2044).
            static_assert(S == 2 && BK == 64, "");
            // arithmetic may move between the rounds where that is faster (32768
            // ragged rows, 16 experts, 2 x 2048 x 7168: int8 800 us against 815,
            // keeping 8 bits 1470 against 1500; the other forms gain nothing)
            constexpr int kMayCross = kI8 || kKeep ? 0x6 : 0;
            constexpr int kReads = NI + NJ;
            // reads and copies before each of the NI rounds of NJ instructions
            // (transposing reads are twice as many, and spread further)
            constexpr int kReadsPer = kQCols ? (kReads + NI - 2) / (NI - 1) : (kReads + 1) / 2;
            constexpr int kPPer = (kPCopies + NI - 1) / NI, kQPer = (kQCopies + NI - 1) / NI;
            bf16x8 pf[2][NI], qf[2][NJ];
            auto read = [&](int set, uint32_t p_at, uint32_t q_at, int c) {
                if (c < NJ)
                    qf[set][c] = read_q(q_at, c, set);
                else
                    pf[set][c - NJ] = read_p(p_at, c - NJ, set);
            };
            const uint32_t lq = lds + 3 * kPBytes;
            uint32_t p0 = lds, p1 = lds + kPBytes, p2 = lds + 2 * kPBytes;   // this step's, the next, the one after
            uint32_t q0 = lq, q1 = lq + kQBytes;
            aim(0);
#pragma unroll
            for (int c = 0; c < kPCopies; ++c)
                copy_p(c, p0);
#pragma unroll
            for (int c = 0; c < kQCopies; ++c)
                copy_q(c, q0);
            aim(1);
#pragma unroll
            for (int c = 0; c < kPCopies; ++c)
                copy_p(c, p1);
#pragma unroll
            for (int c = 0; c < kQCopies; ++c)
                copy_q(c, q1);
            wait_copies<kPCopies + kQCopies>();
#pragma unroll
            for (int c = 0; c < kReads; ++c)
                read(0, p0, q0, c);
            for (int step = 0; step < steps; ++step) {
                aim(step + 2);
#pragma unroll
                for (int i = 0; i < NI; ++i) {
#pragma unroll
                    for (int c = i * kReadsPer; c < (i + 1) * kReadsPer && c < kReads; ++c)
                        read(1, p0, q0, c);
#pragma unroll
                    for (int c = i * kPPer; c < (i + 1) * kPPer && c < kPCopies; ++c)
                        copy_p(c, p2);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        mfma_in_place(acc[i][j], pf[0][i], qf[0][j]);
                    __builtin_amdgcn_sched_barrier(kMayCross);
                }
                wait_copies<kPCopies>();   // all but the ones just made
#pragma unroll
                for (int i = 0; i < NI; ++i) {
#pragma unroll
                    for (int c = i * kReadsPer; c < (i + 1) * kReadsPer && c < kReads; ++c)
                        read(0, p1, q1, c);
#pragma unroll
                    for (int c = i * kQPer; c < (i + 1) * kQPer && c < kQCopies; ++c)
                        copy_q(c, q0);
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        if (i == NI - 1 && j == NJ - 1)
                            mfma_in_place_last(acc[i][j], pf[1][i], qf[1][j], uniform(steps - 1 - step));
                        else
                            mfma_in_place(acc[i][j], pf[1][i], qf[1][j]);
                    }
                    __builtin_amdgcn_sched_barrier(kMayCross);
                }
                const uint32_t free_p = p0, free_q = q0;
                p0 = p1;
                p1 = p2;
                p2 = free_p;
                q0 = q1;
                q1 = free_q;
            }
        } else {
            auto issue = [&](int step, int buf) {
                const uint32_t at = lds + (uint32_t)buf * (kPBytes + kQBytes);
                aim(step);
#pragma unroll
                for (int c = 0; c < kPCopies; ++c)
                    copy_p(c, at);
#pragma unroll
                for (int c = 0; c < kQCopies; ++c)
                    copy_q(c, at + kPBytes);
            };
#pragma unroll
            for (int s = 0; s < S - 1; ++s)
                issue(s, s);
            int buf = 0;
            const int own_steps = (steps + WK - 1) / WK;
            for (int step = 0; step < own_steps; ++step) {
                if constexpr (WK > 1 && kWaves == 1)
                    wait_own_copies<(S - 2) * (kPCopies + kQCopies)>();
                else
                    wait_copies<(S - 2) * (kPCopies + kQCopies)>();
                int into = buf + S - 1;
                into = into >= S ? into - S : into;
                issue(step + S - 1, into);
                const uint32_t at = lds + (uint32_t)buf * (kPBytes + kQBytes);
#pragma unroll
                for (int s = 0; s < BK / 32; ++s) {
                    bf16x8 pf[NI], qf[NJ];
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        pf[i] = read_p(at, i, s);
#pragma unroll
                    for (int j = 0; j < NJ; ++j)
                        qf[j] = read_q(at + kPBytes, j, s);
#pragma unroll
                    for (int i = 0; i < NI; ++i)
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            if constexpr (kInPlace) {
                                if (s == BK / 32 - 1 && i == NI - 1 && j == NJ - 1)
                                    mfma_in_place_last(acc[i][j], pf[i], qf[j], uniform(own_steps - 1 - step));
                                else
                                    mfma_in_place(acc[i][j], pf[i], qf[j]);
                            } else
                                acc[i][j] = product(acc[i][j], pf[i], qf[j]);
                        }
                }
                buf = buf + 1 == S ? 0 : buf + 1;
            }
        }
        drain_copies();

        if constexpr (WK == 1) {
            write<NJ>(a, t, wp, wq, 0, acc);
        } else {
            constexpr int NE = (NJ + WK - 1) / WK;
            Sum all[NI][NE];
            join_groups<WK, kRing, kWaves>(lds_offset(smem), group, wave, acc, all);
            if (group * NE < NJ)
                write<NE>(a, t, wp, wq, group * NE, all);
        }
    }

    // Pre-activations [c, c + 8) of a row (of its gates, or its ups) kept in 8
    // bits. The four lanes of a row hold a block of 32 (np is a multiple of 32).
    static __device__ __forceinline__ void keep(const Args8 &a, int64_t row, int c, const Cols<8> &o, bool ups)
    {
        // (a maximum that hands on a NaN)
        float most = fabsf(o.v[0]);
#pragma unroll
        for (int q = 1; q < 8; ++q)
            most = __builtin_elementwise_maximum(most, fabsf(o.v[q]));
        const uint32_t b = max_of_four(__float_as_uint(most) & 0x7FFFFFFFu) >> 23;
        if (c >= a.np)
            return;
        *(u32x2 *)(a.kept + (row * 2 + ups) * a.np + c) = mxint8_codes(o.v, b);
        if (lane_id() < 16)
            a.kept_scales[(row * 2 + ups) * (a.np / 32) + c / 32] = (uint8_t)b;
    }

    // Gates and ups [c, c + 8) of a row as they were kept.
    struct KeptPair {
        u32x2 code[2];
        uint32_t scale[2];
        // (codes and scale bytes of the tile's rows; past its rows zeros come)
        __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales, int np, int r, int c)
        {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                code[h] = __builtin_amdgcn_raw_buffer_load_b64(codes, (2 * r + h) * np + c, 0, 0);
                scale[h] = __builtin_amdgcn_raw_buffer_load_b8(scales, (2 * r + h) * (np / 32) + c / 32, 0, 0);
            }
        }
        __device__ __forceinline__ Cols<8> values(int h) const
        {
            Cols<8> o;
            const float step = mxint8_step(scale[h]);
#pragma unroll
            for (int q = 0; q < 8; ++q)
                o.v[q] = signed_byte(q < 4 ? code[h].x : code[h].y, q % 4) * step;
            return o;
        }
    };

    template <int N>
    static __device__ __forceinline__ void store(uint16_t *row, int c, int width, const Cols<N> &o)
    {
        if constexpr (OP >= kForwardKeep)
            store_bf16_hw(row, c, width, o);
        else
            store_bf16(row, c, width, o);
    }

    // Results: lane (m, g) of fragment pair (i, j) has row j * 16 + m and
    // columns 4 g .. 4 g + 3 of fragment i. Two fragments are neighbours
    // already where P's rows are read that way (GI), and are merged here
    // otherwise, so that the lanes of a write are neighbours in 64 bytes
    // of a row (float32 results are so as they are).
    template <int N>
    static __device__ __forceinline__ void write(const A &a, const Tile &t, int wp, int wq, int j0, Sum (&acc)[NI][N])
    {
        const int m = lane_id() & 15, g = lane_id() >> 4;
        constexpr int PC = kGlu ? TP / 2 : TP;
        const int col0 = t.p * PC;
        constexpr bool kMerge = kPCols && !is_f32(OP) && NI % 2 == 0;
        constexpr int W = kMerge ? 2 : GI, NG = kHalf / W;
        if constexpr (kMerge && OP != kDgradKept) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    merge_columns(acc[2 * n][j], acc[2 * n + 1][j]);
        }
        // What the rows need from memory is loaded some rows ahead of its use (all
        // of it before the first row is written, for the scales of int8 rows): the
        // compiler moves no load over a store, so that each would wait for its own
        // (input gradient of 32768 rows, 16 experts of 7168 x 2048: 895 against 907
        // us). By 32-bit offsets: 64-bit addresses of rows ahead took 70 registers
        // to memory, and 950 us.
        constexpr int kAhead = OP == kDgradKept ? (N * NG < 8 ? N * NG : 8) : 1;
        [[maybe_unused]] KeptPair pairs[kAhead];
        [[maybe_unused]] __amdgpu_buffer_rsrc_t kept_codes, kept_scales;
        if constexpr (OP == kDgradKept) {
            const uint32_t bytes = (uint32_t)min(t.rows, TQ) * 2u * (uint32_t)a.np;
            kept_codes = read_buffer((const char *)a.kept + (int64_t)t.row0 * 2 * a.np, bytes);
            kept_scales = read_buffer((const char *)a.kept_scales + (int64_t)t.row0 * 2 * (a.np / 32), bytes / 32);
        }
        [[maybe_unused]] auto load_pair = [&](int x) {
            if constexpr (OP == kDgradKept)
                pairs[x % kAhead].load(kept_codes, kept_scales, a.np, wq * (TQ / WQ) + (j0 + x / NG) * 16 + m,
                                       col0 + wp * (PC / WP) + x % NG * 32 + 8 * g);
        };
        if constexpr (OP == kDgradKept) {
            static_assert(W == 2, "");
#pragma unroll
            for (int x = 0; x < kAhead; ++x)
                load_pair(x);
        }
        [[maybe_unused]] float srow[kI8 ? N : 1];
        if constexpr (kI8) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int r = wq * (TQ / WQ) + (j0 + j) * 16 + m;
                srow[j] = r < t.rows ? a.q_scales[(int64_t)t.row0 + r] : 0.0f;
            }
        }
        // int8: the scales of this lane's columns of w
        [[maybe_unused]] Cols<4 * W> su[NG], sv[NG];
        if constexpr (kI8) {
            const float *ps = a.p_scales + (int64_t)t.expert * (kGlu ? 2 * a.np : a.np);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int c = col0 + wp * (PC / WP) + n * 16 * W + 4 * W * g;
                su[n] = load_f32<4 * W>(ps, c, a.np);
                if constexpr (kGlu)
                    sv[n] = load_f32<4 * W>(ps + a.np, c, a.np);
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = wq * (TQ / WQ) + (j0 + j) * 16 + m;
            [[maybe_unused]] const float sr = kI8 ? srow[kI8 ? j : 0] : 0.0f;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int c = col0 + wp * (PC / WP) + n * 16 * W + 4 * W * g;
                Cols<4 * W> u, v;
                if constexpr (kMerge && OP == kDgradKept)   // (here: fewer registers beside what is ahead)
                    merge_columns(acc[2 * n][j], acc[2 * n + 1][j]);
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        u.v[4 * i + q] = (float)acc[n * W + i][j][q];
                        if constexpr (kGlu)
                            v.v[4 * i + q] = (float)acc[kHalf + n * W + i][j][q];
                        // (whole sums to float32, times the row's scale, times the column's)
                        if constexpr (kI8) {
                            u.v[4 * i + q] = u.v[4 * i + q] * sr * su[n].v[4 * i + q];
                            if constexpr (kGlu)
                                v.v[4 * i + q] = v.v[4 * i + q] * sr * sv[n].v[4 * i + q];
                        }
                    }
                if constexpr (kWeights) {
                    const int row = t.q * TQ + r;
                    if (row >= a.nq)
                        continue;
                    const int64_t o = ((int64_t)t.expert * a.nq + row) * a.np;
                    if constexpr (is_f32(OP))
                        store_f32((float *)a.out + o, c, a.np, u, a.accumulate);
                    else
                        store((uint16_t *)a.out + o, c, a.np, u);
                } else {
                    if (r >= t.rows)
                        continue;
                    const int64_t row = t.row0 + r;
                    if constexpr (kKeep) {
                        keep(a, row, c, u, false);
                        keep(a, row, c, v, true);
                    }
                    if constexpr (kGlu) {
                        if constexpr (OP == kForwardGlu) {
                            if (a.preact_out) {
                                store_bf16(a.preact_out + row * 2 * a.np, c, a.np, u);
                                store_bf16(a.preact_out + row * 2 * a.np + a.np, c, a.np, v);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 4 * W; ++q)
                            u.v[q] = swiglu(u.v[q], v.v[q]);
                    }
                    if constexpr (OP == kDgradGlu || OP == kDgradKept) {
                        Cols<4 * W> gate, up;
                        [[maybe_unused]] Cols<4 * W> act;
                        if constexpr (OP == kDgradKept) {
                            gate = pairs[(j * NG + n) % kAhead].values(0);
                            up = pairs[(j * NG + n) % kAhead].values(1);
                            if (j * NG + n + kAhead < N * NG)
                                load_pair(j * NG + n + kAhead);
                        } else {
                            const uint16_t *pre = a.preact_in + row * 2 * a.np;
                            gate = load_bf16<4 * W>(pre, c, a.np);
                            up = load_bf16<4 * W>(pre + a.np, c, a.np);
                        }
#pragma unroll
                        for (int q = 0; q < 4 * W; ++q) {
                            const float s = sigmoid32(gate.v[q]), d = u.v[q];
                            u.v[q] = d * up.v[q] * (s * (1.0f + gate.v[q] * (1.0f - s)));
                            v.v[q] = d * (gate.v[q] * s);
                            if constexpr (OP == kDgradKept)
                                act.v[q] = gate.v[q] * s * up.v[q];
                        }
                        uint16_t *dx = (uint16_t *)a.out + row * 2 * a.np;
                        store(dx, c, a.np, u);
                        store(dx + a.np, c, a.np, v);
                        if constexpr (OP == kDgradKept) {
                            if (a.act)
                                store(a.act + row * a.np, c, a.np, act);
                        }
                    } else {
                        store((uint16_t *)a.out + row * a.np, c, a.np, u);
                    }
                }
            }
        }
    }
};

// The workgroup's tile of a weight gradient; false when there is none for it.
template <int TQ> __device__ __forceinline__ bool weight_tile(const Args &a, Tile &t)
{
    const int64_t tiles = (int64_t)a.pt * a.qt;   // of every expert
    int64_t id, slots;
    if (!spread(tiles * a.r.n, blockIdx.x % kXcds, blockIdx.x / kXcds, id, slots))
        return false;
    t.expert = (int)(id / tiles);
    place(id - t.expert * tiles, a.qt, a.pt, t.p, t.q);
    t.row0 = 0;
    t.sum = uniform(rows_of(a.r, t.expert, t.row0));
    t.row0 = uniform(t.row0);
    t.rows = TQ;
    return true;
}

// The large tiles' kernels carry the smaller ones for an expert's last rows.
template <int OP, int TP, int TQ, int BK, int S, int WP, int WQ, int WK>
__global__ __launch_bounds__(WP *WQ *WK *kWave, (Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>::kPerSimd)) void gemm_kernel(typename Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>::A a)
{
    using K = Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>;
    __shared__ __attribute__((aligned(1024))) char smem[K::kLds];
    Tile t;
    if constexpr (K::kWeights) {
        if (weight_tile<TQ>(a, t))
            K::run(a, t, smem);
    } else {
        if (!find_tile<TQ, K::kDeep>(a.r, a.pt, blockIdx.x, t))
            return;
        if constexpr (K::kDeep) {
            if (t.rows <= TQ / 4)
                Kernel<OP, TP, TQ / 4, BK, S, WP, WQ>::run(a, t, smem);
            else if (t.rows <= TQ / 2)
                Kernel<OP, TP, TQ / 2, BK, S, WP, WQ>::run(a, t, smem);
            else
                K::run(a, t, smem);
        } else {
            K::run(a, t, smem);
        }
    }
}

template <int OP, int TP, int TQ, int BK, int S, int WP, int WQ, int WK = 1>
hipError_t start(typename Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>::A a, int64_t rows_or_n, hipStream_t stream)
{
    constexpr int PC = is_glu(OP) ? TP / 2 : TP;
    a.pt = (a.np + PC - 1) / PC;
    int64_t blocks;
    if (is_weights(OP)) {
        a.qt = (a.nq + TQ - 1) / TQ;
        blocks = tile_blocks(rows_or_n * a.pt * a.qt);
    } else {
        blocks = tile_blocks(most_row_tiles(rows_or_n, a.r.n, TQ) * a.pt);
    }
    if (blocks == 0)
        return hipSuccess;
    constexpr int kThreads = WP * WQ * WK * kWave;
    if (blocks * kThreads > (int64_t)0xFFFFFFFF)
        return hipErrorInvalidConfiguration;
    launch(gemm_kernel<OP, TP, TQ, BK, S, WP, WQ, WK>, dim3((unsigned)blocks), dim3(kThreads), 0,
           stream, a);
    return hipGetLastError();
}

// Where small tiles would leave CUs idle: the largest tile of which there are
// at most 256, one workgroup a CU whose waves divide the sum among them. False
// when there are more of every size. FULL: a tile of 32's columns.
// Measured, us, 32 x 32 / 64 x 32 / 64 x 64 / the tiles that are taken else
// (forward; with how many tiles there are of each): 3 experts of 1 row, gated
// 560 x 3712 (105, 54, 54) 9.4 / 12.7 / 15.5 / 19.3; 1 of 64 rows, gated
// 2048 x 7168 (256, 128, 64) 15.8 / 20.1 / 24.7 / 33.3; 1 of 699 rows, 544 x
// 1016 (374, 198, 99) 10.6 / 8.4 / 8.8 / 9.7; 4 of 256 rows, 1024 x 2048
// (1024, 512, 256) 24.8 / 18.1 / 11.7 / 15.2; 3 of 1000 rows, 512 x 2048 (1536,
// 768, 384) 35.2 / 25.6 / 20.4 / 19.5. Gradient of the input: 1 of 8 rows, 2048
// x 7168 (224, 112, 112) 8.9 / 10.1 / 11.3 / 16.2; 16 of 64 rows, 512 x 1024
// (1024, 512, 256) 19.2 / 11.3 / 8.2 / 8.6.
template <int OP, typename A>
bool start_split(const A &a, int64_t rows, hipStream_t stream, hipError_t &status)
{
    constexpr int FULL = is_glu(OP) ? 16 : 32;
    // (a kept block of 32 columns is wider than the smallest tile's gates)
    if constexpr (!is_keep(OP)) {
        if (tiles_of(a.r, 32, a.np, FULL) <= 256) {
            status = start<OP, 32, 32, 64, 2, 1, 1, 8>(a, rows, stream);
            return true;
        }
    }
    if (tiles_of(a.r, 32, a.np, 2 * FULL) <= 256)
        status = start<OP, 64, 32, 64, 3, 1, 1, 4>(a, rows, stream);
    else if (tiles_of(a.r, 64, a.np, 2 * FULL) <= 256)
        status = start<OP, 64, 64, 64, 2, 1, 1, 4>(a, rows, stream);
    else
        return false;
    return true;
}

// Large tiles (256 x 256, one a CU), square ones (128 x 128, two a CU) or small
// ones (128 x 64, two a CU): what takes the least time by the number of rounds
// of workgroups and the time of a round, which is about linear in the length of
// the sum (16 experts of 2048 rows and 2048 columns, sums of 64 / 256 / 512 /
// 1024 / 2048: large 47 / 73 / 90 / 130 / 230 us in 4 rounds and the last
// tiles', square 50 / 69 / 100 / 158 / 321 in 8, small 70 / 90 / 126 / 203 /
// 394 in 16; a small round is put a quarter higher, for the operands that more
// tiles read again). Large / square / small elsewhere: 2 experts of 6700 rows,
// 1080 x 368 36 / 26 / 35; 13 of 917, 1064 x 1536 76 / 55 / 74; 3 of 3189, 1144
// x 624 26 / 31 / 31; 64 of 96, 1024 x 2048 59 / 61 / 71; 16 of 96, 2048 x 1024
// 19 / 20 / 17. Gradient of the input: 2 of 11246 rows, 4624 x 368 107 / 144 /
// 144; 4 of 2600, 656 x 1120 29 / 34 / 35; 8 of 1500, 1432 x 320 38 / 28 / 31;
// 6 of 700, 1200 x 704 33 / 21 / 19.
// At most one small tile a CU and a sum of 1024 or more: two groups of waves
// divide it (kSmallSplit), us, against one: 1 expert of 4096 rows, 512 x 4096
// (256 tiles) 26.5 / 31.2; 2 of 647, 1408 x 2920 (231) 27.5 / 27.7; gradient of
// the input, 1 of 3000, 7168 x 512 (188) 42.7 / 51.8; 16 of 96, 2048 x 1024
// (256) 17.3 / 18.8; but 8 of 300, 1000 x 1000 (328) 22.3 / 18.3.
enum TileSize { kLarge, kSquare, kSmall, kSmallSplit };
// A round's time for each, ns: a start and its growth with the sum (in 80ths).
struct TileCosts {
    int64_t large, large_sum, square, square_sum, small, small_sum;
};
constexpr TileCosts kCosts = {9000, 1880, 4500, 1320, 4200, 1008};
// Forms in 8 bits, whose small tiles have two buffers for sums up to 1280 (of
// bf16 values, or of pairs of int8), three a CU: one writes while others
// multiply. us, large / square / small with three buffers / with two. Forward,
// kept, gated: 16 experts of 2048 rows, 2048 x 64 110 / 107 / 139 / 106, x 256
// 140 / 144 / 196 / 152, x 512 204 / 245 / 300 / 283; 4 of 1000, 1088 x 256 18.0 /
// 17.7 / 19.1 / 15.9; 2 of 8000, 640 x 320 35 / 28.7 / 36 / 30.6; 37 of 92, 992 x 88
// 15.6 / 13.8 / 15.2 / 12.2; 24 of 83, 544 x 1048 20.9 / 20.4 / 20.3 / 18.7. int8: 16
// of 2048, 2048 x 64 84 / 85 / 132 / 97, x 512 115 / 122 / 176 / 141, x 2048 270 /
// 332 / 414 / 405; 13 of 461, 1280 x 240 13.7 / 13.9 / 14.7 / 12.3; 2 of 1337, 1408 x
// 6512 75 / 70 / 98 / 103; 16 of 96, 2048 x 7168 95 / 100 / 125 / 137.
constexpr TileCosts kCosts8 = {9500, 1520, 4800, 1040, 3900, 1000};
// The gradient through kept pre-activations, which writes both gradients and
// the activation, from codes, at about 170 cycles a result of a wave. As above:
// 16 experts of 2048 rows, 64 x 2048 185 / 173 / 186 / 162, 256 x 2048 192 / 216 /
// 219 / 200, 512 x 2048 221 / 257 / 257 / 246, 1024 x 2048 271 / 327 / 350 / 331; 1 of
// 4632, 192 x 1088 30.9 / 19.7 / 18.1 / 16.5; 4 of 1000, 512 x 1088 36 / 23.6 / 23.0
// / 20.5; 2 of 8000, 320 x 640 35 / 31.6 / 31.0 / 27.8; 37 of 92, 88 x 992 15.9 /
// 15.9 / 15.6 / 13.5; but 24 of 83, 1048 x 544 24 / 22 / 15.0 / 17.2 (above 512 three).
constexpr TileCosts kCostsKept = {36000, 1424, 18000, 1440, 13700, 1304};

// Two buffers for a small tile of the forms in 8 bits (from 64 rows an expert):
// three workgroups a CU in place of two, so a round of them is 768 tiles in
// place of 512. (At 513 to 768 tiles of three buffers, square / small, us, ragged
// rows: forward, kept, 9 experts of 894 rows, 224 x 2760 46.8 / 63.5; int8 gated
// 52 of 70, 576 x 2592 33.9 / 46.4; gradient 27 of 127, 1056 x 3360 65.1 / 83.3.)
template <int OP> bool two_buffers(int64_t sum)
{
    return OP >= kForwardKeep && sum <= (OP == kDgradKept ? 512 : 1280);
}

template <int OP> TileSize best_tiles(const ExpertRows &r, int32_t columns, int columns_of_256, int64_t sum)
{
    constexpr TileCosts c = OP < kForwardKeep ? kCosts : OP == kDgradKept ? kCostsKept : kCosts8;
    auto rounds = [&](int height, int width, int64_t slots) {
        return (tiles_of(r, height, columns, columns_of_256 * width / 256) + slots - 1) / slots;
    };
    const int64_t large = rounds(256, 256, 256) * (c.large + sum * c.large_sum / 80);
    const int64_t square = rounds(128, 128, 512) * (c.square + sum * c.square_sum / 80);
    const int64_t small = rounds(64, 128, two_buffers<OP>(sum) ? 768 : 512) * (c.small + sum * c.small_sum / 80);
    if (large <= square && large <= small)
        return kLarge;
    if (square <= small)
        return kSquare;
    return sum >= 1024 && tiles_of(r, 64, columns, columns_of_256 / 2) <= 256 ? kSmallSplit : kSmall;
}

// A product's tiles. From 64 rows an expert the sizes of best_tiles. Below,
// tiles of 64 rows above the 32 of the smallest (a tile more reads an expert's
// weights again), unless they leave CUs idle (of 64 and 32 rows: 7 experts of
// 2136 rows, 112 x 7160 59 / 78, 2 of 647, 1408 x 2920 27 / 38). Measured, us,
// large / 64 rows / 32 rows, gated:
//   16 experts of 2048 x 7168, 16 rows each 156 / 157 / 157, 48 rows
//   159 / 159 / 198, 96 rows 167 / 219 / 283;
//   64 of 1024 x 2048, 16 rows 128 / 113 / 108, 64 rows 132 / 115 / 121;
//   16 of 512 x 1024 (64 to 128 large tiles), 16 rows 12.1 / 9.5 / 8.3;
//   8 of 2048 x 7168, 256 ragged rows: 106 / 82 / 113.
// Pre-activations kept in 8 bits need 32 gates a wave, so the small tiles'
// waves are two by two there.
template <int OP, typename A> hipError_t start_forward(const A &a, hipStream_t stream)
{
    constexpr int P = is_keep(OP) ? 2 : 4, Q = 4 / P;
    const int64_t rows = a.r.num_rows, n = a.r.n;
    hipError_t status;
    if (start_split<OP>(a, rows, stream, status))
        return status;
    if (rows > 64 * n) {
        const TileSize size = best_tiles<OP>(a.r, a.np, is_glu(OP) ? 128 : 256, a.sum);
        if (size == kLarge)
            return start<OP, 256, 256, 64, 2, 4, 2>(a, rows, stream);
        if (size == kSquare)
            return start<OP, 128, 128, 64, 2, 2, 2>(a, rows, stream);
        if (size == kSmallSplit)
            return start<OP, 128, 64, 64, 3, P, Q, 2>(a, rows, stream);
    }
    const bool wide = rows > 64 * n || (rows > 20 * n && tiles_of(a.r, 64, a.np, is_glu(OP) ? 64 : 128) >= 256);
    if constexpr (OP >= kForwardKeep) {
        // two buffers as said above; sums of few rows an expert, which wait for
        // the weights, up to half as long (int8, 64 of 16 rows, 1024 x 2048 42.0 with
        // three buffers, 45.2 with two; 42 of 20, 416 x 592 6.8 with four, 6.2 with two)
        if (wide && (rows > 64 * n ? two_buffers<OP>(a.sum) : a.sum <= 640))
            return start<OP, 128, 64, 64, 2, P, Q>(a, rows, stream);
        if (!wide && a.sum <= 640)
            return start<OP, 128, 32, 64, 2, P, Q>(a, rows, stream);
    }
    return wide ? start<OP, 128, 64, 64, 3, P, Q>(a, rows, stream) : start<OP, 128, 32, 64, 4, P, Q>(a, rows, stream);
}

// The input gradient's. Few rows an expert, us, large / small tiles: 16 experts
// of 2048 x 7168, 16 rows each 84.5 / 87.1; 64 of 1024 x 2048, 16 rows 44.8 / 43.1.
template <int OP, typename A> hipError_t start_dgrad(const A &a, hipStream_t stream)
{
    const int64_t rows = a.r.num_rows;
    hipError_t status;
    if (start_split<OP>(a, rows, stream, status))
        return status;
    const TileSize size = best_tiles<OP>(a.r, a.np, 256, a.sum);
    if (size == kLarge)
        return start<OP, 256, 256, 64, 2, 4, 2>(a, rows, stream);
    if (size == kSquare)
        return start<OP, 128, 128, 64, 2, 2, 2>(a, rows, stream);
    if (size == kSmallSplit)
        return start<OP, 128, 64, 64, 3, 4, 1, 2>(a, rows, stream);
    if constexpr (OP == kDgradKept) {
        if (two_buffers<OP>(a.sum))
            return start<OP, 128, 64, 64, 2, 4, 1>(a, rows, stream);
    }
    return start<OP, 128, 64, 64, 3, 4, 1>(a, rows, stream);
}

}  // namespace
}  // namespace epx
