// epx_expert_gemm.hip -- the experts' products on ragged row ranges, and
// their gradients, on the matrix cores of gfx950 (bf16 in, float32 sums).
//
//   forward  out[r, n]  = sum_k x[r, k] w[e][n, k]     (P = w, Q = x)
//   dgrad    dx[r, k]   = sum_n dy[r, n] w[e][n, k]    (P = w, Q = dy)
//   wgrad    dw[e][n,k] = sum_r dy[r, n] x[r, k]       (P = x, Q = dy)
//
// Tiles of TP x TQ results; the operands come to LDS in steps of BK along
// the sum, by direct copies (no registers), in a ring of S buffers, so that
// S - 1 steps are under way while one is multiplied.
//
// An operand whose sum index is contiguous in memory is kept as rows of BK
// (a fragment is one 16-byte read); one whose sum index is the row in memory
// as rows of the tile's columns (a fragment is two transposing reads of 8
// bytes). The 16-byte chunks of a row are permuted by an exclusive or with
// bits of the row index, in the copies' source addresses, so that the reads
// of a fragment touch every LDS bank equally.
//
// Few tiles: groups of waves divide a tile's sum among them, each with a ring
// of its own, and add their sums up through LDS in a fixed order; no memory of
// a call's own and no second launch is needed.
//
// Reads past an operand's last row, column or sum index return zeros (the
// buffer descriptors' range check), so ragged tiles need no other code; a
// tile writes the rows and columns that exist.
//
// Few rows an expert: the weights' bytes bound it (256 rows over 8 experts of
// 2 x 2048 x 7168: 80 us, 5.9 TB/s). Many: the matrix cores, at the clock that
// their own load leaves, and the wait for copies at a step's meeting (16
// experts x 2048 rows, 4096 x 7168: forward 1390-1435 us, 1.34-1.38 PFLOP/s;
// dgrad 1420-1480; wgrad 1590-1640; one library product of 32768 rows 1219).
#include "epx_gemm.h"

namespace epx {
namespace {

enum Op { kForward, kForwardGlu, kDgrad, kDgradGlu, kWgrad, kWgradF32 };

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
    static constexpr bool kGlu = OP == kForwardGlu;
    static constexpr bool kPCols = OP >= kDgrad;     // P's sum index is the row in memory
    static constexpr bool kWeights = OP >= kWgrad;
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

    static __device__ __forceinline__ void run(const Args &a, const Tile &t, char *smem)
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

        f32x4 acc[NI][NJ];
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

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
                    __builtin_amdgcn_sched_barrier(0);
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
                    __builtin_amdgcn_sched_barrier(0);
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
                                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[i], qf[j], acc[i][j], 0, 0, 0);
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
            f32x4 all[NI][NE];
            join_groups<WK, kRing, kWaves>(lds_offset(smem), group, wave, acc, all);
            if (group * NE < NJ)
                write<NE>(a, t, wp, wq, group * NE, all);
        }
    }

    // Results: lane (m, g) of fragment pair (i, j) has row j * 16 + m and
    // columns 4 g .. 4 g + 3 of fragment i. Two fragments are neighbours
    // already where P's rows are read that way (GI), and are merged here
    // otherwise, so that the lanes of a write are neighbours in 64 bytes
    // of a row (float32 results are so as they are).
    template <int N>
    static __device__ __forceinline__ void write(const Args &a, const Tile &t, int wp, int wq, int j0, f32x4 (&acc)[NI][N])
    {
        const int m = lane_id() & 15, g = lane_id() >> 4;
        constexpr int PC = kGlu ? TP / 2 : TP;
        const int col0 = t.p * PC;
        constexpr bool kMerge = kPCols && OP != kWgradF32 && NI % 2 == 0;
        constexpr int W = kMerge ? 2 : GI, NG = kHalf / W;
        if constexpr (kMerge) {
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int n = 0; n < NG; ++n)
                    merge_columns(acc[2 * n][j], acc[2 * n + 1][j]);
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int r = wq * (TQ / WQ) + (j0 + j) * 16 + m;
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                const int c = col0 + wp * (PC / WP) + n * 16 * W + 4 * W * g;
                Cols<4 * W> u, v;
#pragma unroll
                for (int i = 0; i < W; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        u.v[4 * i + q] = acc[n * W + i][j][q];
                        if constexpr (kGlu)
                            v.v[4 * i + q] = acc[kHalf + n * W + i][j][q];
                    }
                if constexpr (kWeights) {
                    const int row = t.q * TQ + r;
                    if (row >= a.nq)
                        continue;
                    const int64_t o = ((int64_t)t.expert * a.nq + row) * a.np;
                    if constexpr (OP == kWgradF32)
                        store_f32((float *)a.out + o, c, a.np, u, a.accumulate);
                    else
                        store_bf16((uint16_t *)a.out + o, c, a.np, u);
                } else {
                    if (r >= t.rows)
                        continue;
                    const int64_t row = t.row0 + r;
                    if constexpr (OP == kForwardGlu) {
                        if (a.preact_out) {
                            store_bf16(a.preact_out + row * 2 * a.np, c, a.np, u);
                            store_bf16(a.preact_out + row * 2 * a.np + a.np, c, a.np, v);
                        }
#pragma unroll
                        for (int q = 0; q < 4 * W; ++q)
                            u.v[q] = swiglu(u.v[q], v.v[q]);
                    }
                    if constexpr (OP == kDgradGlu) {
                        const uint16_t *pre = a.preact_in + row * 2 * a.np;
                        const Cols<4 * W> gate = load_bf16<4 * W>(pre, c, a.np), up = load_bf16<4 * W>(pre + a.np, c, a.np);
#pragma unroll
                        for (int q = 0; q < 4 * W; ++q) {
                            const float s = sigmoid32(gate.v[q]), d = u.v[q];
                            u.v[q] = d * up.v[q] * (s * (1.0f + gate.v[q] * (1.0f - s)));
                            v.v[q] = d * (gate.v[q] * s);
                        }
                        uint16_t *dx = (uint16_t *)a.out + row * 2 * a.np;
                        store_bf16(dx, c, a.np, u);
                        store_bf16(dx + a.np, c, a.np, v);
                    } else {
                        store_bf16((uint16_t *)a.out + row * a.np, c, a.np, u);
                    }
                }
            }
        }
    }
};

// The large tiles' kernels carry the smaller ones for an expert's last rows.
template <int OP, int TP, int TQ, int BK, int S, int WP, int WQ, int WK>
__global__ __launch_bounds__(WP *WQ *WK *kWave, (Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>::kPerSimd)) void gemm_kernel(Args a)
{
    using K = Kernel<OP, TP, TQ, BK, S, WP, WQ, WK>;
    __shared__ __attribute__((aligned(1024))) char smem[K::kLds];
    Tile t;
    if constexpr (K::kWeights) {
        const int64_t tiles = (int64_t)a.pt * a.qt;   // of every expert
        int64_t id, slots;
        if (!spread(tiles * a.r.n, blockIdx.x % kXcds, blockIdx.x / kXcds, id, slots))
            return;
        t.expert = (int)(id / tiles);
        place(id - t.expert * tiles, a.qt, a.pt, t.p, t.q);
        t.row0 = 0;
        t.sum = uniform(rows_of(a.r, t.expert, t.row0));
        t.row0 = uniform(t.row0);
        t.rows = TQ;
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
hipError_t start(Args a, int64_t rows_or_n, hipStream_t stream)
{
    constexpr int PC = OP == kForwardGlu ? TP / 2 : TP;
    a.pt = (a.np + PC - 1) / PC;
    int64_t blocks;
    if (OP >= kWgrad) {
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
template <int OP>
bool start_split(const Args &a, int64_t rows, hipStream_t stream, hipError_t &status)
{
    constexpr int FULL = OP == kForwardGlu ? 16 : 32;
    if (tiles_of(a.r, 32, a.np, FULL) <= 256)
        status = start<OP, 32, 32, 64, 2, 1, 1, 8>(a, rows, stream);
    else if (tiles_of(a.r, 32, a.np, 2 * FULL) <= 256)
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
TileSize best_tiles(const ExpertRows &r, int32_t columns, int columns_of_256, int64_t sum)
{
    auto rounds = [&](int height, int width, int64_t slots) {
        return (tiles_of(r, height, columns, columns_of_256 * width / 256) + slots - 1) / slots;
    };
    // ns
    const int64_t large = rounds(256, 256, 256) * (9000 + sum * 47 / 2);
    const int64_t square = rounds(128, 128, 512) * (4500 + sum * 33 / 2);
    const int64_t small = rounds(64, 128, 512) * (4200 + sum * 63 / 5);
    if (large <= square && large <= small)
        return kLarge;
    if (square <= small)
        return kSquare;
    return sum >= 1024 && tiles_of(r, 64, columns, columns_of_256 / 2) <= 256 ? kSmallSplit : kSmall;
}

}  // namespace

hipError_t launch_expert_gemm(const ExpertRows &r, const void *x, const void *w, int32_t width,
                              int32_t inner, bool swiglu, void *preact, void *out,
                              hipStream_t stream)
{
    Args a = {};
    a.r = r;
    a.p = (const char *)w;
    a.q = (const char *)x;
    a.np = width;
    a.sum = inner;
    a.preact_out = (uint16_t *)preact;
    a.out = out;
    // From 64 rows an expert the sizes of best_tiles. Below, tiles of 64 rows
    // above the 32 of the smallest (a tile more reads an expert's weights again),
    // unless they leave CUs idle (of 64 and 32 rows: 7 experts of 2136 rows, 112 x
    // 7160 59 / 78, 2 of 647, 1408 x 2920 27 / 38). Measured, us, large / 64 rows / 32 rows, gated:
    //   16 experts of 2048 x 7168, 16 rows each 156 / 157 / 157, 48 rows
    //   159 / 159 / 198, 96 rows 167 / 219 / 283;
    //   64 of 1024 x 2048, 16 rows 128 / 113 / 108, 64 rows 132 / 115 / 121;
    //   16 of 512 x 1024 (64 to 128 large tiles), 16 rows 12.1 / 9.5 / 8.3;
    //   8 of 2048 x 7168, 256 ragged rows: 106 / 82 / 113.
    const int64_t rows = r.num_rows, n = r.n;
    hipError_t status;
    if (swiglu ? start_split<kForwardGlu>(a, rows, stream, status) : start_split<kForward>(a, rows, stream, status))
        return status;
    if (rows > 64 * n) {
        const TileSize size = best_tiles(r, width, swiglu ? 128 : 256, inner);
        if (size == kLarge)
            return swiglu ? start<kForwardGlu, 256, 256, 64, 2, 4, 2>(a, rows, stream)
                          : start<kForward, 256, 256, 64, 2, 4, 2>(a, rows, stream);
        if (size == kSquare)
            return swiglu ? start<kForwardGlu, 128, 128, 64, 2, 2, 2>(a, rows, stream)
                          : start<kForward, 128, 128, 64, 2, 2, 2>(a, rows, stream);
        if (size == kSmallSplit)
            return swiglu ? start<kForwardGlu, 128, 64, 64, 3, 4, 1, 2>(a, rows, stream)
                          : start<kForward, 128, 64, 64, 3, 4, 1, 2>(a, rows, stream);
    }
    if (rows > 64 * n || (rows > 20 * n && tiles_of(r, 64, width, swiglu ? 64 : 128) >= 256))
        return swiglu ? start<kForwardGlu, 128, 64, 64, 3, 4, 1>(a, rows, stream)
                      : start<kForward, 128, 64, 64, 3, 4, 1>(a, rows, stream);
    return swiglu ? start<kForwardGlu, 128, 32, 64, 4, 4, 1>(a, rows, stream)
                  : start<kForward, 128, 32, 64, 4, 4, 1>(a, rows, stream);
}

hipError_t launch_expert_dgrad(const ExpertRows &r, const void *dy, const void *w, int32_t width,
                               int32_t inner, const void *preact, void *dx, hipStream_t stream)
{
    Args a = {};
    a.r = r;
    a.p = (const char *)w;
    a.q = (const char *)dy;
    a.np = inner;
    a.sum = width;
    a.preact_in = (const uint16_t *)preact;
    a.out = dx;
    // Few rows an expert, us, large / small tiles: 16 experts of 2048 x 7168, 16
    // rows each 84.5 / 87.1; 64 of 1024 x 2048, 16 rows 44.8 / 43.1.
    hipError_t status;
    if (preact ? start_split<kDgradGlu>(a, r.num_rows, stream, status)
               : start_split<kDgrad>(a, r.num_rows, stream, status))
        return status;
    const TileSize size = best_tiles(r, inner, 256, width);
    if (size == kLarge)
        return preact ? start<kDgradGlu, 256, 256, 64, 2, 4, 2>(a, r.num_rows, stream)
                      : start<kDgrad, 256, 256, 64, 2, 4, 2>(a, r.num_rows, stream);
    if (size == kSquare)
        return preact ? start<kDgradGlu, 128, 128, 64, 2, 2, 2>(a, r.num_rows, stream)
                      : start<kDgrad, 128, 128, 64, 2, 2, 2>(a, r.num_rows, stream);
    if (size == kSmallSplit)
        return preact ? start<kDgradGlu, 128, 64, 64, 3, 4, 1, 2>(a, r.num_rows, stream)
                      : start<kDgrad, 128, 64, 64, 3, 4, 1, 2>(a, r.num_rows, stream);
    return preact ? start<kDgradGlu, 128, 64, 64, 3, 4, 1>(a, r.num_rows, stream)
                  : start<kDgrad, 128, 64, 64, 3, 4, 1>(a, r.num_rows, stream);
}

hipError_t launch_expert_wgrad(const ExpertRows &r, const void *dy, const void *x, int32_t width,
                               int32_t inner, bool f32, bool accumulate, void *dw,
                               hipStream_t stream)
{
    Args a = {};
    a.r = r;
    a.p = (const char *)x;
    a.q = (const char *)dy;
    a.np = inner;
    a.nq = width;
    a.out = dw;
    a.accumulate = accumulate;
    // Few tiles, a workgroup a CU at most: 64 x 64 whose waves divide the sum
    // among them, else 64 x 128 with four pairs of waves. Measured, us, 64 x 64 /
    // 64 x 128 / 128 x 128: 2 experts of 376 x 648, 5200 rows each (132 tiles of
    // 64 x 64) 29 / 34 / 68; 4 of 512 x 512, 512 rows (256) 7.0 / 8.0 / 11.9; 4
    // of 512 x 1024 (256 of 64 x 128), 256 rows 10.2 / 7.3 / 9.1, 4096 rows 36 /
    // 28 / 56.
    const auto tiles = [&](int w, int i) { return (int64_t)((width + w - 1) / w) * ((inner + i - 1) / i) * r.n; };
    if (tiles(64, 64) <= 256)
        return f32 ? start<kWgradF32, 64, 64, 64, 2, 1, 1, 4>(a, r.n, stream)
                   : start<kWgrad, 64, 64, 64, 2, 1, 1, 4>(a, r.n, stream);
    if (tiles(64, 128) <= 256)
        return f32 ? start<kWgradF32, 128, 64, 32, 3, 2, 1, 4>(a, r.n, stream)
                   : start<kWgrad, 128, 64, 32, 3, 2, 1, 4>(a, r.n, stream);
    // Else large tiles (one a CU), small ones (128 x 128, three a CU, which
    // covers the start and end of short sums), or those with two groups of waves
    // (one a CU): what takes the least time by the rounds of workgroups and a
    // round's time, about linear in the rows of an expert. Measured, us, large /
    // small / two groups: 2 experts of 4624 x 368, 11246 rows each (222 small
    // tiles) 137 / 143 / 113; 8 of 512 x 1024, 1024 rows (256) 31 / 18.8 / 15.3; 16
    // of 512 x 1024, 128 rows (512) 16.4 / 10.7 / 14.7; 2 of 1408 x 2920, 647 rows
    // (506) 28.2 / 20.2 / 25.6; 7 of 112 x 7160, 2136 rows (392) 55 / 43 / 54; 16 of
    // 2048 x 7168, 64 rows 174 / 155 / -, 256 rows 259 / 238 / - (float32, whose
    // rounds of many tiles write more, 296 / 316), 1024 rows 509 / 546 / - (float32
    // 530 / 637); 64 of 1024 x 2048, 64 rows 105 / 82 / -, 1024 rows 306 / 331 / -.
    const int64_t sum = r.num_rows / r.n, count = tiles(128, 128);
    const auto rounds = [](int64_t t, int64_t slots) { return (t + slots - 1) / slots; };
    // ns
    const int64_t large = rounds(tiles(256, 256), 256) * (8000 + sum * 21);
    const int64_t pairs = rounds(count, 256) * (3000 + sum * 17 / 2);
    const int64_t small = count <= 512 ? 2500 + sum * 33 / 2 : rounds(count, 768) * ((f32 ? 5000 : 2500) + sum * 24);
    if (pairs < small && pairs < large)
        return f32 ? start<kWgradF32, 128, 128, 64, 2, 2, 2, 2>(a, r.n, stream)
                   : start<kWgrad, 128, 128, 64, 2, 2, 2, 2>(a, r.n, stream);
    if (large < small)
        return f32 ? start<kWgradF32, 256, 256, 64, 2, 4, 2>(a, r.n, stream)
                   : start<kWgrad, 256, 256, 64, 2, 4, 2>(a, r.n, stream);
    return f32 ? start<kWgradF32, 128, 128, 32, 3, 2, 2>(a, r.n, stream)
               : start<kWgrad, 128, 128, 32, 3, 2, 2>(a, r.n, stream);
}

}  // namespace epx
