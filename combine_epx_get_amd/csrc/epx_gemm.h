// epx_gemm.h -- pieces shared by the grouped matrix products (internal).
//
// A product's two operands are P, whose index runs along the contiguous
// direction of the output, and Q, whose index is the output row. P is the
// first operand of the matrix instruction, so that the four results of a
// lane are four consecutive elements of an output row.
#pragma once

#include "epx_device.h"
#include "epx_operators.h"

namespace epx {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kXcds = 8;
// A byte offset behind the end of every buffer (buffers hold at most 2^31
// bytes): loads there return zeros.
constexpr uint32_t kOutside = 0x80000000u;

template <int V> using Int = std::integral_constant<int, V>;

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ const char *uniform_ptr(const void *p)
{
    const uint64_t a = (uint64_t)p;
    const uint32_t lo = (uint32_t)uniform((int)a), hi = (uint32_t)uniform((int)(a >> 32));
    return (const char *)(((uint64_t)hi << 32) | lo);
}

// Buffer descriptor of `bytes` bytes from `base`: reads past them give zeros.
__device__ __forceinline__ i32x4 buffer_of(const char *base, uint32_t bytes)
{
    const uint64_t a = (uint64_t)base;
    i32x4 r;
    r.x = uniform((int)a);
    r.y = uniform((int)(a >> 32) & 0xFFFF);
    r.z = uniform((int)bytes);
    r.w = 0x00020000;
    return r;
}

__device__ __forceinline__ uint32_t lds_offset(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char *)p;
}

// 16 bytes a lane from the buffer to LDS at lds + 16 * lane (lds uniform).
// The copy is asynchronous: wait_copies() orders it.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, i32x4 buf, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dwordx4 %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(offset), "s"(buf)
                 : "memory");
}

// 4 bytes a lane to LDS at lds + 4 * lane.
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, i32x4 buf, uint32_t offset)
{
    asm volatile("s_mov_b32 m0, %0\n\t"
                 "s_nop 0\n\t"
                 "buffer_load_dword %1, %2, 0 offen lds"
                 :: "s"(lds), "v"(offset), "s"(buf)
                 : "memory");
}

// Waits until at most PENDING of this wave's copies are under way and its
// own LDS reads are done, then for the workgroup's other waves: afterwards
// every wave's waited-for copies are visible, and what was read before may
// be overwritten.
template <int PENDING> __device__ __forceinline__ void wait_copies()
{
    // the same wait for LDS reads where the compiler counts it (lgkmcnt 0, the
    // other counters at their most): else it waits for them again later
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(PENDING) : "memory");
}

// The same for buffers that only this wave uses.
template <int PENDING> __device__ __forceinline__ void wait_own_copies()
{
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(PENDING) : "memory");
}

// Every copy of this wave is done (before its LDS is given back).
__device__ __forceinline__ void drain_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

template <typename T> __device__ __forceinline__ T lds_read(uint32_t at)
{
    return *(const __attribute__((address_space(3))) T *)(uintptr_t)at;
}

// c += a b with the sum held in the accumulation registers throughout: left
// to itself the compiler moves sums that fill all 256 of them between the two
// register files inside the loop. It does not know this for a matrix
// instruction, so nothing but another one (of another sum, or at least four
// later) may touch a sum until mfma_in_place_last() has waited.
__device__ __forceinline__ void mfma_in_place(f32x4 &c, bf16x8 a, bf16x8 b)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}

// The last of a step. Where no step follows (more is 0), it waits in the same
// statement for the longest time that a result of a 16x16 instruction can
// need, so that whatever reads, copies or spills a sum behind the loop finds
// it done. A statement of its own behind the loop does not order that: the
// compiler read sums, and with the sums as its operands copied them, ahead of
// it, 11 to 18 wait states after the last instruction.
__device__ __forceinline__ void mfma_in_place_last(f32x4 &c, bf16x8 a, bf16x8 b, int more)
{
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\t"
                 "s_cmp_lg_u32 %3, 0\n\t"
                 "s_cbranch_scc1 2\n\t"   // over the two waits
                 "s_nop 15\n\t"
                 "s_nop 15"
                 : "+a"(c)
                 : "v"(a), "v"(b), "s"(more)
                 : "scc");
}

// Sums of WK groups of waves that divided a tile's sum: every group's go to its
// RING bytes of LDS, and each of them adds up, in the order of the groups, NE
// of the NJ columns of fragments, from j0 = group * NE on (groups past the
// last get none). WAVES waves a group; the groups' copies have arrived.
template <int WK, int RING, int WAVES, int NI, int NJ, int NE>
__device__ __forceinline__ void join_groups(uint32_t lds, int group, int wave, const f32x4 (&acc)[NI][NJ],
                                            f32x4 (&all)[NI][NE])
{
    static_assert(NJ % NE == 0 && WK * NE >= NJ && RING >= WAVES * NI * NJ * kWave * 16, "");
    auto at = [&](int of, int i, int j) {
        return lds + (uint32_t)of * RING + (uint32_t)((((wave * NI + i) * NJ + j) * kWave + lane_id()) * 16);
    };
    if constexpr (WAVES > 1)
        __syncthreads();   // a group's waves are done with its buffers
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
            *(__attribute__((address_space(3))) f32x4 *)(uintptr_t)at(group, i, j) = acc[i][j];
    __syncthreads();
    const int j0 = group * NE;
    if (j0 >= NJ)
        return;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NE; ++j) {
            all[i][j] = lds_read<f32x4>(at(0, i, j0 + j));
#pragma unroll
            for (int of = 1; of < WK; ++of)
                all[i][j] += lds_read<f32x4>(at(of, i, j0 + j));
        }
}

// ---------------------------------------------------------------- tiles
// Rows of expert e, 0 for a range outside the buffers.
__device__ __forceinline__ int rows_of(const ExpertRows &r, int e, int &off)
{
    if (e >= r.n)
        return 0;
    off = r.offset[e];
    const int c = r.count[e];
    if (c <= 0)
        return 0;
    if (off < 0 || (int64_t)off + c > r.num_rows) {
        if (kChecked)
            atomicAdd(r.viol, 1ull);
        return 0;
    }
    return c;
}

struct Tile {
    int expert;
    int row0, rows;   // first row of the tile and rows from there to the expert's end
    int p, q;         // tile indexes along P and (within the expert) Q
    int sum;          // the expert's rows, where they are summed over
};

// Row tiles of an expert with c rows. SPLIT: a last tile of at most TQ / 2
// rows is small, and small tiles are counted (and run) apart.
template <int TQ, bool SPLIT> __device__ __forceinline__ int row_tiles(int c, bool small)
{
    const int rem = c % TQ;
    if (!SPLIT)
        return small ? 0 : c / TQ + (rem > 0);
    return small ? rem > 0 && rem <= TQ / 2 : c / TQ + (rem > TQ / 2);
}

// Which of `tiles` tiles an XCD's workgroup number `slot` computes; false when
// none is left for it. `slots` receives the workgroups that every XCD needs
// for all of them.
//
// Neighbours in the order of tiles share operands. They are handed out in
// rounds of about 256, one tile a CU, in which every XCD takes a run of
// neighbours: those share what they read through the XCD's L2, and the runs
// of one round through the memory-side cache (256 MB), which rows and weights
// of a whole batch would not fit. A contiguous eighth of all tiles per XCD
// instead spreads a round over the whole batch and read about twice as much
// from HBM (32768 rows, one matrix of 4096 x 7168: the copies alone took 1310
// us that way, against 1155 us for half as many rows of tiles at a time).
__device__ __forceinline__ bool spread(int64_t tiles, int xcd, int64_t slot, int64_t &id, int64_t &slots)
{
    constexpr int kRound = 256;
    const int64_t rounds = (tiles + kRound - 1) / kRound;
    const int64_t run = rounds == 0 ? 0 : (tiles + kXcds * rounds - 1) / (kXcds * rounds);
    slots = rounds * run;
    if (slot >= slots)
        return false;
    const int64_t round = slot / run;
    id = (round * kXcds + xcd) * run + slot - round * run;
    return id < tiles;
}

// Tile `id` of `total` row tiles by pt column tiles, in the order of tiles:
// GQ row tiles side by side, column after column.
__device__ __forceinline__ void place(int64_t id, int total, int pt, int &p, int &q)
{
    constexpr int GQ = 4;
    const int64_t grp = id / ((int64_t)GQ * pt);
    const int rem = (int)(id - grp * GQ * pt);
    const int q0 = (int)grp * GQ;
    const int gq = total - q0 < GQ ? total - q0 : GQ;
    p = rem / gq;
    q = q0 + rem - p * gq;
}

// Tile of workgroup `b` for products whose row tiles are ragged: expert e has
// ceil(rows / TQ) row tiles with pt column tiles each. Consecutive workgroups
// run on different XCDs. Small tiles come after all others: they fill the
// last round of workgroups, which whole tiles would leave mostly idle (32768
// rows on 16 experts: 136 to 144 row tiles of 256, where 128 would do). Every
// wave computes the same. False when there is no tile for this workgroup.
template <int TQ, bool SPLIT>
__device__ __forceinline__ bool find_tile(const ExpertRows &r, int pt, int b, Tile &t)
{
    const int lane = lane_id();
    int whole = 0, part = 0;
    for (int e0 = 0; e0 < r.n; e0 += kWave) {
        int off;
        const int c = rows_of(r, e0 + lane, off);
        whole += __builtin_amdgcn_readlane(wave_inclusive_scan(row_tiles<TQ, SPLIT>(c, false)), kWave - 1);
        if (SPLIT)
            part += __popcll(__ballot(row_tiles<TQ, SPLIT>(c, true) > 0));
    }
    int64_t slot = b / kXcds, id, slots;
    bool small = false;
    if (!spread((int64_t)whole * pt, b % kXcds, slot, id, slots)) {
        slot -= slots;
        small = true;
        if (!SPLIT || slot < 0 || !spread((int64_t)part * pt, b % kXcds, slot, id, slots))
            return false;
    }
    int q;
    place(id, small ? part : whole, pt, t.p, q);
    int before = 0;
    for (int e0 = 0; e0 < r.n; e0 += kWave) {
        int off = 0;
        const int c = rows_of(r, e0 + lane, off);
        const int nt = row_tiles<TQ, SPLIT>(c, small);
        const int incl = wave_inclusive_scan(nt) + before;
        const uint64_t past = __ballot(incl > q);
        if (past != 0) {
            const int win = __builtin_ctzll(past);
            const int rows = __builtin_amdgcn_readlane(c, win);
            t.expert = e0 + win;
            t.q = small ? rows / TQ
                        : q - (__builtin_amdgcn_readlane(incl, win) - __builtin_amdgcn_readlane(nt, win));
            t.row0 = __builtin_amdgcn_readlane(off, win) + t.q * TQ;
            t.rows = rows - t.q * TQ;
            return true;
        }
        before = __builtin_amdgcn_readlane(incl, kWave - 1);
    }
    return false;
}

// Row tiles of TQ rows that n experts with rows rows in all can have.
inline int64_t most_row_tiles(int64_t rows, int n, int tq)
{
    return rows / tq + (rows < n ? rows : n);
}

// Workgroups for `tiles` tiles at most, whole and small ones handed out apart
// (spread: at most tiles / 8 + tiles / 256 + 2 an XCD for each kind).
inline int64_t tile_blocks(int64_t tiles)
{
    return tiles == 0 ? 0 : (tiles / kXcds + tiles / 256 + 4) * kXcds;
}

// From lane group g holding columns 4 g .. 4 g + 3 of each of two
// neighbouring fragments to holding columns 8 g .. 8 g + 7 of the two: a write
// of 16 bytes a lane is then one of 64 neighbouring bytes a row (bf16).
__device__ __forceinline__ void merge_columns(f32x4 &a, f32x4 &b)
{
    typedef uint32_t u32p __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const float aq = a[q], bq = b[q];
        const u32p h = __builtin_amdgcn_permlane32_swap(__float_as_uint(aq), __float_as_uint(bq), false, false);
        const u32p x = __builtin_amdgcn_permlane16_swap(h.x, h.y, false, false);
        a[q] = __uint_as_float(x.x);
        b[q] = __uint_as_float(x.y);
    }
}

// Tiles of `height` rows and `tile_columns` columns that a product has with
// its experts equally full, each with a last tile half full.
inline int64_t tiles_of(const ExpertRows &r, int height, int64_t columns, int tile_columns)
{
    const int64_t experts = r.n < r.num_rows ? r.n : r.num_rows;
    const int64_t half_full = r.num_rows / height + experts / 2;
    return (half_full > experts ? half_full : experts) * ((columns + tile_columns - 1) / tile_columns);
}

// ---------------------------------------------------------------- activation
// The hardware's reciprocal and base-2 exponential, a step or two each, and
// the rounding of v * log2(e), which grows with v: 2^-22 * (1 + |v|) relative to
// the value at most, far below the bf16 (or E4M3) step of what it is used for.
// Below -87 the reciprocal is subnormal and comes back as 0: silu, which is
// then less than 2^-119, is 0.
__device__ __forceinline__ float sigmoid32(float v) { return __builtin_amdgcn_rcpf(1.0f + __expf(-v)); }
__device__ __forceinline__ float swiglu(float gate, float up) { return gate * sigmoid32(gate) * up; }

__device__ __forceinline__ uint32_t pack2(float a, float b) { return f32_to_bf16(a) | (f32_to_bf16(b) << 16); }

// Widths of the vectors that hold a lane's N consecutive results.
template <int N> struct Cols { float v[N]; };

// Columns [c, c + N) of a bf16 row that has `width` columns (a multiple of 8).
template <int N>
__device__ __forceinline__ void store_bf16(uint16_t *row, int c, int width, const Cols<N> &o)
{
    if constexpr (N == 4) {
        if (c < width)
            *(u32x2 *)(row + c) = u32x2{pack2(o.v[0], o.v[1]), pack2(o.v[2], o.v[3])};
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8)
            if (c + i < width)
                *(u32x4 *)(row + c + i) = u32x4{pack2(o.v[i], o.v[i + 1]), pack2(o.v[i + 2], o.v[i + 3]),
                                                pack2(o.v[i + 4], o.v[i + 5]), pack2(o.v[i + 6], o.v[i + 7])};
    }
}

// The same of a float32 row, written or added.
template <int N>
__device__ __forceinline__ void store_f32(float *row, int c, int width, const Cols<N> &o, bool add)
{
#pragma unroll
    for (int i = 0; i < N; i += 4)
        if (c + i < width) {
            f32x4 *d = (f32x4 *)(row + c + i);
            const f32x4 x = {o.v[i], o.v[i + 1], o.v[i + 2], o.v[i + 3]};
            *d = add ? *d + x : x;
        }
}

// Columns [c, c + N) of a bf16 row; 0 past its `width` columns.
template <int N> __device__ __forceinline__ Cols<N> load_bf16(const uint16_t *row, int c, int width)
{
    Cols<N> o;
    if constexpr (N == 4) {
        const u32x2 v = c < width ? *(const u32x2 *)(row + c) : u32x2{0, 0};
        o.v[0] = bf16_lo(v.x);
        o.v[1] = bf16_hi(v.x);
        o.v[2] = bf16_lo(v.y);
        o.v[3] = bf16_hi(v.y);
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 8) {
            const u32x4 v = c + i < width ? *(const u32x4 *)(row + c + i) : u32x4{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                o.v[i + 2 * q] = bf16_lo(v[q]);
                o.v[i + 2 * q + 1] = bf16_hi(v[q]);
            }
        }
    }
    return o;
}

}  // namespace epx
