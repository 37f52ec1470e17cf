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
#include "epx_expert_tiles.h"

namespace epx {
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
    return swiglu ? start_forward<kForwardGlu>(a, stream) : start_forward<kForward>(a, stream);
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
    return preact ? start_dgrad<kDgradGlu>(a, stream) : start_dgrad<kDgrad>(a, stream);
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
