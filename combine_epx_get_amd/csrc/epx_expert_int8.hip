// epx_expert_int8.hip -- the experts' products of int8 rows and int8 weights,
// with a float32 scale per row and per column, on the matrix cores of gfx950.
//
//   z[r, n] = fl32(sum_k x[r, k] w[e][n, k]) * x_scale[r] * w_scale[e][n]
//
// The tile loop of the bf16 products: a 16-byte chunk holds 16 values in place
// of 8, the matrix instruction (16x16x64) takes chunks as the bf16 one
// (16x16x32) does and multiplies twice the values in the same cycles. Sums are
// whole numbers in 32 bits, exact up to the inner limit of epx.h, so neither
// tiles nor groups of waves change a result; scales, activation and the 8-bit
// form of the pre-activations are applied to them before the one rounding.
//
// Few rows an expert (256 rows over 8 experts of 2 x 2048 x 7168): the weights'
// bytes, 43-44 us, 5.4 TB/s, and 45.5 with the pre-activations kept. Many (32768
// ragged rows, 16 experts of 2 x 2048 x 7168): 760-820 us, 2.3-2.5 POP/s; the
// matrix cores are 64 % busy, waves wait 28 % of their time (a library product of
// one weight, without scales or activation, took 860-875 us there and reached 2.46
// POP/s at 8192^3); 829-835 kept. The second product, without activation: 8 of
// 7168 x 2048, 256 rows 27 us, 4.4 TB/s of weights; 16 of them, 32768 rows 485-490
// us, 2.0 POP/s: half as many steps a tile beside the same results. One row of one
// expert: 7.4 us.
#include "epx_expert_tiles.h"

namespace epx {

hipError_t launch_expert_gemm_int8(const ExpertRows &r, const int8_t *x, const float *x_scales,
                                   const int8_t *w, const float *w_scales, int32_t width,
                                   int32_t inner, bool swiglu, int8_t *kept, uint8_t *kept_scales,
                                   void *out, hipStream_t stream)
{
    Args8 a = {};
    a.r = r;
    a.p = (const char *)w;
    a.q = (const char *)x;
    a.np = width;
    a.sum = inner / 2;
    a.out = out;
    a.q_scales = x_scales;
    a.p_scales = w_scales;
    a.kept = kept;
    a.kept_scales = kept_scales;
    if (kept)
        return start_forward<kInt8Keep>(a, stream);
    return swiglu ? start_forward<kInt8Glu>(a, stream) : start_forward<kInt8>(a, stream);
}

}  // namespace epx
