// epx_operators.h -- launchers of the operators around the exchange: router,
// combine's gradient, the experts' products and 4-bit conversion (internal).
// Apart from epx_internal.h, so that the exchange's kernels keep the sources
// that their profiles were taken on.
#pragma once

#include <type_traits>

#include "epx_internal.h"

namespace epx {

// Router: choice and weights, and the weights' gradient (g gives T, E, k).
hipError_t launch_route(const Geometry &g, const void *logits, bool bf16, bool softmax,
                        const float *bias, bool renormalize, float scale, int32_t *idx,
                        float *weights, hipStream_t stream);
hipError_t launch_route_backward(const Geometry &g, const void *logits, bool bf16, bool softmax,
                                 bool renormalize, float scale, const int32_t *idx,
                                 const float *dweights, void *dlogits, hipStream_t stream);
// dw may be null (y is then not read).
hipError_t launch_combine_backward(const Geometry &g, const epx_layout &L, const void *dout,
                                   const void *y, int64_t y_rows, const float *w, int32_t hidden,
                                   void *dy, float *dw, hipStream_t stream);

// The experts' row ranges as the kernels take them.
struct ExpertRows {
    const int32_t *offset, *count;
    int32_t n, num_rows;
    unsigned long long *viol;   // as in Geometry
};
// Grouped products (width and inner as in epx.h). preact: may be null
// forwards; null when the gradient passes no activation.
hipError_t launch_expert_gemm(const ExpertRows &r, const void *x, const void *w, int32_t width,
                              int32_t inner, bool swiglu, void *preact, void *out,
                              hipStream_t stream);
hipError_t launch_expert_dgrad(const ExpertRows &r, const void *dy, const void *w, int32_t width,
                               int32_t inner, const void *preact, void *dx, hipStream_t stream);
hipError_t launch_expert_wgrad(const ExpertRows &r, const void *dy, const void *x, int32_t width,
                               int32_t inner, bool f32, bool accumulate, void *dw,
                               hipStream_t stream);
hipError_t launch_expert_gemm_mxfp4(const ExpertRows &r, const uint8_t *x, const float *x_scales,
                                    const uint8_t *w, const uint8_t *w_scales, int32_t width,
                                    int32_t inner, bool swiglu, bool fp8_out, void *out,
                                    float *out_scales, hipStream_t stream);
hipError_t launch_mxfp4_quantize(const void *x, int64_t num_rows, int32_t inner, uint8_t *codes,
                                 uint8_t *scales, hipStream_t stream);
hipError_t launch_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t num_rows,
                                   int32_t inner, void *out, hipStream_t stream);

}  // namespace epx
