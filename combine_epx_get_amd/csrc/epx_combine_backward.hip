// epx_combine_backward.hip -- gradient of the combine step on gfx950.
//
// out[t] = sum_j w[t,j] y[slot[t,j]] gives dy[slot[t,j]] = w[t,j] dout[t]
// (a scatter like dispatch's, scaled) and dw[t,j] = <dout[t], y[slot[t,j]]>
// (a gather like combine's). One pass does both: a workgroup holds a token's
// dout chunk in registers, writes the scaled rows and accumulates up to
// kRows dot products while the y rows stream by. Reads T*h*2 + T*k*h*2 bytes
// and writes T*k*h*2: HBM bound (4096 tokens of 7168, top-8: 196 to 200 us, 5.0
// to 5.1 TB/s, the rate of a large copy on this card; more chunks in flight a
// lane measured the same there and 28 us at 384 tokens).
//
// A dot product is summed in a fixed order that depends on the launch shape
// only: ascending chunks in each lane, lanes by xor, waves ascending.
#include "epx_device.h"
#include "epx_operators.h"

namespace epx {
namespace {

constexpr int kRows = 8;   // rows of one token per workgroup pass

__device__ __forceinline__ uint32_t scale2(float w, uint32_t v)
{
    return f32_to_bf16(w * bf16_lo(v)) | (f32_to_bf16(w * bf16_hi(v)) << 16);
}

__device__ __forceinline__ float dot2(uint32_t a, uint32_t b, float acc)
{
    acc = __builtin_fmaf(bf16_lo(a), bf16_lo(b), acc);
    return __builtin_fmaf(bf16_hi(a), bf16_hi(b), acc);
}

// Workgroup (t, s): rows j in [s * per, (s + 1) * per) of token t.
template <bool DOT>
__global__ __launch_bounds__(512) void combine_backward_kernel(
    const u32x4 *__restrict__ dout, const u32x4 *__restrict__ y, int nvec,
    const int32_t *__restrict__ slot, const float *__restrict__ w, int k, int per,
    u32x4 *__restrict__ dy, float *__restrict__ dw, int64_t y_rows, unsigned long long *viol,
    const int32_t *__restrict__ totals, int64_t T)
{
    __shared__ int32_t s_row[kMaxTopk];
    __shared__ float s_w[kMaxTopk];
    __shared__ float s_dot[8][kRows];
    const int64_t t = item_index();
    if (t >= T)
        return;
    const int j_beg = blockIdx.y * per, j_end = min(k, j_beg + per);
    const int bad = totals[3];
    if ((int)threadIdx.x < k) {
        const int r = slot[t * k + threadIdx.x];
        s_row[threadIdx.x] = in_bounds(r, y_rows, viol) ? r : -1;   // checked builds only
        s_w[threadIdx.x] = w[t * k + threadIdx.x];
    }
    __syncthreads();
    if (bad != 0)
        return;   // the layout saw out-of-range expert ids: the slots are undefined
    for (int j0 = j_beg; j0 < j_end; j0 += kRows) {
        const int n = min(kRows, j_end - j0);
        float acc[kRows];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            acc[i] = 0.0f;
        for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
            const u32x4 d = dout[t * nvec + c];
            u32x4 v[kRows];
            if (DOT) {
#pragma unroll
                for (int i = 0; i < kRows; ++i)
                    if (i < n && s_row[j0 + i] >= 0)
                        v[i] = __builtin_nontemporal_load(y + (int64_t)s_row[j0 + i] * nvec + c);
            }
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                if (i >= n || s_row[j0 + i] < 0)
                    continue;
                const float wi = s_w[j0 + i];
                u32x4 o;
                o.x = scale2(wi, d.x);
                o.y = scale2(wi, d.y);
                o.z = scale2(wi, d.z);
                o.w = scale2(wi, d.w);
                __builtin_nontemporal_store(o, dy + (int64_t)s_row[j0 + i] * nvec + c);
                if (DOT)
                    acc[i] = dot2(d.w, v[i].w, dot2(d.z, v[i].z, dot2(d.y, v[i].y, dot2(d.x, v[i].x, acc[i]))));
            }
        }
        if (DOT) {
            const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float a = acc[i];
#pragma unroll
                for (int dd = 32; dd > 0; dd >>= 1)
                    a += __shfl_xor(a, dd, kWave);
                if (lane_id() == 0)
                    s_dot[wave][i] = a;
            }
            __syncthreads();
            if ((int)threadIdx.x < n) {
                float a = 0.0f;
                for (int q = 0; q < waves; ++q)
                    a += s_dot[q][threadIdx.x];
                dw[t * k + j0 + threadIdx.x] = a;
            }
            __syncthreads();   // s_dot is written again by the next rows
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const Geometry &g, const epx_layout &L, const void *dout,
                                   const void *y, int64_t y_rows, const float *w, int32_t hidden,
                                   void *dy, float *dw, hipStream_t stream)
{
    const int nvec = hidden / 8;
    // rows per workgroup: all of a token's, but fewer where that leaves less
    // than 512 workgroups (384 tokens of 7168, top-8: 21.6 us, against 24.0 and
    // 24.8 with 1024 and 2048)
    int per = g.k;
    if (g.T < 512) {
        const int parts = (512 + g.T - 1) / g.T;
        per = (g.k + parts - 1) / parts;
    }
    int threads = (nvec + kWave - 1) / kWave * kWave;
    threads = threads > 512 ? 512 : threads;
    static_assert(kMaxTopk <= kWave, "a thread a choice, from the first wave");
    const dim3 grid = item_grid(g.T, (g.k + per - 1) / per);
    if (dw)
        launch(combine_backward_kernel<true>, grid, dim3(threads), 0, stream, (const u32x4 *)dout,
               (const u32x4 *)y, nvec, (const int32_t *)L.slot, w, g.k, per, (u32x4 *)dy, dw, y_rows,
               g.viol, (const int32_t *)L.totals, (int64_t)g.T);
    else
        launch(combine_backward_kernel<false>, grid, dim3(threads), 0, stream, (const u32x4 *)dout,
               (const u32x4 *)y, nvec, (const int32_t *)L.slot, w, g.k, per, (u32x4 *)dy, dw, y_rows,
               g.viol, (const int32_t *)L.totals, (int64_t)g.T);
    return hipGetLastError();
}

}  // namespace epx
