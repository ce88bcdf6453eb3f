// Gradient of the combine out[t, :] = sum_j w[t, j] y_sorted[p2s[t k + j], :]
// with respect to the expert outputs and the gate weights:
//   d_y[p2s[t k + j], :] = w[t, j] d_out[t, :]          (stored fp16, the type of y)
//   d_w[t, j]            = sum_h d_out[t, h] y_sorted[p2s[t k + j], h]
// Every pair owns its row of y_sorted, so nothing is accumulated across
// tokens and there are no atomics.  Bound by HBM: 2 k H bytes of y read and
// 2 k H of d_y written per token, 4 H of d_out read.  One MI355X, H = 4096,
// k = 8: 16,384 tokens 479 us (5.05 TB/s, what a copy reaches), 1,001 tokens
// 29.8 us.
//
// One block per token; a thread owns 8 columns of a pass, holds their d_out in
// registers and takes CW_J rows at a time, all loaded before the first is used.
// The CW_J products' sums stay in registers over the passes, then go over the
// lanes and, through LDS, over the waves.
#include "common.h"
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int CW_J = 8;

template <int THREADS>
__global__ __launch_bounds__(THREADS)
void combine_backward_kernel(const float* __restrict__ d_out, const uint16_t* __restrict__ y,
                             const float* __restrict__ w, const int32_t* __restrict__ p2s, int T, int k, int H,
                             uint16_t* __restrict__ d_y, float* __restrict__ d_w) {
    constexpr int WAVES = THREADS / WAVE;
    __shared__ float red[WAVES][MAX_TOPK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x) {
        const float* go = d_out + t * H;
        const int32_t* pt = p2s + t * k;
        for (int j0 = 0; j0 < k; j0 += CW_J) {
            float dot[CW_J];
#pragma unroll
            for (int j = 0; j < CW_J; ++j) dot[j] = 0.0f;
            for (int h = tid * 8; h < H; h += THREADS * 8) {
                const float4 ga = *reinterpret_cast<const float4*>(go + h);
                const float4 gb = *reinterpret_cast<const float4*>(go + h + 4);
                u32x4 q[CW_J];
                if (d_w) {
#pragma unroll
                    for (int j = 0; j < CW_J; ++j)
                        if (j0 + j < k) q[j] = ldg16_stream(y + (size_t)pt[j0 + j] * H + h);
                }
                const float v[8] = {ga.x, ga.y, ga.z, ga.w, gb.x, gb.y, gb.z, gb.w};
#pragma unroll
                for (int j = 0; j < CW_J; ++j) {
                    if (j0 + j >= k) break;
                    if (d_y) {
                        const float wj = w[t * k + j0 + j];
                        f16x8 o;
#pragma unroll
                        for (int i = 0; i < 8; ++i) o[i] = (_Float16)(wj * v[i]);
                        stg16(d_y + (size_t)pt[j0 + j] * H + h, __builtin_bit_cast(u32x4, o));
                    }
                    if (d_w) {
                        const f16x8 f = __builtin_bit_cast(f16x8, q[j]);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] = fmaf(v[i], (float)f[i], dot[j]);
                    }
                }
            }
            if (d_w) {
#pragma unroll
                for (int j = 0; j < CW_J; ++j) {
                    if (j0 + j >= k) break;
                    float s = dot[j];
#pragma unroll
                    for (int o = 32; o > 0; o >>= 1) s += __shfl_xor(s, o, 64);
                    if (lane == 0) red[wave][j0 + j] = s;
                }
            }
        }
        if (d_w) {
            __syncthreads();
            if (tid < k) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < WAVES; ++i) s += red[i][tid];
                d_w[t * k + tid] = s;
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const float* d_out, const uint16_t* y, const float* w, const int32_t* p2s, int T,
                                   int k, int H, uint16_t* d_y, float* d_w, hipStream_t s) {
    const unsigned blocks = (unsigned)std::min(T, 1 << 20);
    if (H <= 512) combine_backward_kernel<64><<<blocks, 64, 0, s>>>(d_out, y, w, p2s, T, k, H, d_y, d_w);
    else if (H <= 2048) combine_backward_kernel<256><<<blocks, 256, 0, s>>>(d_out, y, w, p2s, T, k, H, d_y, d_w);
    else combine_backward_kernel<512><<<blocks, 512, 0, s>>>(d_out, y, w, p2s, T, k, H, d_y, d_w);
    return hipGetLastError();
}

}  // namespace moe
