// Gradient of the combine out[t, :] = sum_j w[t, j] y_sorted[p2s[t k + j], :]
// with respect to the expert outputs and the gate weights:
//   d_y[p2s[t k + j], :] = w[t, j] d_out[t, :]          (stored fp16, the type of y)
//   d_w[t, j]            = sum_h d_out[t, h] y_sorted[p2s[t k + j], h]
// Every pair owns its row of y_sorted, so nothing is accumulated across
// tokens and there are no atomics.  Bound by HBM: 2 k H bytes of y read and
// 2 k H of d_y written per token, 4 H of d_out read.
#include "common.h"
#include "kernels.h"

#include <algorithm>

namespace moe {
namespace {

constexpr int CW_THREADS = 256;

__global__ __launch_bounds__(CW_THREADS)
void combine_backward_kernel(const float* __restrict__ d_out, const uint16_t* __restrict__ y,
                             const float* __restrict__ w, const int32_t* __restrict__ p2s, int T, int k, int H,
                             uint16_t* __restrict__ d_y, float* __restrict__ d_w) {
    __shared__ float red[MAX_TOPK][CW_THREADS / WAVE];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (size_t t = blockIdx.x; t < (size_t)T; t += gridDim.x) {
        const float* go = d_out + t * H;
        for (int j = 0; j < k; ++j) {
            const size_t row = (size_t)p2s[t * k + j] * H;
            const float wj = d_y ? w[t * k + j] : 0.0f;
            float dot = 0.0f;
            for (int h = tid * 8; h < H; h += CW_THREADS * 8) {
                const float4 a = *reinterpret_cast<const float4*>(go + h);
                const float4 b = *reinterpret_cast<const float4*>(go + h + 4);
                const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                if (d_w) {
                    const f16x8 q = __builtin_bit_cast(f16x8, ldg16_stream(y + row + h));
#pragma unroll
                    for (int i = 0; i < 8; ++i) dot = fmaf(v[i], (float)q[i], dot);
                }
                if (d_y) {
                    f16x8 o;
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = (_Float16)(wj * v[i]);
                    stg16(d_y + row + h, __builtin_bit_cast(u32x4, o));
                }
            }
            if (d_w) {
#pragma unroll
                for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
                if (lane == 0) red[j][wave] = dot;
            }
        }
        if (d_w) {
            __syncthreads();
            if (tid < k) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < CW_THREADS / WAVE; ++i) v += red[tid][i];
                d_w[t * k + tid] = v;
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const float* d_out, const uint16_t* y, const float* w, const int32_t* p2s, int T,
                                   int k, int H, uint16_t* d_y, float* d_w, hipStream_t s) {
    combine_backward_kernel<<<(unsigned)std::min(T, 1 << 20), CW_THREADS, 0, s>>>(d_out, y, w, p2s, T, k, H, d_y, d_w);
    return hipGetLastError();
}

}  // namespace moe
