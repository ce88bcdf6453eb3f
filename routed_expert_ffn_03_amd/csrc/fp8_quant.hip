// e4m3 codes and block scales of bf16 values: one scale per 128 columns of a
// row (activations) or per 128 x 128 block (weights).
//
// code = e4m3(v / s), s the least power of two >= 2^-126 with max|v| <= 448 s
// over the block's finite values (fp8.h).  Bound by HBM: 2 bytes read, 1
// written per value.  One MI355X: 16,384 rows of 4096 37 us (5.4 TB/s), 32
// weights of 2048 x 4096 142 us (5.7 TB/s); 4 rows 2.7 us, which is a launch.
//
// Rows: 16 lanes per group, 8 values each (one 16-byte load, one 8-byte
// store), the maximum by four lane exchanges.  Weights: one 256-thread block
// per 128 x 128 block, 64 values per thread kept in registers between the
// maximum and the conversion, so the source is read once.
#include "common.h"
#include "fp8.h"

namespace moe {
namespace {

constexpr int QR_THREADS = 256;

__global__ __launch_bounds__(QR_THREADS)
void fp8_quant_rows_kernel(const uint16_t* __restrict__ src, size_t groups, uint8_t* __restrict__ codes,
                           float* __restrict__ scales) {
    const size_t i = (size_t)blockIdx.x * QR_THREADS + threadIdx.x;     // chunk of 8 values
    if (i >= groups * 16) return;                                       // whole groups leave together
    fp8_quant_chunk(src, i, codes, scales);
}

__global__ __launch_bounds__(256)
void fp8_quant_blocks_kernel(const uint16_t* __restrict__ src, int rows, int cols, uint8_t* __restrict__ codes,
                             float* __restrict__ scales) {
    __shared__ float red[4];
    const int nc = cols / FP8_BLOCK;
    const size_t blk = blockIdx.x;                                      // over [mats, rows/128, cols/128]
    const size_t base = blk / nc * FP8_BLOCK * (size_t)cols + blk % nc * FP8_BLOCK;
    const int r0 = threadIdx.x >> 4, c0 = (threadIdx.x & 15) * 8;       // 16 rows x 128 columns per step
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = ldg16_stream(src + base + (size_t)(16 * i + r0) * cols + c0);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(f[j]));
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = top;
    __syncthreads();
    const float s = fp8_scale(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float r = pow2_rcp(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float f[8];
        unpack8(v[i], f);
        *reinterpret_cast<uint2*>(codes + base + (size_t)(16 * i + r0) * cols + c0) = codes8(f, r);
    }
    if (threadIdx.x == 0) scales[blk] = s;
}

}  // namespace

hipError_t launch_quantize_fp8(const uint16_t* src, int64_t mats, int rows, int cols, int block_rows, uint8_t* codes,
                               float* scales, hipStream_t s) {
    const size_t groups = (size_t)mats * rows * (size_t)(cols / FP8_BLOCK);
    if (block_rows == 1) {
        const size_t blocks = (groups * 16 + QR_THREADS - 1) / QR_THREADS;
        fp8_quant_rows_kernel<<<(unsigned)blocks, QR_THREADS, 0, s>>>(src, groups, codes, scales);
    } else {
        fp8_quant_blocks_kernel<<<(unsigned)(groups / FP8_BLOCK), 256, 0, s>>>(src, rows, cols, codes, scales);
    }
    return hipGetLastError();
}

}  // namespace moe
