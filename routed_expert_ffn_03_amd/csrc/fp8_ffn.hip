// Grouped expert FFN on e4m3 weights with one fp32 scale per 128 x 128 block:
//   xq, sx = e4m3 rows of x          (one power-of-two scale per 128 columns)
//   a      = silu(xq Wg^T) * (xq Wu^T)
//   aq, sa = e4m3 rows of a
//   y      = aq Wd^T, stored fp16
// with every 128-column partial product taken in fp32 on the MFMA and
// multiplied by its two scales before it is added (fp8.h).
//
// The weights are the MFMA's A operand and the activation rows its B operand,
// so that a lane's result registers all belong to one activation row: the row
// scale is one value per lane, the weight scale one value per wave, and four
// consecutive result registers are four consecutive output columns.
//
// Work item: (32 rows of a route list, 128 columns of a or 256 of y), one
// 512-thread block; wave w owns 16 gate and the matching 16 up rows (phase 1)
// or 32 rows of W_down (phase 2) over the whole reduction index, so no
// partial sums cross waves; phase 1 exchanges the row maxima of its 128
// columns, which are one scale group of a, and stores codes.
#include "common.h"
#include "ffn_shared.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int F8S_THREADS = 512;

template <int PHASE>
__global__ __launch_bounds__(F8S_THREADS)
void ffn_fp8_rows_kernel(Fp8Args a) {
    __shared__ float top[8][32];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 31, g = lane >> 5;
    const int K = PHASE == 1 ? a.H : a.I, N = PHASE == 1 ? a.I : a.H;
    const int KB = K / FP8_BLOCK;
    const int NT = PHASE == 1 ? N / 128 : N / 256;
    const int n_tiles = a.hdr->n_thin;
    const size_t P = (size_t)a.T * a.k;
    for (int item = blockIdx.x; item < n_tiles * NT; item += gridDim.x) {
        const int q = item / NT, nt = item - q * NT;
        const MTile t = a.thin[q];
        const size_t eoff = (size_t)t.e * N * K;
        const size_t soff = (size_t)t.e * (N / FP8_BLOCK) * KB;
        // this lane's weight row and the scale rows of its block(s)
        const int wrow = PHASE == 1 ? nt * 128 + 16 * wave + (m & 15) : nt * 256 + 32 * wave + m;
        const uint8_t* w = (PHASE == 1 ? (m < 16 ? a.wg : a.wu) : a.wd) + eoff + (size_t)wrow * K + 32 * g;
        const float* s0 = PHASE == 1 ? a.sg + soff + (size_t)nt * KB
                                     : a.sd + soff + (size_t)((nt * 256 + 32 * wave) / FP8_BLOCK) * KB;
        const float* s1 = PHASE == 1 ? a.su + soff + (size_t)nt * KB : s0;
        {
            // rows past the tile repeat its last one; they are never stored
            const int row = t.row0 + min(m, t.rows - 1);
            const size_t src = PHASE == 1 ? (size_t)(a.sorted_pair[row] / a.k) : (size_t)row;
            const uint8_t* x = (PHASE == 1 ? a.xq : a.act) + src * K + 32 * g;
            const float* xs = PHASE == 1 ? a.xs + src * KB : a.as + src;
            const size_t xstep = PHASE == 1 ? 1 : P;
            f32x16 acc = f32x16{};
            for (int b = 0; b < KB; ++b) {
                f32x16 part = f32x16{};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t* wp = w + b * FP8_BLOCK + 64 * h;
                    const uint8_t* xp = x + b * FP8_BLOCK + 64 * h;
                    part = mfma_fp8(pack8(ldg16(wp), ldg16(wp + 16)), pack8(ldg16(xp), ldg16(xp + 16)), part);
                }
                const float sx = xs[b * xstep];
                const float f0 = sx * s0[b], f1 = PHASE == 1 ? sx * s1[b] : f0;
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = fmaf(part[i], i < 8 ? f0 : f1, acc[i]);
            }
            if constexpr (PHASE == 1) {
                float v[8], tp = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = silu_mul(acc[i], acc[i + 8]);
                    tp = fmaxf(tp, finite_abs(v[i]));
                }
                tp = fmaxf(tp, __shfl_xor(tp, 32, 64));
                __syncthreads();
                if (g == 0) top[wave][m] = tp;
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 8; ++i) tp = fmaxf(tp, top[i][m]);
                const float s = fp8_scale(tp), r = pow2_rcp(s);
                if (m < t.rows) {
                    uint8_t* dst = a.act + (size_t)row * a.I + nt * 128 + 16 * wave + 4 * g;
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint32_t*>(dst + 8 * i) =
                            fp8_pack4(v[4 * i] * r, v[4 * i + 1] * r, v[4 * i + 2] * r, v[4 * i + 3] * r);
                    if (wave == 0 && g == 0) a.as[(size_t)nt * P + row] = s;
                }
            } else if (m < t.rows) {
                uint16_t* dst = a.y + (size_t)row * a.H + nt * 256 + 32 * wave + 4 * g;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint2 o;
                    o.x = (uint32_t)f32_to_f16_bits(acc[4 * i]) | ((uint32_t)f32_to_f16_bits(acc[4 * i + 1]) << 16);
                    o.y = (uint32_t)f32_to_f16_bits(acc[4 * i + 2]) | ((uint32_t)f32_to_f16_bits(acc[4 * i + 3]) << 16);
                    *reinterpret_cast<uint2*>(dst + 8 * i) = o;
                }
            }
        }
    }
}

}  // namespace

hipError_t launch_fp8_phase(const Fp8Args& a, int phase, int cus, bool fat, hipStream_t s) {
    if (phase == 1) {
        const hipError_t err = launch_quantize_fp8(a.x, 1, a.T, a.H, 1, a.xq, a.xs, s);
        if (err != hipSuccess) return err;
    }
    if (fat) {
        const hipError_t err = launch_fp8_fat_phase(a, phase, cus, s);
        if (err != hipSuccess) return err;
    }
    if (phase == 1) {
        ffn_fp8_rows_kernel<1><<<2 * cus, F8S_THREADS, 0, s>>>(a);
    } else {
        ffn_fp8_rows_kernel<2><<<2 * cus, F8S_THREADS, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
