// e4m3 helpers and kernel arguments of the 8-bit expert format (internal
// header).
//
// Operands are e4m3 codes (1 sign, 4 exponent, 3 mantissa bits, largest
// finite value 448, no infinities) with one fp32 scale per 128 columns of an
// activation row and per 128 x 128 block of a weight matrix; a value is
// code * scale.  A product over 128 columns takes both scales at once:
//   y[i, n] = sum_b sx[i, b] sw[n / 128, b] sum_{k in b} xq[i, k] wq[n, k],
// the outer sum in fp32.  The inner one: where a kernel streams weights from
// HBM the codes are multiplied as fp16, which holds every code exactly, in the
// fp16 MFMA's fp32 sums.  The M-tiles take the e4m3 MFMA, at twice the rate and
// with fewer bits: it adds the products of eight consecutive k with each cut 13
// bits below the largest of them (measured: next to 2^16 a term of 2^3 is kept
// and 2^2 lost, in every shape of the instruction), and these octets in fp32.
// That is 1.5e-5 rms of a 128-column sum of normally distributed codes; y ends
// 1e-3 of its norm from exact sums, against 3e-2 that rounding x and a to e4m3
// costs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"
#include "ffn_shared.h"

namespace moe {

constexpr int FP8_BLOCK = 128;
constexpr int FP8_BM = 224;              // rows per MFMA M-tile: leaves LDS for the row scales (fp8_fat.hip)

typedef __attribute__((ext_vector_type(8))) int i32x8;

// 16 x 16 x 128 e4m3 products: lane L holds row (A) or column (B) L % 16 and
// 32 bytes of k.  Result element i of lane L is row 4 (L / 16) + i, column
// L % 16.
__device__ __forceinline__ f32x4 mfma16_fp8(i32x8 a, i32x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Eight e4m3 codes as fp16, which holds every one of them exactly.
__device__ __forceinline__ u32x4 fp8_to_f16(uint32_t lo, uint32_t hi) {
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

__device__ __forceinline__ i32x8 pack8(u32x4 lo, u32x4 hi) {
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// |v| where it is finite, else 0: what a block's scale is taken from.
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < __uint_as_float(0x7f800000u) ? a : 0.0f;         // (false for NaN too)
}

// The scale of a block whose largest finite magnitude is `top`: the least
// power of two s >= 2^-126 with top <= 448 s, and 1 for top = 0.  A power of
// two makes v / s exact, so the code of every value is the same in any
// precision; e4m3 keeps its relative step over 14 octaves, so against
// top / 448 this costs at most one octave at the small end.
// top = 2^(p - 127) (1 + f): 448 = 2^8 * 1.75, so the exponent is p - 8, plus
// one where 1 + f > 1.75.  Subnormal tops end at the lower limit.
__device__ __forceinline__ float fp8_scale(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return top > 0.0f ? __uint_as_float((uint32_t)max(e, 1) << 23) : 1.0f;
}

// 1 / s for a power of two s in [2^-126, 2^126].
__device__ __forceinline__ float pow2_rcp(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// Four values (already divided by the scale) as e4m3 codes, nearest even;
// non-finite values become the NaN code.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return (uint32_t)v;
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(v[i] << 16);
        f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float r) {
    return make_uint2(fp8_pack4(f[0] * r, f[1] * r, f[2] * r, f[3] * r),
                      fp8_pack4(f[4] * r, f[5] * r, f[6] * r, f[7] * r));
}

// Chunk i of 8 values of rows of 128-column groups: 16 consecutive lanes hold
// a group, and find its scale by four exchanges.
__device__ __forceinline__ void fp8_quant_chunk(const uint16_t* __restrict__ src, size_t i,
                                                uint8_t* __restrict__ codes, float* __restrict__ scales) {
    float f[8];
    unpack8(ldg16(src + i * 8), f);
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(f[j]));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    const float s = fp8_scale(top);
    *reinterpret_cast<uint2*>(codes + i * 8) = codes8(f, pow2_rcp(s));
    if ((i & 15) == 0) scales[i >> 4] = s;
}

struct Fp8Args {
    const uint16_t* x;                  // bf16 [T, H]
    const uint8_t* wg;                  // e4m3 [E, I, H]
    const uint8_t* wu;
    const uint8_t* wd;                  // e4m3 [E, H, I]
    const float* sg;                    // fp32 [E, I/128, H/128]
    const float* su;
    const float* sd;                    // fp32 [E, H/128, I/128]
    const int32_t* sorted_pair;
    int T, k, H, I, E;
    uint8_t* xq;                        // e4m3 [T, H] and its scales [T, H/128]
    float* xs;
    float* xst;                         // the scales of x by sorted row, [H/128, T*k] (MFMA tiles only)
    uint8_t* act;                       // e4m3 [T*k, I] and its scales [I/128, T*k]
    float* as;
    uint16_t* y;                        // fp16 [T*k, H]
    const FfnHeader* hdr;
    const MTile* fat;
    const MTile* thin;
};

// e4m3 codes and scales of bf16 matrices (fp8_quant.hip): block_rows 1 (rows
// of activations) or 128 (weights).
hipError_t launch_quantize_fp8(const uint16_t* src, int64_t mats, int rows, int cols, int block_rows, uint8_t* codes,
                               float* scales, hipStream_t s);

// One phase of the grouped FFN on e4m3 weights (fp8_ffn.hip): 1 = gate/up
// (quantises x first unless `x_ready`), 2 = down.  `fat` false: no route list
// can be fat.
hipError_t launch_fp8_phase(const Fp8Args& a, int phase, int cus, bool fat, bool x_ready, hipStream_t s);

// ... over the MFMA M-tiles only (fp8_fat.hip)
hipError_t launch_fp8_fat_phase(const Fp8Args& a, int phase, int cus, hipStream_t s);

}  // namespace moe
