// MFMA-tile grouped FFN on e4m3 weights: busy experts' route lists in M-tiles
// of up to 224 rows, each multiplied with 256 weight rows at a time (phase 1:
// 128 gate rows and the matching 128 up rows, so that SwiGLU and the 128-column
// scale group of a stay in one block; phase 2: 256 rows of W_down).
//
//   acc[n, m] += (sum_{k in block b} w[n, k] x[m, k]) * (sx[m, b] * sw[n/128, b])
//
// One 512-thread block per CU, persistent.  A stage is one 128-column block,
// so a row of a stage is one whole 128-byte line: the per-CU load path moves
// about a line per clock however much of it is used.  Operands go through LDS
// by direct-to-LDS loads (8 rows x 128 B per instruction): three slots of
// weight rows (32 KB), which mostly come from HBM and are loaded two stages
// ahead, and two of activation rows (28 KB) with their 224 row scales, loaded
// one stage ahead (mostly L2).  224 rows rather than 256 leave room for the
// scales in the 160 KB of LDS.  16-byte piece c of row r lies at position
// c ^ (r & 7) ^ ((r >> 3) & 1) of its line, so that 8 lanes reading the same
// piece of 8 consecutive rows hit all banks once.
//
// Wave (G, q) owns 64 weight rows (phase 1: gate rows 32 q .. and up rows
// 32 q ..; phase 2: rows 64 q ..) against row tiles G, G + 2, G + 4, G + 6:
// the two waves of a SIMD share the work of any M-tile to within one row
// tile, and while one multiplies its partial sums into the accumulators the
// other's MFMAs run.  The products of one 32 x 32 tile over a stage are two
// 32x32x64 MFMAs into a fresh partial sum, then 16 fmas with the block's
// scale, one value per lane because the activation rows are the MFMA's
// columns.
#include "common.h"
#include "ffn_shared.h"
#include "fp8.h"
#include "kernels.h"
#include "lds_dma.h"

#include <algorithm>
#include <mutex>

namespace moe {
namespace {

constexpr int FF_THREADS = 512;
constexpr uint32_t FF_ROW = 128;                           // bytes of a row per stage
constexpr uint32_t FF_W = 256 * FF_ROW;                    // weight slot
constexpr uint32_t FF_A = FP8_BM * FF_ROW;                 // activation slot
constexpr int FF_NW = 3, FF_NA = 2;
constexpr uint32_t FF_A0 = FF_NW * FF_W;                   // LDS offsets
constexpr uint32_t FF_S0 = FF_A0 + FF_NA * FF_A;
constexpr uint32_t FF_LDS = FF_S0 + FF_NA * 256 * 4;
static_assert(FF_LDS <= 160 * 1024, "LDS of one CU");

// Row pitch of the epilogue staging tile in bytes (16 of padding).
template <int PHASE>
constexpr uint32_t ff_pitch() { return (PHASE == 1 ? 128 : 512) + 16; }
static_assert(FP8_BM * ff_pitch<2>() <= FF_LDS && FP8_BM * ff_pitch<1>() + 4 * 256 * 4 <= FF_LDS, "staging");

template <int PHASE>
__global__ __launch_bounds__(FF_THREADS, 1)
void ffn_fp8_fat_kernel(Fp8Args a) {
    extern __shared__ u32x4 smem[];
    char* const lds = reinterpret_cast<char*>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = wave >> 2, q = wave & 3;
    const int m = lane & 31, g = lane >> 5;
    const int K = PHASE == 1 ? a.H : a.I, N = PHASE == 1 ? a.I : a.H;
    const int KB = K / FP8_BLOCK;
    constexpr int BN = PHASE == 1 ? 128 : 256;
    const int NT = N / BN;
    const int n_items = a.hdr->n_fat * NT;
    const size_t P = (size_t)a.T * a.k;
    const size_t wbytes = (size_t)N * K;
    const __amdgpu_buffer_rsrc_t asrc = PHASE == 1 ? make_rsrc(a.xq, (uint32_t)((size_t)a.T * K))
                                                   : make_rsrc(a.act, (uint32_t)(P * K));
    const __amdgpu_buffer_rsrc_t ssrc = make_rsrc(PHASE == 1 ? a.xst : a.as, (uint32_t)(P * KB * 4));
    const uint32_t sbase = lds_addr(smem);
    // a load instruction moves rows 8 j .. 8 j + 7: lane L row L / 8, position L % 8
    const int lr = lane >> 3;
    auto piece = [&](int row) { return (uint32_t)(((lane & 7) ^ (row & 7) ^ ((row >> 3) & 1)) * 16); };
    // fragment reads: lane (m, g), half h of the stage, 16 bytes j: piece 4 h + 2 g + j of row m
    uint32_t fo[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            fo[h][j] = (uint32_t)m * FF_ROW + (uint32_t)(((4 * h + 2 * g + j) ^ (m & 7) ^ ((m >> 3) & 1)) * 16);
    const uint32_t wfo = (uint32_t)(PHASE == 1 ? 32 * q : 64 * q) * FF_ROW;
    constexpr int WC = (PHASE == 1 ? 128 : 32) * (int)FF_ROW;      // from the wave's first column tile to its second

    for (int item = logical_block(); item < n_items; item += gridDim.x) {
        MTile t;
        int nt;
        fat_item(a.fat, item, NT, t, nt);
        const int rt = (t.rows + 31) >> 5;
        const uint8_t* wmat = PHASE == 1 ? (wave < 4 ? a.wg : a.wu) : a.wd;
        const __amdgpu_buffer_rsrc_t wsrc = make_rsrc(wmat + (size_t)t.e * wbytes, (uint32_t)wbytes);
        // block scales of this wave's column tiles
        const size_t soff = (size_t)t.e * (N / FP8_BLOCK) * KB;
        // (read through the constant address space: scalar loads, which leave the vector loads' count alone)
        typedef const __attribute__((address_space(4))) float* cfloat_t;
        const cfloat_t sw0 = (cfloat_t)(PHASE == 1 ? a.sg + soff + (size_t)nt * KB
                                                   : a.sd + soff + (size_t)(2 * nt + (q >> 1)) * KB);
        const cfloat_t sw1 = PHASE == 1 ? (cfloat_t)(a.su + soff + (size_t)nt * KB) : sw0;
        // activation instruction j of this wave: tile rows 8 (8 j + wave) + L / 8 (rows past the M-tile repeat
        // its last one); weight instruction j: rows 32 wave + 8 j + L / 8 of the slot
        uint32_t aoff[4], woff[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 8 * (8 * j + wave) + lr;
            const int row = t.row0 + min(r, t.rows - 1);
            const uint32_t src = PHASE == 1 ? (uint32_t)(a.sorted_pair[row] / a.k) : (uint32_t)row;
            aoff[j] = src * (uint32_t)K + piece(r);
            const int w = 32 * wave + 8 * j + lr;
            const uint32_t wrow = PHASE == 1 ? (uint32_t)(nt * 128 + (w & 127)) : (uint32_t)(nt * 256 + w);
            woff[j] = wrow * (uint32_t)K + piece(w);
        }
        // row scales [KB][P]: lane L of wave w takes row 64 (w % 4) + L
        const uint32_t srow = (uint32_t)(t.row0 + min(64 * q + lane, t.rows - 1)) * 4u;

        auto kloop = [&](auto rt_c) {
            constexpr int RT = decltype(rt_c)::value;
            constexpr int LA = (RT + 1) / 2;                       // activation loads per wave per stage
            auto issue_w = [&](int kt, int slot) {
                char* st = lds + slot * FF_W + wave * 4096;
#pragma unroll
                for (int j = 0; j < 4; ++j) dma16(wsrc, st + j * 1024, woff[j], kt * FF_ROW);
            };
            auto issue_a = [&](int kt, int slot) {
                __builtin_amdgcn_raw_ptr_buffer_load_lds(ssrc, (lds_ptr_t)(lds + FF_S0 + slot * 1024 + q * 256), 4, srow,
                                                         (uint32_t)(kt * P * 4), 0, 0);
                char* st = lds + FF_A0 + slot * FF_A + wave * 1024;
#pragma unroll
                for (int j = 0; j < LA; ++j)
                    if (8 * j + wave < 4 * RT) dma16(asrc, st + j * 8192, aoff[j], kt * FF_ROW);
            };
            auto run = [&](auto rg_c) {
                constexpr int RG = decltype(rg_c)::value;            // row tiles of this wave
                constexpr int RA = RG > 0 ? RG : 1;
                f32x16 acc[RA][2];
#pragma unroll
                for (int i = 0; i < RA; ++i)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[i][c] = f32x16{};

                issue_w(0, 0);
                issue_a(0, 0);
                if (KB > 1) issue_w(1, 1);
                int wslot = 0, aslot = 0;
                for (int kt = 0; kt < KB; ++kt) {
                    const float s0 = sw0[kt], s1 = sw1[kt];
                    if (kt + 1 < KB) vm_wait<4>(); else vm_wait<0>();    // all but the next stage's weights
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                    if (kt + 1 < KB) issue_a(kt + 1, aslot ^ 1);
                    if (kt + 2 < KB) issue_w(kt + 2, wslot == 0 ? 2 : wslot - 1);
                    if constexpr (RG > 0) {
                        const uint32_t wb = sbase + wslot * FF_W + wfo;
                        const uint32_t ab = sbase + FF_A0 + aslot * FF_A + G * 32 * FF_ROW;
                        const uint32_t sb = sbase + FF_S0 + aslot * 1024 + (32 * G + m) * 4;
                        u32x4 w[2][2][2], x[2][2][2];                // [column tile][half][16 B], [buffer][half][16 B]
                        uint32_t sx[RA];
                        static_for<2>([&](auto h_c) {
                            static_for<2>([&](auto j_c) {
                                constexpr int Hh = decltype(h_c)::value, J = decltype(j_c)::value;
                                w[0][Hh][J] = ds_read16<0>(wb + fo[Hh][J]);
                                x[0][Hh][J] = ds_read16<0>(ab + fo[Hh][J]);
                                w[1][Hh][J] = ds_read16<WC>(wb + fo[Hh][J]);
                            });
                        });
#pragma unroll
                        for (int i = 0; i < RG; ++i) sx[i] = ds_read4(sb + i * 256);
                        lds_wait_all();
                        static_for<2>([&](auto h_c) {
                            static_for<2>([&](auto j_c) {
                                constexpr int Hh = decltype(h_c)::value, J = decltype(j_c)::value;
                                tie_after_wait(w[0][Hh][J]);
                                tie_after_wait(w[1][Hh][J]);
                                tie_after_wait(x[0][Hh][J]);
                            });
                        });
#pragma unroll
                        for (int i = 0; i < RG; ++i) tie_after_wait(sx[i]);
                        static_for<RG>([&](auto i_c) {
                            constexpr int I = decltype(i_c)::value, B = I & 1;
                            if constexpr (I + 1 < RG) {
                                static_for<2>([&](auto h_c) {
                                    static_for<2>([&](auto j_c) {
                                        constexpr int Hh = decltype(h_c)::value, J = decltype(j_c)::value;
                                        x[B ^ 1][Hh][J] = ds_read16<(I + 1) * 64 * (int)FF_ROW>(ab + fo[Hh][J]);
                                    });
                                });
                            }
                            f32x16 p0 = mfma_fp8(pack8(w[0][0][0], w[0][0][1]), pack8(x[B][0][0], x[B][0][1]), f32x16{});
                            f32x16 p1 = mfma_fp8(pack8(w[1][0][0], w[1][0][1]), pack8(x[B][0][0], x[B][0][1]), f32x16{});
                            p0 = mfma_fp8(pack8(w[0][1][0], w[0][1][1]), pack8(x[B][1][0], x[B][1][1]), p0);
                            p1 = mfma_fp8(pack8(w[1][1][0], w[1][1][1]), pack8(x[B][1][0], x[B][1][1]), p1);
                            const float f0 = __uint_as_float(sx[I]) * s0;
                            const float f1 = PHASE == 1 ? __uint_as_float(sx[I]) * s1 : f0;
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[I][0][r] = fmaf(p0[r], f0, acc[I][0][r]);
#pragma unroll
                            for (int r = 0; r < 16; ++r) acc[I][1][r] = fmaf(p1[r], f1, acc[I][1][r]);
                            if constexpr (I + 1 < RG) {
                                lds_wait_all();
                                static_for<2>([&](auto h_c) {
                                    static_for<2>([&](auto j_c) {
                                        tie_after_wait(x[B ^ 1][decltype(h_c)::value][decltype(j_c)::value]);
                                    });
                                });
                            }
                        });
                    }
                    wslot = wslot == 2 ? 0 : wslot + 1;
                    aslot ^= 1;
                }
                __syncthreads();                                     // the ring becomes the staging tile

                // result element r of lane (m, g): row 32 i + m, column 8 (r / 4) + 4 g + r % 4 of the column tile
                constexpr uint32_t PITCH = ff_pitch<PHASE>();
                uint32_t e0 = (uint32_t)(32 * G + m) * PITCH;
                asm volatile("" : "+v"(e0));                         // (addresses derived here, not kept over the items)
                if constexpr (PHASE == 1) {
                    float* top = reinterpret_cast<float*>(lds + FP8_BM * PITCH);      // [4][256] row maxima by q
                    float s[RA];
                    static_for<RG>([&](auto i_c) {
                        constexpr int I = decltype(i_c)::value;
                        float tp = 0.0f;
#pragma unroll
                        for (int r = 0; r < 16; ++r) {
                            const float v = silu_mul(acc[I][0][r], acc[I][1][r]);
                            acc[I][0][r] = v;
                            tp = fmaxf(tp, finite_abs(v));
                        }
                        tp = fmaxf(tp, __shfl_xor(tp, 32, 64));
                        if (g == 0) top[q * 256 + 64 * I + 32 * G + m] = tp;
                    });
                    __syncthreads();
                    static_for<RG>([&](auto i_c) {
                        constexpr int I = decltype(i_c)::value;
                        const float* tr = top + 64 * I + 32 * G + m;
                        s[I] = fp8_scale(fmaxf(fmaxf(tr[0], tr[256]), fmaxf(tr[512], tr[768])));
                        const float rs = pow2_rcp(s[I]);
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            *reinterpret_cast<uint32_t*>(lds + e0 + I * 64 * PITCH + 32 * q + 8 * c + 4 * g) =
                                fp8_pack4(acc[I][0][4 * c] * rs, acc[I][0][4 * c + 1] * rs, acc[I][0][4 * c + 2] * rs,
                                          acc[I][0][4 * c + 3] * rs);
                        const int row = 64 * I + 32 * G + m;
                        if (q == 0 && g == 0 && row < t.rows) a.as[(size_t)nt * P + t.row0 + row] = s[I];
                    });
                } else {
                    static_for<RG>([&](auto i_c) {
                        constexpr int I = decltype(i_c)::value;
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const f32x16& v = acc[I][c];
                                const uint32_t lo = (uint32_t)f32_to_f16_bits(v[4 * j]) |
                                                    ((uint32_t)f32_to_f16_bits(v[4 * j + 1]) << 16);
                                const uint32_t hi = (uint32_t)f32_to_f16_bits(v[4 * j + 2]) |
                                                    ((uint32_t)f32_to_f16_bits(v[4 * j + 3]) << 16);
                                *reinterpret_cast<uint2*>(lds + e0 + I * 64 * PITCH + (64 * q + 32 * c + 8 * j + 4 * g) * 2) =
                                    make_uint2(lo, hi);
                            }
                    });
                }
            };
            if (G == 0) run(std::integral_constant<int, (RT + 1) / 2>{});
            else run(std::integral_constant<int, RT / 2>{});
        };
        switch (rt) {
            case 7: kloop(std::integral_constant<int, 7>{}); break;
            case 6: kloop(std::integral_constant<int, 6>{}); break;
            case 5: kloop(std::integral_constant<int, 5>{}); break;
            case 4: kloop(std::integral_constant<int, 4>{}); break;
            case 3: kloop(std::integral_constant<int, 3>{}); break;
            case 2: kloop(std::integral_constant<int, 2>{}); break;
            default: kloop(std::integral_constant<int, 1>{}); break;
        }
        __syncthreads();
        {
            constexpr uint32_t PITCH = ff_pitch<PHASE>();
            constexpr int BYTES = PHASE == 1 ? 128 : 512;            // of one output row
            constexpr int CPR = BYTES / 16, RPP = FF_THREADS / CPR;
            uint8_t* dst = PHASE == 1 ? a.act : reinterpret_cast<uint8_t*>(a.y);
            const size_t ld = PHASE == 1 ? (size_t)a.I : (size_t)a.H * 2;
            const int ch = tid % CPR;
            for (int r = tid / CPR; r < t.rows; r += RPP)
                stg16(dst + (size_t)(t.row0 + r) * ld + nt * BYTES + ch * 16,
                      *reinterpret_cast<const u32x4*>(lds + r * PITCH + ch * 16));
        }
        __syncthreads();                                             // staging read before the next item's loads
    }
}

// The row scales of x in sorted order, block-major: xst[b, i] = xs[sorted_pair[i] / k, b].
// The MFMA-tile kernel then reads the 32 rows of a tile as one line per block.
__global__ __launch_bounds__(256)
void fp8_sort_scales_kernel(const float* __restrict__ xs, const int32_t* __restrict__ sorted_pair, int P, int k, int KB,
                            float* __restrict__ xst) {
    __shared__ float tile[64][33];
    const int c = threadIdx.x & 31, r0 = threadIdx.x >> 5;           // 8 rows of 32 blocks
    const int l = threadIdx.x & 63, b0 = threadIdx.x >> 6;           // 4 blocks of 64 rows
    for (int base = blockIdx.x * 64; base < P; base += gridDim.x * 64) {
        for (int kb = 0; kb < KB; kb += 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = base + 8 * i + r0;
                if (r < P && kb + c < KB) tile[8 * i + r0][c] = xs[(size_t)(sorted_pair[r] / k) * KB + kb + c];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int b = kb + 4 * i + b0;
                if (base + l < P && b < KB) xst[(size_t)b * P + base + l] = tile[l][b - kb];
            }
            __syncthreads();
        }
    }
}

std::mutex g_ff_mu;
bool g_ff_ready[64] = {};

}  // namespace

hipError_t launch_fp8_fat_phase(const Fp8Args& a, int phase, int cus, hipStream_t s) {
    int dev = 0;
    hipError_t err = hipGetDevice(&dev);
    if (err != hipSuccess) return err;
    if (dev < 0 || dev >= 64) return hipErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lock(g_ff_mu);
        if (!g_ff_ready[dev]) {
            err = hipFuncSetAttribute((const void*)ffn_fp8_fat_kernel<1>, hipFuncAttributeMaxDynamicSharedMemorySize,
                                      (int)FF_LDS);
            if (err == hipSuccess)
                err = hipFuncSetAttribute((const void*)ffn_fp8_fat_kernel<2>,
                                          hipFuncAttributeMaxDynamicSharedMemorySize, (int)FF_LDS);
            if (err != hipSuccess) return err;
            g_ff_ready[dev] = true;
        }
    }
    if (phase == 1) {
        const int P = a.T * a.k;
        const unsigned blocks = (unsigned)std::min((P - 1) / 64 + 1, 8 * cus);
        fp8_sort_scales_kernel<<<blocks, 256, 0, s>>>(a.xs, a.sorted_pair, P, a.k, a.H / FP8_BLOCK, a.xst);
        ffn_fp8_fat_kernel<1><<<cus, FF_THREADS, FF_LDS, s>>>(a);
    } else {
        ffn_fp8_fat_kernel<2><<<cus, FF_THREADS, FF_LDS, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
