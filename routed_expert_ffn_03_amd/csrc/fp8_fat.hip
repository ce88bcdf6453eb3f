// MFMA-tile grouped FFN on e4m3 weights: busy experts' route lists in M-tiles
// of up to 224 rows, each multiplied with 256 weight rows at a time (phase 1:
// 128 gate rows and the matching 128 up rows, so that SwiGLU and the 128-column
// scale group of a stay in one block; phase 2: 256 rows of W_down).
//
//   acc[n, m] += (sum_{k in block b} w[n, k] x[m, k]) * (sx[m, b] * sw[n/128, b])
//
// Products.  A 128-column block is one 16x16x128 MFMA per 16 x 16 tile, into a
// fresh partial sum; its four fmas with the block's scale (one value per lane,
// because the activation rows are the MFMA's columns) follow four products
// later, so they run beside the next tile's.  Register-only probes on random
// codes: 32x32x64 pairs with their fmas 3.0 PF, 16x16x128 with the fmas three
// or four products behind 3.5 PF (4.0 PF without fmas, 5.0 PF on zeros: power
// sets the clock).
//
// Operands.  One 512-thread block per CU, persistent.  A stage is one
// 128-column block, so a row of a stage is one whole 128-byte line.  Weight
// rows (32 KB a stage) go through three LDS slots and activation rows (28 KB)
// with their scales through two, by direct-to-LDS loads of 8 rows x 128 B,
// issued one at a time between the products (all at the stage's start: 5%
// slower).  16-byte piece c of row r lies at position c ^ (r & 7) ^ ((r >> 3)
// & 1) of its line, so that 8 lanes reading the same piece of 8 consecutive
// rows hit all banks once.  224 rows rather than 256 leave room for the scales.
//
// Waves.  Wave (G, q) owns 64 weight rows (phase 1: gate rows 32 q .. and up
// rows 32 q ..; phase 2: rows 64 q ..) against the 16-row tiles G, G + 2, ...:
// the two waves of a SIMD share the work of any M-tile to within one tile.
// The 64 weight rows' fragments stay in registers for a stage, row fragments
// are read two tiles ahead, and one barrier per stage, before its last tile but
// one, says that the next stage's operands have landed and this stage's rows
// have been read.  The next item's first loads go out before the epilogue.
//
// What bounds it (16,384 tokens, 384 experts, 4096 x 2048, top-8, one
// MI355X): gate/up 2.55 ms and down 1.40 ms, 1.67 PF over both.  The MFMAs are
// busy 45% of the cycles at a clock that the power limit holds at 1.83 GHz
// (2.2 GHz with the loads taken out); taking cycles out of a stage or an
// epilogue mostly lowers that clock further.  Loads cost the rest: without
// them gate/up takes 1.7 ms.  Half of the weight reads miss L2, since the two
// blocks that share a weight tile drift apart (11 GB of 6.4 GB).
// Measured and not kept: the two waves of a SIMD in turns with two barriers a
// stage (3.05 / 1.54 ms), 32x32x64 products (2.70 / 1.45), the next stage's
// weights in a second set of registers (3.0 / 1.6), items starting at
// different columns (no change), 192 rows (1.5% slower).
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
constexpr uint32_t FF_S = 256 * 4 + 256;                   // scale slot: 256 row scales, then the two block scales
constexpr uint32_t FF_T0 = FF_S0 + FF_NA * FF_S;           // row maxima of the four column groups
constexpr uint32_t FF_LDS = FF_T0 + 4 * 256 * 4;
static_assert(FF_LDS <= 160 * 1024, "LDS of one CU");
static_assert(FP8_BM <= 224, "at most seven 16-row tiles for a wave");

// Exchanges between lanes that differ in lane bit 5 (or 4): afterwards a lane
// with that bit clear holds both lanes' a, one with it set both lanes' b (in
// the order of the bit).
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
}

template <int PHASE>
__global__ __launch_bounds__(FF_THREADS, 1)
void ffn_fp8_fat_kernel(Fp8Args a) {
    extern __shared__ u32x4 smem[];
    char* const lds = reinterpret_cast<char*>(smem);
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int G = wave >> 2, q = wave & 3;
    const int m = lane & 15, kg = lane >> 4;
    const int K = PHASE == 1 ? a.H : a.I, N = PHASE == 1 ? a.I : a.H;
    const int KB = K / FP8_BLOCK;
    constexpr int BN = PHASE == 1 ? 128 : 256;
    const int NT = N / BN;
    const int n_items = a.hdr->n_fat * NT;
    const size_t P = (size_t)a.T * a.k;
    const size_t wbytes = (size_t)N * K;
    const __amdgpu_buffer_rsrc_t asrc = PHASE == 1 ? make_rsrc(a.xq, (uint32_t)((size_t)a.T * K))
                                                   : make_rsrc(a.act, (uint32_t)(P * K));
    typedef const __attribute__((address_space(1))) void* gptr_t;
    const uint32_t sbase = lds_addr(smem);
    // a load instruction moves rows 8 j .. 8 j + 7: lane L row L / 8, position L % 8
    const int lr = lane >> 3;
    auto piece = [&](int row) { return (uint32_t)(((lane & 7) ^ (row & 7) ^ ((row >> 3) & 1)) * 16); };
    // fragment reads: lane (m, kg), 16 bytes j: piece 2 kg + j of row m
    uint32_t fo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
        fo[j] = sbase + (uint32_t)m * FF_ROW + (uint32_t)(((2 * kg + j) ^ (m & 7) ^ ((m >> 3) & 1)) * 16);
    // column tiles 0, 1 and 2, 3 of this wave: 16 rows of W each (phase 1: gate rows 32 q .. and up rows 32 q ..;
    // phase 2: rows 64 q ..)
    const uint32_t wfo = (uint32_t)(PHASE == 1 ? 32 * q : 64 * q) * FF_ROW;
    constexpr int WC2 = (PHASE == 1 ? 128 : 32) * (int)FF_ROW;

    int item = logical_block();
    if (item >= n_items) return;                                   // the whole block
    MTile t, tn;                                                   // this item's M-tile and the next one's
    int nt, ntn;
    const int second = min(item + (int)gridDim.x, n_items - 1);
    fat_item(a.fat, item, NT, t, nt);
    fat_item(a.fat, second, NT, tn, ntn);

    // Where the loads of an item come from: set up for the item that is
    // loaded next, which is the block's next item once the current one has
    // all its stages under way.
    __amdgpu_buffer_rsrc_t wsrc;
    uint32_t aoff[4], woff[4];
    int na;                                                        // activation instructions of the block per stage
    const float* sp;
    const size_t sstep = wave < 4 ? P : 1;
    // the route-list entries of an M-tile's rows that this lane loads
    auto entries = [&](const MTile& u, int (&en)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int row = u.row0 + min(8 * (8 * j + wave) + lr, u.rows - 1);
            en[j] = PHASE == 1 ? a.sorted_pair[row] : row;
        }
    };
    auto aim = [&](const MTile& u, int un, const int (&en)[4]) {
        const uint8_t* wmat = PHASE == 1 ? (wave < 4 ? a.wg : a.wu) : a.wd;
        wsrc = make_rsrc(wmat + (size_t)u.e * wbytes, (uint32_t)wbytes);
        na = 2 * ((u.rows + 15) >> 4);
        // activation instruction j of this wave: tile rows 8 (8 j + wave) + L / 8 (rows past the M-tile repeat
        // its last one); weight instruction j: rows 32 wave + 8 j + L / 8 of the slot
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t src = (uint32_t)(PHASE == 1 ? en[j] / a.k : en[j]);
            aoff[j] = src * (uint32_t)K + piece(8 * (8 * j + wave) + lr);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int w = 32 * wave + 8 * j + lr;
            const uint32_t wrow = PHASE == 1 ? (uint32_t)(un * 128 + (w & 127)) : (uint32_t)(un * 256 + w);
            woff[j] = wrow * (uint32_t)K + piece(w);
        }
        // Scales of a stage, 4 bytes per lane: waves 0-3 the row scales, 64
        // each, from the block-major array (position 8 (16 G + m) + t holds
        // row 32 t + 16 G + m, so that a lane finds its tiles' scales in a
        // row); wave 4 the two block scales of W (phase 1: gate, up; phase 2:
        // those of the lower and, 8 bytes on, of the upper 128 columns)
        const int pos = 64 * q + lane, r = 32 * (pos & 7) + (pos >> 3);
        const float* rows = (PHASE == 1 ? a.xst : a.as) + u.row0 + min(r, u.rows - 1);
        const size_t soff = (size_t)u.e * (N / FP8_BLOCK) * KB;
        const float* blocks = PHASE == 1 ? (lane == 0 ? a.sg : a.su) + soff + (size_t)un * KB
                                         : a.sd + soff + (size_t)(2 * un + (lane < 2 ? 0 : 1)) * KB;
        sp = wave < 4 ? rows : blocks;
    };
    // slots of stage 0 of the current item: the stages of all items go round
    int w0 = 0, a0 = 0;
    auto wslot = [&](int kt) { return (uint32_t)(w0 + kt) % FF_NW; };
    auto aslot = [&](int kt) { return (uint32_t)(a0 + kt) & 1; };
    auto issue_w = [&](int kt, int j) {                            // weight instruction j of stage kt
        dma16(wsrc, lds + wslot(kt) * FF_W + wave * 4096 + j * 1024, woff[j], kt * FF_ROW);
    };
    auto issue_a = [&](int kt, int j) {                            // activation instruction j, if the M-tile has its rows
        if (8 * j + wave < na) dma16(asrc, lds + FF_A0 + aslot(kt) * FF_A + wave * 1024 + j * 8192, aoff[j], kt * FF_ROW);
    };
    auto issue_s = [&](int kt) {
        if (wave < 5)
            __builtin_amdgcn_global_load_lds((gptr_t)(sp + kt * sstep),
                                             (lds_ptr_t)(lds + FF_S0 + aslot(kt) * FF_S + wave * 256), 4, 0, 0);
    };
    auto issue_rows = [&](int kt) {
        static_for<4>([&](auto j_c) { issue_a(kt, decltype(j_c)::value); });
        issue_s(kt);
    };
    // the first loads of an item: weights of stages 0 and 1, rows of stage 0
    auto issue_first = [&]() {
        static_for<4>([&](auto j_c) { issue_w(0, decltype(j_c)::value); });
        issue_rows(0);
        if (KB > 1) static_for<4>([&](auto j_c) { issue_w(1, decltype(j_c)::value); });
    };
    auto barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };

    {
        int en[4];
        entries(t, en);
        aim(t, nt, en);
    }
    issue_first();
    vm_wait<0>();
    barrier();
    for (;;) {
        const int tt = (t.rows + 15) >> 4;                         // 16-row tiles
        const bool has_next = item + (int)gridDim.x < n_items;
        // ahead of the stages, used after them: the next item's route-list
        // entries and the expert of the item after it
        int en[4];
        entries(tn, en);
        const int ahead = min(item + 2 * (int)gridDim.x, n_items - 1);
        const MTile tq = a.fat[ahead / NT];
        if (KB > 1) issue_rows(1);

        auto run = [&](auto rg_c) {
            constexpr int RG = decltype(rg_c)::value;              // row tiles of this wave: G, G + 2, ...
            constexpr int RA = RG > 0 ? RG : 1;
            // Row fragments: tile i has the same registers in every stage,
            // and any three consecutive tiles (around the stage's end too,
            // where RG > 2) have different ones: 0 1 2, 0 1 2 3, 0 1 2 3 4,
            // 0 1 2 0 1 2, 0 1 2 0 1 2 3.
            constexpr int NB = RG % 3 == 0 ? 3 : RG == 7 ? 4 : RA;
            constexpr auto buffer = [](int i) { return RG == 7 ? (i % 7 == 6 ? 3 : i % 7 % 3) : i % NB; };
            f32x4 acc[RA][4], p[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                p[c] = f32x4{};
#pragma unroll
                for (int i = 0; i < RA; ++i) acc[i][c] = f32x4{};
            }
            float f0 = 0.0f, f1 = 0.0f;                            // scales of the partial sums in p
            u32x4 w[4][2], x[NB][2];                               // weights by column tile, rows in a ring of tiles
            u32x4 sx0, sx1;                                        // row scales of tiles 0-3 and 4-6
            u32x2 swv;                                             // block scales
            auto read_w = [&](auto c_c, int kt) {
                constexpr int C = decltype(c_c)::value;
                const uint32_t wb = wslot(kt) * FF_W + wfo;
                w[C][0] = ds_read16<(C & 1) * 16 * (int)FF_ROW + (C >> 1) * WC2>(wb + fo[0]);
                w[C][1] = ds_read16<(C & 1) * 16 * (int)FF_ROW + (C >> 1) * WC2>(wb + fo[1]);
            };
            auto read_x = [&](auto b_c, auto i_c, int kt) {
                constexpr int B = decltype(b_c)::value, I = decltype(i_c)::value;
                const uint32_t ab = FF_A0 + aslot(kt) * FF_A + G * 16 * FF_ROW;
                x[B][0] = ds_read16<I * 32 * (int)FF_ROW>(ab + fo[0]);
                x[B][1] = ds_read16<I * 32 * (int)FF_ROW>(ab + fo[1]);
            };
            auto read_s = [&](int kt) {                            // three reads
                const uint32_t sb = sbase + FF_S0 + aslot(kt) * FF_S;
                sx0 = ds_read16<0>(sb + (16 * G + m) * 32);
                sx1 = ds_read16<16>(sb + (16 * G + m) * 32);
                swv = ds_read8(sb + 1024 + (PHASE == 2 ? (q >> 1) * 8 : 0));
            };
            auto tie_x = [&](auto b_c) {
                tie_after_wait(x[decltype(b_c)::value][0]);
                tie_after_wait(x[decltype(b_c)::value][1]);
            };
            auto tie_s = [&]() {
                tie_after_wait(sx0);
                tie_after_wait(sx1);
                tie_after_wait(swv);
            };

            // One stage.  LDS returns in order, so a wait for all but the N
            // newest reads is a wait for the older ones.  Reads run two tiles
            // ahead: at tile t those of tile t + 2.  Before the last tile but
            // one every wave has all rows of this stage and the weights of
            // this stage, read in the stage before (barrier: their slots are
            // free); from there on come the next stage's first two tiles and,
            // behind the products that used the old ones, its weights and
            // scales (past the last stage: whatever lies there, unused).
            auto stage = [&](int kt) {
                const bool more = kt + 1 < KB;
                auto boundary = [&]() {
                    // this wave's loads of stage kt + 1: all but the weights of stage kt + 2
                    if (kt + 2 < KB) vm_wait<4>(); else vm_wait<0>();
                    barrier();
                };
                // Loads go out one at a time between the products (a burst of
                // them holds up the wave at its issue): the weights of stage
                // kt + 2 before the boundary, in the slot that stage kt - 1
                // read, and behind it the rows and scales of stage kt + 2.
                constexpr int WT = RG > 3 ? RG - 2 : 1;                    // tiles that the weight loads are spread over
                auto weights = [&](int i) {
                    if (kt + 2 < KB) issue_w(kt + 2, i);
                };
                auto rows = [&](int i) {
                    if (kt + 2 < KB) {
                        issue_a(kt + 2, i);
                        if (i == 3) issue_s(kt + 2);
                    }
                };
                static_for<RG>([&](auto t_c) {
                    constexpr int I = decltype(t_c)::value, B = buffer(I);
                    constexpr bool LAST = I + 1 == RG;
                    constexpr auto B2 = std::integral_constant<int, buffer(I + 2)>{};
                    constexpr auto B1 = std::integral_constant<int, buffer(I + 1)>{};
                    if constexpr (RG <= 2 && I == 0) static_for<4>([&](auto j_c) { weights(decltype(j_c)::value); });
                    if constexpr (I + 2 == RG) {
                        lds_wait_all();
                        if constexpr (I == 0)
                            static_for<4>([&](auto c_c) {
                                tie_after_wait(w[decltype(c_c)::value][0]);
                                tie_after_wait(w[decltype(c_c)::value][1]);
                            });
                        tie_x(std::integral_constant<int, B>{});
                        tie_x(B1);
                        if constexpr (I == 0) tie_s();
                        if (more) boundary();
                        if constexpr (RG > 2) read_x(B2, std::integral_constant<int, 0>{}, kt + 1);
                    }
                    if constexpr (LAST && RG > 2) read_x(B2, std::integral_constant<int, 1>{}, kt + 1);
                    constexpr int O = (I + RG - 1) % RG;           // the tile whose partial sums are in p
                    static_for<4>([&](auto c_c) {
                        constexpr int C = decltype(c_c)::value;
                        if constexpr (I == 0 && RG != 2) {
                            // (the next column tiles' weights and the scales may still be on their way)
                            asm volatile("s_waitcnt lgkmcnt(%0)" : : "n"(9 - 2 * C) : "memory");
                            tie_after_wait(w[C][0]);
                            tie_after_wait(w[C][1]);
                            if constexpr (C == 0) {
                                tie_x(std::integral_constant<int, B>{});
                                if constexpr (RG > 1) tie_x(B1);
                            }
                        }
                        const i32x8 xv = pack8(x[B][0], x[B][1]);
                        __builtin_amdgcn_sched_barrier(0);
                        const float f = PHASE == 1 && C >= 2 ? f1 : f0;
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[O][C][r] = fmaf(p[C][r], f, acc[O][C][r]);
                        asm volatile("" : "+v"(acc[O][C]));        // (here, not sunk to the end of the stage)
                        __builtin_amdgcn_sched_barrier(0);
                        p[C] = mfma16_fp8(pack8(w[C][0], w[C][1]), xv, f32x4{});
                        __builtin_amdgcn_sched_barrier(0);
                        if constexpr (RG > 2 && I < WT && C == 1)
                            static_for<4 * (I + 1) / WT - 4 * I / WT>(
                                [&](auto j_c) { weights(4 * I / WT + decltype(j_c)::value); });
                        if constexpr (LAST && RG > 1) {
                            read_w(c_c, kt + 1);
                            rows(C);
                        }
                    });
                    if constexpr (I + 2 < RG) read_x(B2, std::integral_constant<int, I + 2>{}, kt);
                    if constexpr (RG == 2) read_x(std::integral_constant<int, B>{}, std::integral_constant<int, I>{}, kt + 1);
                    if constexpr (I == 0 && RG != 2) {             // the stage's scales (and with them the next tile)
                        asm volatile("s_waitcnt lgkmcnt(%0)" : : "n"(RG > 2 ? 2 : 0) : "memory");
                        tie_s();
                    } else if constexpr (I + 3 < RG) {             // (the last two tiles wait before the barrier)
                        asm volatile("s_waitcnt lgkmcnt(2)" ::: "memory");
                        tie_x(B1);
                    }
                    const uint32_t sr = I < 4 ? sx0[I & 3] : sx1[I & 3];
                    f0 = __uint_as_float(sr) * __uint_as_float(swv[0]);
                    f1 = PHASE == 1 ? __uint_as_float(sr) * __uint_as_float(swv[1]) : f0;
                    if constexpr (LAST && RG > 1) read_s(kt + 1);
                    if constexpr (RG == 1) {                       // a single tile: everything of the next stage behind the barrier
                        if (more) {
                            boundary();
                            static_for<4>([&](auto j_c) { rows(decltype(j_c)::value); });
                        }
                        read_x(B1, std::integral_constant<int, 0>{}, kt + 1);
                        static_for<4>([&](auto c_c) { read_w(c_c, kt + 1); });
                        read_s(kt + 1);
                    }
                });
                if constexpr (RG == 0) {
                    static_for<4>([&](auto j_c) { weights(decltype(j_c)::value); });
                    if (more) {
                        boundary();
                        static_for<4>([&](auto j_c) { rows(decltype(j_c)::value); });
                    }
                }
            };

            if constexpr (RG > 0) {
                read_x(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{}, 0);
                if constexpr (RG > 1) read_x(std::integral_constant<int, 1>{}, std::integral_constant<int, 1>{}, 0);
                static_for<4>([&](auto c_c) { read_w(c_c, 0); });
                read_s(0);
            }
            int kt = 0;
            do stage(kt); while (++kt < KB);
            if constexpr (RG > 0) {
                // the last stage's reads ahead hold nothing; they land before
                // their registers are used again
                lds_wait_all();
                static_for<4>([&](auto c_c) {
                    tie_after_wait(w[decltype(c_c)::value][0]);
                    tie_after_wait(w[decltype(c_c)::value][1]);
                });
                static_for<NB>([&](auto b_c) { tie_x(b_c); });
                tie_s();
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[RA - 1][c][r] = fmaf(p[c][r], PHASE == 1 && c >= 2 ? f1 : f0, acc[RA - 1][c][r]);
            }

            // The next item's first loads go out here, into slots that no
            // wave reads any more (its stage 0 follows this item's last one),
            // and land over the epilogue.
            if (has_next) {
                aim(tn, ntn, en);
                w0 = (w0 + KB) % FF_NW;
                a0 = (a0 + KB) & 1;
                issue_first();
            }

            // Result element i of tile t, column tile c: row 16 (2 t + G) + m, column 16 c + 4 kg + i
            if constexpr (PHASE == 1) {
                float* top = reinterpret_cast<float*>(lds + FF_T0);
                static_for<RG>([&](auto t_c) {
                    constexpr int I = decltype(t_c)::value;
                    float tp = 0.0f;
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float v = silu_mul(acc[I][c][r], acc[I][c + 2][r]);
                            acc[I][c][r] = v;
                            tp = fmaxf(tp, fabsf(v));              // (NaN is passed over)
                        }
                    if (__builtin_expect(__any(tp == __uint_as_float(0x7f800000u)), 0)) {
                        tp = 0.0f;                                 // an infinity somewhere: over the finite values
#pragma unroll
                        for (int c = 0; c < 2; ++c)
#pragma unroll
                            for (int r = 0; r < 4; ++r) tp = fmaxf(tp, finite_abs(acc[I][c][r]));
                    }
                    tp = fmaxf(tp, __shfl_xor(tp, 16, 64));
                    tp = fmaxf(tp, __shfl_xor(tp, 32, 64));
                    if (kg == 0) top[q * 256 + 32 * I + 16 * G + m] = tp;
                });
                vm_wait<0>();                                      // the next item's loads; the stores below stay behind
                lds_barrier();
                static_for<RG>([&](auto t_c) {
                    constexpr int I = decltype(t_c)::value;
                    const int r = 32 * I + 16 * G + m;
                    const float* tr = top + r;
                    const float s = fp8_scale(fmaxf(fmaxf(tr[0], tr[256]), fmaxf(tr[512], tr[768])));
                    const float rs = pow2_rcp(s);
                    uint32_t v[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        v[c] = fp8_pack4(acc[I][c][0] * rs, acc[I][c][1] * rs, acc[I][c][2] * rs, acc[I][c][3] * rs);
                    swap16(v[0], v[1]);                    // even kg: 8 columns of tile 0, odd kg: of tile 1
                    if (r < t.rows) {
                        *reinterpret_cast<uint2*>(a.act + (size_t)(t.row0 + r) * a.I + nt * 128 + 32 * q + 16 * (kg & 1) +
                                                  4 * (kg & 2)) = make_uint2(v[0], v[1]);
                        if (q == 0 && kg == 0) a.as[(size_t)nt * P + t.row0 + r] = s;
                    }
                });
            } else {
                vm_wait<0>();
                static_for<RG>([&](auto t_c) {
                    constexpr int I = decltype(t_c)::value;
                    const int r = 32 * I + 16 * G + m;
                    // 4 columns of each column tile per lane -> the 16 of tile kg
                    uint32_t v[4][2];
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[c][h] = (uint32_t)f32_to_f16_bits(acc[I][c][2 * h]) |
                                      ((uint32_t)f32_to_f16_bits(acc[I][c][2 * h + 1]) << 16);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        swap32(v[0][h], v[2][h]);
                        swap32(v[1][h], v[3][h]);
                        swap16(v[0][h], v[1][h]);
                        swap16(v[2][h], v[3][h]);
                    }
                    if (r < t.rows) {
                        uint16_t* dst = a.y + (size_t)(t.row0 + r) * a.H + nt * 256 + 64 * q + 16 * kg;
                        stg16(dst, u32x4{v[0][0], v[0][1], v[1][0], v[1][1]});
                        stg16(dst + 8, u32x4{v[2][0], v[2][1], v[3][0], v[3][1]});
                    }
                });
            }
        };
        switch ((tt + 1 - G) >> 1) {
            case 7: run(std::integral_constant<int, 7>{}); break;
            case 6: run(std::integral_constant<int, 6>{}); break;
            case 5: run(std::integral_constant<int, 5>{}); break;
            case 4: run(std::integral_constant<int, 4>{}); break;
            case 3: run(std::integral_constant<int, 3>{}); break;
            case 2: run(std::integral_constant<int, 2>{}); break;
            case 1: run(std::integral_constant<int, 1>{}); break;
            default: run(std::integral_constant<int, 0>{}); break;
        }
        lds_barrier();                                             // everybody's loads have landed; the maxima are free again
        if (!has_next) break;
        item += gridDim.x;
        t = tn;
        nt = ntn;
        fat_item_of(a.fat, tq, ahead, NT, tn, ntn);
    }
}

// The row scales of x in sorted order, block-major: xst[b, i] = xs[sorted_pair[i] / k, b].
// The MFMA-tile kernel then reads the 32 rows of a tile as one line per block.
// Nothing to do where no list became an M-tile.
__global__ __launch_bounds__(256)
void fp8_sort_scales_kernel(const FfnHeader* __restrict__ hdr, const float* __restrict__ xs,
                            const int32_t* __restrict__ sorted_pair, int P, int k, int KB, float* __restrict__ xst) {
    __shared__ float tile[64][33];
    if (hdr->n_fat == 0) return;
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
        fp8_sort_scales_kernel<<<blocks, 256, 0, s>>>(a.hdr, a.xs, a.sorted_pair, P, a.k, a.H / FP8_BLOCK, a.xst);
        ffn_fp8_fat_kernel<1><<<cus, FF_THREADS, FF_LDS, s>>>(a);
    } else {
        ffn_fp8_fat_kernel<2><<<cus, FF_THREADS, FF_LDS, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace moe
