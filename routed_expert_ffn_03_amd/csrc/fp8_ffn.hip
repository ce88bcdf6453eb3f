// Grouped expert FFN on e4m3 weights with one fp32 scale per 128 x 128 block:
//   xq, sx = e4m3 rows of x          (one power-of-two scale per 128 columns)
//   a      = silu(xq Wg^T) * (xq Wu^T)
//   aq, sa = e4m3 rows of a
//   y      = aq Wd^T, stored fp16
// with every 128-column partial product multiplied by its two scales before it
// is added in fp32 (fp8.h).  Busy experts run as MFMA tiles (fp8_fat.hip); here
// are the phases and the streaming kernel of the short route lists, which
// includes all of a decode step.
//
// The weights are the MFMA's A operand and the activation rows its B operand,
// so that a lane's result registers all belong to one activation row: the row
// scale is one value per lane, the weight scale one value per column tile, and
// four consecutive result registers are four consecutive output columns.
//
// Streaming kernel.  Work item: (a tile of up to 32 rows, 128 columns of a or
// 64 of y).  A wave owns 32 gate and the matching 32 up rows (phase 1, four
// waves a block) or 64 rows of W_down (phase 2, one wave a block: with four,
// the 400 items of 4 tokens left a fifth of the CUs' room empty, 40.4 us
// against 39.2; 1 token 21.3 against 18.0) over the whole reduction index, so
// no partial sums cross waves; phase 1 exchanges the row maxima of
// its 128 columns, which are one scale group of a, and stores codes.  Every
// weight is used once, so it is bound by HBM reads: a wave streams its 64 rows
// through its own two-slot LDS ring by direct-to-LDS loads of 8 rows x 128
// bytes with the non-temporal hint (whole lines).  A block of 128 columns
// (8 KB) goes to registers at once, so that two are in flight while it is
// multiplied, across items too.  Activation rows come straight into registers,
// one block ahead; they are a few KB that stay in L2.  The products are fp16
// ones of the converted codes, exact and summed in fp32: half the e4m3 rate
// and two conversions for each pair of codes, which hide under the loads
// (4 tokens on 25 experts of 4096 x 2048, one MI355X: gate/up 70 us and down
// 37 us, 6.0 and 5.7 TB/s of weights, at most 1 us more than with e4m3 products;
// 1,024 tokens, 327 short lists: 0.83 and 0.47 ms, 6.4 TB/s, the same either
// way), and y is five times as close to exact sums.
#include "common.h"
#include "ffn_shared.h"
#include "fp8.h"
#include "kernels.h"
#include "lds_dma.h"

namespace moe {
namespace {

constexpr uint32_t FS_CHUNK = 64 * 128;              // a wave's 64 weight rows of one block
constexpr int FS_SLOTS = 2;
constexpr int FS_CU_WAVES = 8;                       // that fit a CU's LDS

// waves per block
template <int PHASE>
constexpr int fs_waves = PHASE == 1 ? 4 : 1;

template <int PHASE>
__global__ __launch_bounds__(fs_waves<PHASE> * 64, 2)
void ffn_fp8_stream_kernel(Fp8Args a) {
    constexpr int NW = fs_waves<PHASE>;
    constexpr int BN = PHASE == 1 ? 128 : 64 * NW;   // columns of an item
    __shared__ __attribute__((aligned(1024))) char ring[NW * FS_SLOTS * FS_CHUNK];
    __shared__ float top[2][NW][32];                  // phase 1: row maxima by wave, alternating between items
    const int lane = threadIdx.x & 63;
    const int wave = NW > 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
    const int m = lane & 31, g = lane >> 5;
    const int K = PHASE == 1 ? a.H : a.I, N = PHASE == 1 ? a.I : a.H;
    const int KB = K / FP8_BLOCK;
    const int NT = N / BN;
    const int n_mt = a.hdr->n_thin;
    const int n_items = n_mt * NT;
    const size_t P = (size_t)a.T * a.k;
    const size_t wbytes = (size_t)N * K;
    int item = blockIdx.x;
    if (item >= n_items) return;                     // the whole block

    // (read-only here: through the constant address space, so by scalar loads,
    // which leave the vector loads' count alone)
    typedef const __attribute__((address_space(4))) MTile* ctile_t;
    typedef const __attribute__((address_space(4))) float* cfloat_t;
    struct Item {
        int e, row0, rows, nt;
        uint32_t bytes;                              // of its weights that may be loaded
    };
    // items past the end: the last one, with no weights in range (their loads
    // count and go nowhere)
    auto load_item = [&](int it) {
        const int ic = min(it, n_items - 1), nt = ic / n_mt;
        const ctile_t tp = (ctile_t)a.thin + __builtin_amdgcn_readfirstlane(ic - nt * n_mt);
        return Item{tp->e, tp->row0, tp->rows, nt, it < n_items ? (uint32_t)wbytes : 0u};
    };
    // load instruction i moves rows 8 i .. 8 i + 7: lane L row L / 8, position
    // L % 8, which holds piece (L % 8) ^ (row & 7) ^ ((row >> 3) & 1)
    const int lr = lane >> 3;
    uint32_t po[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) po[i] = (uint32_t)(((lane & 7) ^ lr ^ i) * 16);
    auto issue_w = [&](const Item& q, int ch, int sl) {
        const size_t eoff = (size_t)q.e * wbytes;
        const __amdgpu_buffer_rsrc_t w0 = make_rsrc((PHASE == 1 ? a.wg : a.wd) + eoff, q.bytes);
        const __amdgpu_buffer_rsrc_t w1 = PHASE == 1 ? make_rsrc(a.wu + eoff, q.bytes) : w0;
        const uint32_t r0 = (uint32_t)(q.nt * BN + (PHASE == 1 ? 32 : 64) * wave) + lr;
        char* st = ring + (wave * FS_SLOTS + sl) * FS_CHUNK;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(i < 4 ? w0 : w1, (lds_ptr_t)(st + i * 1024), 16,
                                                     (r0 + 8 * (PHASE == 1 ? i & 3 : i)) * (uint32_t)K + po[i & 1],
                                                     ch * FP8_BLOCK, 0, 2);
    };
    // fragment reads: lane (m, g), half h of the block, 16 bytes j: piece 4 h + 2 g + j of row m
    const uint32_t base = lds_addr(ring) + (uint32_t)(wave * FS_SLOTS) * FS_CHUNK + (uint32_t)m * 128;
    uint32_t fo[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) fo[h][j] = base + (uint32_t)(((4 * h + 2 * g + j) ^ (m & 7) ^ ((m >> 3) & 1)) * 16);

    // Loads run two blocks ahead of the products, across items: block
    // (issue, ich) goes out next.
    int issue = item, ich = 0;
    Item qi = load_item(item);
    auto issue_next = [&](int sl) {
        issue_w(qi, ich, sl);
        if (++ich == KB) {
            ich = 0;
            issue += gridDim.x;
            qi = load_item(issue);
        }
    };
    // Activation rows run one block ahead, their route-list entries two.
    // (Rows past a tile repeat its last one; they are never stored.)
    auto entry = [&](const Item& q) {
        const int row = q.row0 + min(m, q.rows - 1);
        return PHASE == 1 ? a.sorted_pair[row] : row;
    };
    Item cur = qi;
    int en = entry(qi), src = PHASE == 1 ? en / a.k : en, xch = 0;
    bool fresh = false;                              // src is of the item before, en of this one
    u32x4 xf[2][2];
    float sx;
    auto issue_x = [&](int ch) {
        const uint8_t* x = (PHASE == 1 ? a.xq : a.act) + (size_t)src * K + ch * FP8_BLOCK + 32 * g;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) xf[h][j] = ldg16(x + 64 * h + 16 * j);
        sx = PHASE == 1 ? a.xs[(size_t)src * KB + ch] : a.as[(size_t)ch * P + src];
    };
    auto next_x = [&]() {                            // rows of block xch; look up those of the block after it
        issue_x(xch);
        xch = ich;
        fresh = ich == 0;
        if (fresh) en = entry(qi);
    };
    issue_next(0);
    next_x();
    __builtin_amdgcn_sched_barrier(0);
    issue_next(1);
    for (int sl = 0, par = 0;; par ^= 1) {
        const Item nxt = load_item(item + gridDim.x);
        const int row = cur.row0 + min(m, cur.rows - 1);
        const size_t soff = (size_t)cur.e * (N / FP8_BLOCK) * KB;
        const cfloat_t s0 = (cfloat_t)(PHASE == 1 ? a.sg + soff + (size_t)cur.nt * KB
                                                  : a.sd + soff + (size_t)((cur.nt * BN + 64 * wave) / FP8_BLOCK) * KB);
        const cfloat_t s1 = PHASE == 1 ? (cfloat_t)(a.su + soff + (size_t)cur.nt * KB) : s0;
        f32x16 acc[2] = {f32x16{}, f32x16{}};
        for (int ch = 0; ch < KB; ++ch) {
            const float f0 = s0[ch], f1 = s1[ch];
            vm_wait<8>();                            // all but the block after this one
            const uint32_t so = (uint32_t)sl * FS_CHUNK;
            u32x4 w[2][2][2];
            static_for<2>([&](auto h_c) {
                static_for<2>([&](auto j_c) {
                    constexpr int Hh = decltype(h_c)::value, J = decltype(j_c)::value;
                    w[0][Hh][J] = ds_read16<0>(fo[Hh][J] + so);
                    w[1][Hh][J] = ds_read16<32 * 128>(fo[Hh][J] + so);
                });
            });
            u32x4 xh[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32x4 v = xf[i >> 2][(i >> 1) & 1];
                xh[i] = fp8_to_f16(v[2 * (i & 1)], v[2 * (i & 1) + 1]);
            }
            const float g0 = sx * f0, g1 = PHASE == 1 ? sx * f1 : g0;
            if (fresh) src = PHASE == 1 ? en / a.k : en;
            next_x();
            lds_wait_all();
            static_for<2>([&](auto h_c) {
                static_for<2>([&](auto j_c) {
                    constexpr int Hh = decltype(h_c)::value, J = decltype(j_c)::value;
                    tie_after_wait(w[0][Hh][J]);
                    tie_after_wait(w[1][Hh][J]);
                });
            });
            __builtin_amdgcn_sched_barrier(0);
            issue_next(sl);                          // the slot is in registers
            __builtin_amdgcn_sched_barrier(0);
            f32x16 p0 = f32x16{}, p1 = f32x16{};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const u32x4 u = w[0][i >> 2][(i >> 1) & 1], v = w[1][i >> 2][(i >> 1) & 1];
                p0 = mfma_f16(fp8_to_f16(u[2 * (i & 1)], u[2 * (i & 1) + 1]), xh[i], p0);
                p1 = mfma_f16(fp8_to_f16(v[2 * (i & 1)], v[2 * (i & 1) + 1]), xh[i], p1);
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                acc[0][r] = fmaf(p0[r], g0, acc[0][r]);
                acc[1][r] = fmaf(p1[r], g1, acc[1][r]);
            }
            sl ^= 1;
        }
        if constexpr (PHASE == 1) {
            float tp = 0.0f;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                acc[0][r] = silu_mul(acc[0][r], acc[1][r]);
                tp = fmaxf(tp, finite_abs(acc[0][r]));
            }
            tp = fmaxf(tp, __shfl_xor(tp, 32, 64));
            if (g == 0) top[par][wave][m] = tp;
            lds_barrier();                           // (the next item's weights stay in flight)
            const float s = fp8_scale(fmaxf(fmaxf(top[par][0][m], top[par][1][m]), fmaxf(top[par][2][m], top[par][3][m])));
            const float r = pow2_rcp(s);
            if (m < cur.rows) {
                uint8_t* dst = a.act + (size_t)row * a.I + cur.nt * 128 + 32 * wave + 4 * g;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<uint32_t*>(dst + 8 * j) =
                        fp8_pack4(acc[0][4 * j] * r, acc[0][4 * j + 1] * r, acc[0][4 * j + 2] * r, acc[0][4 * j + 3] * r);
                if (wave == 0 && g == 0) a.as[(size_t)cur.nt * P + row] = s;
            }
        } else if (m < cur.rows) {
            uint16_t* dst = a.y + (size_t)row * a.H + cur.nt * BN + 64 * wave + 4 * g;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint2 o;
                    o.x = (uint32_t)f32_to_f16_bits(acc[c][4 * j]) | ((uint32_t)f32_to_f16_bits(acc[c][4 * j + 1]) << 16);
                    o.y = (uint32_t)f32_to_f16_bits(acc[c][4 * j + 2]) | ((uint32_t)f32_to_f16_bits(acc[c][4 * j + 3]) << 16);
                    *reinterpret_cast<uint2*>(dst + 32 * c + 8 * j) = o;
                }
        }
        item += gridDim.x;
        if (item >= n_items) break;
        cur = nxt;
    }
    vm_wait<0>();                                    // the unused last blocks have landed
}

}  // namespace

hipError_t launch_fp8_phase(const Fp8Args& a, int phase, int cus, bool fat, bool x_ready, hipStream_t s) {
    if (phase == 1 && !x_ready) {
        const hipError_t err = launch_quantize_fp8(a.x, 1, a.T, a.H, 1, a.xq, a.xs, s);
        if (err != hipSuccess) return err;
    }
    if (fat) {
        const hipError_t err = launch_fp8_fat_phase(a, phase, cus, s);
        if (err != hipSuccess) return err;
    }
    const int waves = FS_CU_WAVES * cus;
    if (phase == 1) ffn_fp8_stream_kernel<1><<<waves / fs_waves<1>, fs_waves<1> * 64, 0, s>>>(a);
    else ffn_fp8_stream_kernel<2><<<waves / fs_waves<2>, fs_waves<2> * 64, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moe
