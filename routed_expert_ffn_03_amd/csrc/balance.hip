// The router's balance loss with per-expert counts, and the gradient of it
// and of the gate weights with respect to the router logits.
//
// With p = softmax of a token's logits over all experts, G groups of L = T/G
// consecutive tokens, n_g the tokens of group g that are not masked, c_ge
// their (token, slot) pairs on expert e and G' the groups with n_g > 0:
//   P_ge = sum_t p_te / n_g
//   loss = coef / G' * sum_g E / (k n_g) * sum_e c_ge P_ge
// The counts carry no gradient, so with s_g = coef E / (k n_g^2 G') (0 for an
// empty group) d loss / d p_te = s_g c_ge, and through the softmax
//   d l_te = p_te (b_te - sum_f p_tf b_tf),  b_te = d_loss s_g c_ge.
// The gate's weights are a softmax over the k selected logits:
//   d l_t,id_j += w_j (dw_j - sum_i w_i dw_i).
//
// Forward: one pass over the logits.  A wave takes two tokens at a time, a
// lane holds NV = ceil(E / 64) of a token's logits; the probabilities are
// added up in registers over the wave's tokens, across the waves in LDS, and
// stored per block.  A second kernel adds the blocks' sums in a fixed order (no
// float atomics: the same bits from run to run), and its last block adds up the
// loss.  Backward: one pass, reading the logits and writing their gradient
// once; the softmax is computed again, which costs no traffic.  Both are bound
// by latency up to about 16k tokens (a token is a load, two or three
// reductions over the wave and an exponential, in turn) and by HBM beyond.
// One MI355X, 384 experts, top-8, the three kernels: 1,024 tokens 4 + 6 + 6
// us, 16,384 tokens 8 + 8 + 14 us, 16 x 4,096 tokens with a fifth of them
// masked 26 + 9 + 39 us (the gradient at 4.7 TB/s).  One token at a
// time, with shuffles for the reductions, the whole took 52 us at 16,384 tokens
// and 99 us at 16 x 4,096, now 28.6 and 75.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int BL_THREADS = 256;
constexpr int BL_WAVES = BL_THREADS / WAVE;
constexpr int BL_ILP = 2;                        // tokens of a wave at a time
constexpr int BR_THREADS = 1024;                 // second kernel: 32 experts x 32 rows of blocks
constexpr int BR_COLS = 32;

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int l) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}

// op over the 64 lanes, the result in every lane: exchanges inside each row
// of 16 lanes (neighbour, pair, half row, row), then the four rows by scalar
// reads (a shuffle per step takes an LDS round trip each)
template <class Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
    v = op(v, dpp<0xB1>(v));                     // quad_perm 1 0 3 2
    v = op(v, dpp<0x4E>(v));                     // quad_perm 2 3 0 1
    v = op(v, dpp<0x141>(v));                    // row_half_mirror
    v = op(v, dpp<0x140>(v));                    // row_mirror
    return op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
}
__device__ __forceinline__ float wave_max(float v) {
    return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ float wave_sum(float v) {
    return wave_reduce(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The LDS accesses of this wave's lanes before it are done before those after.
__device__ __forceinline__ void wave_lds_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The logits of one token: l[i] of expert lane + 64 i, -inf past E.
template <int NV>
__device__ __forceinline__ void token_load(const float* __restrict__ row, int E, int lane, float (&l)[NV]) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < E ? row[e] : -__uint_as_float(0x7f800000u);
    }
}

// l -> softmax(l).  A row whose every logit is -inf has p = 0; NaN or +inf
// make the whole row NaN.
template <int NV>
__device__ __forceinline__ void token_softmax(float (&l)[NV]) {
    float mx = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) mx = fmaxf(mx, l[i]);
    mx = wave_max(mx);
    if (mx == -__uint_as_float(0x7f800000u)) mx = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        l[i] = __expf(l[i] - mx);
        s += l[i];
    }
    s = wave_sum(s);
    const float r = s > 0.0f || s != s ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] *= r;
}

// Tokens of a forward block (all of one group): some 1,024 blocks where there
// are enough tokens, two for each wave at least, 128 at most (each block
// leaves E sums for the second kernel).
int block_tokens(int T, int G) {
    const int per = T / 1024, L = T / G;
    int t = BL_WAVES * BL_ILP;
    while (t < 128 && t < per) t *= 2;
    while (t > BL_WAVES * BL_ILP && t / 2 >= L) t /= 2;
    return t;
}

// Where the workspace keeps the blocks' sums.
struct BalanceWs {
    int* ticket;                                 // blocks of the second kernel that are done
    int* n;                                      // [nb] tokens counted by each block
    int* group_n;                                // [G] tokens counted in each group
    float* part;                                 // [G * col blocks] terms of the loss
    float* prob;                                 // [nb, E]
    int* counts;                                 // [nb, E]
    size_t bytes;
};

size_t balance_blocks(int T, int G) {
    const int bt = block_tokens(T, G);
    return (size_t)G * ((size_t)(T / G) / bt + (T / G % bt ? 1 : 0));
}

BalanceWs balance_ws(int T, int E, int G, void* base) {
    const size_t nb = balance_blocks(T, G);
    auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    char* p = reinterpret_cast<char*>(base);
    BalanceWs w;
    size_t o = 0;
    w.ticket = reinterpret_cast<int*>(p + o); o += 256;
    w.n = reinterpret_cast<int*>(p + o); o += up(nb * 4);
    w.group_n = reinterpret_cast<int*>(p + o); o += up((size_t)G * 4);
    w.part = reinterpret_cast<float*>(p + o); o += up((size_t)G * ((E + BR_COLS - 1) / BR_COLS) * 4);
    w.prob = reinterpret_cast<float*>(p + o); o += up(nb * E * 4);
    w.counts = reinterpret_cast<int*>(p + o); o += up(nb * E * 4);
    w.bytes = o;
    return w;
}

template <int NV>
__global__ __launch_bounds__(BL_THREADS)
void balance_partial_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                            const uint8_t* __restrict__ mask, int E, int k, int L, int bt, int bpg, BalanceWs ws) {
    __shared__ float sp[BL_WAVES][64 * NV];
    __shared__ int sc[64 * NV];
    __shared__ int sn[BL_WAVES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = tid; e < 64 * NV; e += BL_THREADS) sc[e] = 0;
    __syncthreads();
    const int grp = blockIdx.x / bpg, i0 = (blockIdx.x - grp * bpg) * bt;
    const int i1 = min(i0 + bt, L);
    float sum[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) sum[i] = 0.0f;
    int n = 0;
    for (int i = i0 + wave * BL_ILP; i < i1; i += BL_WAVES * BL_ILP) {
        float p[BL_ILP][NV];
        int id[BL_ILP];
        bool on[BL_ILP];
#pragma unroll
        for (int u = 0; u < BL_ILP; ++u) {
            const size_t t = (size_t)grp * L + i + u;
            on[u] = i + u < i1 && (!mask || mask[t] != 0);
            if (!on[u]) continue;                // (masked tokens are not read)
            id[u] = lane < k ? ids[t * k + lane] : -1;
            token_load<NV>(logits + t * E, E, lane, p[u]);
        }
#pragma unroll
        for (int u = 0; u < BL_ILP; ++u) {
            if (!on[u]) continue;
            ++n;
            if (id[u] >= 0 && id[u] < E) atomicAdd(&sc[id[u]], 1);
            token_softmax<NV>(p[u]);
#pragma unroll
            for (int j = 0; j < NV; ++j) sum[j] += p[u][j];
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) sp[wave][lane + 64 * j] = sum[j];
    if (lane == 0) sn[wave] = n;
    __syncthreads();
    for (int e = tid; e < E; e += BL_THREADS) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < BL_WAVES; ++w) v += sp[w][e];
        ws.prob[(size_t)blockIdx.x * E + e] = v;
        ws.counts[(size_t)blockIdx.x * E + e] = sc[e];
    }
    if (tid == 0) {
        int v = 0;
        for (int w = 0; w < BL_WAVES; ++w) v += sn[w];
        ws.n[blockIdx.x] = v;
        if (blockIdx.x == 0) *ws.ticket = 0;
    }
}

// Block (g, c): experts 32 c .. of group g; thread (r, e): blocks r, r + 32, ...
// The block that finishes last knows every group's n_g, so it counts the live
// groups and writes the loss and the group scales.
__global__ __launch_bounds__(BR_THREADS)
void balance_reduce_kernel(BalanceWs ws, int E, int k, int G, int bpg, float coef, int32_t* __restrict__ counts,
                           float* __restrict__ prob, float* __restrict__ group_scale, float* __restrict__ loss) {
    constexpr int R = BR_THREADS / BR_COLS, NW = BR_THREADS / WAVE;
    __shared__ float sp[R][BR_COLS];
    __shared__ int sc[R][BR_COLS];
    __shared__ int sn[NW];
    __shared__ float sl[NW];
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, ncb = gridDim.x / G;
    const int grp = blockIdx.x / ncb, cb = blockIdx.x - grp * ncb;
    const int r = tid / BR_COLS, c = tid % BR_COLS, e = cb * BR_COLS + c;
    int n = 0;
    for (int b = tid; b < bpg; b += BR_THREADS) n += ws.n[(size_t)grp * bpg + b];
    n = wave_sum(n);
    if (lane == 0) sn[wave] = n;
    float p = 0.0f;
    int cnt = 0;
    if (e < E)
#pragma unroll 4
        for (int b = r; b < bpg; b += R) {
            const size_t at = ((size_t)grp * bpg + b) * E + e;
            p += ws.prob[at];
            cnt += ws.counts[at];
        }
    sp[r][c] = p;
    sc[r][c] = cnt;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) n += sn[w];
    float term = 0.0f;
    if (r == 0 && e < E) {
        p = 0.0f;
        cnt = 0;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            p += sp[i][c];
            cnt += sc[i][c];
        }
        p = n > 0 ? p / (float)n : 0.0f;
        prob[(size_t)grp * E + e] = p;
        counts[(size_t)grp * E + e] = cnt;
        term = n > 0 ? (float)cnt * p / (float)n : 0.0f;
    }
    if (tid < 64) {                              // (lanes past BR_COLS hold 0)
        term = wave_sum(term);
        if (tid == 0) {
            __hip_atomic_store(&ws.part[blockIdx.x], term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (cb == 0) __hip_atomic_store(&ws.group_n[grp], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = __hip_atomic_fetch_add(ws.ticket, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
                   (int)gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    int live = 0;
    for (int q = tid; q < G; q += BR_THREADS)
        live += __hip_atomic_load(&ws.group_n[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
    float v = 0.0f;
    for (int i = tid; i < (int)gridDim.x; i += BR_THREADS)
        v += __hip_atomic_load(&ws.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    live = wave_sum(live);
    v = wave_sum(v);
    __syncthreads();                             // sn was read above
    if (lane == 0) {
        sn[wave] = live;
        sl[wave] = v;
    }
    __syncthreads();
    live = 0;
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        live += sn[w];
        v += sl[w];
    }
    const float f = live > 0 ? coef * (float)E / ((float)k * (float)live) : 0.0f;
    if (tid == 0) *loss = f * v;
    for (int q = tid; q < G; q += BR_THREADS) {
        const int m = __hip_atomic_load(&ws.group_n[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        group_scale[q] = m > 0 ? f / ((float)m * (float)m) : 0.0f;
    }
}

struct RouteBwdArgs {
    const float* logits;
    const int32_t* ids;
    const float* w;
    const float* d_w;                            // nullable
    const int32_t* counts;                       // nullable, with the three below
    const float* group_scale;
    const float* d_loss;
    const uint8_t* mask;
    int T, E, k, L, chunk;
    float* d_logits;
};

// A wave takes `chunk` consecutive tokens, two at a time, and keeps the
// group's counts in registers.  The gate's k values are put to their experts
// through a row of LDS per wave and token: added where the ids say (an id that
// appears twice gets both), read back by expert, cleared.
template <int NV>
__global__ __launch_bounds__(BL_THREADS)
void route_backward_kernel(RouteBwdArgs a) {
    __shared__ float row[BL_WAVES][BL_ILP][64 * NV];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
    for (int u = 0; u < BL_ILP; ++u)
#pragma unroll
        for (int i = 0; i < NV; ++i) row[wave][u][lane + 64 * i] = 0.0f;
    const size_t t0 = ((size_t)blockIdx.x * BL_WAVES + wave) * a.chunk;
    const size_t t1 = min(t0 + a.chunk, (size_t)a.T);
    const float dl = a.counts ? *a.d_loss : 0.0f;
    size_t grp = ~(size_t)0;
    float bc[NV];                                // d loss / d p of the group
#pragma unroll
    for (int i = 0; i < NV; ++i) bc[i] = 0.0f;
    for (size_t t = t0; t < t1; t += BL_ILP) {
        float d[BL_ILP][NV], w[BL_ILP], dw[BL_ILP];
        int id[BL_ILP];
        bool on[BL_ILP];
#pragma unroll
        for (int u = 0; u < BL_ILP; ++u) {
            const size_t tu = t + u;
            on[u] = tu < t1 && a.counts && !(a.mask && a.mask[tu] == 0);
            w[u] = dw[u] = 0.0f;
            id[u] = -1;
            if (on[u]) token_load<NV>(a.logits + tu * a.E, a.E, lane, d[u]);
            if (tu < t1 && a.d_w && lane < a.k) {
                w[u] = a.w[tu * a.k + lane];
                dw[u] = a.d_w[tu * a.k + lane];
                id[u] = a.ids[tu * a.k + lane];
            }
        }
#pragma unroll
        for (int u = 0; u < BL_ILP; ++u) {
            const size_t tu = t + u;
            if (tu >= t1) break;
            if (on[u]) {
                const size_t g = tu / (size_t)a.L;
                if (g != grp) {
                    grp = g;
                    const float s = dl * a.group_scale[g];
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int e = lane + 64 * i;
                        bc[i] = e < a.E ? s * (float)a.counts[g * a.E + e] : 0.0f;
                    }
                }
                token_softmax<NV>(d[u]);
                float dot = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) dot = fmaf(d[u][i], bc[i], dot);
                dot = wave_sum(dot);
#pragma unroll
                for (int i = 0; i < NV; ++i) d[u][i] *= bc[i] - dot;
            } else {
#pragma unroll
                for (int i = 0; i < NV; ++i) d[u][i] = 0.0f;
            }
            if (a.d_w) {
                const float v = w[u] * (dw[u] - wave_sum(w[u] * dw[u]));
                const bool in = id[u] >= 0 && id[u] < a.E;
                if (in) atomicAdd(&row[wave][u][id[u]], v);
                wave_lds_order();
#pragma unroll
                for (int i = 0; i < NV; ++i) d[u][i] += row[wave][u][lane + 64 * i];
                wave_lds_order();
                if (in) row[wave][u][id[u]] = 0.0f;
                wave_lds_order();
            }
            float* out = a.d_logits + tu * a.E;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane + 64 * i;
                if (e < a.E) out[e] = d[u][i];
            }
        }
    }
}

// f(number of logits per lane) for E experts
template <class F>
void with_nv(int E, F&& f) {
    const int nv = (E + 63) / 64;
    if (nv <= 1) f(std::integral_constant<int, 1>{});
    else if (nv <= 2) f(std::integral_constant<int, 2>{});
    else if (nv <= 4) f(std::integral_constant<int, 4>{});
    else if (nv <= 6) f(std::integral_constant<int, 6>{});
    else if (nv <= 8) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}

}  // namespace

bool balance_shape_ok(int T, int E, int G) {
    // the launches below stay under 2^32 threads
    const size_t nb = balance_blocks(T, G);
    return nb * BL_THREADS < (1ull << 32) && (size_t)G * ((E + BR_COLS - 1) / BR_COLS) * BR_THREADS < (1ull << 32);
}

size_t balance_ws_bytes(int T, int E, int G) { return balance_ws(T, E, G, nullptr).bytes; }

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int k,
                               int G, float coef, int32_t* counts, float* prob, float* group_scale, float* loss,
                               void* workspace, hipStream_t s) {
    const BalanceWs ws = balance_ws(T, E, G, workspace);
    const int L = T / G, bt = block_tokens(T, G), bpg = (int)(balance_blocks(T, G) / G);
    with_nv(E, [&](auto nv) {
        balance_partial_kernel<decltype(nv)::value><<<(unsigned)G * bpg, BL_THREADS, 0, s>>>(logits, ids, mask, E, k,
                                                                                          L, bt, bpg, ws);
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int ncb = (E + BR_COLS - 1) / BR_COLS;
    balance_reduce_kernel<<<(unsigned)G * ncb, BR_THREADS, 0, s>>>(ws, E, k, G, bpg, coef, counts, prob, group_scale,
                                                                   loss);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* ids, const float* w, const float* d_w,
                                 const int32_t* counts, const float* group_scale, const float* d_loss,
                                 const uint8_t* mask, int T, int E, int k, int G, float* d_logits, hipStream_t s) {
    // up to 2,048 blocks, whole pairs of tokens per wave
    const size_t waves = 2048 * BL_WAVES;
    const int chunk = (int)(((size_t)T + waves * BL_ILP - 1) / (waves * BL_ILP)) * BL_ILP;
    const RouteBwdArgs a{logits, ids, w, d_w, counts, group_scale, d_loss, mask, T, E, k, T / G, chunk, d_logits};
    const unsigned blocks = (unsigned)(((size_t)T + (size_t)chunk * BL_WAVES - 1) / ((size_t)chunk * BL_WAVES));
    with_nv(E, [&](auto nv) { route_backward_kernel<decltype(nv)::value><<<blocks, BL_THREADS, 0, s>>>(a); });
    return hipGetLastError();
}

}  // namespace moe
