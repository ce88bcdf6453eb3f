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
// Forward: one pass over the logits.  A wave takes whole tokens, a lane holds
// NV = ceil(E / 64) of a token's logits; the probabilities are added up in
// registers over the wave's tokens, across the waves in LDS, and stored per
// block.  A second kernel adds the blocks' sums in a fixed order (no float
// atomics: the same bits from run to run), and its last block adds up the
// loss.  Backward: one pass, reading the logits and writing their gradient
// once; the softmax is computed again, which costs no traffic.
#include "common.h"
#include "kernels.h"

#include <algorithm>
#include <type_traits>

namespace moe {
namespace {

constexpr int BL_THREADS = 256;
constexpr int BL_WAVES = BL_THREADS / WAVE;
constexpr int BL_TOKENS = 64;                    // tokens per forward block (one group's)
constexpr int BR_COLS = 32;                      // experts per block of the second kernel

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
    return v;
}
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

// The softmax of one token: p[i] of expert lane + 64 i.  A row whose every
// logit is -inf has p = 0.
template <int NV>
__device__ __forceinline__ void token_softmax(const float* __restrict__ row, int E, int lane, float (&p)[NV]) {
    const float lowest = -__uint_as_float(0x7f800000u);
    float mx = lowest;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        p[i] = e < E ? row[e] : lowest;
        mx = fmaxf(mx, p[i]);
    }
    mx = wave_max(mx);
    if (mx == lowest) mx = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        p[i] = __expf(p[i] - mx);
        s += p[i];
    }
    s = wave_sum(s);
    const float r = s > 0.0f || s != s ? 1.0f / s : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] *= r;
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

BalanceWs balance_ws(int T, int E, int G, void* base) {
    const size_t nb = (size_t)G * ((T / G + BL_TOKENS - 1) / BL_TOKENS);
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
                            const uint8_t* __restrict__ mask, int E, int k, int L, int bpg, BalanceWs ws) {
    __shared__ float sp[BL_WAVES][64 * NV];
    __shared__ int sc[64 * NV];
    __shared__ int sn[BL_WAVES];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < 64 * NV; e += BL_THREADS) sc[e] = 0;
    __syncthreads();
    const int grp = blockIdx.x / bpg, i0 = (blockIdx.x - grp * bpg) * BL_TOKENS;
    const int i1 = min(i0 + BL_TOKENS, L);
    float sum[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) sum[i] = 0.0f;
    int n = 0;
    for (int i = i0 + wave; i < i1; i += BL_WAVES) {
        const size_t t = (size_t)grp * L + i;
        if (mask && mask[t] == 0) continue;
        ++n;
        if (lane < k) {
            const int e = ids[t * k + lane];
            if (e >= 0 && e < E) atomicAdd(&sc[e], 1);
        }
        float p[NV];
        token_softmax<NV>(logits + t * E, E, lane, p);
#pragma unroll
        for (int j = 0; j < NV; ++j) sum[j] += p[j];
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

// Block (g, c): experts 32 c .. of group g; thread (r, e): blocks r, r + 8, ...
// The block that finishes last knows every group's n_g, so it counts the live
// groups and writes the loss and the group scales.
__global__ __launch_bounds__(BL_THREADS)
void balance_reduce_kernel(BalanceWs ws, int E, int k, int G, int bpg, float coef, int32_t* __restrict__ counts,
                           float* __restrict__ prob, float* __restrict__ group_scale, float* __restrict__ loss) {
    constexpr int R = BL_THREADS / BR_COLS;
    __shared__ float sp[R][BR_COLS];
    __shared__ int sc[R][BR_COLS];
    __shared__ int sn[BL_WAVES];
    __shared__ float sl[BL_WAVES];
    __shared__ bool last;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, ncb = gridDim.x / G;
    const int grp = blockIdx.x / ncb, cb = blockIdx.x - grp * ncb;
    const int r = tid / BR_COLS, c = tid % BR_COLS, e = cb * BR_COLS + c;
    int n = 0;
    for (int b = tid; b < bpg; b += BL_THREADS) n += ws.n[(size_t)grp * bpg + b];
    n = wave_sum(n);
    if (lane == 0) sn[wave] = n;
    float p = 0.0f;
    int cnt = 0;
    if (e < E)
        for (int b = r; b < bpg; b += R) {
            const size_t at = ((size_t)grp * bpg + b) * E + e;
            p += ws.prob[at];
            cnt += ws.counts[at];
        }
    sp[r][c] = p;
    sc[r][c] = cnt;
    __syncthreads();
    n = sn[0] + sn[1] + sn[2] + sn[3];
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
    for (int q = tid; q < G; q += BL_THREADS)
        live += __hip_atomic_load(&ws.group_n[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) > 0;
    float v = 0.0f;
    for (int i = tid; i < (int)gridDim.x; i += BL_THREADS)
        v += __hip_atomic_load(&ws.part[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    live = wave_sum(live);
    v = wave_sum(v);
    __syncthreads();                             // sn was read above
    if (lane == 0) {
        sn[wave] = live;
        sl[wave] = v;
    }
    __syncthreads();
    live = sn[0] + sn[1] + sn[2] + sn[3];
    const float f = live > 0 ? coef * (float)E / ((float)k * (float)live) : 0.0f;
    if (tid == 0) *loss = f * (sl[0] + sl[1] + sl[2] + sl[3]);
    for (int q = tid; q < G; q += BL_THREADS) {
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
    int T, E, k, L;
    float* d_logits;
};

template <int NV>
__global__ __launch_bounds__(BL_THREADS)
void route_backward_kernel(RouteBwdArgs a) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (size_t t = (size_t)blockIdx.x * BL_WAVES + wave; t < (size_t)a.T; t += (size_t)gridDim.x * BL_WAVES) {
        float d[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) d[i] = 0.0f;
        if (a.counts && !(a.mask && a.mask[t] == 0)) {
            const size_t grp = t / (size_t)a.L;
            float p[NV], dot = 0.0f;
            token_softmax<NV>(a.logits + t * a.E, a.E, lane, p);
            const float s = *a.d_loss * a.group_scale[grp];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = lane + 64 * i;
                d[i] = e < a.E ? s * (float)a.counts[grp * a.E + e] : 0.0f;
                dot = fmaf(p[i], d[i], dot);
            }
            dot = wave_sum(dot);
#pragma unroll
            for (int i = 0; i < NV; ++i) d[i] = p[i] * (d[i] - dot);
        }
        if (a.d_w) {
            const bool on = lane < a.k;
            const size_t at = t * a.k + lane;
            const float w = on ? a.w[at] : 0.0f, dw = on ? a.d_w[at] : 0.0f;
            const int id = on ? a.ids[at] : -1;
            const float dot = wave_sum(w * dw);
            const float v = w * (dw - dot);
            for (int j = 0; j < a.k; ++j) {
                const int e = __builtin_amdgcn_readfirstlane(__shfl(id, j, 64));
                const float vj = __shfl(v, j, 64);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (e == lane + 64 * i) d[i] += vj;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = lane + 64 * i;
            if (e < a.E) a.d_logits[t * a.E + e] = d[i];
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
    const size_t nb = (size_t)G * ((T / G + BL_TOKENS - 1) / BL_TOKENS);
    return nb * BL_THREADS < (1ull << 32) && (size_t)G * ((E + BR_COLS - 1) / BR_COLS) * BL_THREADS < (1ull << 32);
}

size_t balance_ws_bytes(int T, int E, int G) { return balance_ws(T, E, G, nullptr).bytes; }

hipError_t launch_balance_loss(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E, int k,
                               int G, float coef, int32_t* counts, float* prob, float* group_scale, float* loss,
                               void* workspace, hipStream_t s) {
    const BalanceWs ws = balance_ws(T, E, G, workspace);
    const int L = T / G, bpg = (L + BL_TOKENS - 1) / BL_TOKENS;
    with_nv(E, [&](auto nv) {
        balance_partial_kernel<decltype(nv)::value><<<(unsigned)G * bpg, BL_THREADS, 0, s>>>(logits, ids, mask, E, k,
                                                                                          L, bpg, ws);
    });
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const int ncb = (E + BR_COLS - 1) / BR_COLS;
    balance_reduce_kernel<<<(unsigned)G * ncb, BL_THREADS, 0, s>>>(ws, E, k, G, bpg, coef, counts, prob, group_scale,
                                                                   loss);
    return hipGetLastError();
}

hipError_t launch_route_backward(const float* logits, const int32_t* ids, const float* w, const float* d_w,
                                 const int32_t* counts, const float* group_scale, const float* d_loss,
                                 const uint8_t* mask, int T, int E, int k, int G, float* d_logits, hipStream_t s) {
    const RouteBwdArgs a{logits, ids, w, d_w, counts, group_scale, d_loss, mask, T, E, k, T / G, d_logits};
    const unsigned blocks = (unsigned)std::min((T - 1) / BL_WAVES + 1, 4096);
    with_nv(E, [&](auto nv) { route_backward_kernel<decltype(nv)::value><<<blocks, BL_THREADS, 0, s>>>(a); });
    return hipGetLastError();
}

}  // namespace moe
