// routing.hpp -- each token's experts from a router's logits, the lists that a
// grouped product works on, the sum of a token's experts, and gradients.
//
//   p = softmax(x) or sigmoid(x);  c = p + bias;  x = -inf: closed, never chosen
//   group score = the sum of a group's one or two best open c; the best groups stay
//   experts = the `top` largest c, a tie to the lowest index
//   weight_k = scale p_k / sum_j p_j  or  scale p_k
// c and group scores are binary64: neighbours that binary32 takes for equal would
// change an expert.  Without a bias and sums c is x itself, which orders as p does.
//
// One wave chooses for a token, with V neighbouring experts in each lane.  A
// workgroup takes a stretch of tokens in rounds of up to 64; in a round every expert
// has 64 bits, one for each token that chose it, so a token's place among the
// expert's is a population count, whatever order the waves come in.
#pragma once

#include "gemm_mxfp4.hpp"

namespace lpgemm {

constexpr int kRouteWaves = 16, kRouteThreads = 64 * kRouteWaves;

struct RouteArgs {
    const void *logits;  // [T][ldl]
    const float *bias;   // [E] or null
    int32_t *experts;    // [T][top]
    float *weights;      // [T][top]
    int32_t *rows;       // [T top]
    int32_t *offsets;    // [E + 1]
    int32_t *places;     // [T][top]
    int32_t *counts;     // [workgroups][E], for several workgroups
    int64_t ldl;
    int32_t T, E, top, groups, top_groups, group_top;
    int32_t per_group, stretch;  // experts of a group, tokens of a workgroup
    int32_t sigmoid, renormalise;
    float scale;
};

// Element i of a row as binary32.
template <int IN>
__device__ __forceinline__ float route_load(const void *x, int64_t at)
{
    if (IN == OUT_F32) return static_cast<const float *>(x)[at];
    const uint16_t u = static_cast<const uint16_t *>(x)[at];
    if (IN == OUT_BF16) return __uint_as_float((uint32_t)u << 16);
    return (float)__builtin_bit_cast(_Float16, u);
}

// Unsigned keys that order as the values do: NaN above all, -0 as 0; 0 stands for closed.
__device__ __forceinline__ uint32_t route_key(float x)
{
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return x == -__builtin_inff() ? 0u : (int32_t)u < 0 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t route_key(double x)
{
    if (x != x) return ~0ull;
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.);
    return x == -__builtin_inf() ? 0ull : (int64_t)u < 0 ? ~u : u | 1ull << 63;
}

// The largest of all 64 lanes, in all of them.
__device__ __forceinline__ uint32_t route_largest(uint32_t x)
{
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));  // as mx_scan
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));
    x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

// The lowest lane that holds the largest key, -1 where every key is 0.
__device__ __forceinline__ int route_first(uint32_t key)
{
    const uint32_t m = route_largest(key);
    return m == 0u ? -1 : (int)__builtin_ctzll(__ballot(key == m));
}
__device__ __forceinline__ int route_first(uint64_t key)
{
    const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key, m = route_largest(hi);
    uint64_t at = __ballot(hi == m);
    if (at & (at - 1)) {  // several lanes share the upper half
        const uint32_t n = route_largest(hi == m ? lo : 0u);
        at = __ballot(hi == m && lo == n);
        if (m == 0u && n == 0u) return -1;
    }
    return m == 0u && __builtin_amdgcn_readlane((int)lo, (int)__builtin_ctzll(at)) == 0 ? -1 : (int)__builtin_ctzll(at);
}

__device__ __forceinline__ float route_readlane(float x, int lane) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane)); }
__device__ __forceinline__ double route_readlane(double x, int lane)
{
    const uint64_t u = (uint64_t)__double_as_longlong(x);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = (uint32_t)__builtin_amdgcn_readlane((int)(u >> 32), lane);
    return __longlong_as_double((int64_t)((uint64_t)hi << 32 | lo));
}
__device__ __forceinline__ uint64_t route_readlane(uint64_t x, int lane)
{
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), lane) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, lane);
}

template <typename F>
__device__ __forceinline__ F route_sum(F x)
{
#pragma unroll
    for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
    return x;
}

__device__ __forceinline__ float route_exp(float x) { return expf(x); }
__device__ __forceinline__ double route_exp(double x) { return exp(x); }

template <bool WIDE>
struct RouteTypes {
    typedef float F;
    typedef uint32_t Key;
};
template <>
struct RouteTypes<true> {
    typedef double F;
    typedef uint64_t Key;
};

// The experts of token t: lane k < top ends with expert k (-1: none) and its weight.
// `room`: E doubles of the wave's own in LDS, where groups are left out.
template <int IN, int V, bool WIDE>
__device__ __forceinline__ void route_token(const RouteArgs &g, int64_t t, const int (&group)[V], const float (&bias)[V], double *room, int &expert,
                                            float &weight)
{
    typedef typename RouteTypes<WIDE>::F F;
    typedef typename RouteTypes<WIDE>::Key Key;
    const int lane = threadIdx.x & 63;
    float x[V];
    const float none = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        x[i] = e < g.E ? route_load<IN>(g.logits, t * g.ldl + e) : none;
    }
    F p[V], total = 1;
    if (g.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = x[i] == none ? (F)0 : (F)1 / ((F)1 + route_exp(-(F)x[i]));
    } else {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, route_key(x[i]));
        best = route_largest(best);  // 0: all closed
        const float most = best == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((int32_t)best < 0 ? best ^ 0x80000000u : ~best);
        F sum = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = x[i] == none ? (F)0 : route_exp((F)x[i] - (F)most);
            sum += p[i];
        }
        total = route_sum(sum);
    }
    Key key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (WIDE) {
            const F c = (g.sigmoid ? p[i] : p[i] / total) + (F)bias[i];
            key[i] = (Key)(x[i] == none ? 0 : route_key(c));
        } else {
            key[i] = (Key)route_key(x[i]);
        }
    }
    if (g.top_groups < g.groups) {
        // lane j scores group j
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane * V + i;
            const F c = WIDE ? (g.sigmoid ? p[i] : p[i] / total) + (F)bias[i] : (F)x[i];
            if (e < g.E) room[e] = x[i] == none ? -__builtin_inf() : (double)c;
        }
        __builtin_amdgcn_wave_barrier();
        double first = -__builtin_inf(), second = first;
        uint64_t k1 = 0, k2 = 0;
        if (lane < g.groups)
            for (int j = 0; j < g.per_group; ++j) {
                const double c = room[lane * g.per_group + j];
                const uint64_t k = route_key(c);
                if (k > k1) {
                    second = first, k2 = k1;
                    first = c, k1 = k;
                } else if (k > k2) {
                    second = c, k2 = k;
                }
            }
        const uint64_t score = k1 == 0 ? 0 : route_key(g.group_top > 1 && k2 != 0 ? first + second : first);
        int better = 0;
        for (int j = 0; j < g.groups; ++j) {
            const uint64_t other = route_readlane(score, j);
            better += other > score || (other == score && j < lane) ? 1 : 0;
        }
        const uint64_t kept = __ballot(lane < g.groups && better < g.top_groups);
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (!(kept >> group[i] & 1)) key[i] = 0;
        __builtin_amdgcn_wave_barrier();
    }
    expert = -1;
    F mine = 0, chosen = 0;
    for (int k = 0; k < g.top; ++k) {
        Key best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < V; ++i)
            if (key[i] > best) best = key[i], at = i;
        const int from = __builtin_amdgcn_readfirstlane(route_first(best));
        if (from < 0) break;
        F q = p[0];
#pragma unroll
        for (int i = 1; i < V; ++i) q = at == i ? p[i] : q;
        q = route_readlane(q, from);
        chosen += q;
        const int e = from * V + __builtin_amdgcn_readlane(at, from);  // by all lanes: a branch would leave others' registers
        if (lane == k) {
            expert = e;
            mine = q;
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (lane == from && at == i) key[i] = 0;
    }
    if (g.renormalise) total = chosen == 0 ? (F)1 : chosen;
    weight = expert < 0 ? 0.f : (float)((F)g.scale * (mine / total));
}

// Exclusive sums of n <= 1024 counts in LDS over a workgroup's threads; sums[n] the whole.
__device__ __forceinline__ void route_offsets(const int32_t *count, int32_t *sums, int n, int32_t *part)
{
    const int tid = threadIdx.x, wave = tid >> 6;
    const int own = tid < n ? count[tid] : 0, run = mx_scan(own);
    if ((tid & 63) == 63) part[wave] = run;
    __syncthreads();
    int before = run - own;
    for (int w = 0; w < wave; ++w) before += part[w];
    if (tid < n) sums[tid] = before;
    if (tid == n - 1) sums[n] = before + own;
    __syncthreads();
}

// The places of a workgroup's tokens [t0, t1), whose ranks among their expert's the
// first kernel left there, and the rows' tokens; base[e]: where this workgroup's begin.
__device__ __forceinline__ void route_place(const RouteArgs &g, int64_t t0, int64_t t1, const int32_t *base)
{
    for (int64_t i = t0 * g.top + threadIdx.x; i < t1 * g.top; i += kRouteThreads) {
        const int e = g.experts[i];
        if (e < 0) continue;  // its place is -1 already
        const int at = base[e] + g.places[i];
        g.places[i] = at;
        g.rows[at] = (int32_t)(i / g.top);
    }
}

// Rows behind the last expert's are nobody's.
__device__ __forceinline__ void route_tail(const RouteArgs &g, int used, int block, int blocks)
{
    for (int64_t i = used + (int64_t)block * kRouteThreads + threadIdx.x; i < (int64_t)g.T * g.top; i += (int64_t)blocks * kRouteThreads) g.rows[i] = -1;
}

// LDS: masks [E][2], counts [E], sums [E + 1], part [waves]; room [waves][E] doubles.
__host__ __device__ inline int route_lds(int E, bool groups) { return ((4 * (4 * E + 1 + kRouteWaves) + 7) & ~7) + (groups ? 8 * kRouteWaves * E : 0); }

// Chooses every token's experts; with one workgroup (`alone`) the lists too, else each
// workgroup's counts.  PER: tokens of a wave in a round.
template <int IN, int V, bool WIDE>
__global__ __launch_bounds__(kRouteThreads) void route_choose_kernel(RouteArgs g, int per, int alone)
{
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem);
    int32_t *count = reinterpret_cast<int32_t *>(mask + 2 * g.E), *sums = count + g.E, *part = sums + g.E + 1;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    double *room = reinterpret_cast<double *>(smem + route_lds(g.E, false)) + wave * g.E;
    int group[V];
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        group[i] = e < g.E ? e / g.per_group : 0;
        bias[i] = WIDE && g.bias != nullptr && e < g.E ? g.bias[e] : 0.f;
    }
    for (int i = tid; i < g.E; i += kRouteThreads) {
        count[i] = 0;
        mask[2 * i] = mask[2 * i + 1] = 0;
    }
    __syncthreads();
    const int64_t t0 = (int64_t)blockIdx.x * g.stretch, t1 = min((int64_t)g.T, t0 + g.stretch);
    for (int64_t r0 = t0; r0 < t1; r0 += kRouteWaves * per) {
        int chosen[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            chosen[j] = -1;
            const int local = wave * per + j;
            const int64_t t = r0 + local;
            if (j >= per || t >= t1) continue;
            float weight;
            route_token<IN, V, WIDE>(g, t, group, bias, room, chosen[j], weight);
            if (lane < g.top) {
                g.experts[t * g.top + lane] = chosen[j];
                g.weights[t * g.top + lane] = weight;
                if (chosen[j] >= 0) atomicOr(&mask[2 * chosen[j] + (local >> 5)], 1u << (local & 31));
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int local = wave * per + j;
            const int64_t t = r0 + local;
            if (j >= per || t >= t1 || lane >= g.top) continue;
            int rank = -1;
            if (chosen[j] >= 0) {
                const uint64_t m = (uint64_t)mask[2 * chosen[j] + 1] << 32 | mask[2 * chosen[j]];
                rank = count[chosen[j]] + (int)__popcll(m & ((1ull << local) - 1));
            }
            g.places[t * g.top + lane] = rank;
        }
        __syncthreads();
        for (int i = tid; i < g.E; i += kRouteThreads) {
            count[i] += (int)__popc(mask[2 * i]) + (int)__popc(mask[2 * i + 1]);
            mask[2 * i] = mask[2 * i + 1] = 0;
        }
        __syncthreads();
    }
    if (!alone) {
        for (int i = tid; i < g.E; i += kRouteThreads) g.counts[(int64_t)blockIdx.x * g.E + i] = count[i];
        return;
    }
    route_offsets(count, sums, g.E, part);
    for (int i = tid; i <= g.E; i += kRouteThreads) g.offsets[i] = sums[i];
    route_place(g, t0, t1, sums);  // its own writes of this workgroup, behind barriers
    route_tail(g, sums[g.E], 0, 1);
}

// The lists from the workgroups' counts: each adds up those of the ones before it.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs g)
{
    extern __shared__ __align__(16) uint8_t smem[];
    // before [E], total [E], sums [E + 1], part [waves]
    int32_t *before = reinterpret_cast<int32_t *>(smem), *total = before + g.E, *sums = total + g.E, *part = sums + g.E + 1;
    const int tid = threadIdx.x, blocks = (int)gridDim.x, mine = (int)blockIdx.x;
    for (int i = tid; i < g.E; i += kRouteThreads) before[i] = total[i] = 0;
    __syncthreads();
    const int lanes = min(kRouteThreads, (g.E + 63) / 64 * 64), parts = kRouteThreads / lanes;
    const int e = tid % lanes, first = tid / lanes;
    if (e < g.E && first < parts) {
        int b = 0, a = 0;
        for (int i = first; i < blocks; i += parts) {
            const int c = g.counts[(int64_t)i * g.E + e];
            a += c;
            b += i < mine ? c : 0;
        }
        atomicAdd(&total[e], a);  // whole numbers: any order
        atomicAdd(&before[e], b);
    }
    __syncthreads();
    route_offsets(total, sums, g.E, part);
    for (int i = tid; i < g.E; i += kRouteThreads) before[i] += sums[i];
    if (mine == 0)
        for (int i = tid; i <= g.E; i += kRouteThreads) g.offsets[i] = sums[i];
    __syncthreads();
    const int64_t t0 = (int64_t)mine * g.stretch, t1 = min((int64_t)g.T, t0 + g.stretch);
    route_place(g, t0, t1, before);
    route_tail(g, sums[g.E], mine, blocks);
}

// No tokens: every expert's list is empty.
__global__ __launch_bounds__(256) void route_empty_kernel(int32_t *offsets, int32_t E)
{
    for (int i = threadIdx.x; i <= E; i += 256) offsets[i] = 0;
}

// ---- the logits' gradient --------------------------------------------------------
// With g_k = dL / d weight_k, S = sum of the chosen p, w'_k = p_k / S:
//   dL / dp_k = scale (g_k - sum_j g_j w'_j) / S  or  scale g_k;  0 for the others
//   softmax: dx_i = p_i (dp_i - sum_j p_j dp_j);  sigmoid: dx_i = p_i (1 - p_i) dp_i
// The renormalised softmax has sum p dp = 0 and a gradient at the chosen alone.
struct RouteGradArgs {
    const void *logits;
    const float *dweights;   // [T][top]
    const int32_t *experts;  // [T][top]
    void *dlogits;           // [T][E], dense
    int64_t ldl;
    int32_t T, E, top, sigmoid, renormalise;
    float scale;
};

template <int OUT>
__device__ __forceinline__ void route_store(void *y, int64_t at, float x)
{
    if (OUT == OUT_F32)
        static_cast<float *>(y)[at] = x;
    else
        static_cast<uint16_t *>(y)[at] = (uint16_t)(mx_pack2<OUT>(x, 0.f) & 0xFFFFu);
}

template <int IN, int V>
__global__ __launch_bounds__(256) void route_backward_kernel(RouteGradArgs g)
{
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= g.T) return;
    const float none = -__builtin_inff();
    float p[V], slope[V];  // p and, for sigmoid, p (1 - p)
    float total = 1.f, most = 0.f;
    if (!g.sigmoid) most = none;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = lane * V + i;
        p[i] = e < g.E ? route_load<IN>(g.logits, t * g.ldl + e) : none;
        if (!g.sigmoid) most = p[i] > most || p[i] != p[i] ? p[i] : most;
    }
    if (!g.sigmoid) {
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const float o = __shfl_xor(most, d);
            most = o > most || o != o ? o : most;
        }
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = p[i] == none ? 0.f : expf(p[i] - most);
            sum += p[i];
        }
        total = route_sum(sum);
        if (total == 0.f) total = 1.f;  // all closed
    }
    auto sigmoid = [](float x) { return x == -__builtin_inff() ? 0.f : 1.f / (1.f + expf(-x)); };
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (g.sigmoid) {
            const float s = sigmoid(p[i]);
            slope[i] = p[i] == none ? 0.f : s * (1.f / (1.f + expf(p[i])));
        } else {
            slope[i] = p[i] /= total;
        }
    }
    // lane k: expert k, its p and its weight's gradient
    int e = -1;
    float q = 0.f, d = 0.f;
    if (lane < g.top) {
        e = g.experts[t * g.top + lane];
        if (e < 0 || e >= g.E) e = -1;
        if (e >= 0) {
            const float x = route_load<IN>(g.logits, t * g.ldl + e);
            q = g.sigmoid ? sigmoid(x) : x == none ? 0.f : expf(x - most) / total;
            d = g.scale * g.dweights[t * g.top + lane];
        }
    }
    if (g.renormalise) {
        const float S = route_sum(q), mean = route_sum(d * q);
        d = S == 0.f ? 0.f : (d - mean / S) / S;
    }
    float dp[V];
#pragma unroll
    for (int i = 0; i < V; ++i) dp[i] = 0.f;
    for (int k = 0; k < g.top; ++k) {
        const int to = __builtin_amdgcn_readlane(e, k);
        const float v = route_readlane(d, k);
#pragma unroll
        for (int i = 0; i < V; ++i) dp[i] += to == lane * V + i ? v : 0.f;
    }
    float mean = 0.f;
    if (!g.sigmoid && !g.renormalise) mean = route_sum(e >= 0 ? q * d : 0.f);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int to = lane * V + i;
        if (to < g.E) route_store<IN>(g.dlogits, t * g.E + to, slope[i] * (dp[i] - mean));
    }
}

// ---- a token's experts added up ---------------------------------------------------
//   out[t] = residual[t] + sum_k weights[t][k] y[places[t][k]]
// in binary32, k in order; a place outside [0, R) adds nothing.  Bound by memory.
struct CombineArgs {
    const void *y;          // [R][N]
    const int32_t *places;  // [T][top]
    const float *weights;   // [T][top] or null: ones
    const void *residual;   // [T][N] or null, of the result's type
    void *out;              // [T][N]
    int64_t R, T;
    int32_t N, top, pieces;  // pieces: workgroups of a token's row
};

// Eight values of a row from n on as binary32, zeros from N on.
template <int IN>
__device__ __forceinline__ void route_load8(const void *x, int64_t at, int left, float (&v)[8])
{
    u32x4 w[2];
    mx_load8<IN, false>(x, at, left, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (IN == OUT_F32) {
            v[j] = __uint_as_float(w[j / 4][j % 4]);
        } else {
            const uint32_t d = w[0][j / 2];
            if (IN == OUT_BF16) v[j] = __uint_as_float(j % 2 ? d & 0xFFFF0000u : d << 16);
            else v[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(j % 2 ? d >> 16 : d));
        }
    }
}
template <int OUT>
__device__ __forceinline__ void route_store8(void *y, int64_t at, int n, int N, const float (&v)[8])
{
    mx_store4<OUT>(y, at, n, N, v[0], v[1], v[2], v[3]);
    mx_store4<OUT>(y, at, n + 4, N, v[4], v[5], v[6], v[7]);
}

template <int IN, int OUT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs g)
{
    const int64_t t = blockIdx.x / g.pieces;
    const int n = (int)(blockIdx.x % g.pieces) * 2048 + 8 * (int)threadIdx.x;
    if (n >= g.N) return;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, v[4][8];
    for (int k0 = 0; k0 < g.top; k0 += 4) {
        float w[4];
        bool there[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + j;
            const int at = k < g.top ? g.places[t * g.top + k] : -1;
            there[j] = at >= 0 && at < g.R;
            w[j] = there[j] && g.weights != nullptr ? g.weights[t * g.top + k] : 1.f;
            if (there[j]) route_load8<IN>(g.y, (int64_t)at * g.N + n, g.N - n, v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (there[j])
#pragma unroll
                for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], v[j][i], sum[i]);
    }
    if (g.residual != nullptr) {
        route_load8<OUT>(g.residual, t * g.N + n, g.N - n, v[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += v[0][i];
    }
    route_store8<OUT>(g.out, t * g.N, n, g.N, sum);
}

// dy[places[t][k]] = weights[t][k] dout[t];  dweights[t][k] = <dout[t], y[places[t][k]]>.
// A workgroup takes a token; binary32 sums in a fixed order.
struct CombineGradArgs {
    const void *dout;       // [T][N]
    const void *y;          // [R][N]
    const int32_t *places;  // [T][top]
    const float *weights;   // [T][top] or null: ones
    void *dy;               // [R][N], of y's type; rows in no place are left
    float *dweights;        // [T][top]
    int64_t R, T;
    int32_t N, top;
};

constexpr int kCombineSlots = 8;  // experts at a time

template <int IN, int OUT>
__global__ __launch_bounds__(256) void combine_backward_kernel(CombineGradArgs g)
{
    __shared__ float part[4][kCombineSlots];
    const int64_t t = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int k0 = 0; k0 < g.top; k0 += kCombineSlots) {
        float dot[kCombineSlots], w[kCombineSlots];
        int at[kCombineSlots];
#pragma unroll
        for (int j = 0; j < kCombineSlots; ++j) {
            const int k = k0 + j;
            at[j] = k < g.top ? g.places[t * g.top + k] : -1;
            if (at[j] >= g.R) at[j] = -1;
            w[j] = at[j] >= 0 && g.weights != nullptr ? g.weights[t * g.top + k] : 1.f;
            dot[j] = 0.f;
        }
        for (int n = 8 * (int)threadIdx.x; n < g.N; n += 2048) {
            float d[8];
            route_load8<OUT>(g.dout, t * g.N + n, g.N - n, d);
#pragma unroll
            for (int j = 0; j < kCombineSlots; ++j) {
                if (at[j] < 0) continue;
                float v[8];
                route_load8<IN>(g.y, (int64_t)at[j] * g.N + n, g.N - n, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] = __builtin_fmaf(d[i], v[i], dot[j]);
                    v[i] = w[j] * d[i];
                }
                route_store8<IN>(g.dy, (int64_t)at[j] * g.N, n, g.N, v);
            }
        }
        __syncthreads();  // the last slots' sums have been read
#pragma unroll
        for (int j = 0; j < kCombineSlots; ++j) {
            const float s = route_sum(dot[j]);
            if (lane == 0) part[wave][j] = s;
        }
        __syncthreads();
        const int k = k0 + (int)threadIdx.x;
        if ((int)threadIdx.x < kCombineSlots && k < g.top)
            g.dweights[t * g.top + k] = part[0][threadIdx.x] + part[1][threadIdx.x] + part[2][threadIdx.x] + part[3][threadIdx.x];
    }
}

}  // namespace lpgemm
