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

#include "fp8_block_quantize.hpp"

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
    uint16_t *counts;    // [workgroups][E rounded up to 2], for several workgroups
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

// Unsigned keys that order as the values do: NaN above all, -0 as 0, -inf 0.  Without
// branches, which the compiler makes of conditions on conditions.
__device__ __forceinline__ uint32_t route_key(float x)
{
    const uint32_t u = __float_as_uint(x + 0.f), k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
    return (k | (x != x ? ~0u : 0u)) & (x == -__builtin_inff() ? 0u : ~0u);
}
__device__ __forceinline__ uint64_t route_key(double x)
{
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.);
    const uint32_t sign = (uint32_t)((int32_t)(u >> 32) >> 31), high = x != x ? ~0u : 0u, low = x == -__builtin_inf() ? 0u : ~0u;
    const uint32_t hi = (((uint32_t)(u >> 32) ^ (sign | 0x80000000u)) | high) & low, lo = (((uint32_t)u ^ sign) | high) & low;
    return (uint64_t)hi << 32 | lo;
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

template <int V>
__device__ __forceinline__ void route_exp(float (&x)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = expf(x[i]);
}
// e^x in binary64 to about one step: x = n log 2 + r, |r| <= 0.35, Taylor's series of e^r
// to r^13 (the next term is 5e-18), times 2^n; log 2 in two parts, the first of 32 bits, so
// that n times it is exact.  A third of the library function's instructions.
template <int V>
__device__ __forceinline__ void route_exp(double (&x)[V])
{
    double r[V], p[V];
    int n[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const double whole = __builtin_rint(fmin(fmax(x[i], -1100.), 1100.) * 1.4426950408889634);
        r[i] = __builtin_fma(whole, -1.9082149292705877e-10, __builtin_fma(whole, -0.6931471803691238, x[i]));
        n[i] = (int)whole;
        p[i] = 1. / 6227020800.;
    }
    const double c[13] = {1. / 479001600., 1. / 39916800., 1. / 3628800., 1. / 362880., 1. / 40320., 1. / 5040., 1. / 720.,
                          1. / 120.,       1. / 24.,       1. / 6.,       0.5,          1.,          1.};
#pragma unroll
    for (int j = 0; j < 13; ++j) {
        double k = c[j];
        asm volatile("" : "+s"(k));  // not 26 registers of every lane through the tokens' loop
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = __builtin_fma(p[i], r[i], k);
    }
    // beyond the range the exponent decides (r may be anything there); NaN stays
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = x[i] > 710. ? __builtin_inf() : x[i] < -746. ? 0. : __builtin_ldexp(p[i], n[i]);
}

__device__ __forceinline__ float route_inverse(float x) { return 1.f / x; }
// 1 / x for x >= 1, or x = inf: two Newton steps from the instruction's estimate.
__device__ __forceinline__ double route_inverse(double x)
{
    double y = __builtin_amdgcn_rcp(x);
    y = __builtin_fma(__builtin_fma(-x, y, 1.), y, y);
    y = __builtin_fma(__builtin_fma(-x, y, 1.), y, y);
    return x > 1.7e308 ? 0. : y;
}

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

// The value that a key of binary64 stands for.
__device__ __forceinline__ double route_value(uint64_t key) { return __longlong_as_double((int64_t)(key >> 63 ? key ^ 1ull << 63 : ~key)); }

// Neighbouring V elements of a row from lane V on, -inf past it.
template <int IN, int V>
__device__ __forceinline__ void route_row(const void *x, int64_t at, int left, float (&v)[V])
{
    if (left >= V) {
        typename std::conditional<IN == OUT_F32, uint32_t, uint16_t>::type u[V];
        __builtin_memcpy(u, static_cast<const uint8_t *>(x) + at * (int64_t)sizeof(u[0]), sizeof(u));  // global memory takes any alignment
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = IN == OUT_F32    ? __uint_as_float((uint32_t)u[i])
                   : IN == OUT_BF16 ? __uint_as_float((uint32_t)u[i] << 16)
                                    : (float)__builtin_bit_cast(_Float16, (uint16_t)u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < left ? route_load<IN>(x, at + i) : -__builtin_inff();
    }
}

// The experts of a token with these logits: lane k < top ends with expert k (-1: none) and
// its weight.  `room`: E doubles of the wave's own in LDS, for groups that are not whole lanes.
template <int IN, int V, bool WIDE>
__device__ __forceinline__ void route_token(const RouteArgs &g, const void *logits, double *room, int &expert, float &weight)
{
    typedef typename RouteTypes<WIDE>::F F;
    typedef typename RouteTypes<WIDE>::Key Key;
    const int lane = threadIdx.x & 63;
    const float none = -__builtin_inff();
    const int left = g.E - lane * V;
    float x[V], bias[V], most = 0.f;
    route_row<IN, V>(logits, lane * V, left, x);
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = WIDE && g.bias != nullptr && i < left ? g.bias[lane * V + i] : 0.f;
    F p[V], inverse = 1;
    if (g.sigmoid) {
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = -(F)x[i];
        route_exp(p);
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = route_inverse((F)1 + p[i]);  // closed: 1 / inf
    } else {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) best = max(best, route_key(x[i]));
        best = route_largest(best);  // 0: all closed
        most = best == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u) : __uint_as_float((int32_t)best < 0 ? best ^ 0x80000000u : ~best);
        F sum = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) p[i] = (F)x[i] - (F)most;
        route_exp(p);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            p[i] = x[i] == none ? (F)0 : p[i];  // not NaN where a row's others make it that
            sum += p[i];
        }
        inverse = route_inverse(route_sum(sum));  // the largest alone is 1
    }
    Key key[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        key[i] = WIDE ? (Key)route_key(p[i] * inverse + (F)bias[i]) & (x[i] == none ? (Key)0 : ~(Key)0) : (Key)route_key(x[i]);
    if (g.top_groups < g.groups) {
        const int lanes = g.per_group / V;
        if (lanes * V == g.per_group && (lanes & (lanes - 1)) == 0) {
            // a group is `lanes` neighbouring lanes: its two largest keys meet in all of them
            Key k1 = key[0], k2 = 0;
#pragma unroll
            for (int i = 1; i < V; ++i) {
                k2 = max(k2, min(k1, key[i]));
                k1 = max(k1, key[i]);
            }
            for (int d = 1; d < lanes; d *= 2) {
                const Key o1 = (Key)__shfl_xor((unsigned long long)k1, d), o2 = (Key)__shfl_xor((unsigned long long)k2, d);
                k2 = max(max(k2, o2), min(k1, o1));
                k1 = max(k1, o1);
            }
            // sums are of binary64 scores; one score, as its key
            const uint64_t score = WIDE && g.group_top > 1 && k1 != 0 && k2 != 0 ? route_key(route_value(k1) + route_value(k2)) : (uint64_t)k1;
            const int mine = lane / lanes;
            int better = 0;
            for (int j = 0; j < g.groups; ++j) {
                const uint64_t other = route_readlane(score, j * lanes);
                better += other > score || (other == score && j < mine) ? 1 : 0;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) key[i] = better < g.top_groups ? key[i] : 0;
        } else {
            // lane j scores group j
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                if (e < g.E) reinterpret_cast<uint64_t *>(room)[e] = key[i];
            }
            __builtin_amdgcn_wave_barrier();
            uint64_t k1 = 0, k2 = 0;
            if (lane < g.groups)
                for (int j = 0; j < g.per_group; ++j) {
                    const uint64_t k = reinterpret_cast<const uint64_t *>(room)[lane * g.per_group + j];
                    k2 = max(k2, min(k1, k));
                    k1 = max(k1, k);
                }
            const uint64_t score = WIDE && g.group_top > 1 && k1 != 0 && k2 != 0 ? route_key(route_value(k1) + route_value(k2)) : k1;
            int better = 0;
            for (int j = 0; j < g.groups; ++j) {
                const uint64_t other = route_readlane(score, j);
                better += other > score || (other == score && j < lane) ? 1 : 0;
            }
            const uint64_t kept = __ballot(lane < g.groups && better < g.top_groups);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = lane * V + i;
                key[i] = e < g.E && (kept >> (e / g.per_group) & 1) ? key[i] : 0;
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
    // each lane's keys in order, equal ones by index, by an odd-even merging network (Batcher);
    // their indices, four bits each
    int index[V];
#pragma unroll
    for (int i = 0; i < V; ++i) index[i] = i;
#pragma unroll
    for (int p = 1; p < V; p *= 2)
#pragma unroll
        for (int q = p; q >= 1; q /= 2)
#pragma unroll
            for (int j = q % p; j + q < V; j += 2 * q)
#pragma unroll
                for (int i = 0; i < q; ++i) {
                    const int a = i + j, b = i + j + q;
                    if (b >= V || a / (2 * p) != b / (2 * p)) continue;
                    const bool swap = key[b] > key[a] || (key[b] == key[a] && index[b] < index[a]);
                    const Key hi = swap ? key[b] : key[a], lo = swap ? key[a] : key[b];
                    const int first = swap ? index[b] : index[a], second = swap ? index[a] : index[b];
                    key[a] = hi, key[b] = lo;
                    index[a] = first, index[b] = second;
                }
    typename std::conditional<(V > 8), uint64_t, uint32_t>::type order = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) order |= (decltype(order))index[i] << (4 * i);
    // the lanes' best in turn; lane k takes the k-th
    expert = -1;
    for (int k = 0; k < g.top; ++k) {
        const int from = __builtin_amdgcn_readfirstlane(route_first(key[0]));
        if (from < 0) break;
        const int e = from * V + (__builtin_amdgcn_readlane((int)(uint32_t)order, from) & 15);  // by all lanes: a branch would leave others' registers
        expert = lane == k ? e : expert;
        if (lane == from) {
#pragma unroll
            for (int i = 0; i + 1 < V; ++i) key[i] = key[i + 1];
            key[V - 1] = 0;
            order >>= 4;
        }
    }
    // their scores again, by the same steps: kept meanwhile they would take 2 V registers
    F mine = 0;
    if (expert >= 0) {
        const float y = route_load<IN>(logits, expert);
        F one[1] = {g.sigmoid ? -(F)y : (F)y - (F)most};
        route_exp(one);
        mine = g.sigmoid ? route_inverse((F)1 + one[0]) : one[0];
    }
    F chosen = mine;
    if (g.renormalise)
        for (int d = 1; d < g.top; d *= 2) chosen += __shfl_xor(chosen, d);  // the lanes past the last expert hold 0
    weight = expert < 0 ? 0.f : (float)((F)g.scale * (g.renormalise ? (chosen == 0 ? (F)0 : mine / chosen) : mine * inverse));
}

// Exclusive sums of n <= 1024 counts in LDS over a workgroup's threads; sums[n] the whole
// (the counts may lie there).
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

// Rows behind the last expert's are nobody's.
__device__ __forceinline__ void route_tail(const RouteArgs &g, int used, int block, int blocks)
{
    for (int64_t i = used + (int64_t)block * kRouteThreads + threadIdx.x; i < (int64_t)g.T * g.top; i += (int64_t)blocks * kRouteThreads) g.rows[i] = -1;
}

__host__ __device__ inline int route_pitch(int E) { return (E + 1) & ~1; }

// A workgroup's tokens in a round: its masks have 64 bits.
constexpr int kRouteRound = 64;

// LDS: masks [E][2], counts [E], sums [E + 1], part [waves], chosen [round][top] of 16
// bits; room [waves][E] doubles, where groups are not whole lanes.
__host__ __device__ inline int route_lds(int E, int top, bool room)
{
    return ((4 * (4 * E + 1 + kRouteWaves) + 2 * kRouteRound * top + 7) & ~7) + (room ? 8 * kRouteWaves * E : 0);
}

// Chooses every token's experts; with one workgroup (`alone`, one round) the lists too,
// else each workgroup's counts.  `per`: tokens of a wave in a round.
//
// Bound by instructions, for few tokens by their chain: one token of 256 experts, top 8 of
// 4 groups of 8, sigmoids with a bias 7.6 us; 512 tokens of 64, softmax 6.1; 8192 of 256
// 21.0 (the logits take 1.6 to read).  64 registers for two workgroups a compute unit
// spill: 24 to 32.
template <int IN, int V, bool WIDE>
__global__ __launch_bounds__(kRouteThreads, 4) void route_choose_kernel(RouteArgs g, int per, int alone)
{
    extern __shared__ __align__(16) uint8_t smem[];
    uint32_t *mask = reinterpret_cast<uint32_t *>(smem);
    int32_t *count = reinterpret_cast<int32_t *>(mask + 2 * g.E), *sums = count + g.E, *part = sums + g.E + 1;
    int16_t *chosen = reinterpret_cast<int16_t *>(part + kRouteWaves);
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    double *room = reinterpret_cast<double *>(smem + route_lds(g.E, g.top, false)) + wave * g.E;
    const int64_t t0 = (int64_t)blockIdx.x * g.stretch, t1 = min((int64_t)g.T, t0 + g.stretch);
    for (int i = tid; i < g.E; i += kRouteThreads) {
        count[i] = 0;
        mask[2 * i] = mask[2 * i + 1] = 0;
    }
    __syncthreads();
    for (int64_t r0 = t0; r0 < t1; r0 += kRouteWaves * per) {
        const int tokens = (int)min((int64_t)kRouteWaves * per, t1 - r0);
        for (int local = wave; local < tokens; local += kRouteWaves) {
            const int64_t t = r0 + local;
            int expert;
            float weight;
            route_token<IN, V, WIDE>(g, static_cast<const uint8_t *>(g.logits) + t * g.ldl * (IN == OUT_F32 ? 4 : 2), room, expert, weight);
            if (lane < g.top) {
                g.experts[t * g.top + lane] = expert;
                g.weights[t * g.top + lane] = weight;
                chosen[local * g.top + lane] = (int16_t)expert;
                if (expert >= 0) atomicOr(&mask[2 * expert + (local >> 5)], 1u << (local & 31));
            }
        }
        __syncthreads();
        // an entry's rank: its expert's earlier rounds and earlier tokens of this one
        auto rank = [&](int i) __attribute__((always_inline)) -> int {
            const int e = chosen[i], local = i / g.top;
            if (e < 0) return -1;
            const uint64_t m = (uint64_t)mask[2 * e + 1] << 32 | mask[2 * e];
            return count[e] + (int)__popcll(m & ((1ull << local) - 1));
        };
        if (!alone)
            for (int i = tid; i < tokens * g.top; i += kRouteThreads) g.places[r0 * g.top + i] = rank(i);
        else if (tid < g.E)
            sums[tid] = (int)__popc(mask[2 * tid]) + (int)__popc(mask[2 * tid + 1]);
        __syncthreads();
        if (alone) {  // counts stay 0: a place is the expert's first row and the rank
            route_offsets(sums, sums, g.E, part);
            for (int i = tid; i <= g.E; i += kRouteThreads) g.offsets[i] = sums[i];
            for (int i = tid; i < tokens * g.top; i += kRouteThreads) {
                const int at = rank(i);
                g.places[i] = at < 0 ? -1 : sums[chosen[i]] + at;
                if (at >= 0) g.rows[sums[chosen[i]] + at] = i / g.top;
            }
            route_tail(g, sums[g.E], 0, 1);
            return;
        }
        for (int i = tid; i < g.E; i += kRouteThreads) {
            count[i] += (int)__popc(mask[2 * i]) + (int)__popc(mask[2 * i + 1]);
            mask[2 * i] = mask[2 * i + 1] = 0;
        }
        __syncthreads();
    }
    for (int i = tid; i < g.E; i += kRouteThreads) g.counts[(int64_t)blockIdx.x * route_pitch(g.E) + i] = (uint16_t)count[i];
}

// The lists from the workgroups' counts: each adds up those of the ones before it (512
// tokens 5.2 us, 8192 7.0; from 512 workgroups' counts 10.8): bound by the chain of loads.
__global__ __launch_bounds__(kRouteThreads) void route_place_kernel(RouteArgs g)
{
    extern __shared__ __align__(16) uint8_t smem[];
    // before [E], total [E], sums [E + 1], part [waves]
    int32_t *before = reinterpret_cast<int32_t *>(smem), *total = before + g.E, *sums = total + g.E, *part = sums + g.E + 1;
    const int tid = threadIdx.x, mine = (int)blockIdx.x, blocks = (int)gridDim.x;
    const int64_t t0 = (int64_t)mine * g.stretch, t1 = min((int64_t)g.T, t0 + g.stretch);
    // the first of this thread's entries are on their way meanwhile
    const int64_t own = t0 * g.top + tid;
    int expert = -1, rank = 0;
    if (own < t1 * g.top) {
        expert = g.experts[own];
        rank = g.places[own];
    }
    for (int i = tid; i < g.E; i += kRouteThreads) before[i] = total[i] = 0;
    __syncthreads();
    // two experts a thread, every `parts`-th workgroup
    const int pitch = route_pitch(g.E), lanes = min(kRouteThreads, (pitch / 2 + 63) / 64 * 64), parts = kRouteThreads / lanes;
    const int e = tid % lanes * 2, first = tid / lanes;
    if (e < g.E && first < parts) {
        int b0 = 0, a0 = 0, b1 = 0, a1 = 0;
        for (int i = first; i < blocks; i += 16 * parts) {
            uint32_t c[16];  // on their way together
#pragma unroll
            for (int j = 0; j < 16; ++j)
                c[j] = i + j * parts < blocks ? *reinterpret_cast<const uint32_t *>(g.counts + (int64_t)(i + j * parts) * pitch + e) : 0u;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const bool earlier = i + j * parts < mine;
                a0 += c[j] & 0xFFFFu;
                a1 += c[j] >> 16;
                b0 += earlier ? c[j] & 0xFFFFu : 0u;
                b1 += earlier ? c[j] >> 16 : 0u;
            }
        }
        atomicAdd(&total[e], a0);  // whole numbers: any order
        atomicAdd(&before[e], b0);
        if (e + 1 < g.E) {  // an odd number's last half holds nothing
            atomicAdd(&total[e + 1], a1);
            atomicAdd(&before[e + 1], b1);
        }
    }
    __syncthreads();
    route_offsets(total, sums, g.E, part);
    for (int i = tid; i < g.E; i += kRouteThreads) before[i] += sums[i];
    if (mine == 0)
        for (int i = tid; i <= g.E; i += kRouteThreads) g.offsets[i] = sums[i];
    __syncthreads();
    for (int64_t i = own; i < t1 * g.top; i += kRouteThreads) {
        if (i != own) {
            expert = g.experts[i];
            rank = g.places[i];
        }
        if (expert < 0) continue;  // its place is -1 already
        const int at = before[expert] + rank;
        g.places[i] = at;
        g.rows[at] = (int32_t)(i / g.top);
    }
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
// One wave to a token: 8192 x 256 fp32 9.5 us (1.8 TB/s), a row's loads, exponentials and
// two sums over the wave one after another.
struct RouteGradArgs {
    const void *logits;
    const float *dweights;   // [T][top]
    const int32_t *experts;  // [T][top]
    void *dlogits;           // [T][E], dense
    int64_t ldl;
    int32_t T, E, top, sigmoid, renormalise;
    float scale;
};

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
    // lane k's expert, weight's gradient and logit are on their way beside the row
    int e = -1;
    float d = 0.f, own = none;
    if (lane < g.top) {
        e = g.experts[t * g.top + lane];
        d = g.dweights[t * g.top + lane];
    }
    route_row<IN, V>(g.logits, t * g.ldl + lane * V, g.E - lane * V, p);
    if (e < 0 || e >= g.E) e = -1;
    if (e >= 0) own = route_load<IN>(g.logits, t * g.ldl + e);
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (!g.sigmoid) most = p[i] > most || p[i] != p[i] ? p[i] : most;
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
    // lane k: expert k's p, and its weight's gradient times the scale
    float q = 0.f;
    if (e >= 0) {
        q = g.sigmoid ? sigmoid(own) : own == none ? 0.f : expf(own - most) / total;
        d *= g.scale;
    } else {
        d = 0.f;
    }
    if (g.renormalise) {
        float S = q, mean = d * q;
        for (int i = 1; i < g.top; i *= 2) {  // the lanes past the last expert hold 0
            S += __shfl_xor(S, i);
            mean += __shfl_xor(mean, i);
        }
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
    const int left = g.E - lane * V;
    typename std::conditional<IN == OUT_F32, float, uint16_t>::type out[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float x = slope[i] * (dp[i] - mean);
        if constexpr (IN == OUT_F32) out[i] = x;
        else out[i] = (uint16_t)(mx_pack2<IN>(x, 0.f) & 0xFFFFu);
    }
    auto *to = static_cast<decltype(&out[0])>(g.dlogits) + t * g.E + lane * V;
    if (left >= V) {
        __builtin_memcpy(to, out, sizeof(out));  // global memory takes any alignment
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (i < left) to[i] = out[i];
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
    for (int j = 0; j < 8; ++j) v[j] = f8_element<IN>(w, j);
}
template <int OUT, bool NT>
__device__ __forceinline__ void route_store8(void *y, int64_t at, int n, int N, const float (&v)[8])
{
    if (n + 8 > N) {
        mx_store4<OUT>(y, at, n, N, v[0], v[1], v[2], v[3]);
        mx_store4<OUT>(y, at, n + 4, N, v[4], v[5], v[6], v[7]);
    } else if (OUT == OUT_F32) {
        float *p = static_cast<float *>(y) + at + n;
#pragma unroll
        for (int i = 0; i < 8; i += 4)
            mx_store16<NT>(p + i, u32x4{__float_as_uint(v[i]), __float_as_uint(v[i + 1]), __float_as_uint(v[i + 2]), __float_as_uint(v[i + 3])});
    } else {
        mx_store16<NT>(static_cast<uint16_t *>(y) + at + n,
                       u32x4{mx_pack2<OUT>(v[0], v[1]), mx_pack2<OUT>(v[2], v[3]), mx_pack2<OUT>(v[4], v[5]), mx_pack2<OUT>(v[6], v[7])});
    }
}

// A workgroup takes J pieces of 2048 values of a row.  NT: rows that no cache will keep
// pass by them.  8192 tokens of 4 rows of 4096 bf16 59 us (5.7 TB/s); 16 of 4 2.8.
template <int IN, int OUT, int J, bool NT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs g)
{
    const int64_t t = blockIdx.x / g.pieces;
    const int n0 = (int)(blockIdx.x % g.pieces) * (2048 * J) + 8 * (int)threadIdx.x;
    float sum[J][8];
#pragma unroll
    for (int q = 0; q < J; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[q][i] = 0.f;
    for (int k0 = 0; k0 < g.top; k0 += 4) {
        float w[4];
        int at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = k0 + j;
            at[j] = k < g.top ? g.places[t * g.top + k] : -1;
            w[j] = k < g.top && g.weights != nullptr ? g.weights[t * g.top + k] : 1.f;
            if (at[j] >= g.R) at[j] = -1;
        }
        u32x4 v[J][4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < J; ++q)
                if (at[j] >= 0) mx_load8<IN, NT>(g.y, (int64_t)at[j] * g.N + n0 + 2048 * q, g.N - n0 - 2048 * q, v[q][j]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (at[j] >= 0)
#pragma unroll
                for (int q = 0; q < J; ++q)
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum[q][i] = __builtin_fmaf(w[j], f8_element<IN>(v[q][j], i), sum[q][i]);
    }
#pragma unroll
    for (int q = 0; q < J; ++q) {
        const int n = n0 + 2048 * q;
        if (g.residual != nullptr) {
            u32x4 v[2];
            mx_load8<OUT, false>(g.residual, t * g.N + n, g.N - n, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[q][i] += f8_element<OUT>(v, i);
        }
        route_store8<OUT, false>(g.out, t * g.N, n, g.N, sum[q]);
    }
}

// dy[places[t][k]] = weights[t][k] dout[t];  dweights[t][k] = <dout[t], y[places[t][k]]>.
// A workgroup takes a token; binary32 sums in a fixed order.  NT as above.  Bound by memory:
// 8192 tokens of 4 rows of 4096 bf16 116 us (5.2 TB/s).  One row at a time: with four rows'
// loads ahead, and the registers for them, 128 to 143.
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

template <int IN, int OUT, bool NT>
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
                u32x4 y[2];
                mx_load8<IN, NT>(g.y, (int64_t)at[j] * g.N + n, g.N - n, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] = __builtin_fmaf(d[i], f8_element<IN>(y, i), dot[j]);
                    v[i] = w[j] * d[i];
                }
                route_store8<IN, NT>(g.dy, (int64_t)at[j] * g.N, n, g.N, v);
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
