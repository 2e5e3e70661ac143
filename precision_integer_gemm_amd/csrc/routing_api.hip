// routing_api.hip -- entry points of the experts' routing and of their sum:
// argument checks and launches (contract in include/lpgemm.h).
#include "api_common.hpp"
#include "routing.hpp"

using namespace lpgemm;

namespace {

// Tokens are dealt to this many workgroups (beyond 16 million, to more): every one of the
// second kernel adds up the counts of the others.
constexpr int64_t kMostWorkgroups = 256;

// How T tokens are dealt: tokens of a wave in a round, of a workgroup, workgroups.
struct RoutePlan {
    int per;
    int64_t stretch, blocks;
};
RoutePlan plan_route(int64_t T)
{
    int per = 1;
    while (kRouteWaves * per < kRouteRound && T > kRouteWaves * per * kMostWorkgroups) per *= 2;
    const int64_t round = (int64_t)kRouteWaves * per, rounds = ceil_div(ceil_div(T, round), kMostWorkgroups);
    const int64_t stretch = round * std::min<int64_t>(rounds, UINT16_MAX / round);  // counts of 16 bits
    return {per, stretch, ceil_div(T, stretch)};
}

// Rows of more bytes than this do not stay in the 256 MB last-level cache between a call
// and the next: the sum's loads pass by it, with two pieces of a long row to a workgroup
// (us, kept / past, bf16: 2048 tokens of 4 rows of 4096 16.4 / 17.3, 4096 34.1 / 31.3, 8192
// 78.7 / 59.1; of 2048, 4096 tokens of 8 27.6 / 29.4, 16384 of 4 79.3 / 63.1).  The
// gradients' loads and stores do from twice that on (4096 of 4 of 4096 57.9 / 61.4, 8192
// 131 / 116).
constexpr int64_t kPastCaches = 96 << 20;

size_t route_workspace(int64_t T, int64_t E)
{
    if (T == 0 || E == 0) return 0;
    const RoutePlan p = plan_route(T);
    return p.blocks > 1 ? (size_t)(p.blocks * route_pitch((int)E)) * sizeof(uint16_t) : 0;
}

lpgemm_status check_options(const lpgemm_route_options *o, int64_t T, int64_t E, int64_t ld)
{
    if (o == nullptr || T < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    if ((o->score != LPGEMM_ROUTE_SOFTMAX && o->score != LPGEMM_ROUTE_SIGMOID) || (o->renormalise != 0 && o->renormalise != 1) || o->top < 1 ||
        o->groups < 1 || o->top_groups < 1 || o->top_groups > o->groups || (o->group_top != 1 && o->group_top != 2))
        return LPGEMM_ERR_INVALID_ARG;
    if (E > LPGEMM_ROUTE_MAX_EXPERTS || o->top > LPGEMM_ROUTE_MAX_TOP || o->groups > LPGEMM_ROUTE_MAX_GROUPS || T > INT32_MAX / o->top)
        return LPGEMM_ERR_UNSUPPORTED;
    if (T == 0) return LPGEMM_OK;
    if (E < 1 || E % o->groups != 0 || o->top > E / o->groups * o->top_groups || (T > 1 && (ld < E || ld > (INT64_MAX >> 4) / T))) return LPGEMM_ERR_INVALID_ARG;
    return LPGEMM_OK;
}

template <int IN, int V, bool WIDE>
lpgemm_status launch_choose(const RouteArgs &g, const RoutePlan &p, hipStream_t stream)
{
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &route_choose_kernel<IN, V, WIDE>;
    const lpgemm_status st = allow_lds(kernel, route_lds(64 * V, LPGEMM_ROUTE_MAX_TOP, true), once, err);
    if (st != LPGEMM_OK) return st;
    const int lanes = g.per_group / V;
    const bool room = g.top_groups < g.groups && (lanes * V != g.per_group || (lanes & (lanes - 1)) != 0);
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks), dim3(kRouteThreads), route_lds(g.E, g.top, room), stream, g, p.per, p.blocks == 1 ? 1 : 0);
    return launched();
}

template <int IN, bool WIDE>
lpgemm_status launch_choose_any(const RouteArgs &g, const RoutePlan &p, hipStream_t stream)
{
    if (g.E <= 64) return launch_choose<IN, 1, WIDE>(g, p, stream);
    if (g.E <= 128) return launch_choose<IN, 2, WIDE>(g, p, stream);
    if (g.E <= 256) return launch_choose<IN, 4, WIDE>(g, p, stream);
    if (g.E <= 512) return launch_choose<IN, 8, WIDE>(g, p, stream);
    return launch_choose<IN, 16, WIDE>(g, p, stream);
}

template <int IN>
lpgemm_status launch_route(const RouteArgs &g, hipStream_t stream)
{
    const RoutePlan p = plan_route(g.T);
    const bool wide = g.bias != nullptr || (g.top_groups < g.groups && g.group_top > 1);
    lpgemm_status st = wide ? launch_choose_any<IN, true>(g, p, stream) : launch_choose_any<IN, false>(g, p, stream);
    if (st != LPGEMM_OK || p.blocks == 1) return st;
    hipLaunchKernelGGL(route_place_kernel, dim3((unsigned)p.blocks), dim3(kRouteThreads), 4 * (3 * g.E + 1 + kRouteWaves), stream, g);
    return launched();
}

template <int IN>
lpgemm_status launch_backward(const RouteGradArgs &g, hipStream_t stream)
{
    const auto kernel = g.E <= 64    ? &route_backward_kernel<IN, 1>
                        : g.E <= 128 ? &route_backward_kernel<IN, 2>
                        : g.E <= 256 ? &route_backward_kernel<IN, 4>
                        : g.E <= 512 ? &route_backward_kernel<IN, 8>
                                     : &route_backward_kernel<IN, 16>;
    return launch_rows(g.T, 1, 4, [&](int64_t first, int64_t count, dim3 blocks) {
        RouteGradArgs a = g;
        const int64_t w = (int64_t)element_bytes(IN);
        a.logits = static_cast<const uint8_t *>(g.logits) + first * g.ldl * w;
        a.dlogits = static_cast<uint8_t *>(g.dlogits) + first * g.E * w;
        a.dweights += first * g.top;
        a.experts += first * g.top;
        a.T = (int32_t)count;
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, a);
    });
}

template <int IN>
lpgemm_status launch_combine(CombineArgs g, int out, hipStream_t stream)
{
    const bool past = g.R * g.N * (int64_t)element_bytes(IN) > kPastCaches, two = past && g.N > 2048;
    const auto pick = [&](auto type) {
        constexpr int OUT = decltype(type)::value;
        return two ? &combine_kernel<IN, OUT, 2, true> : past ? &combine_kernel<IN, OUT, 1, true> : &combine_kernel<IN, OUT, 1, false>;
    };
    const auto kernel = out == OUT_F32    ? pick(std::integral_constant<int, OUT_F32>{})
                        : out == OUT_BF16 ? pick(std::integral_constant<int, OUT_BF16>{})
                                          : pick(std::integral_constant<int, OUT_F16>{});
    g.pieces = (int32_t)ceil_div(g.N, two ? 4096 : 2048);
    return launch_rows(g.T, g.pieces, 1, [&](int64_t first, int64_t, dim3 blocks) {
        CombineArgs a = g;
        const int64_t w = out == OUT_F32 ? 4 : 2;
        a.places += first * g.top;
        if (a.weights != nullptr) a.weights += first * g.top;
        if (a.residual != nullptr) a.residual = static_cast<const uint8_t *>(g.residual) + first * g.N * w;
        a.out = static_cast<uint8_t *>(g.out) + first * g.N * w;
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, a);
    });
}

template <int IN>
lpgemm_status launch_combine_backward(const CombineGradArgs &g, int out, hipStream_t stream)
{
    const bool past = g.R * g.N * (int64_t)element_bytes(IN) > 2 * kPastCaches;
    const auto pick = [&](auto type) {
        constexpr int OUT = decltype(type)::value;
        return past ? &combine_backward_kernel<IN, OUT, true> : &combine_backward_kernel<IN, OUT, false>;
    };
    const auto kernel = out == OUT_F32    ? pick(std::integral_constant<int, OUT_F32>{})
                        : out == OUT_BF16 ? pick(std::integral_constant<int, OUT_BF16>{})
                                          : pick(std::integral_constant<int, OUT_F16>{});
    return launch_rows(g.T, 1, 1, [&](int64_t first, int64_t, dim3 blocks) {
        CombineGradArgs a = g;
        a.dout = static_cast<const uint8_t *>(g.dout) + first * g.N * (out == OUT_F32 ? 4 : 2);
        a.places += first * g.top;
        if (a.weights != nullptr) a.weights += first * g.top;
        a.dweights += first * g.top;
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, a);
    });
}

// Sizes that both directions of the sum share.
lpgemm_status check_combine(int64_t R, int64_t T, int64_t top, int64_t N)
{
    if (R < 0 || T < 0 || top < 0 || N < 0) return LPGEMM_ERR_INVALID_ARG;
    if (R > INT32_MAX || N > LPGEMM_COMBINE_MAX_N || top > LPGEMM_COMBINE_MAX_TOP || T > INT32_MAX / std::max<int64_t>(1, top)) return LPGEMM_ERR_UNSUPPORTED;
    return LPGEMM_OK;
}

}  // namespace

extern "C" {

lpgemm_status lpgemm_route_workspace_size(int64_t T, int64_t E, size_t *bytes)
{
    if (bytes == nullptr || T < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (T > INT32_MAX || E > LPGEMM_ROUTE_MAX_EXPERTS) return LPGEMM_ERR_UNSUPPORTED;
    *bytes = route_workspace(T, E);
    return LPGEMM_OK;
}

lpgemm_status lpgemm_route(const void *logits, lpgemm_out_dtype dtype, int64_t ldl, const float *bias, const lpgemm_route_options *options, int32_t *experts,
                           float *weights, int32_t *rows, int32_t *offsets, int32_t *places, int64_t T, int64_t E, void *workspace, size_t workspace_bytes,
                           hipStream_t stream)
{
    const int f = format_of(dtype);
    if (f < 0) return LPGEMM_ERR_INVALID_ARG;
    const lpgemm_status st = check_options(options, T, E, ldl);
    if (st != LPGEMM_OK) return st;
    if (offsets == nullptr || !aligned(offsets, 4)) return LPGEMM_ERR_INVALID_ARG;
    if (T > 0 && (logits == nullptr || experts == nullptr || weights == nullptr || rows == nullptr || places == nullptr ||
                  !aligned(logits, element_bytes(f)) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(rows, 4) || !aligned(places, 4) || !aligned(bias, 4)))
        return LPGEMM_ERR_INVALID_ARG;
    const size_t need = route_workspace(T, E);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 4))) return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    const lpgemm_route_options &o = *options;
    const RouteArgs g{logits, bias, experts, weights, rows, offsets, places, static_cast<uint16_t *>(workspace), ldl, (int32_t)T, (int32_t)E, o.top, o.groups,
                      o.top_groups, o.group_top, (int32_t)std::max<int64_t>(1, E / o.groups), (int32_t)(T > 0 ? plan_route(T).stretch : 0),
                      o.score == LPGEMM_ROUTE_SIGMOID, o.renormalise, o.scale};
    if (T == 0) {
        hipLaunchKernelGGL(route_empty_kernel, dim3(1), dim3(256), 0, stream, offsets, (int32_t)E);
        return launched();
    }
    switch (f) {
    case OUT_F32: return launch_route<OUT_F32>(g, stream);
    case OUT_BF16: return launch_route<OUT_BF16>(g, stream);
    default: return launch_route<OUT_F16>(g, stream);
    }
}

lpgemm_status lpgemm_route_backward(const float *dweights, const void *logits, lpgemm_out_dtype dtype, int64_t ldl, const int32_t *experts,
                                    const lpgemm_route_options *options, void *dlogits, int64_t T, int64_t E, hipStream_t stream)
{
    const int f = format_of(dtype);
    if (f < 0) return LPGEMM_ERR_INVALID_ARG;
    const lpgemm_status st = check_options(options, T, E, ldl);
    if (st != LPGEMM_OK || T == 0) return st;
    if (dweights == nullptr || logits == nullptr || experts == nullptr || dlogits == nullptr || !aligned(dweights, 4) || !aligned(experts, 4) ||
        !aligned(logits, element_bytes(f)) || !aligned(dlogits, element_bytes(f)))
        return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    const lpgemm_route_options &o = *options;
    const RouteGradArgs g{logits, dweights, experts, dlogits, ldl, (int32_t)T, (int32_t)E, o.top, o.score == LPGEMM_ROUTE_SIGMOID, o.renormalise, o.scale};
    switch (f) {
    case OUT_F32: return launch_backward<OUT_F32>(g, stream);
    case OUT_BF16: return launch_backward<OUT_BF16>(g, stream);
    default: return launch_backward<OUT_F16>(g, stream);
    }
}

lpgemm_status lpgemm_combine(const void *Y, lpgemm_out_dtype y_dtype, int64_t R, const int32_t *places, const float *weights, const void *residual, void *out,
                             lpgemm_out_dtype out_dtype, int64_t T, int64_t top, int64_t N, hipStream_t stream)
{
    const int f = format_of(y_dtype), o = format_of(out_dtype);
    if (f < 0 || o < 0) return LPGEMM_ERR_INVALID_ARG;
    const lpgemm_status st = check_combine(R, T, top, N);
    if (st != LPGEMM_OK || T == 0 || N == 0) return st;
    if (out == nullptr || (R > 0 && top > 0 && Y == nullptr) || (top > 0 && places == nullptr) || !aligned(Y, element_bytes(f)) || !aligned(places, 4) ||
        !aligned(weights, 4) || !aligned(residual, element_bytes(o)) || !aligned(out, element_bytes(o)))
        return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    const CombineArgs g{Y, places, weights, residual, out, R, T, (int32_t)N, (int32_t)top, 1};
    switch (f) {
    case OUT_F32: return launch_combine<OUT_F32>(g, o, stream);
    case OUT_BF16: return launch_combine<OUT_BF16>(g, o, stream);
    default: return launch_combine<OUT_F16>(g, o, stream);
    }
}

lpgemm_status lpgemm_combine_backward(const void *dout, lpgemm_out_dtype out_dtype, const void *Y, lpgemm_out_dtype y_dtype, int64_t R, const int32_t *places,
                                      const float *weights, void *dY, float *dweights, int64_t T, int64_t top, int64_t N, hipStream_t stream)
{
    const int f = format_of(y_dtype), o = format_of(out_dtype);
    if (f < 0 || o < 0) return LPGEMM_ERR_INVALID_ARG;
    const lpgemm_status st = check_combine(R, T, top, N);
    if (st != LPGEMM_OK || T == 0 || top == 0) return st;
    if (places == nullptr || dweights == nullptr || (N > 0 && (dout == nullptr || (R > 0 && (Y == nullptr || dY == nullptr)))) || !aligned(Y, element_bytes(f)) ||
        !aligned(dY, element_bytes(f)) || !aligned(places, 4) || !aligned(weights, 4) || !aligned(dweights, 4) || !aligned(dout, element_bytes(o)))
        return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    const CombineGradArgs g{dout, Y, places, weights, dY, dweights, R, T, (int32_t)N, (int32_t)top};
    switch (f) {
    case OUT_F32: return launch_combine_backward<OUT_F32>(g, o, stream);
    case OUT_BF16: return launch_combine_backward<OUT_BF16>(g, o, stream);
    default: return launch_combine_backward<OUT_F16>(g, o, stream);
    }
}

}  // extern "C"
