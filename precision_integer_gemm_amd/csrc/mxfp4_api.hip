// mxfp4_api.hip -- the microscaled 4-bit entry points of the C-ABI: argument
// checks, kernel selection and launches (contract in include/lpgemm.h).
#include "api_common.hpp"
#include "gemm_mxfp4.hpp"
#include "mxfp4_quantize.hpp"

using namespace lpgemm;

namespace {

// rows x K values to or from codes and scales.
lpgemm_status check_values(const void *x, const void *codes, const void *scales, int format, int64_t rows, int64_t K)
{
    if (format < 0 || rows < 0 || K < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_MXFP4_MAX_K || (K > 0 && rows > (INT64_MAX >> 8) / K)) return LPGEMM_ERR_UNSUPPORTED;
    if (rows == 0 || K == 0) return LPGEMM_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr || !aligned(x, element_bytes(format)) ||
        !aligned(codes, 16) || !aligned(scales, 4))
        return LPGEMM_ERR_INVALID_ARG;
    return LPGEMM_OK;
}

// Items of eight values; four a thread where that leaves four workgroups a
// compute unit, else one.
constexpr int64_t kManyItems = 4 * 256 * 4 * 256;
// Values of more bytes than this do not stay in the 256 MB last-level cache
// between a call and the next: they pass by it.  To codes and back, MI355X:
// 16384 x 8192 bf16 (268 MB) 140 us kept, 108 passed by; 3001 x 8191 fp16 (49
// MB, from the cache) 24.7 kept, 28.6 passed by.
// To codes alone, kept / passed by: 16384 x 8192 bf16 63.4 / 59.2, fp32 114 / 113;
// 8192 x 8192 fp32 56.8 / 56.9, 8192 x 8191 (rows at any address) 57.4 / 61.1.
constexpr int64_t kPastCaches = 192 << 20;

template <int IN>
lpgemm_status launch_quantize(const void *x, int64_t ldx, uint8_t *codes, uint8_t *scales, int64_t rows, int64_t K, hipStream_t stream)
{
    const int64_t items = ceil_div(K, kMxUnit) * (kMxUnit / 8), total = rows * items;
    const bool many = total >= kManyItems;
    const bool past = rows * K * (int64_t)element_bytes(IN) > kPastCaches;
    const auto kernel = past ? &mxfp4_quantize_kernel<IN, 4, true> : many ? &mxfp4_quantize_kernel<IN, 4, false> : &mxfp4_quantize_kernel<IN, 1, false>;
    return launch_rows(rows, items, many ? 1024 : 256, [&](int64_t first, int64_t count, dim3 blocks) {
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, static_cast<const uint8_t *>(x) + first * ldx * (int64_t)element_bytes(IN), ldx,
                           reinterpret_cast<uint32_t *>(codes) + first * items, scales + first * (items / 4), count, (int32_t)K, (uint32_t)items);
    });
}

template <int OUT>
lpgemm_status launch_dequantize(const uint8_t *codes, const uint8_t *scales, void *y, int64_t rows, int64_t K, hipStream_t stream)
{
    const int64_t items = ceil_div(K, kMxUnit) * (kMxUnit / 8), total = rows * items;
    const bool many = total >= kManyItems;
    // half as large 16-bit results too: they are written, so the cache has to put
    // them out.  fp32 results leave in two pieces, each half of every 32 bytes,
    // which the caches put together: 8192 x 8192 (268 MB) 75.8 us kept, 109 passed
    // by; in bf16 (134 MB) 31.0 kept, 25.2 passed by
    constexpr bool kMayPass = OUT != OUT_F32;
    const bool past = kMayPass && 2 * rows * K * (int64_t)element_bytes(OUT) > kPastCaches;
    const auto kernel = past ? &mxfp4_dequantize_kernel<OUT, 4, kMayPass> : many ? &mxfp4_dequantize_kernel<OUT, 4, false> : &mxfp4_dequantize_kernel<OUT, 1, false>;
    return launch_rows(rows, items, many ? 1024 : 256, [&](int64_t first, int64_t count, dim3 blocks) {
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, reinterpret_cast<const uint32_t *>(codes) + first * items,
                           scales + first * (items / 4), static_cast<uint8_t *>(y) + first * K * (int64_t)element_bytes(OUT), count, (int32_t)K,
                           (uint32_t)items);
    });
}

template <int HM, int FN, int STAGES, int KG, int OUT>
lpgemm_status launch_tiled(const MxArgs &g, int64_t blocks, hipStream_t stream)
{
    using T = MxTile<HM, FN, STAGES>;
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_mxfp4_tiled_kernel<HM, FN, STAGES, KG, OUT>;
    const lpgemm_status st = allow_lds(kernel, T::lds(LPGEMM_MXFP4_MAX_GROUPS, KG), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256 * KG), T::lds(g.E, KG), stream, g, (int)ceil_div(g.N, 64 * FN), kXcds);
    return launched();
}

template <int OUT>
lpgemm_status launch_large(const MxArgs &g, int64_t blocks, hipStream_t stream)
{
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_mxfp4_large_kernel<OUT>;
    const lpgemm_status st = allow_lds(kernel, MxLarge::lds(LPGEMM_MXFP4_MAX_GROUPS), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), MxLarge::lds(g.E), stream, g, (int)ceil_div(g.N, 256), kXcds);
    return launched();
}

// The narrow kernel's sizes: rows of a product (more only where the tiles are
// few), stages of a wave's registers of A, 32-bit offsets.
constexpr int kNarrowRows = 32, kNarrowMaxRows = 4096, kNarrowStages = 4;

bool narrow_serves(const MxArgs &g)
{
    if (g.offsets != nullptr)
        return g.R <= kMxNarrowRows && g.E <= kMxNarrowGroups && (int64_t)g.T * g.U * kMxUnitCodes <= INT32_MAX &&
               ceil_div(g.N, 16) * (g.R + g.E) <= INT32_MAX / 16;
    return g.R <= kNarrowMaxRows && g.U <= 4 * kMxNarrowWaves * kNarrowStages && g.N <= INT32_MAX / 32;
}

// How the narrow kernel would run: waves to a strip, stages of each, time in
// us; workgroups, and row tiles of the grid.
struct NarrowPlan {
    int kw, stages;
    double time;
    int64_t blocks, tiles;
};
// A strip costs its stages and 1.2 more for its sums and what leads to it, so
// fewer waves for many strips, more where a wave has one.  MI355X, 24 groups of
// 4096 x 4096: 59.8 us with 8 waves, 45.7 with 4, 37.0 with 2; 16 x 28672 x
// 8192: 26.4 us with 8, 24.0 with 4.
NarrowPlan plan_narrow(const MxArgs &g, int64_t cu)
{
    const bool grouped = g.offsets != nullptr;
    const int64_t strips = ceil_div(g.N, 16) * (grouped ? std::min(g.E, g.R) : 1);
    const int64_t per_tile = grouped ? cu : std::max<int64_t>(1, cu / ceil_div(g.R, g.R <= 16 ? 16 : 32));  // workgroups
    NarrowPlan best{kMxNarrowWaves, 1, 0, 0, 0};
    for (int w = kMxNarrowWaves; w > 0; w /= 2) {
        int64_t s = std::max<int64_t>(1, ceil_div(g.U, 4 * w));
        if (!grouped && s > kNarrowStages) continue;
        if (!grouped && s == 3) s = 4;  // registers for 1, 2 or 4
        const double t = 1.35 * (double)ceil_div(strips, per_tile * (kMxNarrowWaves / w)) * ((double)s + 1.2);
        if (best.time == 0 || t < best.time) best = {w, (int)s, t, 0, 0};
    }
    const int64_t items = ceil_div(g.N, 16) * (grouped ? ceil_div(g.R, 16) + std::min(g.E, g.R) : 1);
    best.tiles = grouped ? 1 : ceil_div(g.R, g.R <= 16 ? 16 : 32);
    best.blocks = std::min(ceil_div(items, kMxNarrowWaves / best.kw), std::max<int64_t>(1, cu / best.tiles));
    return best;
}

template <int FA, int S, bool GROUPED, int OUT>
lpgemm_status launch_narrow(const MxArgs &g, const NarrowPlan &p, hipStream_t stream)
{
    using C = MxNarrow<GROUPED>;
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_mxfp4_narrow_kernel<FA, S, GROUPED, OUT>;
    const lpgemm_status st = allow_lds(kernel, C::lds(kMxNarrowGroups), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks, (unsigned)p.tiles), dim3(64 * kMxNarrowWaves), C::lds(g.E), stream, g, p.kw, p.stages);
    return launched();
}

template <int OUT>
lpgemm_status launch_narrow_any(const MxArgs &g, const NarrowPlan &p, hipStream_t stream)
{
    if (g.offsets != nullptr) return launch_narrow<1, 1, true, OUT>(g, p, stream);
    if (g.R <= 16)
        return p.stages == 1   ? launch_narrow<1, 1, false, OUT>(g, p, stream)
               : p.stages == 2 ? launch_narrow<1, 2, false, OUT>(g, p, stream)
                               : launch_narrow<1, 4, false, OUT>(g, p, stream);
    return p.stages == 1   ? launch_narrow<2, 1, false, OUT>(g, p, stream)
           : p.stages == 2 ? launch_narrow<2, 2, false, OUT>(g, p, stream)
                           : launch_narrow<2, 4, false, OUT>(g, p, stream);
}

// The tiled kernels' shapes and what one of their tiles costs in time: us for
// a stage (256 k) at heights of 64, 128, 192 and 256 rows, and for a tile.  A
// compute unit draws about 60 GB/s of codes from beyond its XCD's L2 and 100
// from it, so small tiles pay for their copies and large ones, one to a
// compute unit, for a tile's beginning and end.  Fitted on MI355X; where they
// meet (us, 64 x 64 / 64 x 128 / 128 x 128 / 128 x 128 with four stages / 256 x 256):
//     1024 x 1024 x 4096     8.5 /  9.8 / 12.6 / 13.1 /  26
//     513 x 6086 x 384       9.2 /  6.3 /  6.7 /  7.4 /   -
//     199 x 8582 x 6277       23 /   22 /   23 /   19 /  40
//     2848 x 2880 x 3200      41 /   39 /   34 /   36 /  31
//     4096 x 4096 x 4096      88 /    - /   50 /    - /  41
// 64 x 64 with K in one / two halves: 1024 x 1024 x 4096 9.6 / 8.9, 2000 x 200
// x 4096 8.9 / 7.9, 333 x 1001 x 2897 7.5 / 7.5, 700 x 1400 x 2560 7.6 / 7.9.
struct Shape {
    int high, wide, stages;
    double stage[4], tile;
};
constexpr Shape kShapes[] = {{64, 64, 4, {0.25}, 1.2},
                             {64, 64, 4, {0.21}, 1.7},  // K in two halves side by side
                             {64, 128, 2, {0.42}, 1.1},
                             {128, 128, 2, {0.45, 0.70}, 1.5},
                             {128, 128, 4, {0.50, 0.62}, 2.0},
                             {256, 256, 2, {0.80, 1.10, 1.45, 1.75}, 9.0}};
constexpr int kSplitUnits = 8;  // two pairs of stages for each half
// A ring of two stages hides a copy's way only behind a second workgroup.
constexpr double kAlone = 1.6;
// And groups' matrices come from further away than a product's shared columns.
constexpr double kGrouped = 1.15;
enum { kShape64, kShape64Split, kShape64x128, kShape128, kShape128Deep, kShape256, kShapeCount };

// The shape that should take the least time for R rows in equal groups; *time in us.
int choose_shape(const MxArgs &g, int64_t cu, double *time)
{
    const int64_t groups = g.offsets ? std::min(g.E, g.R) : 1, rows = ceil_div(g.R, groups), stages = ceil_div(g.U, 2);
    int best = kShape64;
    double least = 0;
    for (int i = 0; i < kShapeCount; ++i) {
        const Shape &s = kShapes[i];
        if (i == kShape256 && g.U < MxLarge::kMinUnits) continue;
        const int64_t c = ceil_div(rows, s.high), blocks = ceil_div(ceil_div(rows, 64), c);  // tiles of a group, their height / 64
        const int64_t tiles = groups * c * ceil_div(g.N, s.wide);
        if ((i == kShape128Deep || i == kShape64Split) && tiles > cu) continue;  // one to a compute unit
        if (i == kShape64Split && g.U < kSplitUnits) continue;
        const bool two = i != kShape256 && s.stages == 2;
        const double per_stage = s.stage[blocks - 1] * (two && tiles <= cu ? kAlone : 1.0) * (two && g.offsets ? kGrouped : 1.0);
        const double t = (double)ceil_div(tiles, cu) * ((double)stages * per_stage + s.tile);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    *time = least;
    return best;
}

// Whether the narrow kernel takes a call that it can serve.  Few rows are its
// own (grouped: up to eight a group on average); beyond, it wins where the tiles
// are few and K long, as its waves split K (us, 64 x 64 tiles / narrow):
//     96 x 80 x 5753        10.4 /  6.0        200 x 300 x 8192     12.8 /  8.9
//     100 x 100 x 16384     22.9 / 13.1        1000 x 64 x 16384    22.2 / 14.2
//     64 x 8192 x 8192      13.3 / 18.1        333 x 1001 x 2897     7.5 /  8.5
// Few rows, best tiles / narrow, weights from memory, as in use: 16 x 28672 x
// 8192 29.5 / 23.9, 16 x 12313 x 7906 15.4 / 14.4 (weights that the last-level
// cache holds: 16 x 28672 x 8192 21.2 / 23.0).  With 17 to 32 rows it wins where
// its strips fill their rounds, and loses up to 18% where they do not:
//     17 x 4096 x 4096       7.6 /  5.3        17 x 12313 x 7906    15.5 / 16.7
//     32 x 4096 x 4096       7.7 /  6.3        25 x 12313 x 7906    15.9 / 17.6
//     24 x 28672 x 8192     30.3 / 27.8        32 x 12313 x 7906    16.3 / 19.2
//     32 x 28672 x 8192     30.7 / 29.4        32 x 8192 x 8192     15.4 / 15.8
//     24 x 4096 x 14336     20.6 / 13.3        32 x 4096 x 14336    21.5 / 14.9
// (the estimates are of weights in the caches and do not tell these apart).
// Grouped, the host knows the groups' average alone.  32 groups of 4096 x 4096,
// best tiles / narrow by rows a group, shared out evenly, by chance (the largest
// has 6, 22, 55, 69, 107 rows), and all rows in one group:
//     1    53.8 / 44.4     25.2 / 23.3      9.8 / 12.8
//     4    54.9 / 45.6     42.6 / 35.0     13.0 / 11.3
//     8    54.7 / 49.6     43.0 / 46.9     13.6 / 23.3
//     12   56.1 / 53.9     44.0 / 60.2     14.4 / 35.0
//     16   55.6 / 57.6     47.4 / 73.1     14.8 / 46.8
// 64 groups of 2048 x 4096 and 8 of 4096 x 4096 meet in the same places (8 rows:
// 55.3 / 50.1, 42.8 / 49.0, 13.6 / 23.5; 16.7 / 15.1, 14.6 / 14.5, 10.9 / 12.8).
bool narrow_pays(const MxArgs &g, int64_t cu, double tiled)
{
    if (g.offsets != nullptr) return g.R <= 8 * (int64_t)g.E;
    return g.R <= kNarrowRows || plan_narrow(g, cu).time + 0.5 < tiled;
}

// What runs a product: the narrow kernel, or a shape of the tiled ones on so
// many workgroups of so many threads.
struct MxPlan {
    int shape;  // kShapeCount: narrow
    NarrowPlan narrow;
    int64_t blocks;
    int threads;
};

lpgemm_status plan_shape(const MxArgs &g, int shape, int64_t cu, MxPlan *p)
{
    const Shape &s = kShapes[shape];
    const int64_t tiles_n = ceil_div(g.N, s.wide);
    // 32-bit tile counts; at most one ragged row tile a group more than the rows fill
    if (ceil_div(g.R, s.high) + g.E > INT32_MAX / tiles_n) return LPGEMM_ERR_UNSUPPORTED;
    const int64_t most = (ceil_div(g.R, s.high) + (g.offsets ? std::min(g.E, g.R) : 0)) * tiles_n;
    const int lds = shape == kShape64         ? MxTile<1, 1, 4>::lds(g.E, 1)
                    : shape == kShape64Split  ? MxTile<1, 1, 4>::lds(g.E, 2)
                    : shape == kShape64x128   ? MxTile<1, 2, 2>::lds(g.E, 1)
                    : shape == kShape128      ? MxTile<2, 2, 2>::lds(g.E, 1)
                    : shape == kShape128Deep  ? MxTile<2, 2, 4>::lds(g.E, 1)
                                              : MxLarge::lds(g.E);
    *p = MxPlan{shape, {}, std::min(most, (lds > 80 * 1024 ? 1 : 2) * cu), shape == kShape64Split ? 512 : 256};
    return LPGEMM_OK;
}

lpgemm_status plan_product(const MxArgs &g, int64_t cu, int forced, MxPlan *p)
{
    const auto narrow = [&] {
        const NarrowPlan n = plan_narrow(g, cu);
        *p = MxPlan{kShapeCount, n, n.blocks * n.tiles, 64 * kMxNarrowWaves};
        return LPGEMM_OK;
    };
    if (forced == LPGEMM_KERNEL_AUTO || forced == LPGEMM_KERNEL_TILED) {
        double time = 0;
        const int shape = choose_shape(g, cu, &time);
        if (forced == LPGEMM_KERNEL_AUTO && narrow_serves(g) && narrow_pays(g, cu, time)) return narrow();
        return plan_shape(g, shape, cu, p);
    }
    switch (forced) {
    case LPGEMM_KERNEL_TILED_64: return plan_shape(g, g.R * (int64_t)g.N > 64 * 64 * cu || g.U < kSplitUnits ? kShape64 : kShape64Split, cu, p);
    case LPGEMM_KERNEL_TILED_128: return plan_shape(g, g.R * (int64_t)g.N > 128 * 128 * cu ? kShape128 : kShape128Deep, cu, p);
    case LPGEMM_KERNEL_TILED_256: return plan_shape(g, g.U < MxLarge::kMinUnits ? kShape128 : kShape256, cu, p);
    case LPGEMM_KERNEL_SKINNY: return narrow_serves(g) ? narrow() : LPGEMM_ERR_UNSUPPORTED;
    default: return LPGEMM_ERR_UNSUPPORTED;
    }
}

template <int OUT>
lpgemm_status launch_product(const MxArgs &g, hipStream_t stream)
{
    MxPlan p;
    const lpgemm_status st = plan_product(g, compute_units(), forced_kernel(), &p);
    if (st != LPGEMM_OK) return st;
    switch (p.shape) {
    case kShape64: return launch_tiled<1, 1, 4, 1, OUT>(g, p.blocks, stream);
    case kShape64Split: return launch_tiled<1, 1, 4, 2, OUT>(g, p.blocks, stream);
    case kShape64x128: return launch_tiled<1, 2, 2, 1, OUT>(g, p.blocks, stream);
    case kShape128: return launch_tiled<2, 2, 2, 1, OUT>(g, p.blocks, stream);
    case kShape128Deep: return launch_tiled<2, 2, 4, 1, OUT>(g, p.blocks, stream);
    case kShape256: return launch_large<OUT>(g, p.blocks, stream);
    default: return launch_narrow_any<OUT>(g, p.narrow, stream);
    }
}

// Sizes and pointers that both products share; R rows of D.
lpgemm_status check_product(const void *A, const void *SFA, const void *B, const void *SFB, const void *D, int format,
                            int64_t T, int64_t R, int64_t N, int64_t K, int64_t E)
{
    if (format < 0 || T < 0 || R < 0 || N < 0 || K < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_MXFP4_MAX_K || T > LPGEMM_MXFP4_MAX_ROWS || R > LPGEMM_MXFP4_MAX_ROWS || N > LPGEMM_MXFP4_MAX_ROWS)
        return LPGEMM_ERR_UNSUPPORTED;
    if (R == 0 || N == 0) return LPGEMM_OK;
    if (D == nullptr || !aligned(D, 16)) return LPGEMM_ERR_INVALID_ARG;
    if (K > 0 && ((T > 0 && (A == nullptr || SFA == nullptr)) || (E > 0 && (B == nullptr || SFB == nullptr)) ||
                  !aligned(A, 16) || !aligned(B, 16) || !aligned(SFA, 4) || !aligned(SFB, 4)))
        return LPGEMM_ERR_INVALID_ARG;
    return LPGEMM_OK;
}

lpgemm_status run_product(const MxArgs &g, int format, hipStream_t stream)
{
    (void)hipGetLastError();
    switch (format) {
    case OUT_F32: return launch_product<OUT_F32>(g, stream);
    case OUT_BF16: return launch_product<OUT_BF16>(g, stream);
    default: return launch_product<OUT_F16>(g, stream);
    }
}

}  // namespace

extern "C" {

lpgemm_status lpgemm_mxfp4_quantize(const void *X, lpgemm_out_dtype x_dtype, int64_t ldx, uint8_t *codes,
                                    uint8_t *scales, int64_t rows, int64_t K, hipStream_t stream)
{
    const int f = format_of(x_dtype);
    const lpgemm_status st = check_values(X, codes, scales, f, rows, K);
    if (st != LPGEMM_OK || rows == 0 || K == 0) return st;
    if (ldx < (rows > 1 ? K : 0) || (rows > 1 && ldx > (INT64_MAX >> 4) / rows)) return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    switch (f) {
    case OUT_F32: return launch_quantize<OUT_F32>(X, ldx, codes, scales, rows, K, stream);
    case OUT_BF16: return launch_quantize<OUT_BF16>(X, ldx, codes, scales, rows, K, stream);
    default: return launch_quantize<OUT_F16>(X, ldx, codes, scales, rows, K, stream);
    }
}

lpgemm_status lpgemm_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, void *Y, lpgemm_out_dtype y_dtype,
                                      int64_t rows, int64_t K, hipStream_t stream)
{
    const int f = format_of(y_dtype);
    const lpgemm_status st = check_values(Y, codes, scales, f, rows, K);
    if (st != LPGEMM_OK || rows == 0 || K == 0) return st;
    (void)hipGetLastError();
    switch (f) {
    case OUT_F32: return launch_dequantize<OUT_F32>(codes, scales, Y, rows, K, stream);
    case OUT_BF16: return launch_dequantize<OUT_BF16>(codes, scales, Y, rows, K, stream);
    default: return launch_dequantize<OUT_F16>(codes, scales, Y, rows, K, stream);
    }
}

lpgemm_status lpgemm_mxfp4(const uint8_t *A, const uint8_t *SFA, const uint8_t *B, const uint8_t *SFB, void *D,
                           lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K, void *workspace,
                           size_t workspace_bytes, hipStream_t stream)
{
    const int f = format_of(out_dtype);
    const lpgemm_status st = check_product(A, SFA, B, SFB, D, f, M, M, N, K, 1);
    if (st != LPGEMM_OK) return st;
    if (workspace_bytes > 0 && (workspace == nullptr || !aligned(workspace, 256))) return LPGEMM_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return LPGEMM_OK;
    const MxArgs g{A, SFA, B, SFB, D, nullptr, nullptr, (int32_t)M, (int32_t)M, (int32_t)N, (int32_t)ceil_div(K, kMxUnit), 1};
    return run_product(g, f, stream);
}

lpgemm_status lpgemm_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K, int32_t cu_count, size_t *bytes)
{
    (void)cu_count;
    if (bytes == nullptr || M < 0 || N < 0 || K < 0) return LPGEMM_ERR_INVALID_ARG;
    *bytes = 0;
    if (K > LPGEMM_MXFP4_MAX_K || M > LPGEMM_MXFP4_MAX_ROWS || N > LPGEMM_MXFP4_MAX_ROWS) return LPGEMM_ERR_UNSUPPORTED;
    return LPGEMM_OK;
}

lpgemm_status lpgemm_mxfp4_plan(int64_t R, int64_t N, int64_t K, int64_t E, int32_t cu_count, lpgemm_plan_info *info)
{
    if (info == nullptr || R < 0 || N < 0 || K < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_MXFP4_MAX_K || R > LPGEMM_MXFP4_MAX_ROWS || N > LPGEMM_MXFP4_MAX_ROWS || E > LPGEMM_MXFP4_MAX_GROUPS)
        return LPGEMM_ERR_UNSUPPORTED;
    *info = lpgemm_plan_info{};
    if (R == 0 || N == 0) return LPGEMM_OK;
    static const int32_t some = 0;  // offsets are there or not, nobody reads them
    const MxArgs g{nullptr, nullptr, nullptr, nullptr, nullptr, E > 0 ? &some : nullptr, nullptr,
                   (int32_t)R, (int32_t)R, (int32_t)N, (int32_t)ceil_div(K, kMxUnit), (int32_t)std::max<int64_t>(E, 1)};
    MxPlan p;
    const lpgemm_status st = plan_product(g, cu_count > 0 ? cu_count : 256, forced_kernel(), &p);
    if (st != LPGEMM_OK) return st;
    const bool narrow = p.shape == kShapeCount;
    info->kernel = narrow ? LPGEMM_KERNEL_SKINNY : LPGEMM_KERNEL_TILED;
    info->tile_m = !narrow ? kShapes[p.shape].high : E > 0 || R <= 16 ? 16 : 32;
    info->tile_n = narrow ? 16 : kShapes[p.shape].wide;
    info->k_split = narrow ? p.narrow.kw : p.shape == kShape64Split ? 2 : 1;
    info->workgroups = p.blocks;
    info->threads = p.threads;
    info->k_chunks = 1;
    return LPGEMM_OK;
}

lpgemm_status lpgemm_mxfp4_grouped(const uint8_t *A, const uint8_t *SFA, int64_t T, const int32_t *rows,
                                   const uint8_t *B, const uint8_t *SFB, int64_t E, const int32_t *offsets, void *D,
                                   lpgemm_out_dtype out_dtype, int64_t R, int64_t N, int64_t K, hipStream_t stream)
{
    const int f = format_of(out_dtype);
    const lpgemm_status st = check_product(A, SFA, B, SFB, D, f, T, R, N, K, E);
    if (st != LPGEMM_OK) return st;
    if (rows == nullptr && T != R) return LPGEMM_ERR_INVALID_ARG;
    if (E > LPGEMM_MXFP4_MAX_GROUPS) return LPGEMM_ERR_UNSUPPORTED;
    const int64_t units = ceil_div(K, kMxUnit);
    if (rows != nullptr && T * units * kMxUnitCodes > INT32_MAX) return LPGEMM_ERR_UNSUPPORTED;
    if (R == 0 || N == 0 || E == 0) return LPGEMM_OK;
    if (offsets == nullptr || !aligned(offsets, 4) || !aligned(rows, 4)) return LPGEMM_ERR_INVALID_ARG;
    if (T == 0) {  // every row of D is of zeros; the kernels' dead reads of A need an address
        A = B;
        SFA = SFB;
    }
    const MxArgs g{A, SFA, B, SFB, D, offsets, rows, (int32_t)T, (int32_t)R, (int32_t)N, (int32_t)units, (int32_t)E};
    return run_product(g, f, stream);
}

}  // extern "C"
