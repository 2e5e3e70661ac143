// fp8_block_api.hip -- entry points of the e4m3 operators with a scale per block
// of 128: argument checks, kernel selection and launches (contract in
// include/lpgemm.h).
#include "api_common.hpp"
#include "gemm_fp8_block.hpp"

using namespace lpgemm;

namespace {

// 0 for a scale per row, 7 per 128 rows, -1 for anything else.
int shift_of(int64_t block_rows) { return block_rows == 1 ? 0 : block_rows == 128 ? 7 : -1; }

int64_t units_of(int64_t K) { return ceil_div(K, kF8Unit); }

// rows x K values to or from codes and scales.
lpgemm_status check_values(const void *x, const void *codes, const void *scales, int format, int shift, int64_t rows, int64_t K)
{
    if (format < 0 || shift < 0 || rows < 0 || K < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_FP8_BLOCK_MAX_K || (K > 0 && rows > (INT64_MAX >> 8) / K)) return LPGEMM_ERR_UNSUPPORTED;
    if (rows == 0 || K == 0) return LPGEMM_OK;
    if (x == nullptr || codes == nullptr || scales == nullptr || !aligned(x, element_bytes(format)) || !aligned(codes, 16) || !aligned(scales, 4))
        return LPGEMM_ERR_INVALID_ARG;
    return LPGEMM_OK;
}

// Codes back to values: from so many items on, four a thread, and values that pass by the
// caches (us, one kept / four past: 1001 x 2897 bf16 3.25 / 3.57, 1024 x 4096 bf16 3.65 /
// 3.21, 2048 x 4096 bf16 5.75 / 4.12, 8192 x 8192 fp32 67.9 / 48.5).
constexpr int64_t kManyItems = 2 * 256 * 4 * 256;
// Values of more bytes than this do not stay in the 256 MB last-level cache
// between a call and the next: to codes, they pass by it (us, kept / past: a scale per row,
// 4096 x 4096 fp32 13.3 / 16.0, 16384 x 8192 bf16 72.3 / 70.8; per 128 rows 14.2 / 16.8,
// 72.8 / 62.7, 8192 x 8192 fp32 59.4 / 57.3).
constexpr int64_t kPastCaches = 192 << 20;

template <int IN, bool POW2>
lpgemm_status launch_quantize(const void *x, int64_t ldx, uint8_t *codes, float *scales, int shift, int64_t rows, int64_t K, hipStream_t stream)
{
    const int64_t units = units_of(K), items = 16 * units, width = (int64_t)element_bytes(IN);
    const bool past = rows * K * width > kPastCaches;
    uint64_t *to = reinterpret_cast<uint64_t *>(codes);
    if (shift != 0) {
        const auto kernel = past ? &fp8_block_quantize_square_kernel<IN, true, POW2> : &fp8_block_quantize_square_kernel<IN, false, POW2>;
        return launch_rows(ceil_div(rows, 128), units, 1, [&](int64_t first, int64_t, dim3 blocks) {
            hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, static_cast<const uint8_t *>(x) + 128 * first * ldx * width, ldx, to + 128 * first * items,
                               scales + first * units, rows - 128 * first, (int32_t)K, (uint32_t)units);
        });
    }
    const auto kernel = past ? &fp8_block_quantize_kernel<IN, true, POW2> : &fp8_block_quantize_kernel<IN, false, POW2>;
    return launch_rows(rows, items, 256, [&](int64_t first, int64_t count, dim3 blocks) {
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, static_cast<const uint8_t *>(x) + first * ldx * width, ldx, to + first * items,
                           scales + first * units, count, (int32_t)K, (uint32_t)items);
    });
}

template <int IN>
lpgemm_status launch_quantize_any(const void *x, int64_t ldx, uint8_t *codes, float *scales, int shift, bool pow2, int64_t rows, int64_t K, hipStream_t stream)
{
    return pow2 ? launch_quantize<IN, true>(x, ldx, codes, scales, shift, rows, K, stream) : launch_quantize<IN, false>(x, ldx, codes, scales, shift, rows, K, stream);
}

template <int OUT>
lpgemm_status launch_dequantize(const uint8_t *codes, const float *scales, int shift, void *y, int64_t rows, int64_t K, hipStream_t stream)
{
    const int64_t items = units_of(K) * (kF8Unit / f8_item<OUT>()), width = (int64_t)element_bytes(OUT);
    const bool many = rows * items >= kManyItems;
    const auto kernel = many ? &fp8_block_dequantize_kernel<OUT, 4, true> : &fp8_block_dequantize_kernel<OUT, 1, false>;
    return launch_rows(rows, items, many ? 1024 : 256, [&](int64_t first, int64_t count, dim3 blocks) {
        hipLaunchKernelGGL(kernel, blocks, dim3(256), 0, stream, reinterpret_cast<const uint32_t *>(codes + first * items * f8_item<OUT>()), scales,
                           static_cast<uint8_t *>(y) + first * K * width, first, count, (int32_t)K, (uint32_t)items, shift);
    });
}

template <int HM, int FN, int STAGES, int KG, bool ROWS, int OUT>
lpgemm_status launch_tiled(const F8Args &g, int64_t blocks, hipStream_t stream)
{
    using T = F8Tile<HM, FN, STAGES>;
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_fp8_block_tiled_kernel<HM, FN, STAGES, KG, ROWS, OUT>;
    const lpgemm_status st = allow_lds(kernel, T::lds(LPGEMM_FP8_BLOCK_MAX_GROUPS, KG), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256 * KG), T::lds(g.E, KG), stream, g, (int)ceil_div(g.N, 64 * FN), kXcds);
    return launched();
}

template <int OUT>
lpgemm_status launch_large(const F8Args &g, int64_t blocks, hipStream_t stream)
{
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_fp8_block_large_kernel<OUT>;
    const lpgemm_status st = allow_lds(kernel, F8Large::lds(LPGEMM_FP8_BLOCK_MAX_GROUPS), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(512), F8Large::lds(g.E), stream, g, (int)ceil_div(g.N, 256), kXcds);
    return launched();
}

// ---- the narrow kernel --------------------------------------------------------
// Sizes it takes: rows of a product, stages of a wave's registers of A for up to 16 rows
// and for more (beyond them A comes through the ring, as it does for groups), 32-bit
// offsets.  Four stages of 32 rows would not fit the registers.
constexpr int kNarrowMaxRows = 4096;
int narrow_stages(int64_t rows) { return rows <= 16 ? 4 : 2; }
int64_t narrow_units(int64_t rows) { return kF8NarrowUnits * kMxNarrowWaves * narrow_stages(rows); }

bool narrow_serves(const F8Args &g)
{
    if (g.offsets != nullptr)
        return g.R <= kMxNarrowRows && g.E <= kMxNarrowGroups && (int64_t)g.T * g.U * kF8UnitCodes <= INT32_MAX &&
               ceil_div(g.N, 16) * (g.R + g.E) <= INT32_MAX / 16;
    return g.R <= kNarrowMaxRows && g.N <= INT32_MAX / 32 && ceil_div(g.N, 16) * ceil_div(g.R, 16) <= INT32_MAX / 16;
}

// How it would run: waves to a strip, stages of each, time in us; workgroups,
// row tiles of the grid, and whether A comes through the ring.
struct NarrowPlan {
    int kw, stages;
    double time;
    int64_t blocks, tiles;
    bool ring;
};

NarrowPlan plan_narrow(const F8Args &g, int64_t cu)
{
    const bool grouped = g.offsets != nullptr, ring = grouped || g.U > narrow_units(g.R);
    const int64_t row_tiles = ceil_div(g.R, g.R <= 16 ? 16 : 32);
    const int64_t strips = ceil_div(g.N, 16) * (grouped ? std::min(g.E, g.R) : ring ? ceil_div(g.R, 16) : 1);
    const int64_t per_tile = ring ? cu : std::max<int64_t>(1, cu / row_tiles);  // workgroups
    NarrowPlan best{kMxNarrowWaves, 1, 0, 0, 0, ring};
    for (int w = kMxNarrowWaves; w > 0; w /= 2) {
        int64_t s = std::max<int64_t>(1, ceil_div(g.U, kF8NarrowUnits * w));
        if (!ring && s > narrow_stages(g.R)) continue;
        if (!ring && s == 3) s = 4;  // registers for 1, 2 or 4
        const double t = 1.35 * (double)ceil_div(strips, per_tile * (kMxNarrowWaves / w)) * ((double)s + 1.2);
        if (best.time == 0 || t < best.time) best = {w, (int)s, t, 0, 0, ring};
    }
    const int64_t items = ceil_div(g.N, 16) * (grouped ? ceil_div(g.R, 16) + std::min(g.E, g.R) : ring ? ceil_div(g.R, 16) : 1);
    best.tiles = ring ? 1 : row_tiles;
    best.blocks = std::min(ceil_div(items, kMxNarrowWaves / best.kw), std::max<int64_t>(1, cu / best.tiles));
    return best;
}

template <int FA, int S, bool RING, int OUT>
lpgemm_status launch_narrow(const F8Args &g, const NarrowPlan &p, hipStream_t stream)
{
    using C = F8Narrow<RING>;
    static std::once_flag once[kMaxDevices];
    static hipError_t err[kMaxDevices];
    const auto kernel = &gemm_fp8_block_narrow_kernel<FA, S, RING, OUT>;
    const lpgemm_status st = allow_lds(kernel, C::lds(kMxNarrowGroups), once, err);
    if (st != LPGEMM_OK) return st;
    hipLaunchKernelGGL(kernel, dim3((unsigned)p.blocks, (unsigned)p.tiles), dim3(64 * kMxNarrowWaves), C::lds(g.E), stream, g, p.kw, p.stages);
    return launched();
}

template <int OUT>
lpgemm_status launch_narrow_any(const F8Args &g, const NarrowPlan &p, hipStream_t stream)
{
    if (p.ring) return launch_narrow<1, 1, true, OUT>(g, p, stream);
    if (g.R <= 16)
        return p.stages == 1   ? launch_narrow<1, 1, false, OUT>(g, p, stream)
               : p.stages == 2 ? launch_narrow<1, 2, false, OUT>(g, p, stream)
                               : launch_narrow<1, 4, false, OUT>(g, p, stream);
    return p.stages == 1 ? launch_narrow<2, 1, false, OUT>(g, p, stream) : launch_narrow<2, 2, false, OUT>(g, p, stream);
}

// ---- the choice ---------------------------------------------------------------
// The tiled kernels' shapes and what one of their tiles costs: us for a stage at heights
// of 64, 128, 192 and 256 rows with every compute unit busy, where tiles are fewer than
// those, and for a tile.  Fitted on MI355X; where they meet (us, bf16, 64 x 64 / 128 x 128
// / 256 x 256):
//     1024 x 1024 x 4096   12.8 / 23.5 / 42.4     2048 x 4096 x 4096   66.5 / 40.6 / 44.7
//     512 x 4096 x 4096    20.3 / 23.8 / 42.7     2848 x 2880 x 3200   53.9 / 48.5 / 39.0
//     1024 x 4096 x 4096   35.9 / 25.6 / 43.3     4096 x 4096 x 4096      - / 77.9 / 61.4
//     200 x 8582 x 6277    36.4 / 34.0 / 64.0     513 x 6086 x 384     10.2 /  8.1 /    -
// 32 groups of 4096 x 4096, rows shared out by chance:
//     1024 rows  111 / 121 / 129    4096 rows  223 / 157 / 142    16384 rows  646 / 403 / 296
// Binary32 results convert codes on the vector ALU and have costs of their own (64 x 64 /
// 128 x 128):
//     512 x 2048 x 4096    15.7 / 37.3    1500 x 1500 x 1500   17.7 / 19.6
//     1024 x 2048 x 512     7.8 / 10.9    2048 x 2048 x 256    12.2 / 10.7
//     2048 x 2048 x 2048   28.3 / 24.4    1024 x 4096 x 4096   49.9 / 41.6
//     513 x 6086 x 384     13.4 / 12.0    4096 x 4096 x 4096    193 / 156
// and 256 x 4096 x 4096, 64 x 64 whole / in two halves: 18.7 / 16.4, bf16 14.0 / 12.4.
struct Shape {
    int high, wide, lds;
    double stage[4], few, tile;
};
enum { kShape64, kShape64Split, kShape128, kShape128Deep, kShape256, kShapeCount };
Shape shape_of(int shape, int groups, int format)
{
    const bool f32 = format == OUT_F32;
    switch (shape) {
    case kShape64: return {64, 64, F8Tile<1, 1, 4>::lds(groups, 1), {f32 ? 0.36 : 0.26}, f32 ? 0.38 : 0.34, 1.5};
    case kShape64Split: return {64, 64, F8Tile<1, 1, 4>::lds(groups, 2), {f32 ? 0.30 : 0.22}, f32 ? 0.30 : 0.26, 2.5};
    case kShape128: return {128, 128, F8Tile<2, 2, 2>::lds(groups, 1), {0.45, 0.60}, 0.72, 2.0};
    case kShape128Deep:
        if (f32) return {128, 128, F8Tile<2, 2, 4>::lds(groups, 1), {0.70, 0.98}, 0.98, 6.0};
        return {128, 128, F8Tile<2, 2, 4>::lds(groups, 1), {0.50, 0.72}, 0.72, 2.0};
    default: return {256, 256, F8Large::lds(groups), {0.85, 1.10, 1.40, 1.72}, 1.40, 4.0};
    }
}
constexpr int kSplitUnits = 16;       // two windows of scales for each half
constexpr double kMemory = 4.9e6;     // bytes of matrices a us, whatever the shape

// Which results and scales a shape has: the large kernel's K loop has registers for one
// scale a tile's columns and 16-bit results alone; a scale for every row of B takes 64 x 64;
// binary32 results' 128 x 128 take more registers than two workgroups have, so one with
// the deeper ring (4096^3 172 us as two that spill, 1024 x 4096 x 4096 61 -> 42).
bool serves(const F8Args &g, int format, int shape)
{
    if (shape == kShape256) return format != OUT_F32 && g.sb_shift != 0 && g.U >= F8Large::kMinUnits;
    return shape == kShape64 || (shape == kShape64Split ? g.U >= kSplitUnits : g.sb_shift != 0 && (shape == kShape128Deep || format != OUT_F32));
}

int64_t tiles_of(const F8Args &g, const Shape &s, int64_t *blocks)
{
    const int64_t groups = g.offsets ? std::min(g.E, g.R) : 1, rows = ceil_div(g.R, groups);
    // groups of different sizes have half a tile more than their average's rows fill
    const int64_t tiles = g.offsets ? std::max<int64_t>(groups, (2 * (int64_t)g.R + groups * s.high) / (2 * s.high)) : ceil_div(rows, s.high);
    *blocks = std::min<int64_t>(4, ceil_div(ceil_div(rows, 64), ceil_div(rows, s.high)));
    return tiles * ceil_div(g.N, s.wide);
}

// The shape that should take the least time; the smaller of equal ones.
int choose_shape(const F8Args &g, int format, int64_t cu)
{
    int best = kShape64;
    double best_time = 0;
    for (int i = 0; i < kShapeCount; ++i) {
        if (!serves(g, format, i)) continue;
        const Shape s = shape_of(i, 0, format);
        int64_t blocks;
        const int64_t tiles = tiles_of(g, s, &blocks);
        // one tile to a compute unit: K in two halves, a ring of four stages
        if ((i == kShape64Split || (i == kShape128Deep && serves(g, format, kShape128))) && tiles > cu) continue;
        if (i == kShape128 && tiles <= cu) continue;
        const double stage = tiles < cu * 3 / 4 ? std::min(s.few, s.stage[blocks - 1] * 1.3) : s.stage[blocks - 1];
        const double own = (double)ceil_div(tiles, cu) * ((double)g.U * stage + s.tile);
        const double t = std::max(own, (double)std::min(g.E, g.R) * g.N * g.U * kF8UnitCodes / kMemory);
        if (best_time == 0 || t < best_time) {
            best = i;
            best_time = t;
        }
    }
    return best;
}

// Whether the narrow kernel takes a call that it can serve: up to 16 rows, up to 32 with
// A in registers, and few tiles with long K, which its waves split (us, best tiles /
// narrow):
//     16 x 28672 x 8192   50.5 / 40.6      32 x 28672 x 8192   50.9 / 74.5
//     1 x 4096 x 4096     11.1 /  5.6      64 x 4096 x 4096    11.6 / 17.9
//     32 x 4096 x 4096    11.3 /  9.6      100 x 100 x 16384   30.1 / 15.3
// Grouped, up to eight rows a group on average (32 groups of 4096 x 4096 by chance):
//     32 rows  83.4 / 73.1     256 rows  113 / 94     384 rows  117 / 115     512 rows  116 / 133
bool narrow_pays(const F8Args &g, int64_t cu)
{
    if (g.offsets != nullptr) return g.R <= 8 * (int64_t)g.E;
    if (g.R <= 32) return g.R <= 16 || g.U <= narrow_units(g.R);
    return g.U >= 32 && ceil_div(g.R, 64) * ceil_div(g.N, 64) <= cu / 16;
}

struct F8Plan {
    int shape;  // kShapeCount: narrow
    NarrowPlan narrow;
    int64_t blocks;
    int threads;
};

lpgemm_status plan_shape(const F8Args &g, int format, int shape, int64_t cu, F8Plan *p)
{
    const Shape s = shape_of(shape, g.E, format);
    const int64_t tiles_n = ceil_div(g.N, s.wide);
    // 32-bit tile counts; at most one ragged row tile a group more than the rows fill
    if (ceil_div(g.R, s.high) + g.E > INT32_MAX / tiles_n) return LPGEMM_ERR_UNSUPPORTED;
    const int64_t most = (ceil_div(g.R, s.high) + (g.offsets ? std::min(g.E, g.R) : 0)) * tiles_n;
    *p = F8Plan{shape, {}, std::min(most, (s.lds > 80 * 1024 ? 1 : 2) * cu), shape == kShape64Split || shape == kShape256 ? 512 : 256};
    return LPGEMM_OK;
}

lpgemm_status plan_product(const F8Args &g, int format, int64_t cu, int forced, F8Plan *p)
{
    const auto narrow = [&] {
        const NarrowPlan n = plan_narrow(g, cu);
        *p = F8Plan{kShapeCount, n, n.blocks * n.tiles, 64 * kMxNarrowWaves};
        return LPGEMM_OK;
    };
    switch (forced) {
    case LPGEMM_KERNEL_AUTO:
    case LPGEMM_KERNEL_TILED:
        if (forced == LPGEMM_KERNEL_AUTO && narrow_serves(g) && narrow_pays(g, cu)) return narrow();
        return plan_shape(g, format, choose_shape(g, format, cu), cu, p);
    case LPGEMM_KERNEL_TILED_256:
        if (serves(g, format, kShape256)) return plan_shape(g, format, kShape256, cu, p);
        [[fallthrough]];
    case LPGEMM_KERNEL_TILED_128:
        if (serves(g, format, kShape128Deep))
            return plan_shape(g, format, g.R * (int64_t)g.N > 128 * 128 * cu && serves(g, format, kShape128) ? kShape128 : kShape128Deep, cu, p);
        [[fallthrough]];
    case LPGEMM_KERNEL_TILED_64:
        return plan_shape(g, format, g.R * (int64_t)g.N > 64 * 64 * cu || !serves(g, format, kShape64Split) ? kShape64 : kShape64Split, cu, p);
    case LPGEMM_KERNEL_SKINNY: return narrow_serves(g) ? narrow() : LPGEMM_ERR_UNSUPPORTED;
    default: return LPGEMM_ERR_UNSUPPORTED;
    }
}

template <int OUT>
lpgemm_status launch_product(const F8Args &g, hipStream_t stream)
{
    F8Plan p;
    const lpgemm_status st = plan_product(g, OUT, compute_units(), forced_kernel(), &p);
    if (st != LPGEMM_OK) return st;
    const bool rows = g.sb_shift == 0;
    switch (p.shape) {
    case kShape64: return rows ? launch_tiled<1, 1, 4, 1, true, OUT>(g, p.blocks, stream) : launch_tiled<1, 1, 4, 1, false, OUT>(g, p.blocks, stream);
    case kShape64Split: return rows ? launch_tiled<1, 1, 4, 2, true, OUT>(g, p.blocks, stream) : launch_tiled<1, 1, 4, 2, false, OUT>(g, p.blocks, stream);
    case kShape128:
        if constexpr (OUT != OUT_F32) return launch_tiled<2, 2, 2, 1, false, OUT>(g, p.blocks, stream);
        return LPGEMM_ERR_UNSUPPORTED;
    case kShape128Deep: return launch_tiled<2, 2, 4, 1, false, OUT>(g, p.blocks, stream);
    case kShape256:
        if constexpr (OUT != OUT_F32) return launch_large<OUT>(g, p.blocks, stream);
        return LPGEMM_ERR_UNSUPPORTED;
    default: return launch_narrow_any<OUT>(g, p.narrow, stream);
    }
}

// Sizes and pointers that both products share; R rows of D.
lpgemm_status check_product(const void *A, const void *SFA, const void *B, const void *SFB, int shift, const void *D, int format, int64_t T, int64_t R,
                            int64_t N, int64_t K, int64_t E)
{
    if (format < 0 || shift < 0 || T < 0 || R < 0 || N < 0 || K < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_FP8_BLOCK_MAX_K || T > LPGEMM_FP8_BLOCK_MAX_ROWS || R > LPGEMM_FP8_BLOCK_MAX_ROWS || N > LPGEMM_FP8_BLOCK_MAX_ROWS ||
        E > LPGEMM_FP8_BLOCK_MAX_GROUPS)
        return LPGEMM_ERR_UNSUPPORTED;
    if (R == 0 || N == 0) return LPGEMM_OK;
    if (D == nullptr || !aligned(D, 16)) return LPGEMM_ERR_INVALID_ARG;
    if (K > 0 && ((T > 0 && (A == nullptr || SFA == nullptr)) || (E > 0 && (B == nullptr || SFB == nullptr)) || !aligned(A, 16) || !aligned(B, 16) ||
                  !aligned(SFA, 4) || !aligned(SFB, 4)))
        return LPGEMM_ERR_INVALID_ARG;
    return LPGEMM_OK;
}

F8Args args_of(const uint8_t *A, const float *SFA, int64_t T, const int32_t *rows, const uint8_t *B, const float *SFB, int shift, int64_t E,
               const int32_t *offsets, void *D, int64_t R, int64_t N, int64_t K)
{
    F8Args g;
    static_cast<MxArgs &>(g) = MxArgs{A, reinterpret_cast<const uint8_t *>(SFA), B, reinterpret_cast<const uint8_t *>(SFB), D, offsets, rows,
                                      (int32_t)T, (int32_t)R, (int32_t)N, (int32_t)units_of(K), (int32_t)E};
    g.sb_shift = shift;
    g.sb_rows = (int32_t)(shift != 0 ? ceil_div(N, 128) : N);
    return g;
}

lpgemm_status run_product(const F8Args &g, int format, hipStream_t stream)
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

lpgemm_status lpgemm_fp8_block_quantize(const void *X, lpgemm_out_dtype x_dtype, int64_t ldx, int64_t block_rows, int32_t power_of_two, uint8_t *codes,
                                        float *scales, int64_t rows, int64_t K, hipStream_t stream)
{
    const int f = format_of(x_dtype), shift = shift_of(block_rows);
    const lpgemm_status st = check_values(X, codes, scales, f, shift, rows, K);
    if (st != LPGEMM_OK) return st;
    if (power_of_two != 0 && power_of_two != 1) return LPGEMM_ERR_INVALID_ARG;
    if (rows == 0 || K == 0) return LPGEMM_OK;
    if (ldx < (rows > 1 ? K : 0) || (rows > 1 && ldx > (INT64_MAX >> 4) / rows)) return LPGEMM_ERR_INVALID_ARG;
    (void)hipGetLastError();
    switch (f) {
    case OUT_F32: return launch_quantize_any<OUT_F32>(X, ldx, codes, scales, shift, power_of_two, rows, K, stream);
    case OUT_BF16: return launch_quantize_any<OUT_BF16>(X, ldx, codes, scales, shift, power_of_two, rows, K, stream);
    default: return launch_quantize_any<OUT_F16>(X, ldx, codes, scales, shift, power_of_two, rows, K, stream);
    }
}

lpgemm_status lpgemm_fp8_block_dequantize(const uint8_t *codes, const float *scales, int64_t block_rows, void *Y, lpgemm_out_dtype y_dtype, int64_t rows,
                                          int64_t K, hipStream_t stream)
{
    const int f = format_of(y_dtype), shift = shift_of(block_rows);
    const lpgemm_status st = check_values(Y, codes, scales, f, shift, rows, K);
    if (st != LPGEMM_OK || rows == 0 || K == 0) return st;
    (void)hipGetLastError();
    switch (f) {
    case OUT_F32: return launch_dequantize<OUT_F32>(codes, scales, shift, Y, rows, K, stream);
    case OUT_BF16: return launch_dequantize<OUT_BF16>(codes, scales, shift, Y, rows, K, stream);
    default: return launch_dequantize<OUT_F16>(codes, scales, shift, Y, rows, K, stream);
    }
}

lpgemm_status lpgemm_fp8_block(const uint8_t *A, const float *SFA, const uint8_t *B, const float *SFB, int64_t b_block_rows, void *D,
                               lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K, hipStream_t stream)
{
    const int f = format_of(out_dtype), shift = shift_of(b_block_rows);
    const lpgemm_status st = check_product(A, SFA, B, SFB, shift, D, f, M, M, N, K, 1);
    if (st != LPGEMM_OK || M == 0 || N == 0) return st;
    return run_product(args_of(A, SFA, M, nullptr, B, SFB, shift, 1, nullptr, D, M, N, K), f, stream);
}

lpgemm_status lpgemm_fp8_block_grouped(const uint8_t *A, const float *SFA, int64_t T, const int32_t *rows, const uint8_t *B, const float *SFB,
                                       int64_t b_block_rows, int64_t E, const int32_t *offsets, void *D, lpgemm_out_dtype out_dtype, int64_t R, int64_t N,
                                       int64_t K, hipStream_t stream)
{
    const int f = format_of(out_dtype), shift = shift_of(b_block_rows);
    const lpgemm_status st = check_product(A, SFA, B, SFB, shift, D, f, T, R, N, K, E);
    if (st != LPGEMM_OK) return st;
    if (rows == nullptr && T != R) return LPGEMM_ERR_INVALID_ARG;
    if (rows != nullptr && T * units_of(K) * (int64_t)kF8UnitCodes > INT32_MAX) return LPGEMM_ERR_UNSUPPORTED;
    if (R == 0 || N == 0 || E == 0) return LPGEMM_OK;
    if (offsets == nullptr || !aligned(offsets, 4) || !aligned(rows, 4)) return LPGEMM_ERR_INVALID_ARG;
    if (T == 0) {  // every row of D is of zeros; the kernels' dead reads of A need an address
        A = B;
        SFA = SFB;
    }
    return run_product(args_of(A, SFA, T, rows, B, SFB, shift, E, offsets, D, R, N, K), f, stream);
}

lpgemm_status lpgemm_fp8_block_plan(int64_t R, int64_t N, int64_t K, int64_t E, int32_t cu_count, lpgemm_plan_info *info)
{
    if (info == nullptr || R < 0 || N < 0 || K < 0 || E < 0) return LPGEMM_ERR_INVALID_ARG;
    if (K > LPGEMM_FP8_BLOCK_MAX_K || R > LPGEMM_FP8_BLOCK_MAX_ROWS || N > LPGEMM_FP8_BLOCK_MAX_ROWS || E > LPGEMM_FP8_BLOCK_MAX_GROUPS)
        return LPGEMM_ERR_UNSUPPORTED;
    *info = lpgemm_plan_info{};
    if (R == 0 || N == 0) return LPGEMM_OK;
    static const int32_t some = 0;  // offsets are there or not, nobody reads them
    const F8Args g = args_of(nullptr, nullptr, R, nullptr, nullptr, nullptr, 7, std::max<int64_t>(E, 1), E > 0 ? &some : nullptr, nullptr, R, N, K);
    F8Plan p;
    const lpgemm_status st = plan_product(g, OUT_BF16, cu_count > 0 ? cu_count : 256, forced_kernel(), &p);
    if (st != LPGEMM_OK) return st;
    const bool narrow = p.shape == kShapeCount;
    const Shape s = shape_of(p.shape, 0, OUT_BF16);
    info->kernel = narrow ? LPGEMM_KERNEL_SKINNY : LPGEMM_KERNEL_TILED;
    info->tile_m = !narrow ? s.high : p.narrow.ring || R <= 16 ? 16 : 32;
    info->tile_n = narrow ? 16 : s.wide;
    info->k_split = narrow ? p.narrow.kw : p.shape == kShape64Split ? 2 : 1;
    info->workgroups = p.blocks;
    info->threads = p.threads;
    info->k_chunks = 1;
    return LPGEMM_OK;
}

}  // extern "C"
