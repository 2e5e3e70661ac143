// gemm_mxfp4.hpp -- products of microscaled 4-bit float operands,
//     D[m][n] = out( sum_j 2^(sa[m][j] - 127) 2^(sb[n][j] - 127) sum_{k in block j} a[m][k] b[n][k] )
// over blocks of 32 k, one pair of matrices or one matrix of B per group of
// rows.  gfx950's v_mfma_scale_f32_*_f8f6f4 multiplies e2m1 operands with one
// e8m0 scale byte per row and block: the format's definition, in one
// instruction.  Products of a block are exact and sums are binary32; the one
// rounding to fewer bits is that of the result.
//
// Three kernels (the choice between them: mxfp4_api.hip):
//  - tiled, 64 x 64 to 128 x 128 tiles: bound by what a compute unit draws from
//    its L2 and beyond (60-100 GB/s): 1110 rows on 13 groups of 1001 x 2897
//    12.4 us, 4096 on 64 of 2048 x 4096 77 us (3.9 TB/s), 333 x 1001 x 2897 7.2 us.
//  - large, tiles of 256 columns: bound by the one stream of instructions of a
//    SIMD's one wave, which issues copies, reads and MFMAs, and by a tile's
//    beginning and end.  8192^3 261 us, 4.2 PFLOP/s, with the matrix cores 57%
//    busy at 1.74 GHz (the same MFMAs on registers alone: 6.2-6.5 PFLOP/s at
//    1.59-1.66 GHz); 3000 x 5120 x 6144 50 us; 16384 rows on 32 groups of 4096 x
//    4096 190-202 us (2.8 PFLOP/s, 35% busy at 2.03 GHz).
//  - narrow, few rows: bound by memory: 16 x 28672 x 8192 23.9 us (5.3 TB/s), 64
//    rows on 24 of 32 groups of 4096 x 4096 36 us (6.0 TB/s), 1 x 4096 x 4096
//    4.3 us on the device.
#pragma once

#include "device_common.hpp"
#include "mxfp4_quantize.hpp"

namespace lpgemm {

constexpr int kMxFormat = 4;  // e2m1 operand format of the f8f6f4 MFMA

struct MxArgs {
    const uint8_t *A, *SFA;   // [T][64 U], [T][4 U]
    const uint8_t *B, *SFB;   // [E][N][64 U], [E][N][4 U]
    void *D;                  // [R][N]
    const int32_t *offsets;   // [E + 1]: group e is rows [offsets[e], offsets[e + 1]); null: one group of all rows
    const int32_t *rows;      // [R]: row of A for each row of D; null: the same row
    int32_t T, R, N, U, E;
};

// Group e's rows [begin, end): each offset taken into [0, R], and one below an
// offset before it to that one, so that no row is in two groups and the groups
// have at most R / height + E row tiles whatever the offsets hold.  `ordered`:
// no offset is below the one before it; false comes back where e's are not.
__device__ __forceinline__ bool mx_group(const MxArgs &g, int e, bool ordered, int &begin, int &end)
{
    const int first = g.offsets[e], after = g.offsets[e + 1];  // both on their way at once
    const int next = min(max(after, 0), g.R);
    begin = min(max(first, 0), g.R);
    if (__builtin_expect(!ordered, 0))
        for (int i = 0; i < e; ++i) begin = max(begin, min(g.offsets[i], g.R));
    end = max(begin, next);
    return next >= begin;
}

__device__ __forceinline__ i32x8 mx_operand(i32x4 c) { return i32x8{c.x, c.y, c.z, c.w, 0, 0, 0, 0}; }

// ---- tiled kernel ------------------------------------------------------------
// 16 bytes (4 bytes) per lane from rsrc[voffset] into LDS at lds_base + 16 (4) lane;
// offsets at or past the resource's size read zeros.
__device__ __forceinline__ void mx_dma16(i32x4 rsrc, uint32_t voffset, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 : : "v"(voffset), "s"(rsrc), "s"(lds_base) : "memory", "m0");
}
// mx_dma16 from rsrc[voffset + soffset].
__device__ __forceinline__ void mx_dma16_at(i32x4 rsrc, uint32_t voffset, uint32_t soffset, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
                 : : "v"(voffset), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soffset)), "s"(__builtin_amdgcn_readfirstlane(lds_base))
                 : "memory", "m0");
}
// mx_dma16 of data that is read once: it need not stay in the caches.
__device__ __forceinline__ void mx_dma16_nt(i32x4 rsrc, uint32_t voffset, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen nt lds"
                 : : "v"(voffset), "s"(rsrc), "s"(lds_base) : "memory", "m0");
}
__device__ __forceinline__ void mx_dma4(i32x4 rsrc, uint32_t voffset, uint32_t lds_base)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 : : "v"(voffset), "s"(rsrc), "s"(lds_base) : "memory", "m0");
}


// Two binary32 values as two bf16 or fp16, nearest even, in one dword.
template <int OUT>
__device__ __forceinline__ uint32_t mx_pack2(float a, float b)
{
    const mx_f32x2 v = {a, b};
    if (OUT == OUT_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, mx_bf16x2));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, mx_f16x2));
}

// The sum over the lanes up to this one, all 64 active: within rows of 16 lanes,
// then the rows' last lanes into the rows behind them.  Every instruction before
// the first copy costs its fetch: 1105 rows on 13 groups of 1001 x 2897 take 10.7
// us on the device, 11.0 with a permutation through LDS for each of the six steps.
__device__ __forceinline__ int mx_scan(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr:1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast:15 to rows 1, 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // row_bcast:31 to rows 2, 3
    return x;
}

// Row tiles of `high` rows before each group, summed into cum[0 .. E], and
// their number: thread t takes groups t P .. t P + P - 1.  cum has WAVES words
// more for the waves' sums.  The groups are counted as if their offsets were
// `ordered` and, where a wave finds some that are not (-1 in its sum's place),
// once more.  bounds, if any: begin | end << 16 of every group.
template <int WAVES>
__device__ __forceinline__ int mx_tiles_before(const MxArgs &g, int high, int32_t *cum, uint32_t *bounds, bool &ordered)
{
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int32_t *part = cum + g.E + 1;
    const int P = (g.E + 64 * WAVES - 1) / (64 * WAVES);
    int before = 0;
    for (ordered = true;; ordered = false) {
        int sum = 0;
        bool fell = false;
        for (int i = 0; i < P; ++i) {
            int b = 0, f = 0;
            if (tid * P + i < g.E) fell |= !mx_group(g, tid * P + i, ordered, b, f);
            sum += (f - b + high - 1) / high;
        }
        const int run = mx_scan(sum);
        const bool again = ordered && __ballot(fell) != 0;
        if (lane == 63) part[wave] = again ? -1 : run;
        __syncthreads();
        before = run - sum;
        int all = 0;  // negative: a wave's offsets fall
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int p = part[w];
            all |= p;
            before += w < wave ? p : 0;
        }
        if (__builtin_expect(__builtin_amdgcn_readfirstlane(all) >= 0, 1)) break;
        __syncthreads();  // every wave has read the sums
    }
    for (int i = 0; i < P; ++i) {
        const int e = tid * P + i;
        if (e >= g.E) break;
        int b, f;
        mx_group(g, e, ordered, b, f);
        cum[e] = before;
        if (bounds != nullptr) bounds[e] = (uint32_t)b | (uint32_t)f << 16;
        before += (f - b + high - 1) / high;
        if (e == g.E - 1) cum[g.E] = before;
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(cum[g.E]);
}

// The groups' row tiles.  Up to 64 groups are held by the lanes of every wave
// by itself, one load and a scan away (no barrier, nothing in LDS); more in
// `cum`, whose bounds are read again where a tile needs them.
struct MxGroups {
    int begin = 0, end = 0, before = 0, total = 0;  // lane e: group e
    const int32_t *cum = nullptr;
    const uint32_t *bounds = nullptr;  // in LDS, where a kernel has room for them
    bool ordered = true;

    template <int WAVES>
    __device__ __forceinline__ void init(const MxArgs &g, int high, int32_t *table, uint32_t *room = nullptr)
    {
        const int lane = threadIdx.x & 63;
        cum = table;
        bounds = room;
        if (g.E > 64) {
            total = mx_tiles_before<WAVES>(g, high, table, room, ordered);
            return;
        }
        const bool fell = lane < g.E && !mx_group(g, lane, true, begin, end);
        if (__builtin_expect(__ballot(fell) != 0, 0) && lane < g.E) mx_group(g, lane, false, begin, end);
        const int own = (end - begin + high - 1) / high, run = mx_scan(own);
        before = run - own;
        total = __builtin_amdgcn_readlane(run, 63);
    }
    // The group that row tile rt belongs to, the last that begins at or before
    // it: its rows [b, f) and the tiles before it.
    __device__ __forceinline__ int of(const MxArgs &g, int rt, int &b, int &f, int &first) const
    {
        const int lane = threadIdx.x & 63;
        int n = 0;
        if (g.E > 64) {
            for (int i = 0; i < g.E; i += 64) n += (int)__popcll(__ballot(i + lane < g.E && cum[i + lane] <= rt));
            const int e = __builtin_amdgcn_readfirstlane(n - 1);
            first = __builtin_amdgcn_readfirstlane(cum[e]);
            if (bounds != nullptr) {
                const uint32_t bound = __builtin_amdgcn_readfirstlane(bounds[e]);
                b = (int)(bound & 0xFFFFu);
                f = (int)(bound >> 16);
            } else {
                mx_group(g, e, ordered, b, f);
                b = __builtin_amdgcn_readfirstlane(b);
                f = __builtin_amdgcn_readfirstlane(f);
            }
            return e;
        }
        n = (int)__popcll(__ballot(lane < g.E && before <= rt));
        const int e = __builtin_amdgcn_readfirstlane(n - 1);
        first = __builtin_amdgcn_readlane(before, e);
        b = __builtin_amdgcn_readlane(begin, e);
        f = __builtin_amdgcn_readlane(end, e);
        return e;
    }
};

// Tile v of `total`: group e, rows [m0, m1) of D, height 64 fm, columns from
// n0, for tiles of up to 64 HM rows and 64 FN columns.
template <int HM, int FN>
__device__ __forceinline__ void mx_find_tile(const MxArgs &g, int v, int total, int tiles_n, int xcds, const MxGroups &groups, int &e,
                                             int &m0, int &m1, int &n0, int &fm)
{
    // XCD-contiguous: workgroups v, v + 8, .. share an L2 and take neighbouring tiles
    const int whole = total - total % xcds;
    const int id = v < whole ? (v % xcds) * (whole / xcds) + v / xcds : v;
    int begin = 0, end = g.R, first = 0;
    e = 0;
    if (g.offsets != nullptr) e = groups.of(g, id / tiles_n, begin, end, first);
    const int blocks = (end - begin + 63) / 64, c = (blocks + HM - 1) / HM;  // of 64 rows; tiles
    // bands of four row tiles, the band's tiles of one column together
    const int in_group = id - first * tiles_n;
    const int band = in_group / (4 * tiles_n), high = min(4, c - 4 * band);
    const int in_band = in_group - band * 4 * tiles_n;
    const int j = 4 * band + in_band % high;
    n0 = in_band / high * 64 * FN;
    // the group's blocks, shared out evenly
    fm = blocks / c + (j < blocks % c ? 1 : 0);
    m0 = begin + 64 * (j * (blocks / c) + min(j, blocks % c));
    m1 = min(end, m0 + 64 * fm);
}

// Eight or four neighbouring values of a row as OUT, from column n on; those
// from N on are skipped.  Whole pieces go out in 16-byte (four of a 16-bit type:
// 8-byte) stores whatever the row's alignment: global memory takes them at any
// address of the element's alignment, and single stores of rows of odd length
// cost more than the product (5314 x 845 x 1825: 30 us).
template <int OUT>
__device__ __forceinline__ void mx_store8(void *d, int64_t at, int n, int N, i32x4 packed)
{
    uint16_t *p = static_cast<uint16_t *>(d) + at + n;
    if (n + 8 <= N) {
        __builtin_memcpy(p, &packed, 16);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (n + i < N) p[i] = (uint16_t)((uint32_t)packed[i / 2] >> (16 * (i % 2)));
    }
}
template <int OUT>
__device__ __forceinline__ void mx_store4(void *d, int64_t at, int n, int N, float x0, float x1, float x2, float x3)
{
    if (OUT == OUT_F32) {
        float *p = static_cast<float *>(d) + at + n;
        const float x[4] = {x0, x1, x2, x3};
        if (n + 4 <= N) {
            __builtin_memcpy(p, x, 16);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (n + i < N) p[i] = x[i];
        }
    } else {
        uint16_t *p = static_cast<uint16_t *>(d) + at + n;
        const uint32_t w[2] = {mx_pack2<OUT>(x0, x1), mx_pack2<OUT>(x2, x3)};
        if (n + 4 <= N) {
            __builtin_memcpy(p, w, 8);
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (n + i < N) p[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
        }
    }
}

// 32 rows x 32 W columns of D, blocks c(0) .. c(W - 1) side by side, through the
// wave's own `stage` of LDS (mx_stage_bytes), so that a store instruction writes
// whole rows of them.  In the MFMA's layout it writes 32 bytes of each of 32
// rows, which memory takes far more slowly: 2848 x 2880 fp32 went out at 2 TB/s.
template <int OUT, int W>
__host__ __device__ constexpr int mx_stage_pitch() { return 32 * W * (OUT == OUT_F32 ? 4 : 2) + 16; }
template <int OUT, int W>
__host__ __device__ constexpr int mx_stage_bytes() { return 32 * mx_stage_pitch<OUT, W>(); }
template <int OUT, int W, typename Block>
__device__ __forceinline__ void mx_store_rows(const MxArgs &g, uint8_t *stage, Block c, int m0, int m1, int nb)
{
    constexpr int kPitch = mx_stage_pitch<OUT, W>();
    int lane = (int)threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // addresses are computed here, not kept through the K loop
    uint8_t *mine = stage + (lane & 31) * kPitch;
    const int h = lane >> 5;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const f32x16 &x = c(w);
#pragma unroll
        for (int rg = 0; rg < 4; ++rg) {
            const int col = 32 * w + 8 * rg + 4 * h;
            if (OUT == OUT_F32) {
                const i32x4 v = {(int32_t)__float_as_uint(x[4 * rg]), (int32_t)__float_as_uint(x[4 * rg + 1]),
                                 (int32_t)__float_as_uint(x[4 * rg + 2]), (int32_t)__float_as_uint(x[4 * rg + 3])};
                *reinterpret_cast<i32x4 *>(mine + 4 * col) = v;
            } else {
                *reinterpret_cast<uint64_t *>(mine + 2 * col) =
                    (uint64_t)mx_pack2<OUT>(x[4 * rg + 2], x[4 * rg + 3]) << 32 | mx_pack2<OUT>(x[4 * rg], x[4 * rg + 1]);
            }
        }
    }
    // the wave's own writes, read by its other lanes
    __builtin_amdgcn_wave_barrier();
    constexpr int kPiece = OUT == OUT_F32 ? 4 : 8, kLanes = 32 * W / kPiece, kRows = 64 / kLanes;  // columns a lane; lanes a row; rows at a time
    const int sub = lane / kLanes, n = nb + lane % kLanes * kPiece;
#pragma unroll
    for (int i = 0; i < 32 / kRows; ++i) {
        const int row = i * kRows + sub, m = m0 + row;
        const i32x4 v = *reinterpret_cast<const i32x4 *>(stage + row * kPitch + lane % kLanes * 16);
        if (m >= m1) continue;
        if (OUT == OUT_F32)
            mx_store4<OUT>(g.D, (int64_t)m * g.N, n, g.N, __int_as_float(v[0]), __int_as_float(v[1]), __int_as_float(v[2]), __int_as_float(v[3]));
        else
            mx_store8<OUT>(g.D, (int64_t)m * g.N, n, g.N, v);
    }
    __builtin_amdgcn_wave_barrier();
}

// A workgroup of four waves (2 x 2) computes tiles of 64 FM x 64 FN, FM = 1 ..
// FN chosen tile by tile from its group's rows, so a group wastes less than 64
// rows whatever its size; a wave holds FM x FN blocks of 32 x 32.
//
// A stage is two units (256 k) of every row: 128 code bytes, one cache line,
// and 8 scale bytes.  Lane half h of a wave takes unit h of the stage, MFMA
// step s its block s, so one dword of scales serves a lane's four steps, the
// MFMA picking byte s.  In LDS a row's eight 16-byte chunks are permuted by
// c -> c ^ (row / 2) % 8: both the copies (8 rows of 128 bytes each) and the
// fragment reads (16 rows of one chunk) touch all banks once.
//
// Scales come for two stages at a time, 16 bytes of every row: a copy of
// scattered rows costs a cycle for each, whatever it brings (8192^3 lost 67 us
// of 414 to copies of a dword).  The window is the row's last four units where
// fewer are left; a scale past the row is then another of that row's: it meets
// zero codes, and it is NaN only where the row's results are anyway.
__device__ __forceinline__ int mx_scale_window(int q, int U) { return max(0, min(4 * q, U - 4)); }
// Dword of a window that belongs to unit u.
__device__ __forceinline__ int mx_scale_at(int u, int q, int U)
{
    const int first = mx_scale_window(q, U);
    return min(u - first, min(3, U - 1 - first));
}

template <int HM, int FN, int STAGES>
struct MxTile {
    static_assert((FN == 1 || FN == 2) && HM <= FN && (STAGES == 2 || STAGES == 4), "heights up to HM, 64 or 128 columns");
    static constexpr int BN = 64 * FN;
    static constexpr int kStages = STAGES;
    static constexpr int NB = 2 * FN;                            // a wave's copies of B per stage
    static constexpr int copies(int fm) { return NB + 2 * fm; }  // of codes; and one of scales in even stages
    static constexpr int kCodes = (BN + 64 * HM) * 128;          // of a stage: B's rows, then A's
    // scales of two stages: 1 KB a wave, of its 32 FN rows; two pairs are in flight, and the one being read
    static constexpr int kPairs = kStages / 2 + 1, kScales = 4096;
    static constexpr int kRing = kStages * kCodes + kPairs * kScales;
    static constexpr int lds(int groups, int kgroups) { return kgroups * kRing + 4 * (groups + 1 + 4 * kgroups); }
};

// KG == 2: eight waves, the second four on the second half of K with a ring of
// their own; their sums are added at the end, through LDS.  A stage of a small
// tile is a chain of waits (a copy's, a barrier's, a fragment's: 0.25 us, of
// which its MFMAs are 0.06), so where there is one tile to a compute unit two
// chains side by side are shorter, by what the copies leave: 60 x 60 x 16384
// 22.0 -> 16.6 us, 1024 x 1024 x 4096 9.6 -> 8.9 us.
template <int HM, int FN, int STAGES, int KG, int OUT>
__global__ __launch_bounds__(256 * KG, KG == 1 ? 2 : 1) void gemm_mxfp4_tiled_kernel(MxArgs g, int tiles_n, int xcds)
{
    using T = MxTile<HM, FN, STAGES>;
    static_assert(4 * mx_stage_bytes<OUT, FN>() <= T::kStages * T::kCodes, "the ring holds the rows on their way out");
    constexpr int ST = T::kStages;
    extern __shared__ __align__(1024) uint8_t smem_all[];
    int32_t *cum = reinterpret_cast<int32_t *>(smem_all + KG * T::kRing);  // [E + 1]: row tiles before group e

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
    const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
    uint8_t *smem = smem_all + kg * T::kRing;
    const int wm = wave >> 1, wn = wave & 1;
    const int r32 = lane & 31, h = lane >> 5;
    // this half's stages: k0 .. k0 + ktiles - 1, whole pairs (scales come for two)
    const int U = g.U, ktiles = KG == 1 ? (U + 1) / 2 : 2 * ((U + 7) / 8), k0 = kg * ktiles;
    const uint32_t ldc = (uint32_t)U * kMxUnitCodes, lds_ = (uint32_t)U * kMxUnitScales;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    MxGroups groups;
    if (g.offsets != nullptr) groups.init<4 * KG>(g, 64 * HM, cum);
    const int total = (g.offsets == nullptr ? (g.R + 64 * HM - 1) / (64 * HM) : groups.total) * tiles_n;

    // The current tile: group e, rows [m0, m1) of D, columns from n0, height 64 fm.
    int e = 0, m0 = 0, m1 = 0, n0 = 0, fm = 0;
    auto find = [&](int v) __attribute__((always_inline)) {
        mx_find_tile<HM, FN>(g, v, total, tiles_n, xcds, groups, e, m0, m1, n0, fm);
    };

    // Source offsets of this lane in each copy of a stage, and of its row in
    // the copy of scales: waves 0, 1 serve A's rows, 32 FN each, waves 2, 3 B's.
    i32x4 rsrc_a, rsrc_b, rsrc_s;
    uint32_t a_off[2 * HM], b_off[T::NB], s_off;
    const int c8 = lane & 7;
    // chunk of the row's 128 bytes that goes to position c8 of row 8 p + lane / 8
    auto chunk = [&](int p) { return c8 ^ ((4 * p + (lane >> 4)) & 7); };
#pragma unroll
    for (int i = 0; i < T::NB; ++i) {
        const int p = wave * T::NB + i;
        b_off[i] = (uint32_t)(8 * p + (lane >> 3)) * ldc + 16u * (uint32_t)chunk(p);
    }
    auto place = [&]() __attribute__((always_inline)) {  // resources and A's offsets of the current tile
        const int64_t brow = (int64_t)e * g.N + n0;
        const uint32_t nrows = (uint32_t)min(T::BN, g.N - n0);
        const int64_t arow = g.rows == nullptr ? m0 : 0;
        const uint32_t mrows = (uint32_t)(g.rows == nullptr ? m1 - m0 : g.T);
        rsrc_b = make_rsrc(g.B + brow * ldc, nrows * ldc);
        rsrc_a = make_rsrc(g.A + arow * ldc, mrows * ldc);
        rsrc_s = make_rsrc(wave < 2 ? g.SFA + arow * lds_ : g.SFB + brow * lds_, (wave < 2 ? mrows : nrows) * lds_);
        auto row_offset = [&](int r, uint32_t ld) __attribute__((always_inline)) -> uint32_t {  // of tile row r of A
            if (g.rows == nullptr) return (uint32_t)r * ld;
            const int at = m0 + r < m1 ? g.rows[m0 + r] : -1;
            return at >= 0 && at < g.T ? (uint32_t)at * ld : kOutOfRange;
        };
#pragma unroll
        for (int i = 0; i < 2 * HM; ++i) {
            const int p = wave * 2 * fm + i;
            if (i < 2 * fm) a_off[i] = row_offset(8 * p + (lane >> 3), ldc) + 16u * (uint32_t)chunk(p);
        }
        const int r = (wave & 1) * 32 * FN + lane;  // FN == 1: 32 rows, the upper lanes' zeros go nowhere
        s_off = lane >= 32 * FN ? kOutOfRange : wave < 2 ? row_offset(r, lds_) : (uint32_t)r * lds_;
    };

    // Copy j of stage kt's copies into its slot, for tiles of height 64 f.
    // Units past the row read zeros.
    auto issue = [&](int j, int f, int local, uint32_t base) __attribute__((always_inline)) {
        const int kt = k0 + local;
        const uint32_t koff = (uint32_t)kt * 128u;
        if (j < T::NB) {
            const int p = wave * T::NB + j;
            const bool in = 2 * kt + (chunk(p) >> 2) < U;
            mx_dma16_at(rsrc_b, in ? b_off[j] : kOutOfRange, koff, base + (uint32_t)p * 1024u);
        } else {
            const int i = j - T::NB, p = wave * 2 * f + i;
            const bool in = 2 * kt + (chunk(p) >> 2) < U;
            mx_dma16_at(rsrc_a, in ? a_off[i] : kOutOfRange, koff, base + T::BN * 128 + (uint32_t)p * 1024u);
        }
    };
    // The scales of stages 2 q and 2 q + 1.  Rows of fewer than four units have
    // no window of 16 bytes: theirs are written by hand, and these copies bring
    // zeros to a place that is not read.
    auto issue_scales = [&](int q) __attribute__((always_inline)) {
        const int at = k0 / 2 + q;
        const bool copied = U >= 4 && 4 * at < U;
        mx_dma16_at(rsrc_s, copied ? s_off : kOutOfRange, (uint32_t)mx_scale_window(at, U) * 4u,
                    lds0 + (uint32_t)(ST * T::kCodes + (U >= 4 ? q % T::kPairs : 1) * T::kScales) + (uint32_t)wave * 1024u);
    };
    // dispatch on the height; bodies see it as a constant
    auto with_height = [&](auto body) __attribute__((always_inline)) {
        if (HM >= 2 && fm == 2) body(std::integral_constant<int, HM >= 2 ? 2 : 1>{});
        else body(std::integral_constant<int, 1>{});
    };
    auto prologue = [&]() __attribute__((always_inline)) {
        if (U < 4) {
            const uint8_t *sf = wave < 2 ? g.SFA + (g.rows == nullptr ? (int64_t)m0 * lds_ : 0) : g.SFB + ((int64_t)e * g.N + n0) * lds_;
            const uint32_t size = (wave < 2 ? (uint32_t)(g.rows == nullptr ? m1 - m0 : g.T) : (uint32_t)min(T::BN, g.N - n0)) * lds_;
            for (int u = 0; u < 4; ++u) {
                uint32_t x = 0;
                if (u < U && s_off < size) x = *reinterpret_cast<const uint32_t *>(sf + s_off + 4 * u);
                *reinterpret_cast<uint32_t *>(smem + ST * T::kCodes + wave * 1024 + lane * 16 + 4 * u) = x;
            }
        }
        with_height([&](auto height) __attribute__((always_inline)) {
            constexpr int FM = decltype(height)::value;
#pragma unroll
            for (int st = 0; st < ST; ++st) {
                if (st % 2 == 0) issue_scales(st / 2);
#pragma unroll
                for (int j = 0; j < T::copies(FM); ++j) issue(j, FM, st, lds0 + (uint32_t)(st * T::kCodes));
            }
        });
    };

    f32x16 acc[FN][HM];  // [n block][m block]
    auto contract = [&](auto height) __attribute__((always_inline)) {
        constexpr int FM = decltype(height)::value;
        constexpr int C = T::copies(FM);
        constexpr uint32_t kA = T::BN * 128;
        constexpr int kBlocks = FM * FN, kReads = FM + FN;
        // copies younger than stage 0's; at a stage's end, than the next one's
        constexpr int kFirst = (ST - 1) * C + (ST - 1) / 2, kSteady = (ST - 2) * C + (ST - 2) / 2;
        wait_vmcnt<kFirst>();
        lds_barrier();

#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

        i32x4 fb[2][FN], fa[2][FM];
        uint32_t sb[FN], sa[FM], sb_next[FN], sa_next[FM];
        const int swz = (r32 >> 1) & 7;
        // fragment i of step s: B's blocks, then A's
        auto read = [&](int s, int i, const uint8_t *base) __attribute__((always_inline)) {
            const uint32_t at = (uint32_t)r32 * 128u + 16u * (uint32_t)((4 * h + s) ^ swz);
            if (i < FN)
                fb[s & 1][i] = load16(base + (wn * FN + i) * 4096 + at);
            else
                fa[s & 1][i - FN] = load16(base + kA + (wm * FM + i - FN) * 4096 + at);
        };
        // row r of a half of FN blocks sits in that half's wave's kilobyte;
        // A's rows are dealt out by FN blocks whatever the tile's height
        auto read_scales = [&](int kt) __attribute__((always_inline)) {
            const int q = kt >> 1, d = mx_scale_at(2 * (k0 + kt) + h, k0 / 2 + q, U);
            const uint8_t *base = smem + ST * T::kCodes + (q % T::kPairs) * T::kScales + 4 * d;
#pragma unroll
            for (int i = 0; i < FN; ++i)
                sb_next[i] = *reinterpret_cast<const uint32_t *>(base + (2 + wn) * 1024 + (32 * i + r32) * 16);
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int blk = wm * FM + i;
                sa_next[i] = *reinterpret_cast<const uint32_t *>(base + blk / FN * 1024 + (32 * (blk % FN) + r32) * 16);
            }
        };
        auto take_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < FN; ++i) sb[i] = sb_next[i];
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] = sa_next[i];
        };
        read_scales(0);
#pragma unroll
        for (int i = 0; i < kReads; ++i) read(0, i, smem);
        take_scales();
        // Step S: the next step's reads go out after the first MFMAs, the
        // copies that refill the stage's slot between all of the last step's.
        constexpr int kPer = (kReads + kBlocks - 1) / kBlocks;
        auto step = [&](auto index, const uint8_t *next, bool reads, bool refill, int kt, uint32_t slot_base) __attribute__((always_inline)) {
            constexpr int S = decltype(index)::value;
            if (S == 3 && refill && (kt & 1) == 0) issue_scales((kt + ST) >> 1);
            if (S == 3 && reads) read_scales(kt + 1);
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int fn = b / FM, f = b % FM;
                acc[fn][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(fb[S & 1][fn]), mx_operand(fa[S & 1][f]),
                                                                             acc[fn][f], kMxFormat, kMxFormat, S, sb[fn], S, sa[f]);
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    if (reads && i / kPer == b) read((S + 1) & 3, i, next);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    if (refill && j >= b * C / kBlocks && j < (b + 1) * C / kBlocks) issue(j, FM, kt + ST, slot_base);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using i0 = std::integral_constant<int, 0>;
        using i1 = std::integral_constant<int, 1>;
        using i2 = std::integral_constant<int, 2>;
        using i3 = std::integral_constant<int, 3>;
        int slot = 0;
        for (int kt = 0; kt + 1 < ktiles; ++kt) {
            const uint8_t *base = smem + slot * T::kCodes;
            const uint32_t lbase = lds0 + (uint32_t)(slot * T::kCodes);
            slot = slot + 1 == ST ? 0 : slot + 1;
            const uint8_t *next = smem + slot * T::kCodes;
            step(i0{}, base, true, false, kt, 0);
            step(i1{}, base, true, false, kt, 0);
            step(i2{}, base, true, false, kt, 0);
            wait_vmcnt<kSteady>();
            lds_barrier();
            step(i3{}, next, true, true, kt, lbase);
            take_scales();
        }
        const uint8_t *base = smem + slot * T::kCodes;
        step(i0{}, base, true, false, 0, 0);
        step(i1{}, base, true, false, 0, 0);
        step(i2{}, base, true, false, 0, 0);
        step(i3{}, base, false, false, 0, 0);
        wait_vmcnt<0>();  // copies past the last stage
    };

    for (int v = blockIdx.x; v < total; v += (int)gridDim.x) {
        find(v);
        place();
        prologue();
        with_height(contract);
        lds_barrier();  // every wave is done with the ring
        if (KG == 2) {
            // the second half's sums, 16 bytes a lane at a time
            i32x4 *sums = reinterpret_cast<i32x4 *>(smem_all + T::kRing) + wave * (HM * FN * 4 * 64) + lane;
#pragma unroll
            for (int i = 0; i < HM * FN * 4; ++i) {
                const f32x16 &x = acc[i / 4 % FN][i / 4 / FN];
                if (kg == 1)
                    sums[i * 64] = i32x4{__float_as_int(x[4 * (i % 4)]), __float_as_int(x[4 * (i % 4) + 1]),
                                         __float_as_int(x[4 * (i % 4) + 2]), __float_as_int(x[4 * (i % 4) + 3])};
            }
            lds_barrier();
            if (kg == 0) {
#pragma unroll
                for (int i = 0; i < HM * FN * 4; ++i) {
                    const i32x4 y = sums[i * 64];
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[i / 4 % FN][i / 4 / FN][4 * (i % 4) + q] += __int_as_float(y[q]);
                }
            }
        }
        uint8_t *out_stage = smem + wave * mx_stage_bytes<OUT, FN>();
#pragma unroll
        for (int f = 0; f < HM; ++f) {
            if (f >= fm || kg != 0) break;
            mx_store_rows<OUT, FN>(g, out_stage, [&](int w) -> const f32x16 & { return acc[w][f]; }, m0 + (wm * fm + f) * 32, m1,
                                   n0 + wn * FN * 32);
        }
        lds_barrier();  // every wave's rows have left it
    }
}

// ---- large tiles -----------------------------------------------------------
// Tiles of 64 FM x 256, FM = 1 .. 4 by the group's rows, four waves (2 x 2) of
// FM x 4 blocks of 32 x 32, one workgroup per compute unit.  A stage is two
// units (256 k) as above.
//
// Each wave reads the next stage's fragments into registers while it
// contracts this one: in step s (FM x 4 MFMAs on block s of every unit) all of
// block s of its half of A and of B.  After the step's barrier these rows'
// place in LDS is free, and the copies of the stage after the next go there:
// four a wave and step (wave w serves half w % 2 of A or B), spread between
// the MFMAs, with seven steps for them to arrive.  With all of a stage's
// copies behind its last step, as the smaller tiles have them, the one wave of
// a SIMD stood still for them: 8192^3 took 400 us.
//
// Scales as in the smaller tiles; U >= 4.
struct MxLarge {
    // Codes: 32 KB for each half of A and of B, in it 8 KB for each block of 32
    // rows, 4 KB a slot (a read's slot and block fit its offset field);
    // scales: 4 KB for each half, 2 KB a slot.
    static constexpr int kHalf = 32768, kBlock = 8192, kSlot = 4096;
    static constexpr int kScales = 4 * kHalf, kScaleHalf = 4096, kScaleSlot = 2048;
    static constexpr int kTables = kScales + 4 * kScaleHalf;
    static constexpr int lds(int groups) { return kTables + 4 * (groups + 1 + 4); }
    static constexpr int kMinUnits = 4;
};

template <int OUT>
__global__ __launch_bounds__(256, 1) void gemm_mxfp4_large_kernel(MxArgs g, int tiles_n, int xcds)
{
    using C = MxLarge;
    extern __shared__ __align__(1024) uint8_t smem[];
    int32_t *cum = reinterpret_cast<int32_t *>(smem + C::kTables);

    // What depends on the lane is computed afresh where it is used, from an
    // opaque copy of its number: kept through the K loop it would not fit the
    // registers, and a spilled value that is read back waits for every copy
    // in flight.
    auto opaque_lane = [&]() __attribute__((always_inline)) {
        int l = (int)threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        return l;
    };
    const int lane0 = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const int U = g.U, pairs = (U + 3) / 4;  // of stages
    const uint32_t ldc = (uint32_t)U * kMxUnitCodes, lds_ = (uint32_t)U * kMxUnitScales;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    MxGroups groups;
    if (g.offsets != nullptr) groups.init<4>(g, 256, cum);
    const int total = (g.offsets == nullptr ? (g.R + 255) / 256 : groups.total) * tiles_n;

    // The current tile: group e, rows [m0, m1) of D, columns from n0, height 64 fm.
    int e = 0, m0 = 0, m1 = 0, n0 = 0, fm = 0;
    auto find = [&](int v) __attribute__((always_inline)) {
        mx_find_tile<4, 4>(g, v, total, tiles_n, xcds, groups, e, m0, m1, n0, fm);
    };

    // This wave's copies: half `wave % 2` of A (waves 0, 1) or B.
    const bool of_b = wave >= 2;
    const int half = wave & 1;
    const uint32_t lds_mine = lds0 + (uint32_t)(wave * C::kHalf);
    const uint32_t lds_scales = lds0 + (uint32_t)(C::kScales + wave * C::kScaleHalf);
    i32x4 rsrc, rsrc_s;
    uint32_t off[4][4], s_off[2];
    int upper[2];  // unit of the stage that copies p = 0, 2 (1, 3) bring to this lane
#pragma unroll
    for (int p = 0; p < 2; ++p) upper[p] = ((lane0 & 7) ^ ((4 * p + (lane0 >> 4)) & 7)) >> 2;
    auto place = [&]() __attribute__((always_inline)) {
        const int lane = opaque_lane();
        const int64_t brow = (int64_t)e * g.N + n0;
        const uint32_t nrows = (uint32_t)min(256, g.N - n0);
        const bool gather = !of_b && g.rows != nullptr;
        const int64_t arow = gather ? 0 : m0;
        const uint32_t mrows = (uint32_t)(gather ? g.T : m1 - m0);
        rsrc = make_rsrc(of_b ? g.B + brow * ldc : g.A + arow * ldc, (of_b ? nrows : mrows) * ldc);
        rsrc_s = make_rsrc(of_b ? g.SFB + brow * lds_ : g.SFA + arow * lds_, (of_b ? nrows : mrows) * lds_);
        const int blocks = of_b ? 4 : fm;  // of 32 rows in this half
        // source row of row r of the half, or -1
        auto row = [&](int r) __attribute__((always_inline)) -> int {
            if (r >= 32 * blocks) return -1;
            const int at = half * 32 * blocks + r;
            if (!gather) return at;
            const int i = m0 + at < m1 ? g.rows[m0 + at] : -1;
            return i < g.T ? i : -1;
        };
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const int at = row(32 * s + 8 * p + (lane >> 3));
                off[s][p] = at >= 0 ? (uint32_t)at * ldc + 16u * (uint32_t)((lane & 7) ^ ((4 * p + (lane >> 4)) & 7)) : kOutOfRange;
            }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int at = row(64 * i + lane);
            s_off[i] = at >= 0 ? (uint32_t)at * lds_ : kOutOfRange;
        }
    };
    // Copy p of block s of stage k; stages and units past the row read zeros.
    auto copy = [&](int s, int p, int k) __attribute__((always_inline)) {
        const uint32_t o = upper[p & 1] < U - 2 * k ? off[s][p] : kOutOfRange;
        mx_dma16_at(rsrc, o, (uint32_t)k * 128u, lds_mine + (uint32_t)(s * C::kBlock + (k & 1) * C::kSlot + p * 1024));
    };
    auto copy_scales = [&](int i, int q) __attribute__((always_inline)) {
        const uint32_t o = 4 * q < U ? s_off[i] : kOutOfRange;
        mx_dma16_at(rsrc_s, o, (uint32_t)mx_scale_window(q, U) * 4u, lds_scales + (uint32_t)((q & 1) * C::kScaleSlot + i * 1024));
    };
    auto prologue = [&]() __attribute__((always_inline)) {
        copy_scales(0, 0);
        copy_scales(1, 0);
#pragma unroll
        for (int s = 0; s < 8; ++s)
#pragma unroll
            for (int p = 0; p < 4; ++p) copy(s & 3, p, s >> 2);
    };

    int v = blockIdx.x;
    if (v >= total) return;
    find(v);
    place();
    prologue();

    auto run_tile = [&](auto height) __attribute__((always_inline)) {
        constexpr int FM = decltype(height)::value;
        const int lane = opaque_lane(), r32 = lane & 31, h = lane >> 5;
        f32x16 acc[4][FM];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

        struct Frags {
            i32x4 a[4][4], b[4][4];  // [block][step]
            uint32_t sa[4], sb[4];
        };
        Frags x, y;
        // this lane's place in a block of A's and B's halves: row r32, block t of unit h
        uint32_t at_a[4], at_b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const uint32_t at = (uint32_t)(r32 * 128 + 16 * ((4 * h + t) ^ ((r32 >> 1) & 7)));
            at_a[t] = (uint32_t)(wm * C::kHalf) + at;
            at_b[t] = (uint32_t)((2 + wn) * C::kHalf) + at;
        }
        const uint32_t at_sa = (uint32_t)(C::kScales + wm * C::kScaleHalf + r32 * 16);
        const uint32_t at_sb = (uint32_t)(C::kScales + (2 + wn) * C::kScaleHalf + r32 * 16);
        // read j of block s of stage k (its parity odd): four fragments of B, four of A, their scales
        constexpr int kReads = 10;
        auto read = [&](Frags &f, int j, int s, int odd, int k) __attribute__((always_inline)) {
            const int slot = s * C::kBlock + odd * C::kSlot;
            if (j < 4) {
                f.b[s][j] = load16(smem + at_b[j] + slot);
            } else if (j < 8) {
                if (s < FM) f.a[s][j - 4] = load16(smem + at_a[j - 4] + slot);
            } else {
                const int q = k >> 1, i = mx_scale_at(2 * k + h, q, U);
                const uint32_t at = (uint32_t)((q & 1) * C::kScaleSlot + 4 * i);
                if (j == 8)
                    f.sb[s] = *reinterpret_cast<const uint32_t *>(smem + at_sb + at + s * 512);
                else if (s < FM)
                    f.sa[s] = *reinterpret_cast<const uint32_t *>(smem + at_sa + at + s * 512);
            }
        };

        // stage 0 into registers, then its place to stage 2
        wait_vmcnt<16>();
        lds_barrier();
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int j = 0; j < kReads; ++j) read(x, j, s, 0, 0);
        lds_barrier();
#pragma unroll
        for (int s = 0; s < 3; ++s) {
#pragma unroll
            for (int p = 0; p < 4; ++p) copy(s, p, 2);
            if (s == 0) {
                copy_scales(0, 1);
                copy_scales(1, 1);
            }
        }

        // Step S of stage k (cur: its fragments): the next stage's block S into
        // nxt; copies of block S - 1 of the stage after that one's successor
        // (step 0: of block 3 of the stage after the next), and of the scales.
        // The wait leaves the last six steps' copies in flight: 24, and two of
        // scales where step 1 of an odd stage is among them.
        auto step = [&](auto index, auto parity, const Frags &cur, Frags &nxt, int k) __attribute__((always_inline)) {
            constexpr int S = decltype(index)::value, ODD = decltype(parity)::value;
            constexpr int kAt = 4 * ODD + S;
            wait_vmcnt<(kAt == 4 || kAt == 5) ? 24 : 26>();
            lds_barrier();
            constexpr int kBlocks = 4 * FM, kCopies = (ODD && S == 1) ? 6 : 4;
            constexpr int kPer = (kReads + kBlocks - 1) / kBlocks;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int fn = b / FM, f = b % FM;
                acc[fn][f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(cur.b[fn][S]), mx_operand(cur.a[f][S]),
                                                                             acc[fn][f], kMxFormat, kMxFormat, S, cur.sb[fn], S, cur.sa[f]);
#pragma unroll
                for (int j = 0; j < kReads; ++j)
                    if (j / kPer == b) read(nxt, j, S, 1 - ODD, k + 1);
#pragma unroll
                for (int c = 0; c < kCopies; ++c)
                    if (c * kBlocks / kCopies == b) {
                        if (c >= 4)
                            copy_scales(c - 4, (k + 3) >> 1);
                        else if (S == 0)
                            copy(3, c, k + 2);
                        else
                            copy(S - 1, c, k + 3);
                    }
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using i0 = std::integral_constant<int, 0>;
        using i1 = std::integral_constant<int, 1>;
        using i2 = std::integral_constant<int, 2>;
        using i3 = std::integral_constant<int, 3>;
        for (int k = 0; k < 2 * pairs; k += 2) {
            step(i0{}, i0{}, x, y, k);
            step(i1{}, i0{}, x, y, k);
            step(i2{}, i0{}, x, y, k);
            step(i3{}, i0{}, x, y, k);
            step(i0{}, i1{}, y, x, k + 1);
            step(i1{}, i1{}, y, x, k + 1);
            step(i2{}, i1{}, y, x, k + 1);
            step(i3{}, i1{}, y, x, k + 1);
        }
        wait_vmcnt<0>();  // copies past the last stage

        const int tm0 = m0, tm1 = m1, tn0 = n0;
        v += (int)gridDim.x;
        lds_barrier();  // every wave is done with the ring
        // Whole rows through the ring, then the next tile's first copies.  The
        // other way round, results in the MFMA's layout behind the copies, 16-bit
        // types took as long and fp32 far longer (8192 x 8192 x 4096: 272 / 190 us).
        uint8_t *out_stage = smem + wave * mx_stage_bytes<OUT, 4>();
#pragma unroll
        for (int f = 0; f < FM; ++f)
            mx_store_rows<OUT, 4>(g, out_stage, [&](int w) -> const f32x16 & { return acc[w][f]; }, tm0 + (wm * FM + f) * 32, tm1,
                                  tn0 + wn * 128);
        if (v >= total) return;
        lds_barrier();  // every wave's rows have left
        find(v);
        place();
        prologue();
    };

    while (v < total) {
        if (fm == 4) run_tile(std::integral_constant<int, 4>{});
        else if (fm == 3) run_tile(std::integral_constant<int, 3>{});
        else if (fm == 2) run_tile(std::integral_constant<int, 2>{});
        else run_tile(std::integral_constant<int, 1>{});
    }
    wait_vmcnt<0>();
}

// ---- narrow kernel -------------------------------------------------------------
// Few rows of A: bound by reading B once.  A workgroup of eight waves takes
// strips of 16 rows of B; KW neighbouring waves split a strip's K, and 8 / KW
// strips are worked on at a time.  Every wave streams its own part: a stage is
// 16 rows x 4 units (256 contiguous bytes a row, 4 KB of codes and 256 bytes of
// scales) copied straight into the wave's own ring of D slots, so no wave
// waits for another's copies.  v_mfma_scale_f32_16x16x128 takes unit g of the
// stage in lane group g and its block s in step s, one scale dword per lane and
// stage.  In LDS chunk c of row r sits at c ^ r: the 16 rows of a fragment read
// touch all banks once.  The KW partial tiles are added in LDS in a fixed
// order, by the subgroup's waves in turn.
//
// A stays in registers (product: 16 FA rows, S stages a wave; more rows are
// the grid's second dimension, each tile reading B for itself) or, where it
// changes from strip to strip (grouped: tiles of up to 16 rows of one group,
// gathered), comes through the ring beside B.
constexpr int kMxNarrowWaves = 8;
// Grouped calls keep what an item looks up in LDS: a load from memory would wait
// behind the copies in flight.  A row number takes 16 bits there.
constexpr int kMxNarrowRows = 896;
constexpr int kMxNarrowGroups = 512;

template <bool GROUPED>
struct MxNarrow {
    static constexpr int kSide = 4096 + 256;                     // a stage's codes and scales
    static constexpr int kStage = kSide * (GROUPED ? 2 : 1);
    static constexpr int kPer = GROUPED ? 10 : 5;                // copies of a stage
    static constexpr int D = GROUPED ? 2 : 4;
    static constexpr int kRing = kMxNarrowWaves * D * kStage;
    static constexpr int kSums = 2 * kMxNarrowWaves * 64 * 16;
    static constexpr int lds(int groups) { return kRing + kSums + (GROUPED ? 4 * (2 * groups + 1 + kMxNarrowWaves + kMxNarrowRows) : 0); }
};

typedef float mx_f32x4 __attribute__((ext_vector_type(4)));

template <int FA, int S, bool GROUPED, int OUT>
__global__ __launch_bounds__(64 * kMxNarrowWaves) void gemm_mxfp4_narrow_kernel(MxArgs g, int kw, int stages)
{
    static_assert(!GROUPED || (FA == 1 && S == 1), "grouped: one row tile, stages counted at run time");
    using C = MxNarrow<GROUPED>;
    if (!GROUPED) {  // a workgroup's row tile, as a product of its own
        const int m0 = (int)blockIdx.y * 16 * FA;
        g.A += (int64_t)m0 * g.U * kMxUnitCodes;
        g.SFA += (int64_t)m0 * g.U * kMxUnitScales;
        g.D = static_cast<uint8_t *>(g.D) + (int64_t)m0 * g.N * (OUT == OUT_F32 ? 4 : 2);
        g.R = min(g.R - m0, 16 * FA);
    }
    extern __shared__ __align__(1024) uint8_t smem[];
    mx_f32x4 *sums = reinterpret_cast<mx_f32x4 *>(smem + C::kRing);  // [2][waves][64]
    int32_t *cum = reinterpret_cast<int32_t *>(smem + C::kRing + C::kSums);
    uint32_t *bounds = reinterpret_cast<uint32_t *>(cum + g.E + 1 + kMxNarrowWaves);  // begin | end << 16
    int32_t *index = reinterpret_cast<int32_t *>(bounds + g.E);

    const int lane = threadIdx.x & 63, r16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % kw, sub = wave / kw, side_by_side = kMxNarrowWaves / kw;
    const int U = g.U, strips = (g.N + 15) / 16;
    const int n_stages = GROUPED ? stages : S;
    const uint32_t ldc = (uint32_t)U * kMxUnitCodes, lds_ = (uint32_t)U * kMxUnitScales;
    const uint32_t ring = (uint32_t)(wave * C::D * C::kStage);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem) + ring;
    const uint8_t *mine = smem + ring;

    int items = strips;
    MxGroups groups;
    if (GROUPED) {
        if (g.rows != nullptr)
            for (int i = threadIdx.x; i < g.R; i += 64 * kMxNarrowWaves) index[i] = g.rows[i];
        groups.init<kMxNarrowWaves>(g, 16, cum, bounds);
        items = groups.total * strips;
        __syncthreads();  // the indices
    }
    const int rounds = (items - (int)blockIdx.x * side_by_side + (int)gridDim.x * side_by_side - 1) / ((int)gridDim.x * side_by_side);
    if (rounds <= 0) return;

    // This lane's part of each copy: rows 4 t + lg, chunk r16 ^ row of its 256
    // bytes; scales: row lane / 4, unit lane % 4.
    uint32_t b_off[4], chunk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        chunk[t] = (uint32_t)(r16 ^ (4 * t + lg));
        b_off[t] = (uint32_t)(4 * t + lg) * ldc + 16u * chunk[t];
    }
    const uint32_t sb_off = (uint32_t)(lane >> 2) * lds_ + 4u * (uint32_t)(lane & 3);

    // Where an item's copies come from, set as its first stage is issued.
    struct Item {
        int strip, m0, m1;  // m0 < 0: none
    };
    auto item_of = [&](int round) __attribute__((always_inline)) {
        Item it;
        const int id = (round * (int)gridDim.x + (int)blockIdx.x) * side_by_side + sub;
        it.m0 = id < items ? 0 : -1;
        it.m1 = g.R;
        it.strip = id;
        if (GROUPED && id < items) {
            int begin, end, first;
            const int e = groups.of(g, id / strips, begin, end, first);
            const int tiles = (end - begin + 15) / 16, in_group = id - first * strips;
            // a strip's row tiles one after another: its later reads come from the caches
            it.strip = e * strips + in_group / tiles;
            it.m0 = begin + 16 * (in_group % tiles);
            it.m1 = min(end, it.m0 + 16);
        }
        return it;
    };
    i32x4 rsrc_b, rsrc_sb, rsrc_a, rsrc_sa;
    uint32_t a_off[4], sa_off;
    if (GROUPED) {
        rsrc_a = make_rsrc(g.A, (uint32_t)g.T * ldc);
        rsrc_sa = make_rsrc(g.SFA, (uint32_t)g.T * lds_);
    }
    auto aim = [&](const Item &it) __attribute__((always_inline)) {
        const int e = GROUPED ? it.strip / strips : 0, n0 = 16 * (it.strip - e * strips);
        const int64_t brow = (int64_t)e * g.N + n0;
        const uint32_t n = it.m0 < 0 ? 0u : (uint32_t)min(16, g.N - n0);
        rsrc_b = make_rsrc(g.B + brow * ldc, n * ldc);
        rsrc_sb = make_rsrc(g.SFB + brow * lds_, n * lds_);
        if (GROUPED) {
            auto row = [&](int r) __attribute__((always_inline)) -> int {
                if (it.m0 < 0 || it.m0 + r >= it.m1) return -1;
                const int at = g.rows == nullptr ? it.m0 + r : index[it.m0 + r];
                return at < g.T ? at : -1;
            };
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = row(4 * t + lg);
                a_off[t] = at >= 0 ? (uint32_t)at * ldc + 16u * chunk[t] : kOutOfRange;
            }
            const int at = row(lane >> 2);
            sa_off = at >= 0 ? (uint32_t)at * lds_ + 4u * (uint32_t)(lane & 3) : kOutOfRange;
        }
    };
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        const int u0 = 4 * (part * n_stages + s);
        const uint32_t base = lds0 + (uint32_t)(slot * C::kStage);
        const uint32_t koff = (uint32_t)u0 * kMxUnitCodes, soff = (uint32_t)u0 * kMxUnitScales;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            mx_dma16_nt(rsrc_b, u0 + (int)(chunk[t] >> 2) < U ? b_off[t] + koff : kOutOfRange, base + (uint32_t)t * 1024u);
        mx_dma4(rsrc_sb, u0 + (lane & 3) < U ? sb_off + soff : kOutOfRange, base + 4096u);
        if (GROUPED) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                mx_dma16(rsrc_a, u0 + (int)(chunk[t] >> 2) < U ? a_off[t] + koff : kOutOfRange, base + C::kSide + (uint32_t)t * 1024u);
            mx_dma4(rsrc_sa, u0 + (lane & 3) < U ? sa_off + soff : kOutOfRange, base + C::kSide + 4096u);
        }
    };

    // A in registers: lane (r16, lg), stage s, unit lg: 64 code bytes, one scale dword.
    i32x4 a[FA][S][4];
    uint32_t sa[FA][S];
    if (!GROUPED) {
        const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.A, (uint32_t)g.R * ldc);
        const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(g.SFA, (uint32_t)g.R * lds_);
#pragma unroll
        for (int f = 0; f < FA; ++f)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int u = 4 * (part * S + s) + lg;
                const uint32_t row = (uint32_t)(16 * f + r16);
                const bool in = u < U && (int)row < g.R;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    a[f][s][q] = buffer_load16(ra, in ? row * ldc + (uint32_t)u * kMxUnitCodes + 16u * q : kOutOfRange);
                sa[f][s] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsa, in ? row * lds_ + (uint32_t)u * kMxUnitScales : kOutOfRange, 0, 0);
            }
    }

    // The copies run D stages ahead of the arithmetic, over the item borders.
    int ahead_round = 0, ahead_stage = 0;
    Item next = item_of(0), cur = next;
    aim(next);
    auto advance = [&](int slot) __attribute__((always_inline)) {
        if (ahead_round < rounds) issue(ahead_stage, slot);
        if (++ahead_stage == n_stages) {
            ahead_stage = 0;
            if (++ahead_round < rounds) {
                next = item_of(ahead_round);
                aim(next);
            }
        }
    };
    // grouped: the items between the arithmetic's and the copies' are looked up again
#pragma unroll
    for (int d = 0; d < C::D; ++d) advance(d);
    if (!GROUPED) {
        // A is waited for here, once
#pragma unroll
        for (int f = 0; f < FA; ++f)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                asm volatile("" : "+v"(sa[f][s]));
#pragma unroll
                for (int q = 0; q < 4; ++q) asm volatile("" : "+v"(a[f][s][q]));
            }
    }

    int slot = 0, issued_left = rounds * n_stages;  // stages not yet contracted
    for (int round = 0; round < rounds; ++round) {
        mx_f32x4 acc[FA];
#pragma unroll
        for (int f = 0; f < FA; ++f) acc[f] = mx_f32x4{0.f, 0.f, 0.f, 0.f};
        auto contract = [&](int s) __attribute__((always_inline)) {
            // D stages are in flight while there are as many left
            if (issued_left >= C::D)
                wait_vmcnt<(C::D - 1) * C::kPer>();
            else
                wait_vmcnt<0>();
            const uint8_t *base = mine + slot * C::kStage;
            i32x4 b[4], ar[4];
            uint32_t sar = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) b[q] = load16(base + r16 * 256 + 16 * ((4 * lg + q) ^ r16));
            const uint32_t sb = *reinterpret_cast<const uint32_t *>(base + 4096 + 16 * r16 + 4 * lg);
            if (GROUPED) {
#pragma unroll
                for (int q = 0; q < 4; ++q) ar[q] = load16(base + C::kSide + r16 * 256 + 16 * ((4 * lg + q) ^ r16));
                sar = *reinterpret_cast<const uint32_t *>(base + C::kSide + 4096 + 16 * r16 + 4 * lg);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read out before the slot is filled again
            advance(slot);
            slot = slot + 1 == C::D ? 0 : slot + 1;
            --issued_left;
#pragma unroll
            for (int f = 0; f < FA; ++f) {
#define LPGEMM_MX_STEP(q)                                                                                                 \
    acc[f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(mx_operand(b[q]), mx_operand(GROUPED ? ar[q] : a[f][s][q]), \
                                                              acc[f], kMxFormat, kMxFormat, q, sb, q, GROUPED ? sar : sa[f][s]);
                LPGEMM_MX_STEP(0) LPGEMM_MX_STEP(1) LPGEMM_MX_STEP(2) LPGEMM_MX_STEP(3)
#undef LPGEMM_MX_STEP
            }
        };
        if (GROUPED) {
            for (int s = 0; s < n_stages; ++s) contract(0);
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) contract(s);
        }
        cur = item_of(round);
        auto store = [&](int f, const mx_f32x4 &x) __attribute__((always_inline)) {
            const int e = GROUPED ? cur.strip / strips : 0;
            const int m = cur.m0 + 16 * f + r16;
            if (cur.m0 < 0 || m >= cur.m1) return;
            mx_store4<OUT>(g.D, (int64_t)m * g.N, 16 * (cur.strip - e * strips) + 4 * lg, g.N, x.x, x.y, x.z, x.w);
        };
        if (kw == 1) {
#pragma unroll
            for (int f = 0; f < FA; ++f) store(f, acc[f]);
            continue;
        }
#pragma unroll
        for (int f = 0; f < FA; ++f) {
            // one row tile at a time through the sums' two halves in turn
            const int half = (round * FA + f) & 1;
            sums[(half * kMxNarrowWaves + wave) * 64 + lane] = acc[f];
            lds_barrier();
            if (part == (round * FA + f) % kw) {
                mx_f32x4 x = sums[(half * kMxNarrowWaves + sub * kw) * 64 + lane];
                for (int w = 1; w < kw; ++w) x += sums[(half * kMxNarrowWaves + sub * kw + w) * 64 + lane];
                store(f, x);
            }
        }
    }
}

}  // namespace lpgemm
