// gemm_fp8_block.hpp -- products of e4m3 operands with a binary32 scale per 128
// values of a row (B: or per 128 x 128),
//     D[m][n] = out( sum_j SFA[m][j] SFB[n][j] sum_{k in block j} a[m][k] b[n][k] ),
// one pair of matrices or one matrix of B per group of rows.
//
// A block's 128 products are summed on the matrix cores from zero, and the sum
// goes into binary32 accumulators with one fused multiply-add by fl(sa sb).  16-bit
// results take v_mfma_scale_f32_*_f8f6f4, whose sums of eight products keep 13 bits
// below the largest (2e-5 of the result, a tenth of fp16's rounding); binary32
// results keep binary32 sums: their codes become bf16, which holds every e4m3
// value, and go through the bf16 matrix cores at half the rate.
#pragma once

#include "fp8_block_quantize.hpp"

namespace lpgemm {

// An operand row is U units of 128 code bytes; its scales are U floats.  Fields as
// in MxArgs, whose group and store helpers serve here too.
struct F8Args : MxArgs {
    int32_t sb_shift;  // rows of B that share a scale: 1 << sb_shift (0 or 7)
    int32_t sb_rows;   // rows of each matrix's scales
};

constexpr uint32_t kF8UnitCodes = 128, kF8UnitScales = 4;

typedef __bf16 f8_bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes of two dwords as bf16 (exact: three bits of mantissa, exponents -9 .. 8).
__device__ __forceinline__ f8_bf16x8 f8_bf16(int32_t lo, int32_t hi)
{
    const mx_bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true),
                    c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
    return f8_bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// 32 codes of a row or column, the lane's part of 64 k (32 x 32 blocks) or 128 k (16 x 16).
struct F8Frag {
    i32x4 lo, hi;
    __device__ __forceinline__ i32x8 all() const { return i32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w}; }
    __device__ __forceinline__ f8_bf16x8 part(int q) const
    {
        const i32x4 x = q < 2 ? lo : hi;
        return q % 2 ? f8_bf16(x.z, x.w) : f8_bf16(x.x, x.y);
    }
};

// p + the products of 64 k, 32 x 32.  Constant scale operands of 0 select the MFMA
// without scales, half the scaled one's code.
template <bool FINE>
__device__ __forceinline__ f32x16 f8_mfma32(const F8Frag &b, const F8Frag &a, f32x16 p)
{
    if (FINE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_32x32x16_bf16(b.part(q), a.part(q), p, 0, 0, 0);
        return p;
    }
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b.all(), a.all(), p, 0, 0, 0, 0, 0, 0);
}
// The products of 128 k, 16 x 16.
template <bool FINE>
__device__ __forceinline__ mx_f32x4 f8_mfma16(const F8Frag &b, const F8Frag &a)
{
    mx_f32x4 p = {0.f, 0.f, 0.f, 0.f};
    if (FINE) {
#pragma unroll
        for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.part(q), a.part(q), p, 0, 0, 0);
        return p;
    }
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b.all(), a.all(), p, 0, 0, 0, 0, 0, 0);
}

// ---- tiled kernel ------------------------------------------------------------
// A workgroup of four waves (2 x 2) computes tiles of 64 FM x 64 FN, FM = 1 .. HM
// chosen tile by tile from its group's rows; a wave holds FM x FN blocks of 32 x 32.
//
// A stage is one unit (128 k) of every row, one cache line.  MFMA step s takes 64 k of
// it, lane half h 32 of those.  In LDS a row's eight 16-byte chunks are permuted by
// c -> c ^ (row / 2) % 8, so that copies and reads touch all banks once.
//
// Scales come for four stages at a time, 16 bytes of every row: a copy of scattered
// rows costs a cycle for each, whatever it brings.  The window is the row's last four
// units where fewer are left.
__device__ __forceinline__ int f8_scale_window(int q, int U) { return max(0, min(4 * q, U - 4)); }
// Float of a window that belongs to unit u (past the row: another of that row's; it meets zero codes).
__device__ __forceinline__ int f8_scale_at(int u, int q, int U)
{
    const int first = f8_scale_window(q, U);
    return min(u - first, min(3, U - 1 - first));
}

template <int HM, int FN, int STAGES>
struct F8Tile {
    static_assert((FN == 1 || FN == 2) && HM <= FN && (STAGES == 2 || STAGES == 4), "heights up to HM, 64 or 128 columns");
    static constexpr int BN = 64 * FN;
    static constexpr int kStages = STAGES;
    static constexpr int NB = 2 * FN;                            // a wave's copies of B per stage
    static constexpr int copies(int fm) { return NB + 2 * fm; }  // of codes; before them one of scales, or of nothing
    static constexpr int kCodes = (BN + 64 * HM) * 128;          // of a stage: B's rows, then A's
    static constexpr int kScales = 4096;                         // of four stages: 1 KB a wave, of its 32 FN rows
    // 1 KB that nobody reads, and what the lanes hold of up to 64 groups
    static constexpr int kNowhere = kStages * kCodes + 2 * kScales, kRing = kNowhere + 1024, kGroups = 768;
    static constexpr int lds(int groups, int kgroups) { return kgroups * kRing + kGroups + 4 * (groups + 1 + 4 * kgroups); }
};

// KG == 2: eight waves, the second four on the second half of K with a ring of their
// own; their sums are added at the end, through LDS.
// ROWS: B has a scale for every row.  Binary32 results' larger tiles keep their codes' bf16
// forms too, in twice the registers: one workgroup to a compute unit.
template <int HM, int FN, int STAGES, int KG, bool ROWS, int OUT>
__global__ __launch_bounds__(256 * KG, KG == 1 && !(OUT == OUT_F32 && HM == 2) ? 2 : 1) void gemm_fp8_block_tiled_kernel(F8Args g, int tiles_n, int xcds)
{
    using T = F8Tile<HM, FN, STAGES>;
    static_assert(4 * mx_stage_bytes<OUT, FN>() <= T::kStages * T::kCodes, "the ring holds the rows on their way out");
    constexpr int ST = T::kStages;
    constexpr bool FINE = OUT == OUT_F32;
    extern __shared__ __align__(1024) uint8_t smem_all[];
    int32_t *table = reinterpret_cast<int32_t *>(smem_all + KG * T::kRing), *cum = table + T::kGroups / 4;  // [E + 1]: row tiles before group e

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
    const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
    uint8_t *smem = smem_all + kg * T::kRing;
    const int wm = wave >> 1, wn = wave & 1;
    const int r32 = lane & 31, h = lane >> 5;
    // this half's stages: k0 .. k0 + ktiles - 1, whole windows of scales
    const int U = g.U, ktiles = KG == 1 ? U : 4 * ((U + 7) / 8), k0 = kg * ktiles;
    const uint32_t ldc = (uint32_t)U * kF8UnitCodes, lds_ = (uint32_t)U * kF8UnitScales;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    MxGroups groups;
    if (g.offsets != nullptr) groups.init<4 * KG>(g, 64 * HM, cum);
    const int total = (g.offsets == nullptr ? (g.R + 64 * HM - 1) / (64 * HM) : groups.total) * tiles_n;
    // the lanes' part is put away between tiles: the K loop has few registers for it
    table[lane] = groups.begin;  // by every wave, the same
    table[64 + lane] = groups.end;
    table[128 + lane] = groups.before;

    // The current tile: group e, rows [m0, m1) of D, columns from n0, height 64 fm.
    int e = 0, m0 = 0, m1 = 0, n0 = 0, fm = 0;
    auto find = [&](int v) __attribute__((always_inline)) {
        int at = (int)threadIdx.x & 63;
        asm volatile("" : "+v"(at));
        groups.begin = table[at];
        groups.end = table[64 + at];
        groups.before = table[128 + at];
        mx_find_tile<HM, FN>(g, v, total, tiles_n, xcds, groups, e, m0, m1, n0, fm);
    };

    // Source offsets of this lane in each copy of a stage, and of its row in
    // the copy of scales: waves 0, 1 serve A's rows, 32 FN each, waves 2, 3 B's.
    i32x4 rsrc_a, rsrc_b, rsrc_s;
    uint32_t a_off[2 * HM], b_off[T::NB], s_off, s_size;
    const uint8_t *s_base;
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
        // a tile's columns lie in one block of 128 rows of B
        const int64_t srow = (int64_t)e * g.sb_rows + (ROWS ? n0 : n0 >> 7);
        s_base = wave < 2 ? g.SFA + arow * lds_ : g.SFB + srow * lds_;
        s_size = (wave < 2 ? mrows : ROWS ? nrows : 1u) * lds_;
        rsrc_s = make_rsrc(s_base, s_size);
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
        s_off = lane >= 32 * FN ? kOutOfRange : wave < 2 ? row_offset(r, lds_) : ROWS ? (uint32_t)r * lds_ : 0u;
    };

    // Copy j of stage `local`'s copies into its slot, for tiles of height 64 f.
    // Units past the row read zeros: their resources are empty.
    auto issue = [&](int j, int f, int local, uint32_t base) __attribute__((always_inline)) {
        const int kt = k0 + local;
        const uint32_t koff = (uint32_t)kt * kF8UnitCodes;
        const int i = j - T::NB, p = j < T::NB ? wave * T::NB + j : wave * 2 * f + i;
        i32x4 rsrc = j < T::NB ? rsrc_b : rsrc_a;
        rsrc.z = kt < U ? rsrc.z : 0;
        mx_dma16_at(rsrc, j < T::NB ? b_off[j < T::NB ? j : 0] : a_off[j < T::NB ? 0 : i], koff, base + (j < T::NB ? 0u : T::BN * 128u) + (uint32_t)p * 1024u);
    };
    // The scales of the window that stage `local` begins, if it begins one; else zeros to
    // nowhere: a branch in the K loop would let the compiler move the sums past it.  Rows
    // of fewer than four units have no window of 16 bytes: theirs are written by hand.
    auto issue_scales = [&](int local) __attribute__((always_inline)) {
        const int q = local >> 2, at = k0 / 4 + q;
        const bool due = (local & 3) == 0 && U >= 4;
        i32x4 rsrc = rsrc_s;
        rsrc.z = due && 4 * at < U ? rsrc.z : 0;
        mx_dma16_at(rsrc, s_off, (uint32_t)f8_scale_window(at, U) * 4u,
                    lds0 + (uint32_t)(due ? ST * T::kCodes + (q & 1) * T::kScales + wave * 1024 : T::kNowhere));
    };
    auto with_height = [&](auto body) __attribute__((always_inline)) {
        if (HM >= 2 && fm == 2) body(std::integral_constant<int, HM >= 2 ? 2 : 1>{});
        else body(std::integral_constant<int, 1>{});
    };
    auto prologue = [&]() __attribute__((always_inline)) {
        if (U < 4) {
            for (int u = 0; u < 4; ++u) {
                uint32_t x = 0;
                if (u < U && s_off < s_size) x = *reinterpret_cast<const uint32_t *>(s_base + s_off + 4 * u);
                *reinterpret_cast<uint32_t *>(smem + ST * T::kCodes + wave * 1024 + lane * 16 + 4 * u) = x;
            }
        }
        with_height([&](auto height) __attribute__((always_inline)) {
            constexpr int FM = decltype(height)::value;
#pragma unroll
            for (int st = 0; st < ST; ++st) {
                issue_scales(st);
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
        constexpr int kBlocks = FM * FN;
        wait_vmcnt<(ST - 1) * (C + 1)>();  // the first stage and its scales
        lds_barrier();

#pragma unroll
        for (int i = 0; i < FN; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

        struct Stage {
            F8Frag b[FN][2], a[FM][2];  // [block][step]
            float sa[FM], sb[ROWS ? FN * 16 : 1];
        };
        Stage x, y;
        const int swz = (r32 >> 1) & 7;
        // 16-byte read i of a stage: B's blocks, then A's, four each
        constexpr int kReads = 4 * (FM + FN);
        auto read = [&](Stage &f, int i, const uint8_t *base) __attribute__((always_inline)) {
            const int blk = i / 4, s = i / 2 % 2, c = i % 2;
            const uint32_t at = (uint32_t)r32 * 128u + 16u * (uint32_t)((4 * s + 2 * h + c) ^ swz);
            F8Frag &to = blk < FN ? f.b[blk][s] : f.a[blk - FN][s];
            const i32x4 v = load16(base + (blk < FN ? (wn * FN + blk) * 4096 : (int)kA + (wm * FM + blk - FN) * 4096) + at);
            if (c == 0) to.lo = v;
            else to.hi = v;
        };
        // row r of a half of FN blocks sits in that half's wave's kilobyte;
        // A's rows are dealt out by FN blocks whatever the tile's height
        auto read_scales = [&](Stage &f, int kt) __attribute__((always_inline)) {
            const int q = kt >> 2, d = f8_scale_at(k0 + kt, k0 / 4 + q, U);
            const uint8_t *base = smem + ST * T::kCodes + (q & 1) * T::kScales + 4 * d;
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int blk = wm * FM + i;
                f.sa[i] = *reinterpret_cast<const float *>(base + blk / FN * 1024 + (32 * (blk % FN) + r32) * 16);
            }
            if (ROWS) {
#pragma unroll
                for (int i = 0; i < 16 * FN; ++i)
                    f.sb[ROWS ? i : 0] = *reinterpret_cast<const float *>(base + (2 + wn) * 1024 +
                                                                         (32 * (i / 16) + 8 * (i / 4 % 4) + 4 * h + i % 4) * 16);
            } else {
                f.sb[0] = *reinterpret_cast<const float *>(base + 2 * 1024);
            }
        };
        read_scales(x, 0);
#pragma unroll
        for (int i = 0; i < kReads; ++i) read(x, i, smem);

        // Stage kt from cur: the next one's reads go out between the MFMAs, and the copies
        // that refill this one's slot, which all waves have read out before the barrier.
        int slot = 0;
        auto stage = [&](const Stage &cur, Stage &nxt, int kt) __attribute__((always_inline)) {
            wait_vmcnt<(ST - 2) * (C + 1)>();  // the next stage and its scales
            lds_barrier();
            const uint32_t refill = lds0 + (uint32_t)(slot * T::kCodes);
            slot = slot + 1 == ST ? 0 : slot + 1;
            const uint8_t *next = smem + slot * T::kCodes;
            issue_scales(kt + ST);
            read_scales(nxt, kt + 1);
            constexpr int kPer = (kReads + kBlocks - 1) / kBlocks;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const int fn = b / FM, f = b % FM;
                f32x16 p = f8_mfma32<FINE>(cur.b[fn][0], cur.a[f][0], f32x16{});
#pragma unroll
                for (int i = 0; i < kReads; ++i)
                    if (i / kPer == b) read(nxt, i, next);
                p = f8_mfma32<FINE>(cur.b[fn][1], cur.a[f][1], p);
#pragma unroll
                for (int j = 0; j < C; ++j)
                    if (j >= b * C / kBlocks && j < (b + 1) * C / kBlocks) issue(j, FM, kt + ST, refill);
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    acc[fn][f][i] = __builtin_fmaf(p[i], cur.sa[f] * cur.sb[ROWS ? 16 * fn + i : 0], acc[fn][f][i]);
            }
        };
        int kt = 0;
        for (; kt + 1 < ktiles; kt += 2) {
            stage(x, y, kt);
            stage(y, x, kt + 1);
        }
        if (kt < ktiles) stage(x, y, kt);
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
// Tiles of 64 FM x 256, FM = 1 .. 4 by the group's rows, one workgroup of eight waves (2
// x 4) per compute unit; a wave holds FM x 2 blocks of 32 x 32 (FM = 4: 128 accumulators,
// which the scaling's fused multiply-adds need in plain registers, two waves a SIMD).
//
// A stage is one unit (128 k), two slots.  A wave keeps its two blocks of B for the stage
// and reads its FM blocks of A one ahead.  Block FM - 1 of a stage is contracted while the
// next stage's first blocks are read, behind a barrier: there the next stage has landed, and
// this one's A has been read out by all waves and is filled again; its B has been since the
// second block, behind a barrier of its own.  Copies go out one or two between two blocks of
// MFMAs all through the stage: 8192^3 takes 475 us with all of them behind the one barrier,
// 443 with B's behind the other, two at a time, 435 so; asked for half a stage earlier
// still, but three at a time, 465.  A block's sum is scaled and added while the next
// block's MFMAs run.
//
// Bound by the power that the matrix cores draw and by what the waves wait for at the
// barriers: 8192^3 435 us (2.53 PFLOP/s; the library's product with one scale for a whole
// matrix 359), the matrix cores busy 68% of the cycles at 1.63 GHz; 16384 rows on 32 groups
// of 4096 x 4096 292 us.  Dealing the groups' tiles out by height, tallest first, evened the
// workgroups' rows and cost what they share in the L2: 305 -> 323 us.
struct F8Large {
    // Codes: 32 KB a slot for A, then for B (a slot and block fit a read's offset field);
    // scales: 4 KB a window for A's rows and 1 KB for B's; 1 KB that nobody reads; what
    // the lanes hold of up to 64 groups.
    static constexpr int kSlot = 32768, kB = 2 * kSlot, kScales = 4 * kSlot, kScaleSlot = 4096 + 1024;
    static constexpr int kNowhere = kScales + 2 * kScaleSlot, kGroups = kNowhere + 1024, kTables = kGroups + 768;
    static constexpr int lds(int groups) { return kTables + 4 * (groups + 1 + 8); }
    static constexpr int kMinUnits = 4;
};

template <int OUT>
__global__ __launch_bounds__(512, 1) void gemm_fp8_block_large_kernel(F8Args g, int tiles_n, int xcds)
{
    using C = F8Large;
    static_assert(OUT != OUT_F32, "binary32 sums' operands take more registers than are left");
    extern __shared__ __align__(1024) uint8_t smem[];
    int32_t *cum = reinterpret_cast<int32_t *>(smem + C::kTables);

    // computed afresh where it is used: kept through the K loop it would not fit the registers
    auto opaque_lane = [&]() __attribute__((always_inline)) {
        int l = (int)threadIdx.x & 63;
        asm volatile("" : "+v"(l));
        return l;
    };
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const int U = g.U;
    const uint32_t ldc = (uint32_t)U * kF8UnitCodes, lds_ = (uint32_t)U * kF8UnitScales;
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem);

    MxGroups groups;
    if (g.offsets != nullptr) groups.init<8>(g, 256, cum);
    const int total = (g.offsets == nullptr ? (g.R + 255) / 256 : groups.total) * tiles_n;
    // the lanes' part is put away between tiles: the K loop has no registers for it
    int32_t *held = reinterpret_cast<int32_t *>(smem + C::kGroups) + (threadIdx.x & 63);
    held[0] = groups.begin;  // by every wave, the same
    held[64] = groups.end;
    held[128] = groups.before;

    // The current tile: group e, rows [m0, m1) of D, columns from n0, height 64 fm.
    int e = 0, m0 = 0, m1 = 0, n0 = 0, fm = 0;
    auto find = [&](int v) __attribute__((always_inline)) {
        const int32_t *held = reinterpret_cast<const int32_t *>(smem + C::kGroups) + opaque_lane();
        groups.begin = held[0];
        groups.end = held[64];
        groups.before = held[128];
        mx_find_tile<4, 4>(g, v, total, tiles_n, xcds, groups, e, m0, m1, n0, fm);
    };

    // This wave's copies of a stage: rows 32 wave .. + 31 of B, 8 fm wave .. of A; of a
    // window of scales waves 0 .. 3 64 rows of A each, wave 4 B's.
    i32x4 rsrc_a, rsrc_b, rsrc_s;
    uint32_t a_off[4], b_off[2], s_off;
    auto place = [&]() __attribute__((always_inline)) {
        const int lane = opaque_lane();
        const int64_t brow = (int64_t)e * g.N + n0;
        const uint32_t nrows = (uint32_t)min(256, g.N - n0);
        const int64_t arow = g.rows == nullptr ? m0 : 0;
        const uint32_t mrows = (uint32_t)(g.rows == nullptr ? m1 - m0 : g.T);
        rsrc_b = make_rsrc(g.B + brow * ldc, nrows * ldc);
        rsrc_a = make_rsrc(g.A + arow * ldc, mrows * ldc);
        const int64_t srow = (int64_t)e * g.sb_rows + (n0 >> 7);
        rsrc_s = make_rsrc(wave < 4 ? g.SFA + arow * lds_ : g.SFB + srow * lds_, (wave < 4 ? mrows : (nrows + 127) / 128) * lds_);
        auto row = [&](int r) __attribute__((always_inline)) -> int {  // source row of tile row r of A, or -1
            if (r >= 64 * fm) return -1;
            if (g.rows == nullptr) return r;
            const int at = m0 + r < m1 ? g.rows[m0 + r] : -1;
            return at < g.T ? at : -1;
        };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c < 2) b_off[c] = (uint32_t)(32 * wave + 8 * c + (lane >> 3)) * ldc + 16u * (uint32_t)((lane & 7) ^ ((4 * c + (lane >> 4)) & 7));
            // copy c of A brings rows 8 p .. 8 p + 7, p = fm wave + c
            const int p = fm * wave + c, at = c < fm ? row(8 * p + (lane >> 3)) : -1;
            a_off[c] = at >= 0 ? (uint32_t)at * ldc + 16u * (uint32_t)((lane & 7) ^ ((4 * p + (lane >> 4)) & 7)) : kOutOfRange;
        }
        const int at = wave < 4 ? row(64 * wave + lane) : wave == 4 && lane < 2 ? lane : -1;
        s_off = at >= 0 ? (uint32_t)at * lds_ : kOutOfRange;
    };
    // Copies of stage k; stages past the row read zeros from a resource without bytes.
    auto copy_b = [&](int c, int k) __attribute__((always_inline)) {
        i32x4 rsrc = rsrc_b;
        rsrc.z = k < U ? rsrc.z : 0;
        // copies 2 and 3: 16 rows on, the same chunks
        mx_dma16_at(rsrc, b_off[c & 1] + (c < 2 ? 0u : 16u * ldc), (uint32_t)k * kF8UnitCodes,
                    lds0 + (uint32_t)(C::kB + (k & 1) * C::kSlot + (4 * wave + c) * 1024));
    };
    auto copy_a = [&](int c, int k) __attribute__((always_inline)) {
        i32x4 rsrc = rsrc_a;
        rsrc.z = k < U ? rsrc.z : 0;
        mx_dma16_at(rsrc, a_off[c], (uint32_t)k * kF8UnitCodes, lds0 + (uint32_t)((k & 1) * C::kSlot + (fm * wave + c) * 1024));
    };
    // The window that stage k begins, if it begins one, by waves 0 .. 4; else zeros to
    // nowhere: a branch in the K loop would let the compiler move the sums past it.
    auto copy_scales = [&](int k) __attribute__((always_inline)) {
        const int q = k >> 2;
        const bool due = (k & 3) == 0 && wave < 5;
        i32x4 rsrc = rsrc_s;
        rsrc.z = due && k < U ? rsrc.z : 0;
        mx_dma16_at(rsrc, s_off, (uint32_t)f8_scale_window(q, U) * 4u,
                    lds0 + (uint32_t)(due ? C::kScales + (q & 1) * C::kScaleSlot + wave * 1024 : C::kNowhere));
    };
    auto begin_stage = [&](int k) __attribute__((always_inline)) {
        if (k == 0) copy_scales(0);
#pragma unroll
        for (int c = 0; c < 4; ++c) copy_b(c, k);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            if (c < fm && (k == 0 || c < 2)) copy_a(c, k);  // the second stage's others: in the first
    };

    int v = blockIdx.x;
    if (v >= total) return;
    find(v);
    place();
    begin_stage(0);
    begin_stage(1);

    auto run_tile = [&](auto height) __attribute__((always_inline)) {
        constexpr int FM = decltype(height)::value;
        const int lane = opaque_lane(), r32 = lane & 31, h = lane >> 5;
        f32x16 acc[2][FM];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < FM; ++j) acc[i][j] = f32x16{};

        F8Frag fb[2][2], fa[2][2];  // [block][step]; A's in turn
        float s[FM], waiting = 0.f;  // a stage's scales; the waiting sum's
        f32x16 p[2];
        // this lane's chunks of a row of A: 4 step + 2 h + half, permuted
        uint32_t at[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            at[q] = (uint32_t)(wm * FM * 4096 + r32 * 128 + 16 * ((4 * (q >> 1) + 2 * h + (q & 1)) ^ ((r32 >> 1) & 7)));
        auto read = [&](F8Frag (&f)[2], int q, uint32_t from, int slot) __attribute__((always_inline)) {
            const i32x4 x = load16(smem + from + slot);
            if (q & 1) f[q >> 1].hi = x;
            else f[q >> 1].lo = x;
        };
        auto read_a = [&](F8Frag (&f)[2], int q, int j, int odd) __attribute__((always_inline)) { read(f, q, at[q], odd * C::kSlot + j * 4096); };
        // B's are as far behind them for every lane
        auto read_b = [&](int i, int odd) __attribute__((always_inline)) {
            uint32_t behind = (uint32_t)(C::kB + wn * 8192 - wm * FM * 4096);
            asm volatile("" : "+s"(behind));  // four more registers through the loop would not fit
#pragma unroll
            for (int q = 0; q < 4; ++q) read(fb[i], q, at[q] + behind, odd * C::kSlot + i * 4096);
        };
        auto read_scales = [&](float (&to)[FM], int k) __attribute__((always_inline)) {
            const int q = k >> 2, d = f8_scale_at(k, q, U);
            const uint8_t *base = smem + C::kScales + (q & 1) * C::kScaleSlot + 4 * d;
            const float sb = *reinterpret_cast<const float *>(base + 4096 + 16 * (wn >> 1));
#pragma unroll
            for (int j = 0; j < FM; ++j) to[j] = *reinterpret_cast<const float *>(base + (32 * (wm * FM + j) + r32) * 16) * sb;
        };

        wait_vmcnt<4 + (FM < 2 ? FM : 2)>();
        lds_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) read_a(fa[0], q, 0, 0);
        read_b(0, 0);
        read_b(1, 0);
        read_scales(s, 0);
        p[1] = f32x16{};  // the block before the first: nothing

        // Stage k, its parity ODD; A's block j sits in fa[(ODD * FM + j) & 1].
        auto stage = [&](auto parity, int k) __attribute__((always_inline)) {
            constexpr int ODD = decltype(parity)::value;
#pragma unroll
            for (int j = 0; j < FM; ++j) {
                constexpr int kTurn = ODD * FM;
                F8Frag(&cur)[2] = fa[(kTurn + j) & 1];
                F8Frag(&nxt)[2] = fa[(kTurn + j + 1) & 1];
                const bool last = j == FM - 1;
                if (last) {
                    // the next stage has landed; the copies of B behind it stay in flight
                    wait_vmcnt<FM == 1 ? 0 : 4>();
                    lds_barrier();
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    // every wave has read this stage's B
                    if (FM == 2 ? j == 0 && i == 1 : j == 1 && FM > 2 && i == 0) lds_barrier();
                    // the block before this one: its sum, accumulator and scale
                    const int pj = i == 1 ? j : j == 0 ? FM - 1 : j - 1, pi = 1 - i;
                    const float ps = i == 1 || j > 0 ? s[pj] : waiting;
                    p[i] = f8_mfma32<false>(fb[i][0], cur[0], f32x16{});
                    __builtin_amdgcn_sched_barrier(0);
                    read_a(nxt, 2 * i, last ? 0 : j + 1, last ? 1 - ODD : ODD);
                    read_a(nxt, 2 * i + 1, last ? 0 : j + 1, last ? 1 - ODD : ODD);
#pragma unroll
                    for (int r = 0; r < 8; ++r) acc[pi][pj][r] = __builtin_fmaf(p[pi][r], ps, acc[pi][pj][r]);
                    __builtin_amdgcn_sched_barrier(0);
                    p[i] = f8_mfma32<false>(fb[i][1], cur[1], p[i]);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int r = 8; r < 16; ++r) acc[pi][pj][r] = __builtin_fmaf(p[pi][r], ps, acc[pi][pj][r]);
                    if (FM > 2 && j == 0 && 2 + i < FM) copy_a(2 + i, k + 1);
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        if (FM == 4 ? j == 1 + c / 2 && i == c % 2 : FM == 3 ? j == 1 && i == c / 2 : FM == 2 && j == 0 && i == 1) copy_b(c, k + 2);
                    if (last) {
                        read_b(i, 1 - ODD);
                        if (i == 0) {
                            waiting = s[FM - 1];
                            copy_scales(k + 2);
                        } else {
                            read_scales(s, k + 1);
                        }
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            if (c < FM && c < 2 && c == i) copy_a(c, k + 2);
                            if (FM == 1 && c / 2 == i) copy_b(c, k + 2);
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        };
        using even = std::integral_constant<int, 0>;
        using odd = std::integral_constant<int, 1>;
        int k = 0;
        for (; k + 1 < U; k += 2) {
            stage(even{}, k);
            stage(odd{}, k + 1);
        }
        if (k < U) stage(even{}, k);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[1][FM - 1][r] = __builtin_fmaf(p[1][r], waiting, acc[1][FM - 1][r]);
        wait_vmcnt<0>();  // copies past the last stage

        const int tm0 = m0, tm1 = m1, tn0 = n0;
        v += (int)gridDim.x;
        lds_barrier();  // every wave is done with the ring
        // the next tile's first stage is on its way while the rows leave through the second slot
        const bool more = v < total;
        if (more) {
            find(v);
            place();
            begin_stage(0);
        }
        static_assert(4 * mx_stage_bytes<OUT, 2>() <= C::kSlot, "half of the second slot holds four waves' rows");
        uint8_t *out_stage = smem + C::kSlot + wn * mx_stage_bytes<OUT, 2>() + wm * C::kB;
#pragma unroll
        for (int f = 0; f < FM; ++f)
            mx_store_rows<OUT, 2>(g, out_stage, [&](int w) -> const f32x16 & { return acc[w][f]; }, tm0 + (wm * FM + f) * 32, tm1, tn0 + wn * 64);
        if (!more) return;
        lds_barrier();  // every wave's rows have left
        begin_stage(1);
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
// Few rows of A: bound by reading B once.  A workgroup of eight waves takes strips of
// 16 rows of B; KW neighbouring waves split a strip's K, and 8 / KW strips are worked
// on at a time.  Every wave streams its own part: a stage is 16 rows x 2 units (256
// contiguous bytes a row, 4 KB of codes, and their scales) copied straight into the
// wave's own ring of D slots, so no wave waits for another's copies.  The 16 x 16 x 128
// MFMA takes a unit whole, 32 of its codes in lane group g.  In LDS chunk c of row r
// sits at c ^ r.  The KW partial tiles are added in LDS in a fixed order, by the
// subgroup's waves in turn.
//
// A stays in registers (16 FA rows, S stages a wave; more rows are the grid's second
// dimension) or, with RING (groups: tiles of up to 16 rows of one group, gathered;
// and long K), comes through the ring beside B.
constexpr int kF8NarrowUnits = 2;  // of a stage

template <bool RING>
struct F8Narrow {
    static constexpr int kSide = 4096 + 256;                     // a stage's codes and scales
    static constexpr int kStage = kSide * (RING ? 2 : 1);
    static constexpr int kPer = RING ? 10 : 5;                   // copies of a stage
    static constexpr int D = RING ? 2 : 4;
    static constexpr int kRing = kMxNarrowWaves * D * kStage;
    static constexpr int kSums = 2 * kMxNarrowWaves * 64 * 16;
    static constexpr int lds(int groups) { return kRing + kSums + (RING ? 4 * (2 * groups + 1 + kMxNarrowWaves + kMxNarrowRows) : 0); }
};

template <int FA, int S, bool RING, int OUT>
__global__ __launch_bounds__(64 * kMxNarrowWaves) void gemm_fp8_block_narrow_kernel(F8Args g, int kw, int stages)
{
    static_assert(!RING || (FA == 1 && S == 1), "ring: one row tile, stages counted at run time");
    using C = F8Narrow<RING>;
    constexpr bool FINE = OUT == OUT_F32;
    const bool grouped = RING && g.offsets != nullptr;
    if (!RING) {  // a workgroup's row tile, as a product of its own
        const int m0 = (int)blockIdx.y * 16 * FA;
        g.A += (int64_t)m0 * g.U * kF8UnitCodes;
        g.SFA += (int64_t)m0 * g.U * kF8UnitScales;
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
    const int n_stages = RING ? stages : S;
    const uint32_t ldc = (uint32_t)U * kF8UnitCodes, lds_ = (uint32_t)U * kF8UnitScales;
    const uint32_t ring = (uint32_t)(wave * C::D * C::kStage);
    const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(smem) + ring;
    const uint8_t *mine = smem + ring;

    int items = strips * (RING ? (g.R + 15) / 16 : 1);
    MxGroups groups;
    if (grouped) {
        if (g.rows != nullptr)
            for (int i = threadIdx.x; i < g.R; i += 64 * kMxNarrowWaves) index[i] = g.rows[i];
        groups.init<kMxNarrowWaves>(g, 16, cum, bounds);
        items = groups.total * strips;
        __syncthreads();  // the indices
    }
    const int rounds = (items - (int)blockIdx.x * side_by_side + (int)gridDim.x * side_by_side - 1) / ((int)gridDim.x * side_by_side);
    if (rounds <= 0) return;

    // This lane's part of each copy: rows 4 t + lg, chunk r16 ^ row of its 256 bytes;
    // scales: lane 2 r + u takes row r's of unit u (where 128 rows share one, every
    // row's is that), the upper lanes none.
    uint32_t b_off[4], chunk[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        chunk[t] = (uint32_t)(r16 ^ (4 * t + lg));
        b_off[t] = (uint32_t)(4 * t + lg) * ldc + 16u * chunk[t];
    }
    const int s_row = lane >> 1, s_unit = lane & 1;  // s_row above 15: none
    const uint32_t sb_off = s_row > 15 ? kOutOfRange : (g.sb_shift != 0 ? 0u : (uint32_t)s_row * lds_) + 4u * (uint32_t)s_unit;

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
        if (RING && id < items) {
            int begin = 0, end = g.R, first = 0, e = 0;
            if (grouped) e = groups.of(g, id / strips, begin, end, first);
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
    if (grouped) {
        rsrc_a = make_rsrc(g.A, (uint32_t)g.T * ldc);
        rsrc_sa = make_rsrc(g.SFA, (uint32_t)g.T * lds_);
    }
    auto aim = [&](const Item &it) __attribute__((always_inline)) {
        const int e = grouped ? it.strip / strips : 0, n0 = 16 * (it.strip - e * strips);
        const int64_t brow = (int64_t)e * g.N + n0, srow = (int64_t)e * g.sb_rows + (n0 >> g.sb_shift);
        const uint32_t n = it.m0 < 0 ? 0u : (uint32_t)min(16, g.N - n0);
        rsrc_b = make_rsrc(g.B + brow * ldc, n * ldc);
        rsrc_sb = make_rsrc(g.SFB + srow * lds_, (g.sb_shift != 0 ? min(n, 1u) : n) * lds_);
        if (RING) {
            const int64_t arow = grouped ? 0 : max(it.m0, 0);  // a product's rows from its tile on: any size
            if (!grouped) {
                const uint32_t m = it.m0 < 0 ? 0u : (uint32_t)(it.m1 - it.m0);
                rsrc_a = make_rsrc(g.A + arow * ldc, m * ldc);
                rsrc_sa = make_rsrc(g.SFA + arow * lds_, m * lds_);
            }
            auto row = [&](int r) __attribute__((always_inline)) -> int {
                if (it.m0 < 0 || it.m0 + r >= it.m1) return -1;
                if (!grouped) return r;
                const int at = g.rows == nullptr ? it.m0 + r : index[it.m0 + r];
                return at < g.T ? at : -1;
            };
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int at = row(4 * t + lg);
                a_off[t] = at >= 0 ? (uint32_t)at * ldc + 16u * chunk[t] : kOutOfRange;
            }
            const int at = s_row > 15 ? -1 : row(s_row);
            sa_off = at >= 0 ? (uint32_t)at * lds_ + 4u * (uint32_t)s_unit : kOutOfRange;
        }
    };
    auto issue = [&](int s, int slot) __attribute__((always_inline)) {
        const int u0 = kF8NarrowUnits * (part * n_stages + s);
        const uint32_t base = lds0 + (uint32_t)(slot * C::kStage);
        const uint32_t koff = (uint32_t)u0 * kF8UnitCodes, soff = (uint32_t)u0 * kF8UnitScales;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            mx_dma16_nt(rsrc_b, u0 + (int)(chunk[t] >> 3) < U ? b_off[t] + koff : kOutOfRange, base + (uint32_t)t * 1024u);
        mx_dma4(rsrc_sb, u0 + s_unit < U ? sb_off + soff : kOutOfRange, base + 4096u);
        if (RING) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
                mx_dma16(rsrc_a, u0 + (int)(chunk[t] >> 3) < U ? a_off[t] + koff : kOutOfRange, base + C::kSide + (uint32_t)t * 1024u);
            mx_dma4(rsrc_sa, u0 + s_unit < U ? sa_off + soff : kOutOfRange, base + C::kSide + 4096u);
        }
    };

    // A in registers: lane (r16, lg), unit u: codes 32 lg .. 32 lg + 31, one scale.
    F8Frag a[FA][S][kF8NarrowUnits];
    float sa[FA][S][kF8NarrowUnits];
    if (!RING) {
        const __amdgpu_buffer_rsrc_t ra = buffer_rsrc(g.A, (uint32_t)g.R * ldc);
        const __amdgpu_buffer_rsrc_t rsa = buffer_rsrc(g.SFA, (uint32_t)g.R * lds_);
#pragma unroll
        for (int f = 0; f < FA; ++f)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int q = 0; q < kF8NarrowUnits; ++q) {
                    const int u = kF8NarrowUnits * (part * S + s) + q;
                    const uint32_t row = (uint32_t)(16 * f + r16);
                    const bool in = u < U && (int)row < g.R;
                    const uint32_t at = in ? row * ldc + (uint32_t)u * kF8UnitCodes + 32u * (uint32_t)lg : kOutOfRange;
                    a[f][s][q].lo = buffer_load16(ra, at);
                    a[f][s][q].hi = buffer_load16(ra, in ? at + 16u : kOutOfRange);
                    sa[f][s][q] = __int_as_float((int)__builtin_amdgcn_raw_buffer_load_b32(rsa, in ? row * lds_ + (uint32_t)u * kF8UnitScales : kOutOfRange, 0, 0));
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
#pragma unroll
    for (int d = 0; d < C::D; ++d) advance(d);
    if (!RING) {
        // A is waited for here, once
#pragma unroll
        for (int f = 0; f < FA; ++f)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int q = 0; q < kF8NarrowUnits; ++q) {
                    asm volatile("" : "+v"(sa[f][s][q]));
                    asm volatile("" : "+v"(a[f][s][q].lo));
                    asm volatile("" : "+v"(a[f][s][q].hi));
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
            F8Frag b[kF8NarrowUnits], ar[kF8NarrowUnits];
            float sar[kF8NarrowUnits];
            // both units' scales of rows 4 lg .. 4 lg + 3, two floats a row
            const i32x4 t0 = load16(base + 4096 + 32 * lg), t1 = load16(base + 4096 + 32 * lg + 16);
#pragma unroll
            for (int q = 0; q < kF8NarrowUnits; ++q) {
                const int c = 8 * q + 2 * lg;
                b[q].lo = load16(base + r16 * 256 + 16 * (c ^ r16));
                b[q].hi = load16(base + r16 * 256 + 16 * ((c + 1) ^ r16));
                if (RING) {
                    ar[q].lo = load16(base + C::kSide + r16 * 256 + 16 * (c ^ r16));
                    ar[q].hi = load16(base + C::kSide + r16 * 256 + 16 * ((c + 1) ^ r16));
                    sar[q] = *reinterpret_cast<const float *>(base + C::kSide + 4096 + 8 * r16 + 4 * q);
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read out before the slot is filled again
            advance(slot);
            slot = slot + 1 == C::D ? 0 : slot + 1;
            --issued_left;
#pragma unroll
            for (int q = 0; q < kF8NarrowUnits; ++q) {
                const float sb[4] = {__int_as_float(q ? t0.y : t0.x), __int_as_float(q ? t0.w : t0.z), __int_as_float(q ? t1.y : t1.x),
                                     __int_as_float(q ? t1.w : t1.z)};
#pragma unroll
                for (int f = 0; f < FA; ++f) {
                    const mx_f32x4 p = f8_mfma16<FINE>(b[q], RING ? ar[q] : a[f][s][q]);
                    const float sf = RING ? sar[q] : sa[f][s][q];
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[f][i] = __builtin_fmaf(p[i], sf * sb[i], acc[f][i]);
                }
            }
        };
        if (RING) {
            for (int s = 0; s < n_stages; ++s) contract(0);
        } else {
#pragma unroll
            for (int s = 0; s < S; ++s) contract(s);
        }
        cur = item_of(round);
        auto store = [&](int f, const mx_f32x4 &x) __attribute__((always_inline)) {
            const int e = grouped ? cur.strip / strips : 0;
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
