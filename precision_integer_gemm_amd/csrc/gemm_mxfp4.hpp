// gemm_mxfp4.hpp -- products of microscaled 4-bit float operands,
//     D[m][n] = out( sum_j 2^(sa[m][j] - 127) 2^(sb[n][j] - 127) sum_{k in block j} a[m][k] b[n][k] )
// over blocks of 32 k, one pair of matrices or one matrix of B per group of
// rows.  gfx950's v_mfma_scale_f32_*_f8f6f4 multiplies e2m1 operands with one
// e8m0 scale byte per row and block: the format's definition, in one instruction.
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

// Group e's rows [begin, end), each offset taken into [0, R].
__device__ __forceinline__ void mx_group(const MxArgs &g, int e, int &begin, int &end)
{
    begin = 0;
    end = g.R;
    if (g.offsets != nullptr) {
        begin = min(max(g.offsets[e], 0), g.R);
        end = min(max(g.offsets[e + 1], begin), g.R);
    }
}

__device__ __forceinline__ i32x8 mx_operand(i32x4 c) { return i32x8{c.x, c.y, c.z, c.w, 0, 0, 0, 0}; }

// One wave per 32 x 32 block of D, operands straight from memory: lane l holds
// row l % 32 of each operand and, of every 128-k unit, the two blocks
// 2 (l / 32) and 2 (l / 32) + 1, one per MFMA.  B is the MFMA's row operand,
// so a lane ends with four consecutive n of one m.
template <int OUT>
__global__ __launch_bounds__(256) void gemm_mxfp4_simple_kernel(MxArgs g)
{
    const int lane = threadIdx.x & 63;
    const int r32 = lane & 31, h = lane >> 5;
    const int e = blockIdx.z;
    const int n0 = ((int)blockIdx.x * 4 + (int)(threadIdx.x >> 6)) * 32;
    int begin, end;
    mx_group(g, e, begin, end);
    if (n0 >= g.N) return;
    const int64_t brow = (int64_t)e * g.N + min(n0 + r32, g.N - 1);
    const uint8_t *pb = g.B + brow * g.U * kMxUnitCodes + 32 * h;
    const uint8_t *psb = g.SFB + brow * g.U * kMxUnitScales;
    for (int m0 = begin + (int)blockIdx.y * 32; m0 < end; m0 += (int)gridDim.y * 32) {
        const int m = m0 + r32;
        int64_t arow = min(m, end - 1);
        if (g.rows != nullptr) arow = g.rows[arow];
        const bool live = arow >= 0 && arow < g.T;
        if (!live) arow = 0;
        const uint8_t *pa = g.A + arow * g.U * kMxUnitCodes + 32 * h;
        const uint8_t *psa = g.SFA + arow * g.U * kMxUnitScales;
        f32x16 acc = {};
        for (int u = 0; u < g.U; ++u) {
            uint32_t sa = *reinterpret_cast<const uint32_t *>(psa + u * 4) >> (16 * h);
            const uint32_t sb = *reinterpret_cast<const uint32_t *>(psb + u * 4) >> (16 * h);
            if (!live) sa = 0;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                i32x4 a = load16(pa + u * kMxUnitCodes + 16 * s);
                if (!live) a = i32x4{0, 0, 0, 0};
                const i32x4 b = load16(pb + u * kMxUnitCodes + 16 * s);
                if (s == 0)
                    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(b), mx_operand(a), acc, kMxFormat,
                                                                          kMxFormat, 0, sb, 0, sa);
                else
                    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(mx_operand(b), mx_operand(a), acc, kMxFormat,
                                                                          kMxFormat, 1, sb, 1, sa);
            }
        }
        if (m < end) {
            Epilogue epi{g.D, nullptr, nullptr};
#pragma unroll
            for (int rg = 0; rg < 4; ++rg) {
                const float v[4] = {acc[4 * rg], acc[4 * rg + 1], acc[4 * rg + 2], acc[4 * rg + 3]};
                store_row4f<OUT>(epi, m, g.N, n0 + 8 * rg + 4 * h, v);
            }
        }
    }
}

}  // namespace lpgemm
