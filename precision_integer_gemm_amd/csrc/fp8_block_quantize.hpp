// fp8_block_quantize.hpp -- to and from e4m3 codes with one binary32 scale for
// each block of 128 values of a row, or of 128 x 128 values.
//
// A row of K values becomes U = ceil(K / 128) units of 128 code bytes, zeros
// past K.  For a block with a = max |x| and l = max(a, 2^-100),
//     s = fl(l / 448), or the smallest power of two with l / s <= 448,
//     code = e4m3(fl(x * fl(1 / s)))      fl: binary32, nearest even
// The largest value lands on 448 (the last step's error of 2^-23 is far below
// the next code's border at 464), so nothing saturates; 2^-100 keeps 1 / s
// finite.  A block that holds a NaN or an infinity gets s = NaN and codes 0.
#pragma once

#include "gemm_mxfp4.hpp"

namespace lpgemm {

constexpr int kF8Unit = 128;  // values, and code bytes, of a row per unit
constexpr float kF8Most = 448.f;

// The largest of 16 neighbouring lanes, in all of them.
__device__ __forceinline__ uint32_t f8_largest16(uint32_t a)
{
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x128, 0xF, 0xF, false));  // row_ror:8, 4, 2, 1
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x124, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x122, 0xF, 0xF, false));
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x121, 0xF, 0xF, false));
    return a;
}

// The binary32 value of a magnitude's bits in IN.
template <int IN>
__device__ __forceinline__ float f8_value(uint32_t a)
{
    if (IN == OUT_F32) return __uint_as_float(a);
    if (IN == OUT_BF16) return __uint_as_float(a << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)a);
}

// A block's scale and its inverse; not finite: (NaN, -) and false.
template <bool POW2>
__device__ __forceinline__ bool f8_scale(float a, float &scale, float &inverse)
{
    const bool fine = __float_as_uint(a) < 0x7F800000u;
    const float l = fmaxf(a, 0x1p-100f);
    if (POW2) {
        // 448 = 1.75 2^8: l = m 2^e takes 2^(e - 8), or twice that above 1.75
        const uint32_t u = __float_as_uint(l);
        scale = __uint_as_float((u & 0x7F800000u) + ((u & 0x007FFFFFu) > 0x00600000u ? (1u << 23) : 0u) - (8u << 23));
    } else {
        scale = __fdiv_rn(l, kF8Most);
    }
    inverse = __fdiv_rn(1.f, scale);
    if (!fine) scale = __uint_as_float(0x7FC00000u);
    return fine;
}

// Value j of eight.
template <int IN>
__device__ __forceinline__ float f8_element(const u32x4 (&w)[2], int j)
{
    if (IN == OUT_F32) return __uint_as_float(w[j / 4][j % 4]);
    const uint32_t d = w[0][j / 2];
    if (IN == OUT_BF16) return __uint_as_float(j % 2 ? d & 0xFFFF0000u : d << 16);
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(j % 2 ? d >> 16 : d));
}

// Eight codes of the values times `inverse`.
template <int IN>
__device__ __forceinline__ uint64_t f8_codes(const u32x4 (&w)[2], float inverse)
{
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int d = 0;
        d = __builtin_amdgcn_cvt_pk_fp8_f32(f8_element<IN>(w, 4 * h) * inverse, f8_element<IN>(w, 4 * h + 1) * inverse, d, false);
        d = __builtin_amdgcn_cvt_pk_fp8_f32(f8_element<IN>(w, 4 * h + 2) * inverse, f8_element<IN>(w, 4 * h + 3) * inverse, d, true);
        c[h] = (uint32_t)d;
    }
    return (uint64_t)c[1] << 32 | c[0];
}

// One row to a block.  A workgroup takes 256 items of eight values; 16 neighbouring lanes
// share a block.  `items` = 16 units of a row.  Bound by memory: 8192 x 8192 fp32 57.8 us
// (5.8 TB/s), bf16 37.3; four items a thread took 60.9 and 39.7, 1001 x 2897 fp32 3.8 for 3.2.
template <int IN, bool NT, bool POW2>
__global__ __launch_bounds__(256) void fp8_block_quantize_kernel(const void *__restrict__ X, int64_t ldx, uint64_t *__restrict__ codes,
                                                                 float *__restrict__ scales, int64_t rows, int32_t K, uint32_t items)
{
    const int64_t total = rows * items;  // a multiple of 16
    const int64_t first = (int64_t)blockIdx.x * 256, i = first + threadIdx.x;
    const int64_t row0 = first / items;
    const MxItem it = mx_item(row0, (uint32_t)(first - row0 * items) + threadIdx.x, items);
    u32x4 w[2];
    mx_load8<IN, NT>(X, it.row * ldx + it.k0, i < total ? K - it.k0 : 0, w);
    float scale, inverse;
    const bool fine = f8_scale<POW2>(f8_value<IN>(f8_largest16(mx_largest<IN>(w))), scale, inverse);
    const uint64_t c = fine ? f8_codes<IN>(w, inverse) : 0u;
    if (i < total) {
        codes[i] = c;
        if ((i & 15) == 0) scales[i >> 4] = scale;
    }
}

// 128 rows to a block: a workgroup takes one block, 16 lanes to a row's 128
// values, and holds it in registers between the maximum and the codes.  Bound by memory:
// 8192 x 8192 fp32 57.3 us (5.9 TB/s).
template <int IN, bool NT, bool POW2>
__global__ __launch_bounds__(256) void fp8_block_quantize_square_kernel(const void *__restrict__ X, int64_t ldx, uint64_t *__restrict__ codes,
                                                                        float *__restrict__ scales, int64_t rows, int32_t K, uint32_t units)
{
    __shared__ uint32_t part[4];
    const uint32_t tile = blockIdx.x / units, unit = blockIdx.x - tile * units;
    const int sub = threadIdx.x >> 4, k0 = (int)(unit * kF8Unit) + 8 * (int)(threadIdx.x & 15);
    const int64_t r0 = (int64_t)tile * kF8Unit + sub;
    u32x4 w[8][2];
    uint32_t a = 0;
#pragma unroll
    for (int p = 0; p < 8; ++p) mx_load8<IN, NT>(X, (r0 + 16 * p) * ldx + k0, r0 + 16 * p < rows ? K - k0 : 0, w[p]);
#pragma unroll
    for (int p = 0; p < 8; ++p) a = max(a, mx_largest<IN>(w[p]));
    a = f8_largest16(a);
    a = max(a, (uint32_t)__shfl_xor((int)a, 16));
    a = max(a, (uint32_t)__shfl_xor((int)a, 32));
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
    __syncthreads();
    a = max(max(part[0], part[1]), max(part[2], part[3]));
    float scale, inverse;
    const bool fine = f8_scale<POW2>(f8_value<IN>(a), scale, inverse);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int64_t row = r0 + 16 * p;
        if (row < rows) codes[(row * units + unit) * 16 + (threadIdx.x & 15)] = fine ? f8_codes<IN>(w[p], inverse) : 0u;
    }
    if (threadIdx.x == 0) scales[blockIdx.x] = scale;
}

// Codes back to values: fl(e4m3 * s), rounded to OUT.  Items of V codes, four
// where a value takes four bytes, so that a store instruction writes whole
// lines (with eight a lane it wrote half of every 32 bytes).  Bound by the stores: 8192 x
// 8192 to fp32 48.5 us (6.9 TB/s), to bf16 30.1.
// `shift`: 0, or 7 where 128 rows share a scale.
template <int OUT>
constexpr int f8_item() { return OUT == OUT_F32 ? 4 : 8; }

template <int OUT, int J, bool NT>
__global__ __launch_bounds__(256) void fp8_block_dequantize_kernel(const uint32_t *__restrict__ codes, const float *__restrict__ scales,
                                                                   void *__restrict__ Y, int64_t row_base, int64_t rows, int32_t K, uint32_t items,
                                                                   int shift)
{
    constexpr int V = f8_item<OUT>(), kPerUnit = kF8Unit / V;
    const int64_t total = rows * items;
    const int64_t first = (int64_t)blockIdx.x * (256 * J);
    const int64_t row0 = first / items;
    const uint32_t rest0 = (uint32_t)(first - row0 * items);
    uint32_t c[J][2];
    float s[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t local = (uint32_t)min((int64_t)(256 * j + threadIdx.x), total - 1 - first);
        const uint32_t at = rest0 + local, r = at / items;
        if (V == 8) {
            const uint2 d = reinterpret_cast<const uint2 *>(codes)[first + local];
            c[j][0] = d.x;
            c[j][1] = d.y;
        } else {
            c[j][0] = codes[first + local];
        }
        s[j] = scales[((row_base + row0 + r) >> shift) * (items / kPerUnit) + (at - r * items) / kPerUnit];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t local = 256 * j + threadIdx.x;
        const uint32_t at = rest0 + local, r = at / items;
        const int k0 = V * (int)(at - r * items), left = first + local < total ? K - k0 : 0;
        float v[V];
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const mx_f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j][h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j][h], true);
            v[4 * h] = lo.x * s[j];
            v[4 * h + 1] = lo.y * s[j];
            v[4 * h + 2] = hi.x * s[j];
            v[4 * h + 3] = hi.y * s[j];
        }
        u32x4 w;
        if (OUT == OUT_F32)
            w = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        else
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = mx_pack2<OUT>(v[(2 * q) % V], v[(2 * q + 1) % V]);
        const int64_t to = (row0 + r) * K + k0;
        if (left >= V) {
            if (OUT == OUT_F32)
                mx_store16<NT>(static_cast<float *>(Y) + to, w);
            else
                mx_store16<NT>(static_cast<uint16_t *>(Y) + to, w);
        } else {
#pragma unroll
            for (int k = 0; k < V - 1; ++k) {
                if (k >= left) break;
                if (OUT == OUT_F32)
                    static_cast<float *>(Y)[to + k] = v[k];
                else
                    static_cast<uint16_t *>(Y)[to + k] = (uint16_t)(w[k / 2] >> (16 * (k % 2)));
            }
        }
    }
}

}  // namespace lpgemm
