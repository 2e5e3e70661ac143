// mxfp4_quantize.hpp -- to and from the microscaled 4-bit float format.
//
// A row of K values becomes U = ceil(K / 128) units of 64 code bytes and 4
// scale bytes.  For each block of 32 consecutive values, with a = max |x|,
//     e = max(floor(log2 a) - 2, -127)        (the largest value lands in [4, 8))
//     scale byte = e + 127 (e8m0),  code = e2m1(x / 2^e)
// where e2m1 rounds to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, a tie going
// to the even code, and magnitudes above 6 become 6; bit 3 is the sign.  With
// E the exponent field of a in binary32, the scale byte is max(E, 2) - 2.  A
// block that holds a NaN or an infinity gets scale byte 255 (NaN) and codes 0.
//
// Bound by memory: 8192 x 8192 fp32 57 us (5.4 TB/s read and written), back to
// bf16 25 us (6.8 TB/s; its codes come from the caches), 82 us together; 90 with
// loads and stores that the caches keep, 197 with seven compares a value in
// place of the conversion instructions and a 64-bit division for each item.
// Back to fp16 25 us, to fp32 76 us (4.0 TB/s: a store instruction writes half of
// every 32 bytes).  A row of 8192 takes 2 us; the call, 5 us.
#pragma once

#include "device_common.hpp"

namespace lpgemm {

constexpr int kMxUnit = 128;        // values of a row per unit
constexpr int kMxUnitCodes = 64;    // code bytes per unit
constexpr int kMxUnitScales = 4;    // scale bytes per unit
constexpr int kMxUnitE8M0 = 127;    // scale byte of 1.0

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 mx_f16x2 __attribute__((ext_vector_type(2)));
typedef float mx_f32x2 __attribute__((ext_vector_type(2)));

// The scale operand of the fp4 conversions for an e8m0 byte below 255: they
// take 2^(s - 127) from the exponent field.
__device__ __forceinline__ float mx_scale(uint32_t s) { return __uint_as_float(s == 0u ? 0x00400000u : s << 23); }

// 16 bytes at any address of the element's alignment (global memory takes
// unaligned vector accesses).  NT: data that no cache will keep anyway passes
// by them, so that the codes stay.
typedef u32x4 mx_loose __attribute__((aligned(2)));
template <bool NT>
__device__ __forceinline__ u32x4 mx_load16(const void *p)
{
    if (NT) return __builtin_nontemporal_load(static_cast<const mx_loose *>(p));
    return *static_cast<const mx_loose *>(p);
}
template <bool NT>
__device__ __forceinline__ void mx_store16(void *p, u32x4 v)
{
    if (NT)
        __builtin_nontemporal_store(v, static_cast<mx_loose *>(p));
    else
        *static_cast<mx_loose *>(p) = v;
}

// Eight values of a row from k0 on, zeros from K on: IN is OUT_F32, OUT_BF16
// or OUT_F16; 16-bit types in w[0].
template <int IN, bool NT>
__device__ __forceinline__ void mx_load8(const void *x, int64_t at, int left, u32x4 (&w)[2])
{
    w[0] = w[1] = u32x4{0, 0, 0, 0};
    if (IN == OUT_F32) {
        const float *p = static_cast<const float *>(x) + at;
        if (left >= 8) {
            w[0] = mx_load16<NT>(p);
            w[1] = mx_load16<NT>(p + 4);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) w[j / 4][j % 4] = __float_as_uint(p[j]);
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(x) + at;
        if (left >= 8) {
            w[0] = mx_load16<NT>(p);
        } else {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < left) w[0][j / 2] |= (uint32_t)p[j] << (16 * (j % 2));
        }
    }
}

// Largest magnitude of the eight as its bits: they order as the values do.
template <int IN>
__device__ __forceinline__ uint32_t mx_largest(const u32x4 (&w)[2])
{
    uint32_t a = 0;
    if (IN == OUT_F32) {
#pragma unroll
        for (int j = 0; j < 8; ++j) a = max(a, w[j / 4][j % 4] & 0x7FFFFFFFu);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) a = max(a, max(w[0][j] & 0x7FFFu, (w[0][j] >> 16) & 0x7FFFu));
    }
    return a;
}

// Exponent field in binary32 of the magnitude with these bits.
template <int IN>
__device__ __forceinline__ uint32_t mx_exponent(uint32_t a)
{
    if (IN == OUT_F32) return a >> 23;
    if (IN == OUT_BF16) return a >> 7;
    return __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)a)) >> 23;
}

// Eight e2m1 codes of the values over 2^(s - 127): the conversion divides,
// rounds to nearest even and takes what is beyond 6 to 6.
template <int IN>
__device__ __forceinline__ uint32_t mx_codes(const u32x4 (&w)[2], float scale)
{
    uint32_t c = 0;
    if (IN == OUT_F32) {
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[0][0]), __uint_as_float(w[0][1]), scale, 0);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[0][2]), __uint_as_float(w[0][3]), scale, 1);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[1][0]), __uint_as_float(w[1][1]), scale, 2);
        c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(w[1][2]), __uint_as_float(w[1][3]), scale, 3);
    } else {
        // scalars first: a bit cast of a vector's element takes the vector's first
        const uint32_t d0 = w[0][0], d1 = w[0][1], d2 = w[0][2], d3 = w[0][3];
        if (IN == OUT_BF16) {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_bf16x2, d0), scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_bf16x2, d1), scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_bf16x2, d2), scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(mx_bf16x2, d3), scale, 3);
        } else {
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_f16x2, d0), scale, 0);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_f16x2, d1), scale, 1);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_f16x2, d2), scale, 2);
            c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(c, __builtin_bit_cast(mx_f16x2, d3), scale, 3);
        }
    }
    return c;
}

// A workgroup takes 256 J items of eight values, neighbouring ones at a time;
// an item is four code bytes, and four neighbouring lanes share a block and
// its maximum.  `items` = 16 units of a row.
struct MxItem {
    int64_t row;
    int32_t k0;
};
__device__ __forceinline__ MxItem mx_item(int64_t row0, uint32_t rest, uint32_t items)
{
    const uint32_t rows = rest / items;
    return MxItem{row0 + rows, (int32_t)(8 * (rest - rows * items))};
}

template <int IN, int J, bool NT>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const void *__restrict__ X, int64_t ldx,
                                                             uint32_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales, int64_t rows,
                                                             int32_t K, uint32_t items)
{
    const int64_t total = rows * items;  // a multiple of 16
    const int64_t first = (int64_t)blockIdx.x * (256 * J);
    const int64_t row0 = first / items;
    const uint32_t rest0 = (uint32_t)(first - row0 * items);
    u32x4 w[J][2];
    bool pad[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t local = 256 * j + threadIdx.x;
        const MxItem it = mx_item(row0, rest0 + local, items);
        pad[j] = (it.k0 & ~31) >= K;
        mx_load8<IN, NT>(X, it.row * ldx + it.k0, first + local < total ? K - it.k0 : 0, w[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t i = first + 256 * j + threadIdx.x;
        uint32_t a = mx_largest<IN>(w[j]);
        a = max(a, (uint32_t)__shfl_xor((int)a, 1));
        a = max(a, (uint32_t)__shfl_xor((int)a, 2));
        const uint32_t E = mx_exponent<IN>(a);
        const uint32_t s = E == 255u ? 255u : pad[j] ? (uint32_t)kMxUnitE8M0 : max(E, 2u) - 2u;
        const uint32_t c = s == 255u ? 0u : mx_codes<IN>(w[j], mx_scale(s));
        if (i < total) {
            codes[i] = c;
            if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
        }
    }
}

// Eight values of a code dword as OUT, times 2^(s - 127); s = 255: NaN.
template <int OUT>
__device__ __forceinline__ void mx_values(uint32_t c, uint32_t s, u32x4 (&w)[2])
{
    const float scale = mx_scale(s);
    if (OUT == OUT_F32) {
#define LPGEMM_MX_PAIR(q)                                                                     \
        {                                                                                     \
            const mx_f32x2 v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, scale, q);          \
            w[(q) / 2][2 * ((q) % 2)] = s == 255u ? 0x7FC00000u : __float_as_uint(v.x);        \
            w[(q) / 2][2 * ((q) % 2) + 1] = s == 255u ? 0x7FC00000u : __float_as_uint(v.y);    \
        }
        LPGEMM_MX_PAIR(0) LPGEMM_MX_PAIR(1) LPGEMM_MX_PAIR(2) LPGEMM_MX_PAIR(3)
#undef LPGEMM_MX_PAIR
    } else if (OUT == OUT_BF16) {
        w[0] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3))};
        if (s == 255u) w[0] = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    } else {
        w[0] = u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 0)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 1)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 2)),
                     __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, 3))};
        if (s == 255u) w[0] = u32x4{0x7E007E00u, 0x7E007E00u, 0x7E007E00u, 0x7E007E00u};
    }
}

template <int OUT, int J, bool NT>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales,
                                                               void *__restrict__ Y, int64_t rows, int32_t K,
                                                               uint32_t items)
{
    const int64_t total = rows * items;
    const int64_t first = (int64_t)blockIdx.x * (256 * J);
    const int64_t row0 = first / items;
    const uint32_t rest0 = (uint32_t)(first - row0 * items);
    uint32_t c[J], s[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t i = min(first + 256 * j + threadIdx.x, total - 1);
        c[j] = codes[i];
        s[j] = scales[i >> 2];
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const uint32_t local = 256 * j + threadIdx.x;
        const MxItem it = mx_item(row0, rest0 + local, items);
        const int left = first + local < total ? K - it.k0 : 0;
        u32x4 w[2];
        mx_values<OUT>(c[j], s[j], w);
        const int64_t at = it.row * K + it.k0;
        if (OUT == OUT_F32) {
            float *p = static_cast<float *>(Y) + at;
            if (left >= 8) {
                mx_store16<NT>(p, w[0]);
                mx_store16<NT>(p + 4, w[1]);
            } else {
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (k < left) p[k] = __uint_as_float(w[k / 4][k % 4]);
            }
        } else {
            uint16_t *p = static_cast<uint16_t *>(Y) + at;
            if (left >= 8) {
                mx_store16<NT>(p, w[0]);
            } else {
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (k < left) p[k] = (uint16_t)(w[0][k / 2] >> (16 * (k % 2)));
            }
        }
    }
}

}  // namespace lpgemm
