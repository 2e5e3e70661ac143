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
#pragma once

#include "device_common.hpp"

namespace lpgemm {

constexpr int kMxUnit = 128;        // values of a row per unit
constexpr int kMxUnitCodes = 64;    // code bytes per unit
constexpr int kMxUnitScales = 4;    // scale bytes per unit
constexpr int kMxUnitE8M0 = 127;    // scale byte of 1.0

// e2m1 code (3 bits) of a magnitude m >= 0, nearest, ties to the even code.
__device__ __forceinline__ uint32_t e2m1_code(float m)
{
    return (uint32_t)(m > 0.25f) + (uint32_t)(m >= 0.75f) + (uint32_t)(m > 1.25f) + (uint32_t)(m >= 1.75f) +
           (uint32_t)(m > 2.5f) + (uint32_t)(m >= 3.5f) + (uint32_t)(m > 5.0f);
}

// 2^(s - 127) of an e8m0 byte (255: NaN); s = 0 is subnormal in binary32.
__device__ __forceinline__ float e8m0_value(uint32_t s)
{
    return s == 255u ? __uint_as_float(0x7FC00000u) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// Value of an e2m1 code: 0, 0.5, 1, 1.5, 2, 3, 4, 6 with the sign in bit 3.
__device__ __forceinline__ float e2m1_value(uint32_t c)
{
    const uint32_t e = (c >> 1) & 3u, m = c & 1u;
    const uint32_t mag = e ? ((126u + e) << 23) | (m << 22) : (m ? 0x3F000000u : 0u);
    return __uint_as_float(mag | ((c & 8u) << 28));
}

// An input value as binary32 (exact): IN is OUT_F32, OUT_BF16 or OUT_F16.
template <int IN>
__device__ __forceinline__ float mx_load(const void *x, int64_t i)
{
    if (IN == OUT_F32) return static_cast<const float *>(x)[i];
    const uint16_t h = static_cast<const uint16_t *>(x)[i];
    if (IN == OUT_BF16) return __uint_as_float((uint32_t)h << 16);
    return (float)__builtin_bit_cast(_Float16, h);
}

// One thread per 8 values (4 code bytes); four neighbouring lanes share a
// block and its maximum.
template <int IN>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const void *__restrict__ X, int64_t ldx,
                                                             uint32_t *__restrict__ codes,
                                                             uint8_t *__restrict__ scales, int64_t rows,
                                                             int64_t K, int64_t units)
{
    const int64_t total = rows * units * 16;  // threads with work; a multiple of 16
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t row = i / (units * 16);
        const int64_t k0 = (i - row * units * 16) * 8;
        float x[8];
        uint32_t a = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[j] = k0 + j < K ? mx_load<IN>(X, row * ldx + k0 + j) : 0.f;
            a = max(a, __float_as_uint(x[j]) & 0x7FFFFFFFu);
        }
        a = max(a, (uint32_t)__shfl_xor((int)a, 1));
        a = max(a, (uint32_t)__shfl_xor((int)a, 2));
        const uint32_t E = a >> 23;
        const bool whole_pad = (k0 & ~(int64_t)31) >= K;
        const uint32_t s = E == 255u ? 255u : whole_pad ? (uint32_t)kMxUnitE8M0 : max(E, 2u) - 2u;
        // 2^(127 - s): normal for every s <= 252, so the products below are exact
        // except where they fall far under 0.25
        const float inv = __uint_as_float((254u - min(s, 252u)) << 23);
        uint32_t out = 0;
        if (s != 255u) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = fabsf(x[j]) * inv;
                out |= (e2m1_code(m) | ((__float_as_uint(x[j]) >> 28) & 8u)) << (4 * j);
            }
        }
        codes[i] = out;
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)s;
    }
}

// One thread per 8 values.
template <int OUT>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint32_t *__restrict__ codes,
                                                               const uint8_t *__restrict__ scales,
                                                               void *__restrict__ Y, int64_t rows, int64_t K,
                                                               int64_t units)
{
    const int64_t total = rows * units * 16;
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += step) {
        const int64_t row = i / (units * 16);
        const int64_t k0 = (i - row * units * 16) * 8;
        const uint32_t c = codes[i];
        const float S = e8m0_value(scales[i >> 2]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (k0 + j >= K) break;
            float v = e2m1_value((c >> (4 * j)) & 15u) * S;
            // the product itself is converted: folded into one operation with the
            // conversion to fp16 it would lose the sign of a result that rounds to zero
            asm volatile("" : "+v"(v));
            if (OUT == OUT_F32)
                static_cast<float *>(Y)[row * K + k0 + j] = v;
            else
                static_cast<uint16_t *>(Y)[row * K + k0 + j] = (uint16_t)out_bits<OUT>(v);
        }
    }
}

}  // namespace lpgemm
