/*
 * lpgemm.h -- low-precision integer GEMM for AMD Instinct MI355X (gfx950)
 *
 *     C[M,N] = A[M,K] . B[N,K]^T     exact, int32 result
 *
 * Two operand formats, both "NT" (every operand row is contiguous along K):
 *
 *   int4 x int4  both A and B are signed 4-bit values packed two per byte.
 *   W4A8         A is int8, B is packed signed 4-bit.
 *
 * Packing (both pages that define it agree): logical element k of a row lives
 * in byte k/2 of that row; even k in the low nibble, odd k in the high nibble;
 * each nibble is a two's-complement value in [-8, 7].  A packed row of K
 * logical elements therefore occupies K/2 bytes, and K must be even.
 *   - TileLang tutorial, ch. 14 sec. 5 "low_precision_gemm.py": pack_int4
 *     (byte = (x[2j] & 0xF) | ((x[2j+1] & 0xF) << 4); odd last dim rejected)
 *     and matmul_int4 (int4 operands, int32 accumulator).
 *   - tilelang PR "[Example] add w4a8 gemm kernel" (#815): torch_convert
 *     (byte j//2, nibble j%2, sign-extended) and ref_program (C = A . B^T of
 *     int8 A and the unpacked int4 B); K given to the kernel is the logical,
 *     unpacked length.
 *   - tilelang PR "[CUDA] Support int4 T.gemm" (#2063), example gemm_int4:
 *     matmul_nt_int4, A[M,K] and B[N,K] int4, C[M,N] int32,
 *     T.gemm(A, B, C, transpose_B=True).
 *
 * Conventions shared by every entry point
 *   - All data pointers are DEVICE pointers owned by the caller; the library
 *     keeps no pointer after the call returns.
 *   - The library never allocates device memory.  Two faster paths need
 *     scratch memory, which only the "_ws" entry points take, from the
 *     caller: large int4 x int4 calls (LPGEMM_KERNEL_FP6, below) re-encode A
 *     and B into a workspace, and int32 calls with long K over few 64 x 64 or
 *     128 x 128 tiles keep one M x N int32 slice of partial sums per K range.
 *     lpgemm_workspace_size gives the bytes a call can use; with less (or
 *     none, as in the entry points without "_ws") the call takes a path that
 *     fits, with the same result.
 *   - Matrices are dense and row-major with no padding: A row stride is K/2
 *     bytes (packed) or K bytes (int8), B row stride K/2 bytes, C row stride
 *     N int32.
 *   - C is overwritten (no alpha/beta) and must not overlap A or B.
 *   - Calls are asynchronous on `stream` (0 = the null stream).  A return of
 *     LPGEMM_OK means the work was validated and enqueued; faults during
 *     execution surface at the caller's next synchronisation.
 *   - Argument checks happen on the host before any HIP call, so an invalid
 *     call touches no device state.
 *   - Calls are thread-safe (lpgemm_set_kernel_override, a test hook,
 *     acts on the calling thread only).  Any alignment is accepted; 16-byte aligned
 *     bases with K a multiple of 32 take the fast kernels, anything else a
 *     slower general kernel with the same results.
 *   - Exactness: the int8 kernels pre-scale 4-bit values by 16 inside int32,
 *     which is exact while 16384*K < 2^31, i.e. K <= 131070.  Larger K
 *     returns LPGEMM_ERR_UNSUPPORTED.  Within that range every result fits
 *     int32 (|C| <= 64*K for int4 x int4, <= 1024*K for W4A8).  The FP6 path
 *     is exact over the same range, although the matrix cores do not add in
 *     IEEE binary32: measured on MI355X, one instruction sums its products
 *     in groups of 8 consecutive k on a grid of 2^-14 of the group's largest
 *     product (lower bits truncated), then combines the group sums and the
 *     accumulator with binary32 round-to-nearest-even.  int4 values are exact
 *     in FP6 E3M2, each product is an integer of magnitude <= 64, so the
 *     grid step is below 1 and no integer bit is dropped, and every combined
 *     value is an integer below 2^23, exact in binary32.  Checked bit for bit
 *     against the oracle on the whole 8192^3 product and on closed forms at
 *     K = 131040 with a single odd product next to partial sums of
 *     64 (K - 1) = 8386496, placed in the first, a middle and the last 64-k
 *     block.
 */
#ifndef LPGEMM_H
#define LPGEMM_H

#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The enumerations are int-sized in C and C++ alike; compiled as C++ they have
 * int as their underlying type, so any int a C caller passes is a value of the
 * type and an unknown one can be rejected. */
#ifdef __cplusplus
#define LPGEMM_ENUM_BASE : int
#else
#define LPGEMM_ENUM_BASE
#endif

typedef enum lpgemm_status LPGEMM_ENUM_BASE {
    LPGEMM_OK = 0,
    LPGEMM_ERR_INVALID_ARG = 1, /* negative size, odd K, null pointer, bad enum  */
    LPGEMM_ERR_UNSUPPORTED = 2, /* valid request the library cannot serve        */
    LPGEMM_ERR_HIP = 3,         /* the HIP runtime reported an error at launch   */
    LPGEMM_ERR_SCRATCH_LIMIT = 4 /* lpgemm_int4_int4_noalloc: the call needs more */
                                 /* than LPGEMM_STATIC_SCRATCH_BYTES of scratch   */
} lpgemm_status;

/* Largest supported K (logical elements); see "Exactness" above. */
#define LPGEMM_MAX_K 131070

/*
 * int4 x int4:  C[m][n] = sum_k a(m,k) * b(n,k)
 *   A_packed  device, bytes [M][K/2] (int8 or uint8 storage, same bits)
 *   B_packed  device, bytes [N][K/2]
 *   C         device, int32 [M][N], written
 *   M, N, K   logical sizes; K even, 0 <= K <= LPGEMM_MAX_K
 * Returns LPGEMM_OK (also for M == 0 or N == 0: nothing is done; K == 0
 * writes zeros), LPGEMM_ERR_INVALID_ARG for negative sizes, odd K or a null
 * pointer that would be dereferenced, LPGEMM_ERR_UNSUPPORTED for K above the
 * limit, LPGEMM_ERR_HIP if the launch failed.
 * Defined by the int4 GEMM example of "[CUDA] Support int4 T.gemm" and the
 * tutorial's matmul_int4 with its pack_int4 layout.
 */
lpgemm_status lpgemm_int4_int4(const void *A_packed, const void *B_packed, int32_t *C,
                               int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * W4A8:  C[m][n] = sum_k A[m][k] * b(n,k)
 *   A         device, int8 [M][K]
 *   B_packed  device, bytes [N][K/2], nibbles sign-extended on unpack
 *   C         device, int32 [M][N], written
 * Sizes, return codes and behaviour as for lpgemm_int4_int4.
 * Defined by "[Example] add w4a8 gemm kernel": ref_program and the kernel's
 * in_dtype int8 / accum_dtype int32 with the u8 -> i4 -> i8 unpack of B.
 */
lpgemm_status lpgemm_w4a8(const int8_t *A, const uint8_t *B_packed, int32_t *C,
                          int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- caller-provided workspace -------------------------------------------- */

/*
 * Bytes of workspace that a call with these sizes can use: of
 * lpgemm_int4_int4_ws / lpgemm_w4a8_ws (scaled == 0) or of
 * lpgemm_int4_int4_scaled_ws (scaled == 1).  0 when the call's fastest path
 * needs none.  Host only: no HIP call, no device access.  The planning
 * assumes 16-byte aligned operands and `cu_count` compute units (0 = 256, an
 * MI355X); a call on a device that plans differently still runs correctly
 * with this workspace, taking only paths that fit in it.
 *   variant   LPGEMM_VARIANT_I4I4 or LPGEMM_VARIANT_W4A8 (declared below)
 *   bytes     written with the size
 * Returns LPGEMM_ERR_INVALID_ARG for a null `bytes`, an unknown variant,
 * `scaled` other than 0 or 1, or sizes the GEMM calls reject as invalid;
 * LPGEMM_ERR_UNSUPPORTED for K above LPGEMM_MAX_K.
 */
typedef enum lpgemm_variant LPGEMM_ENUM_BASE { LPGEMM_VARIANT_I4I4 = 0, LPGEMM_VARIANT_W4A8 = 1 } lpgemm_variant;

lpgemm_status lpgemm_workspace_size(lpgemm_variant variant, int32_t scaled, int64_t M, int64_t N,
                                    int64_t K, int32_t cu_count, size_t *bytes);

/*
 * lpgemm_int4_int4 / lpgemm_w4a8 with a caller-owned workspace:
 *   workspace        device memory, 256-byte aligned, or NULL
 *   workspace_bytes  its size in bytes (0 with NULL)
 * The library uses the workspace during the call's kernels on `stream` only
 * (the caller must not reuse it until the call's work on `stream` has
 * finished, and two calls in flight at once need two workspaces); nothing
 * has to be initialised and its contents afterwards are unspecified.  With
 * workspace_bytes >= lpgemm_workspace_size(...) the call takes the fastest
 * path for its shape; with less it takes the fastest path that fits (the FP6
 * path needs the whole re-encoding, K ranges are cut to the slices that fit).
 * Results are identical whatever the workspace.  Returns
 * LPGEMM_ERR_INVALID_ARG for a NULL or misaligned workspace with
 * workspace_bytes > 0, otherwise as the calls without workspace.
 */
lpgemm_status lpgemm_int4_int4_ws(const void *A_packed, const void *B_packed, int32_t *C,
                                  int64_t M, int64_t N, int64_t K, void *workspace,
                                  size_t workspace_bytes, hipStream_t stream);

lpgemm_status lpgemm_w4a8_ws(const int8_t *A, const uint8_t *B_packed, int32_t *C, int64_t M,
                             int64_t N, int64_t K, void *workspace, size_t workspace_bytes,
                             hipStream_t stream);

/*
 * lpgemm_int4_int4_ws for callers that cannot allocate device memory at all
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc): the workspace is the library's own static scratch, a device
 * array of LPGEMM_STATIC_SCRATCH_BYTES that each GPU the library runs on
 * holds from the library's load until the process ends.  The call allocates
 * nothing and calls no allocating routine; the caller still provides A, B
 * and C.  It takes the path lpgemm_int4_int4_ws takes with unlimited
 * workspace and returns LPGEMM_ERR_SCRATCH_LIMIT, before any launch, when
 * that path needs more scratch than the array holds (lpgemm_workspace_size
 * gives the need: 8192^3 needs 96 MiB and fits, 16384 x 16384 x 8192 needs
 * 192 MiB and is rejected).  Every call on one GPU shares that GPU's scratch, which
 * keeps the last call's contents (nothing in it needs to start at zero):
 * calls that overlap on one GPU -- on different streams, or from different
 * threads -- race and must be serialised by the caller.  Other arguments,
 * sizes and return codes as for lpgemm_int4_int4.
 */
#define LPGEMM_STATIC_SCRATCH_BYTES (128u << 20)

lpgemm_status lpgemm_int4_int4_noalloc(const void *A_packed, const void *B_packed, int32_t *C,
                                       int64_t M, int64_t N, int64_t K, hipStream_t stream);

/* ---- per-channel scaled output ---------------------------------------------- */

/* Element type of a scaled result. */
typedef enum lpgemm_out_dtype LPGEMM_ENUM_BASE {
    LPGEMM_OUT_F32 = 0,     /* IEEE binary32                               */
    LPGEMM_OUT_BF16 = 1,    /* bfloat16 bits (upper half of a binary32)    */
    LPGEMM_OUT_F16 = 2,     /* IEEE binary16                               */
    LPGEMM_OUT_FP8_E4M3 = 3, /* e4m3 byte (lpgemm_fp8_e4m3 only)           */
    LPGEMM_OUT_FP8_E5M2 = 4  /* e5m2 byte (lpgemm_fp8_e5m2 only)           */
} lpgemm_out_dtype;

/*
 * Scaled product with one scale per row of A and one per row of B:
 *
 *     D[m][n] = out( ((float)C[m][n] * scale_a[m]) * scale_b[n] )
 *
 * where C[m][n] is the exact integer result of lpgemm_int4_int4 /
 * lpgemm_w4a8, (float) converts it to binary32 rounding to nearest even
 * (exact while |C| < 2^24), each * is a binary32 multiply rounding to nearest
 * even, and out() converts the binary32 value to out_dtype rounding to
 * nearest even (F32: unchanged; BF16: a NaN stays a quiet NaN, values past the
 * largest finite bf16 become infinities; F16: likewise for binary16).  This is
 * the tutorial's gemm_blockscaled (ch. 14 sec. 5, "low_precision_gemm.py":
 * SFA / SFB scales applied per K block, fp32 accumulation, out_dtype result)
 * with a single K block: per-row and per-column scales.  The integer sum
 * stays exact; only the epilogue rounds.
 *   scale_a   device, float [M] (4-byte aligned)
 *   scale_b   device, float [N] (4-byte aligned)
 *   D         device, [M][N] of out_dtype, row stride N elements, written;
 *             aligned to its element size
 * Other arguments, sizes and return codes as for the unscaled calls; also
 * LPGEMM_ERR_INVALID_ARG for an unknown out_dtype, a null or misaligned scale
 * vector or D.  K == 0 gives out(((float)0 * scale_a[m]) * scale_b[n]).
 */
lpgemm_status lpgemm_int4_int4_scaled(const void *A_packed, const void *B_packed,
                                      const float *scale_a, const float *scale_b, void *D,
                                      lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K,
                                      hipStream_t stream);

lpgemm_status lpgemm_w4a8_scaled(const int8_t *A, const uint8_t *B_packed, const float *scale_a,
                                 const float *scale_b, void *D, lpgemm_out_dtype out_dtype,
                                 int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * lpgemm_int4_int4_scaled with a caller-owned workspace (the FP6 path for
 * large shapes), under the rules of lpgemm_int4_int4_ws.  The W4A8 scaled
 * product has no path that uses a workspace.
 */
lpgemm_status lpgemm_int4_int4_scaled_ws(const void *A_packed, const void *B_packed,
                                         const float *scale_a, const float *scale_b, void *D,
                                         lpgemm_out_dtype out_dtype, int64_t M, int64_t N,
                                         int64_t K, void *workspace, size_t workspace_bytes,
                                         hipStream_t stream);

/*
 * Per-K-block scaled product (the tutorial's gemm_blockscaled, ch. 14 sec. 5,
 * "low_precision_gemm.py": scale tables SFA[M, ceil(K/g)] and SFB[N, ceil(K/g)]
 * in the float32 accumulator type, applied along K one block of
 * sf_granularity_k = g at a time into a float32 accumulator, result in
 * out_dtype), for the integer operands of lpgemm_int4_int4 / lpgemm_w4a8:
 *
 *     C_j[m][n] = sum over k in [j g, min(K, (j+1) g)) of a(m,k) b(n,k)   (exact)
 *     term_j    = ((float)C_j[m][n] * SFA[m][j]) * SFB[n][j]
 *     acc       = term_0 + term_1 + ... + term_(nb-1), added left to right
 *     D[m][n]   = out(acc)
 *
 * with nb = ceil(K / g) blocks (the last one shorter when g does not divide
 * K); (float) converts to binary32 rounding to nearest even (exact while
 * |C_j| < 2^24), each * and + is a binary32 operation rounding to nearest
 * even (no fused multiply-add), and out() is the conversion of the scaled
 * entry points.  The order of the additions is fixed, so the result is
 * unique.  With g >= K (one block) this is the per-channel product of
 * lpgemm_int4_int4_scaled / lpgemm_w4a8_scaled.  K == 0 gives +0.
 *   A / A_packed  as for the unscaled call
 *   B_packed      device, packed int4 [N][K/2]
 *   SFA           device, float [M][nb] row-major (4-byte aligned)
 *   SFB           device, float [N][nb] row-major (4-byte aligned)
 *   g             block length in k: a power of two, 32 <= g <= 2^30 (the
 *                 page names 128 and 32)
 *   D             device, [M][N] of out_dtype (F32, BF16 or F16), written;
 *                 aligned to its element size
 * Returns LPGEMM_ERR_INVALID_ARG for negative sizes, odd K, a bad g or
 * out_dtype, a null or misaligned pointer that would be dereferenced;
 * LPGEMM_ERR_UNSUPPORTED for K above LPGEMM_MAX_K or a forced kernel other
 * than GENERAL / TILED / TILED_128 / TILED_64; LPGEMM_ERR_HIP if a launch
 * failed.  K % 32 == 0 with 16-byte aligned A and B (and D aligned to 16
 * bytes for F32, 8 for BF16 / F16) takes the tiled matrix-core kernel (the
 * integer partial of each block in int32 matrix-core accumulators, added
 * where the block ends), anything else a one-thread-per-element kernel; both
 * give the same bits.  The library allocates nothing.
 */
lpgemm_status lpgemm_int4_int4_blockscaled(const void *A_packed, const void *B_packed, const float *SFA,
                                           const float *SFB, int64_t g, void *D,
                                           lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K,
                                           hipStream_t stream);

lpgemm_status lpgemm_w4a8_blockscaled(const int8_t *A, const uint8_t *B_packed, const float *SFA,
                                      const float *SFB, int64_t g, void *D, lpgemm_out_dtype out_dtype,
                                      int64_t M, int64_t N, int64_t K, hipStream_t stream);

/*
 * fp8 GEMM (second workload):  C[m][n] = out( sum_k a(m,k) * b(n,k) )
 *   A          device, e4m3 bytes [M][K]
 *   B          device, e4m3 bytes [N][K]
 *   C          device, [M][N] binary32 (LPGEMM_OUT_F32) or e4m3 bytes
 *              (LPGEMM_OUT_FP8_E4M3), written
 *   M, N, K    any sizes >= 0, K <= LPGEMM_MAX_K
 * E4M3 is the OCP 8-bit format without infinities: sign, 4 exponent bits
 * (bias 7), 3 mantissa bits; exponent 0 is subnormal; S.1111.111 is NaN; the
 * largest finite magnitude is 448.  Every product is exact in binary32.  Let
 * S be the exact sum and P = sum_k |a(m,k) b(n,k)|.
 *   - The one-thread-per-element kernel adds the products in binary32 in k
 *     order: |C - S| <= 1.01 * K * 2^-24 * P.
 *   - The matrix-core kernel runs v_mfma_scale_f32_32x32x64_f8f6f4, whose
 *     summation is not IEEE binary32 and not published.  Measured on MI355X:
 *     an instruction takes 64 k in groups of 8 consecutive k; in a group every
 *     product is truncated toward zero to a multiple of 2^(E-13), E the largest
 *     e(a) + e(b) over the group's nonzero products (e: the binary exponent of
 *     an e4m3 code, -6 for subnormals); the group sums and the accumulator are
 *     added in binary32, rounding to nearest even.  Hence
 *         |C - S| <= 7 * sum_groups 2^(EA + EB - 13) + 1.01 * K * 2^-24 * P
 *     with EA, EB the largest exponents of the group's nonzero codes of A's
 *     row m and B's row n (E <= EA + EB).  Products of small integers (E <= 6)
 *     lose nothing; a large product and much smaller ones in one group lose
 *     up to about 2^-10 of the large one, whatever the exact sum.
 * An e4m3 result rounds the binary32 result to nearest, ties to even,
 * saturating at +-448 (NaN stays NaN).  K == 0 writes zeros.
 * Returns LPGEMM_ERR_INVALID_ARG for negative sizes, a null pointer that would
 * be dereferenced, or an out_dtype other than the two above;
 * LPGEMM_ERR_UNSUPPORTED for K above LPGEMM_MAX_K; LPGEMM_ERR_HIP if a launch
 * failed.  16-byte aligned A and B with K % 16 == 0 (and C aligned to 16 bytes
 * for binary32, 4 for e4m3) take the tiled matrix-core kernel, anything else
 * a slower one-thread-per-element kernel.
 * Defined by the TileLang tutorial's gemm_fp8 (chapter 14): A[M,K] and B[N,K]
 * in the fp8 dtype (e4m3), T.gemm(..., transpose_B=True) into a float32
 * accumulator, C stored in the fp8 dtype.
 */
lpgemm_status lpgemm_fp8_e4m3(const uint8_t *A, const uint8_t *B, void *C,
                              lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K,
                              hipStream_t stream);

/*
 * fp8 GEMM with e5m2 operands (the tutorial's gemm_fp8 takes "e4m3 / e5m2"
 * into a float32 accumulator):  C[m][n] = out( sum_k a(m,k) * b(n,k) )
 *   A          device, e5m2 bytes [M][K]
 *   B          device, e5m2 bytes [N][K]
 *   C          device, [M][N] binary32 (LPGEMM_OUT_F32) or e5m2 bytes
 *              (LPGEMM_OUT_FP8_E5M2), written
 *   M, N, K    any sizes >= 0, K <= LPGEMM_MAX_K
 * E5M2 is the OCP 8-bit format with infinities (the upper byte of an IEEE
 * binary16): sign, 5 exponent bits (bias 15), 2 mantissa bits; exponent 0 is
 * subnormal (smallest 2^-16); exponent 31 is infinity (mantissa 0) or NaN;
 * the largest finite magnitude is 57344.  Every product is exact in binary32
 * and no sum of finite products overflows it.  Infinities and NaNs follow
 * IEEE arithmetic: an infinite operand gives an infinite product (NaN against
 * zero), opposite infinities in one sum give NaN, a NaN operand gives NaN.
 * The accuracy of finite results is that of lpgemm_fp8_e4m3, with e(x) the
 * binary exponent of an e5m2 code (-14 for subnormals): measured on MI355X,
 * the matrix-core instruction sums e5m2 products in the same groups of 8 k
 * with the same truncation to a multiple of 2^(E-13), so
 *     |C - S| <= 7 * sum_groups 2^(EA + EB - 13) + 1.01 * K * 2^-24 * P
 * for the matrix-core kernel and |C - S| <= 1.01 * K * 2^-24 * P for the
 * one-thread-per-element kernel.
 * An e5m2 result rounds the binary32 result to nearest, ties to even;
 * magnitudes from 61440 (the midpoint above 57344) become infinities, NaN
 * stays NaN.  K == 0 writes zeros.  Return codes and the choice of kernel as
 * for lpgemm_fp8_e4m3 (with LPGEMM_OUT_FP8_E5M2 as the only fp8 out_dtype;
 * C aligned to 16 bytes for binary32, 4 for e5m2, for the tiled kernel).
 */
lpgemm_status lpgemm_fp8_e5m2(const uint8_t *A, const uint8_t *B, void *C,
                              lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K,
                              hipStream_t stream);

/*
 * Pack logical int4 values (held one per int8) into bytes, on the device:
 *   logical  device, int8 [rows][K], each value in [-8, 7] (only the low four
 *            bits of each value are kept, as the tutorial's pack_int4 does)
 *   packed   device, bytes [rows][K/2], written
 * K must be even (LPGEMM_ERR_INVALID_ARG otherwise, as pack_int4 raises on an
 * odd last dimension); rows * K/2 beyond the int64 range returns
 * LPGEMM_ERR_UNSUPPORTED.  The tutorial's pack_int4 defines the layout.
 */
lpgemm_status lpgemm_pack_int4(const int8_t *logical, uint8_t *packed, int64_t rows, int64_t K,
                               hipStream_t stream);

/*
 * Unpack bytes into logical int4 values, one per int8, sign-extended:
 *   packed   device, bytes [rows][K/2]
 *   logical  device, int8 [rows][K], written
 * Argument errors as for lpgemm_pack_int4.  The dequantise-only test kernel
 * of "[Example] add w4a8 gemm kernel" (u8 -> i4 -> i8 of byte j//2, nibble
 * j%2) defines the operation.
 */
lpgemm_status lpgemm_unpack_int4(const uint8_t *packed, int8_t *logical, int64_t rows, int64_t K,
                                 hipStream_t stream);

/* ---- microscaled 4-bit floating point (mxfp4) -----------------------------
 *
 * The OCP microscaling format with 4-bit elements: a row of K values is cut
 * into blocks of 32 consecutive values; every value is an e2m1 code (0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives; sign in bit 3) and every block has
 * one e8m0 scale byte s standing for 2^(s - 127), 255 for NaN:
 *     value(k) = e2m1(code(k)) * 2^(s(k / 32) - 127)
 * A row holds U = ceil(K / 128) units, 64 code bytes and 4 scale bytes each:
 *     codes   [rows][64 U]   element k in byte k / 2, even k in the low nibble
 *     scales  [rows][4 U]    block j in byte j
 * Codes past K are zero, and so every value past K is; a block that lies past
 * K has scale 127.  With K % 128 == 0 there is no padding.
 * Codes are 16-byte aligned, scales 4-byte aligned, D 16-byte aligned and
 * other values to their element (LPGEMM_ERR_INVALID_ARG otherwise).
 */
#define LPGEMM_MXFP4_MAX_K (1 << 20)
#define LPGEMM_MXFP4_MAX_ROWS (1 << 30)   /* of D, A and B (each group's) */
#define LPGEMM_MXFP4_MAX_GROUPS 1024

/*
 * Rows of F32, BF16 or F16 values -> codes and scales.
 *   X       device, x_dtype [rows][K], row r at X + r * ldx elements
 *           (ldx >= K; any alignment of the element size)
 *   codes, scales   device, written whole, the padding of each row included
 * With a = max |x| of a block, s = max(floor(log2 a) - 2, -127) + 127 (a = 0:
 * s = 0) and code = the e2m1 value nearest to x / 2^(s - 127), a tie going to
 * the even code, magnitudes above 6 becoming 6.  A block that holds a NaN or
 * an infinity gets s = 255 and zero codes: all its values become NaN.
 * LPGEMM_ERR_INVALID_ARG for negative sizes, another x_dtype, ldx < K with
 * several rows, a null or misaligned pointer; LPGEMM_ERR_UNSUPPORTED for K
 * above LPGEMM_MXFP4_MAX_K or more code bytes than any device holds.
 */
lpgemm_status lpgemm_mxfp4_quantize(const void *X, lpgemm_out_dtype x_dtype, int64_t ldx, uint8_t *codes,
                                    uint8_t *scales, int64_t rows, int64_t K, hipStream_t stream);

/*
 * Codes and scales -> the values they stand for, y_dtype [rows][K] dense.
 * Exact for F32 and BF16 (every value has at most two significant bits);
 * F16 rounds to nearest even.  Errors as for lpgemm_mxfp4_quantize.
 */
lpgemm_status lpgemm_mxfp4_dequantize(const uint8_t *codes, const uint8_t *scales, void *Y, lpgemm_out_dtype y_dtype,
                                      int64_t rows, int64_t K, hipStream_t stream);

/*
 * D[m][n] = out( sum_k a(m,k) b(n,k) )   of mxfp4 operands
 *   A, SFA   device, codes and scales of M rows of K values
 *   B, SFB   device, codes and scales of N rows of K values
 *   D        device, [M][N] F32, BF16 or F16, written
 * Products of one block are exact; the matrix cores add them in groups of 8 k
 * (each group exact: its products are multiples of 1/4 of at most 36, times
 * one power of two) and the groups to a binary32 accumulator, rounding to
 * nearest even; partial sums of K ranges, where a kernel takes them, are added
 * in binary32 in a fixed order.  So |D - S| <= 1.01 (K / 8 + 16) 2^-24 P before
 * out(), with S the exact sum and P = sum |a b|, while no scale product leaves
 * binary32's normal range.  A block of scale 255 makes its row (A) or column
 * (B) of D NaN.  K == 0 writes zeros.
 * lpgemm_mxfp4_workspace_size gives the bytes of scratch memory that a call
 * can use; no kernel uses any at present, so it is 0.  A workspace that is
 * passed is 256-byte aligned, and a call runs without one (null, 0).
 * LPGEMM_ERR_INVALID_ARG for negative sizes, another out_dtype, a null or
 * misaligned pointer that would be dereferenced; LPGEMM_ERR_UNSUPPORTED above
 * the limits; LPGEMM_ERR_HIP if a launch failed.
 */
lpgemm_status lpgemm_mxfp4(const uint8_t *A, const uint8_t *SFA, const uint8_t *B, const uint8_t *SFB, void *D,
                           lpgemm_out_dtype out_dtype, int64_t M, int64_t N, int64_t K, void *workspace,
                           size_t workspace_bytes, hipStream_t stream);
lpgemm_status lpgemm_mxfp4_workspace_size(int64_t M, int64_t N, int64_t K, int32_t cu_count, size_t *bytes);

/*
 * The product of every group of rows with that group's matrix: for row i of D
 * in group e, offsets[e] <= i < offsets[e + 1],
 *     D[i][n] = out( sum_k a(rows[i], k) b_e(n, k) )
 *   A, SFA    device, codes and scales of T rows
 *   rows      device, int32 [R], the row of A for each row of D, or null (row
 *             i is row i; T == R).  An index outside [0, T) stands for a row
 *             of zeros.  With rows, A's codes span at most 2^31 - 1 bytes.
 *   B, SFB    device, codes and scales of E matrices of N rows, one after another
 *   offsets   device, int32 [E + 1], non-decreasing from 0 to R; groups may be
 *             empty.  Read on the device, so a call needs no synchronisation.
 *             Each offset is taken into [0, R], and one below an offset before
 *             it to that one: no row is in two groups and nothing outside D is
 *             written.  Rows of D in no group are left as they are.
 *   D         device, [R][N], written
 * Accuracy and errors as for lpgemm_mxfp4; E above LPGEMM_MXFP4_MAX_GROUPS
 * is LPGEMM_ERR_UNSUPPORTED.
 */
lpgemm_status lpgemm_mxfp4_grouped(const uint8_t *A, const uint8_t *SFA, int64_t T, const int32_t *rows,
                                   const uint8_t *B, const uint8_t *SFB, int64_t E, const int32_t *offsets, void *D,
                                   lpgemm_out_dtype out_dtype, int64_t R, int64_t N, int64_t K, hipStream_t stream);

/* Static, human-readable name of a status code (never NULL). */
const char *lpgemm_status_string(lpgemm_status status);

/* ---- kernel selection: host-only, for tests and measurement -------------- */

typedef enum lpgemm_kernel LPGEMM_ENUM_BASE {
    LPGEMM_KERNEL_AUTO = 0,      /* choose by shape and alignment (default)      */
    LPGEMM_KERNEL_GENERAL = 1,   /* any shape and alignment; slow                */
    LPGEMM_KERNEL_TILED = 2,     /* block-tiled MFMA kernel, tile size by shape   */
    LPGEMM_KERNEL_SKINNY = 3,    /* narrow-M kernel (M <= 64) streaming B once   */
    LPGEMM_KERNEL_TILED_128 = 4, /* block-tiled, 128 x 128 output tiles          */
    LPGEMM_KERNEL_TILED_256 = 5, /* block-tiled, 256 x 256 output tiles          */
    LPGEMM_KERNEL_TILED_64 = 6,  /* block-tiled, 64 x 64 output tiles            */
    LPGEMM_KERNEL_FP6 = 7        /* int4 x int4: A, B re-encoded as FP6 E3M2,    */
                                 /* 256 x 256 tiles on the FP6 matrix cores       */
} lpgemm_kernel;
/* The mxfp4 products have TILED, TILED_64, TILED_128, TILED_256 (tiles of up to
 * that many rows and columns; TILED_256 with K <= 384 runs as TILED_128, whose
 * ring takes rows of fewer than four units) and SKINNY (product: K <= 16384, up
 * to 4096 rows; grouped: up to 896 rows of D and 512 groups); anything else
 * forced on them is LPGEMM_ERR_UNSUPPORTED. */
/* LPGEMM_KERNEL_AUTO picks FP6 for int4 x int4 when the fast path applies,
 * the call's workspace holds the re-encoded operands, M > 128, and either the
 * 256 x 256 output tiles number at least twice the compute units with
 * K >= 2048, or three quarters of them with K >= 3072 (there the re-encoding
 * pass costs less than the matrix cores save).  Up to 128 rows of
 * A it takes the tiled kernel with 128 x 128 or 64 x 64 tiles (B is read
 * once), or the narrow-M kernel for M <= 16, either format, and up to 64 rows
 * where the tiled kernel would have few workgroups.  With an int32 result and
 * K > 8192 on the narrow-M kernel, K is cut into ranges whose sums are added
 * into C, which the call zeroes first; scaled results with K > 8192 take each
 * range in turn inside one workgroup when there are enough strips, else the
 * tiled kernel.  With an int32 result, K >= 12288 and fewer 64 x 64 tiles than
 * two per compute unit (or fewer 128 x 128 tiles than two thirds of the
 * compute units), the tiles are split over K ranges whose partial sums go to
 * slices of the call's workspace (as many ranges as slices fit, none below
 * two) and are summed into C by a second kernel.  LPGEMM_KERNEL_SKINNY serves
 * up to 64 rows (row groups of 16). */

/* How a call would be executed. */
typedef struct lpgemm_plan_info {
    int32_t kernel;        /* lpgemm_kernel actually used                        */
    int32_t tile_m;        /* output rows per workgroup                          */
    int32_t tile_n;        /* output columns per workgroup                       */
    int32_t k_split;       /* waves that split K inside one workgroup (skinny)   */
    int64_t workgroups;    /* workgroups launched                                */
    int32_t threads;       /* threads per workgroup                              */
    int32_t k_chunks;      /* K ranges contracted separately and summed into  */
                           /* C (narrow-M with K > 8192; 64- or 128-tiles     */
                           /* with long K over few tiles), else 1             */
    int64_t workspace_bytes; /* workspace the call uses (0: none)             */
} lpgemm_plan_info;

/*
 * Fill *info with the kernel and launch shape a call with these arguments,
 * an int32 result and `workspace_bytes` of workspace (0: a call without
 * workspace; SIZE_MAX: every path available) would use, without touching the
 * device (pointers are only inspected for alignment).  `cu_count` is the
 * number of compute units to plan for (0 = 256, an MI355X).  Returns what
 * the call would return for argument errors, LPGEMM_ERR_UNSUPPORTED if a
 * forced kernel cannot run this shape (LPGEMM_KERNEL_FP6 also without the
 * workspace it needs).
 */
lpgemm_status lpgemm_plan(lpgemm_variant variant, const void *A, const void *B, const void *C,
                          int64_t M, int64_t N, int64_t K, size_t workspace_bytes,
                          int32_t cu_count, lpgemm_plan_info *info);

/*
 * The same for an mxfp4 product of R rows: E == 0 lpgemm_mxfp4, E > 0
 * lpgemm_mxfp4_grouped with E groups and R rows of A and D.  info->kernel is TILED or
 * SKINNY, tile_m the most rows of a tile, k_split the waves (SKINNY) or halves
 * of a workgroup that split K.
 */
lpgemm_status lpgemm_mxfp4_plan(int64_t R, int64_t N, int64_t K, int64_t E, int32_t cu_count, lpgemm_plan_info *info);

/*
 * Force a kernel for the later calls made on the calling thread
 * (LPGEMM_KERNEL_AUTO restores the default; other threads are not
 * affected).  A forced kernel that cannot serve a shape makes the call return
 * LPGEMM_ERR_UNSUPPORTED.  Returns LPGEMM_ERR_INVALID_ARG for an unknown
 * value.  Meant for tests and benchmarks.
 */
lpgemm_status lpgemm_set_kernel_override(lpgemm_kernel kernel);

#ifdef __cplusplus
}
#endif

#endif /* LPGEMM_H */
