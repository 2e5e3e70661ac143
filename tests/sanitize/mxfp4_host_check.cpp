// Drives the host-side paths of the microscaled 4-bit entry points -- argument
// checks, the choice of kernel, shape and grid -- over a wide grid of shapes,
// for a host-only build with AddressSanitizer and UndefinedBehaviorSanitizer.
// No call here reaches a kernel launch: shapes are planned, and the entry
// points are called only with arguments they reject, or with nothing to do,
// before any HIP call.  Exit status 0 when all checks pass.
#include <cstdint>
#include <cstdio>

#include "host_common.hpp"
#include "lpgemm.h"

// what the source of the integer products gives the others
static int forced = LPGEMM_KERNEL_AUTO;
int lpgemm::forced_kernel() { return forced; }
int lpgemm::compute_units() { return 256; }

static int failures = 0;
#define CHECK(c)                                                                  \
    do {                                                                          \
        if (!(c)) {                                                               \
            std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #c); \
            ++failures;                                                           \
        }                                                                         \
    } while (0)

int main()
{
    const int64_t sizes[] = {-1, 0, 1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 896, 897, 1000, 4096, 4097, 8192, 28672, 1 << 20,
                             (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (int64_t)INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 4, INT64_MAX};
    const int64_t ks[] = {-1, 0, 1, 128, 129, 384, 385, 512, 1024, 2897, 4096, 8192, 16384, 16385, 28672, 65536, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, INT64_MAX};
    const int64_t groups[] = {-1, 0, 1, 2, 13, 64, 65, 512, 513, 1024, 1025, INT64_MAX};
    const int cus[] = {-1, 0, 1, 8, 256, 304, INT32_MAX};
    const lpgemm_kernel kernels[] = {LPGEMM_KERNEL_AUTO, LPGEMM_KERNEL_GENERAL, LPGEMM_KERNEL_TILED, LPGEMM_KERNEL_SKINNY,
                                     LPGEMM_KERNEL_TILED_128, LPGEMM_KERNEL_TILED_256, LPGEMM_KERNEL_TILED_64, LPGEMM_KERNEL_FP6};
    long planned = 0;
    for (lpgemm_kernel kernel : kernels) {
        forced = kernel;
        for (int64_t R : sizes)
            for (int64_t N : sizes)
                for (int64_t K : ks)
                    for (int64_t E : groups)
                        for (int cu : cus) {
                            lpgemm_plan_info info{};
                            const lpgemm_status st = lpgemm_mxfp4_plan(R, N, K, E, cu, &info);
                            CHECK(st == LPGEMM_OK || st == LPGEMM_ERR_INVALID_ARG || st == LPGEMM_ERR_UNSUPPORTED);
                            if (R < 0 || N < 0 || K < 0 || E < 0) CHECK(st == LPGEMM_ERR_INVALID_ARG);
                            if (st == LPGEMM_OK && R > 0 && N > 0) {
                                CHECK(info.kernel == LPGEMM_KERNEL_TILED || info.kernel == LPGEMM_KERNEL_SKINNY);
                                CHECK(info.workgroups >= 1 && (info.threads == 256 || info.threads == 512));
                                CHECK(info.tile_m >= 16 && info.tile_n >= 16 && info.k_split >= 1 && info.k_split <= 8);
                                // a launch's threads are counted in 32 bits
                                if (cu > 0 && cu < 1024) CHECK(info.workgroups * info.threads < (int64_t)1 << 32);
                            }
                            ++planned;
                        }
    }
    forced = LPGEMM_KERNEL_AUTO;
    CHECK(lpgemm_mxfp4_plan(4, 4, 128, 0, 0, nullptr) == LPGEMM_ERR_INVALID_ARG);
    for (int64_t M : sizes)
        for (int64_t N : sizes)
            for (int64_t K : ks) {
                size_t b = 7;
                const lpgemm_status st = lpgemm_mxfp4_workspace_size(M, N, K, 0, &b);
                CHECK(st == LPGEMM_OK || st == LPGEMM_ERR_INVALID_ARG || st == LPGEMM_ERR_UNSUPPORTED);
                if (st == LPGEMM_OK) CHECK(b == 0);
            }
    // entry points: arguments rejected, or nothing to do, before any HIP call
    uint8_t *P = reinterpret_cast<uint8_t *>(uintptr_t{4096});
    uint8_t *U = P + 1;  // misaligned for everything but bytes
    const int32_t *I = reinterpret_cast<const int32_t *>(P);
    for (int64_t r : sizes)
        for (int64_t K : ks) {
            const bool empty = r == 0 || K == 0;
            for (int type = -1; type < 6; ++type) {
                const auto t = (lpgemm_out_dtype)type;
                const lpgemm_status q = lpgemm_mxfp4_quantize(U, t, K, U, U, r, K, nullptr);
                const lpgemm_status d = lpgemm_mxfp4_dequantize(U, U, U, t, r, K, nullptr);
                CHECK(q == d);
                CHECK(q == LPGEMM_ERR_INVALID_ARG || q == LPGEMM_ERR_UNSUPPORTED || (q == LPGEMM_OK && empty));
            }
            if (r > 1 && K > 1 && K <= 1 << 20) {
                CHECK(lpgemm_mxfp4_quantize(P, LPGEMM_OUT_BF16, K - 1, P, P, r, K, nullptr) != LPGEMM_OK);
                CHECK(lpgemm_mxfp4_quantize(P, LPGEMM_OUT_BF16, INT64_MAX, P, P, r, K, nullptr) != LPGEMM_OK);
            }
            // more code bytes than any device holds
            if (r >= INT64_MAX / 4 && K >= 0) CHECK(lpgemm_mxfp4_dequantize(P, P, P, LPGEMM_OUT_F32, r, K, nullptr) == (K == 0 ? LPGEMM_OK : LPGEMM_ERR_UNSUPPORTED));
            for (int64_t N : sizes) {
                const bool none = r == 0 || N == 0;
                const lpgemm_status p = lpgemm_mxfp4(P, P, P, P, U, LPGEMM_OUT_F32, r, N, K, nullptr, 0, nullptr);
                CHECK(p == LPGEMM_ERR_INVALID_ARG || p == LPGEMM_ERR_UNSUPPORTED || (p == LPGEMM_OK && none));
                for (int64_t E : groups) {
                    const lpgemm_status g = lpgemm_mxfp4_grouped(P, P, r, nullptr, P, P, E, I, U, LPGEMM_OUT_F32, r, N, K, nullptr);
                    CHECK(g == LPGEMM_ERR_INVALID_ARG || g == LPGEMM_ERR_UNSUPPORTED || (g == LPGEMM_OK && none));
                    const lpgemm_status i = lpgemm_mxfp4_grouped(P, P, r, I, P, P, E, nullptr, P, LPGEMM_OUT_F32, 5, N, K, nullptr);
                    CHECK(i == LPGEMM_ERR_INVALID_ARG || i == LPGEMM_ERR_UNSUPPORTED || (i == LPGEMM_OK && (N == 0 || E == 0)));
                }
            }
        }
    if (failures)
        std::fprintf(stderr, "%d checks failed\n", failures);
    else
        std::printf("microscaled host-path sanitizer run: %ld plans, all checks passed\n", planned);
    return failures ? 1 : 0;
}
