// Drives the host-side paths of the block-scaled e4m3 and routing entry points --
// argument checks, the choice of kernel, shape and grid -- over a wide grid of
// shapes, for a host-only build with AddressSanitizer and
// UndefinedBehaviorSanitizer.  No call here reaches a kernel launch.
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

static bool known(lpgemm_status st) { return st == LPGEMM_OK || st == LPGEMM_ERR_INVALID_ARG || st == LPGEMM_ERR_UNSUPPORTED; }

int main()
{
    const int64_t sizes[] = {-1, 0, 1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 896, 897, 1000, 4096, 4097, 8192, 28672, 1 << 20,
                             (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (int64_t)INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX / 4, INT64_MAX};
    const int64_t ks[] = {-1, 0, 1, 128, 129, 384, 385, 2048, 2049, 4096, 8192, 8193, 28672, 1 << 20, (1 << 20) + 1, INT64_MAX};
    const int64_t groups[] = {-1, 0, 1, 2, 13, 64, 65, 512, 513, 1024, 1025, INT64_MAX};
    const int cus[] = {-1, 0, 1, 8, 256, INT32_MAX};
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
                            const lpgemm_status st = lpgemm_fp8_block_plan(R, N, K, E, cu, &info);
                            CHECK(known(st));
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
    CHECK(lpgemm_fp8_block_plan(4, 4, 128, 0, 0, nullptr) == LPGEMM_ERR_INVALID_ARG);
    // entry points: arguments rejected, or nothing to do, before any HIP call
    uint8_t *P = reinterpret_cast<uint8_t *>(uintptr_t{4096});
    uint8_t *U = P + 1;  // misaligned for everything but bytes
    float *F = reinterpret_cast<float *>(P), *UF = reinterpret_cast<float *>(U);
    int32_t *I = reinterpret_cast<int32_t *>(P), *UI = reinterpret_cast<int32_t *>(U);
    for (int64_t r : sizes)
        for (int64_t K : ks) {
            const bool empty = r == 0 || K == 0;
            for (int64_t block : {INT64_MIN, (int64_t)0, (int64_t)1, (int64_t)128, INT64_MAX})
                for (int type = -1; type < 6; ++type) {
                    const auto t = (lpgemm_out_dtype)type;
                    const lpgemm_status q = lpgemm_fp8_block_quantize(U, t, K, block, 1, U, UF, r, K, nullptr);
                    const lpgemm_status d = lpgemm_fp8_block_dequantize(U, UF, block, U, t, r, K, nullptr);
                    CHECK(q == d && known(q) && (q != LPGEMM_OK || empty));
                }
            if (r > 1 && K > 1 && K <= 1 << 20) {
                CHECK(lpgemm_fp8_block_quantize(P, LPGEMM_OUT_BF16, K - 1, 1, 0, P, F, r, K, nullptr) != LPGEMM_OK);
                CHECK(lpgemm_fp8_block_quantize(P, LPGEMM_OUT_BF16, INT64_MAX, 128, 0, P, F, r, K, nullptr) != LPGEMM_OK);
            }
            for (int64_t N : sizes) {
                const bool none = r == 0 || N == 0;
                const lpgemm_status p = lpgemm_fp8_block(P, F, P, F, 128, U, LPGEMM_OUT_F32, r, N, K, nullptr);
                CHECK(known(p) && (p != LPGEMM_OK || none));
                for (int64_t E : groups) {
                    const lpgemm_status g = lpgemm_fp8_block_grouped(P, F, r, nullptr, P, F, 1, E, I, U, LPGEMM_OUT_F32, r, N, K, nullptr);
                    CHECK(known(g) && (g != LPGEMM_OK || none));
                    const lpgemm_status i = lpgemm_fp8_block_grouped(P, F, r, I, P, F, 128, E, nullptr, P, LPGEMM_OUT_F32, 5, N, K, nullptr);
                    CHECK(known(i) && (i != LPGEMM_OK || N == 0 || E == 0));
                }
                for (int64_t top : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)32, (int64_t)1024, (int64_t)1025, INT64_MAX}) {
                    const lpgemm_status c = lpgemm_combine(U, LPGEMM_OUT_BF16, r, UI, nullptr, nullptr, U, LPGEMM_OUT_BF16, N, top, K, nullptr);
                    CHECK(known(c) && (c != LPGEMM_OK || N == 0 || K == 0));
                    const lpgemm_status b = lpgemm_combine_backward(U, LPGEMM_OUT_BF16, U, LPGEMM_OUT_F32, r, UI, nullptr, U, UF, N, top, K, nullptr);
                    CHECK(known(b) && (b != LPGEMM_OK || N == 0 || top == 0));
                }
            }
        }
    for (int64_t T : sizes)
        for (int64_t E : groups) {
            size_t bytes = 7;
            CHECK(known(lpgemm_route_workspace_size(T, E, &bytes)));
            CHECK(lpgemm_route_workspace_size(T, E, nullptr) == LPGEMM_ERR_INVALID_ARG);
            for (int top : {INT32_MIN, -1, 0, 1, 2, 32, 33, INT32_MAX})
                for (int count : {INT32_MIN, 0, 1, 2, 13, 64, 65, INT32_MAX})
                    for (int64_t ld : {INT64_MIN, (int64_t)0, E, INT64_MAX}) {
                        const lpgemm_route_options o{LPGEMM_ROUTE_SIGMOID, top, count, 1, 2, 1, 1.f};
                        const lpgemm_status st = lpgemm_route(U, LPGEMM_OUT_F32, ld, nullptr, &o, I, F, I, UI, I, T, E, nullptr, 0, nullptr);
                        CHECK(st == LPGEMM_ERR_INVALID_ARG || st == LPGEMM_ERR_UNSUPPORTED);
                        const lpgemm_status b = lpgemm_route_backward(UF, P, LPGEMM_OUT_F32, ld, I, &o, P, T, E, nullptr);
                        CHECK(known(b) && (b != LPGEMM_OK || T == 0));
                    }
        }
    if (failures)
        std::fprintf(stderr, "%d checks failed\n", failures);
    else
        std::printf("experts' host-path sanitizer run: %ld plans, all checks passed\n", planned);
    return failures ? 1 : 0;
}
