// api_common.hpp -- what the float operators' entry points share on the host.
#pragma once

#include "lpgemm.h"

#include <algorithm>
#include <mutex>

#include "device_common.hpp"
#include "host_common.hpp"

namespace lpgemm {

inline int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }
inline bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline lpgemm_status launched() { return hipGetLastError() == hipSuccess ? LPGEMM_OK : LPGEMM_ERR_HIP; }

// lpgemm_out_dtype -> OutFormat; -1 for anything but F32, BF16 and F16.
inline int format_of(lpgemm_out_dtype d)
{
    switch (d) {
    case LPGEMM_OUT_F32: return OUT_F32;
    case LPGEMM_OUT_BF16: return OUT_BF16;
    case LPGEMM_OUT_F16: return OUT_F16;
    default: return -1;
    }
}

inline uintptr_t element_bytes(int format) { return format == OUT_F32 ? 4u : 2u; }

// A launch has fewer than 2^32 threads, of 256 to a workgroup: launch(first,
// count, blocks) for the rows in ranges that one holds (2^30 - 64 rows of up to
// 128 values).
template <typename Launch>
lpgemm_status launch_rows(int64_t rows, int64_t items, int64_t block_items, Launch launch)
{
    constexpr int64_t kMostBlocks = (1 << 24) - 1;
    if (rows * items > INT32_MAX * block_items) return LPGEMM_ERR_UNSUPPORTED;
    const int64_t most = kMostBlocks * block_items / items;
    for (int64_t first = 0; first < rows; first += most) {
        const int64_t count = std::min(most, rows - first);
        launch(first, count, dim3((unsigned)ceil_div(count * items, block_items)));
        const lpgemm_status st = launched();
        if (st != LPGEMM_OK) return st;
    }
    return LPGEMM_OK;
}

constexpr int kMaxDevices = 64;
constexpr int kXcds = 8;  // MI355X: 8 XCDs, workgroup ids dealt round robin over them

// Dynamic LDS above 64 KB has to be asked for, once per kernel and device.
template <typename Kernel>
lpgemm_status allow_lds(Kernel kernel, int bytes, std::once_flag *once, hipError_t *err)
{
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return LPGEMM_ERR_HIP;
    std::call_once(once[dev], [&] {
        err[dev] = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    return err[dev] == hipSuccess ? LPGEMM_OK : LPGEMM_ERR_HIP;
}

}  // namespace lpgemm
