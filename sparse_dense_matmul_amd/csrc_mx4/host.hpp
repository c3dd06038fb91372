// Argument checks and dispatch shared by the 4-bit products and the experts' layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "vspmm.h"

#include "mx4.hpp"

namespace vspmm {
namespace {

constexpr int64_t kI32Max = 2147483647;
constexpr int64_t kRowsMax = 1 << 30;   // rows of an array: the kernels' row numbers run past the end by a tile
constexpr int64_t kWidthMax = 1 << 24;  // elements of a row
constexpr int64_t kThreadsMax = 0xffffffff;  // threads of a launch along x: more are refused by the runtime

vspmm_status launched() { return hipGetLastError() == hipSuccess ? VSPMM_OK : VSPMM_ERR_HIP; }

bool fits(int64_t x) { return x >= 0 && x <= kI32Max; }
bool dense_elt(int elt) { return elt == VSPMM_ELT_BF16 || elt == VSPMM_ELT_F16; }

template <typename F>
auto with_dense(int elt, F &&f) {
    return elt == VSPMM_ELT_BF16 ? f(bf16{}) : f(f16{});
}

// A kernel that may use more LDS than the default limit of 64 KB, up to `most` bytes of its launch's and 1 KB of its own
// (a vote of a block's threads has 256 bytes), says so once for each device (a call on the host of 1.7 us, where a launch
// takes 3).
template <auto Kernel>
void allow_lds(size_t most) {
    static std::atomic<uint64_t> done{0};
    int device = 0;
    if (most <= 63 * 1024 || hipGetDevice(&device) != hipSuccess) return;
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device < 64 && (done.load(std::memory_order_relaxed) & bit)) return;
    if (hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                            int(most)) == hipSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
}

vspmm_status check_dense(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (!fits(n) || !fits(width) || ld < 0) return VSPMM_ERR_DIM;
    if (n > kRowsMax || width > kWidthMax) return VSPMM_ERR_UNSUPPORTED;
    if (n > 0 && width > 0 && !p) return VSPMM_ERR_NULL;
    return VSPMM_OK;
}
// Rows that are written must not overlap.
vspmm_status check_written(int64_t n, int64_t width, int64_t ld, const void *p) {
    if (n > 1 && ld < width) return VSPMM_ERR_DIM;
    return check_dense(n, width, ld, p);
}
[[maybe_unused]] vspmm_status check_mx4(const vspmm_mx4 *a, int64_t n, int64_t width) {
    if (!a) return VSPMM_ERR_NULL;
    if (!fits(n) || !fits(width) || a->ld_codes < 0 || a->ld_scales < 0) return VSPMM_ERR_DIM;
    if (n > kRowsMax || width > kWidthMax) return VSPMM_ERR_UNSUPPORTED;
    if (n > 0 && width > 0 && (!a->codes || !a->scales)) return VSPMM_ERR_NULL;
    return VSPMM_OK;
}

}  // namespace
}  // namespace vspmm
