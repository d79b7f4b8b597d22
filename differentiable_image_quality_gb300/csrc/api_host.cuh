// Host-side helpers shared by the entry points of the C ABI.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "gbssim.h"

namespace gbssim {

// An NVTX range named after the entry point, open for the call's host-side work
// (argument checks, planning, launches), so that a profiler's timeline shows
// which call issued which kernels.  With no profiler attached both NVTX calls
// return at once.
struct CallRange {
    explicit CallRange(const char *name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange &) = delete;
    CallRange &operator=(const CallRange &) = delete;
};

inline int cuda_fail(cudaError_t e)
{
    (void)cudaGetLastError();  // clear a sticky launch error so the next call starts clean
    return e == cudaSuccess ? GBSSIM_OK : GBSSIM_ECUDA;
}

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Number of SMs of the current device (a launch fact, read once per device).
inline cudaError_t current_sm_count(int *out, int *device = nullptr)
{
    constexpr int kMost = 64;
    static std::atomic<int> known[kMost];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (device) *device = dev;
    if (dev < kMost && (*out = known[dev].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < kMost) known[dev].store(*out, std::memory_order_relaxed);
    return e;
}

}  // namespace gbssim
