// Host helpers shared by the translation units that implement the C ABI.
#pragma once

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "rkv.h"

namespace rkv {
namespace api {

// An NVTX range around one entry point, so a profile of the whole path splits by API call.
// Costs a few nanoseconds when no profiler is attached.
struct ApiRange {
    explicit ApiRange(const char* name) { nvtxRangePushA(name); }
    ~ApiRange() { nvtxRangePop(); }
    ApiRange(const ApiRange&) = delete;
    ApiRange& operator=(const ApiRange&) = delete;
};

inline uint64_t align_up(uint64_t x, uint64_t a) { return (x + a - 1) / a * a; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// A failed CUDA call becomes RKV_ERR_CUDA; with RKV_DEBUG set in the environment its
// CUDA error string is also printed to stderr.
inline rkv_status cuda_status(cudaError_t e)
{
    if (e == cudaSuccess)
        return RKV_OK;
    static const bool verbose = std::getenv("RKV_DEBUG") != nullptr;
    if (verbose)
        std::fprintf(stderr, "librkv: CUDA error %d: %s\n", static_cast<int>(e), cudaGetErrorString(e));
    return RKV_ERR_CUDA;
}

}  // namespace api
}  // namespace rkv
