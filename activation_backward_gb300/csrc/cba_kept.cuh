// cba_kept.cuh -- values that the runtime is asked for once per process.
#pragma once

#include <atomic>
#include <cuda_runtime_api.h>

namespace cba {

// The positive number that `query(&n)` gives: asked for until it has succeeded
// once, then kept in `kept` (0 at first).  A failure is returned and not kept, so
// that a call after it starts afresh.
template <typename Query>
cudaError_t kept_value(std::atomic<int> &kept, int *value, Query query) {
    int n = kept.load(std::memory_order_relaxed);
    if (n == 0) {
        const cudaError_t e = query(&n);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        kept.store(n, std::memory_order_relaxed);
    }
    *value = n;
    return cudaSuccess;
}

}  // namespace cba
