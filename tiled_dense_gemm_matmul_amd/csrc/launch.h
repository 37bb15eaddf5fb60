// Launches of any number of workgroups.
#ifndef LAUNCH_H
#define LAUNCH_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gemm_fwd.h"

namespace {

// Calls launch(first, count) for `groups` workgroups of `threads` threads, in
// slices of 2^31 threads: a grid has to stay below 2^32 (from there on it was
// taken without an error and its last workgroups never ran).  Stops at a slice
// that the runtime does not take.
template <class F>
int in_slices(int64_t groups, int threads, F launch) {
    const int64_t most = ((int64_t)1 << 31) / threads;
    for (int64_t first = 0; first < groups; first += most) {
        launch(first, (unsigned)std::min(groups - first, most));
        if (hipGetLastError() != hipSuccess) return GEMM_ERR_LAUNCH;
    }
    return GEMM_OK;
}

}  // namespace

#endif /* LAUNCH_H */
