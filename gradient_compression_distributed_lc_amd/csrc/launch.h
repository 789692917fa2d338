// launch.h -- kernel launches of the library: one place that reports a failed
// launch and, while profiling is on, brackets the kernel with events.
#ifndef TLC_LAUNCH_H
#define TLC_LAUNCH_H

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <mutex>
#include <vector>

#include "tlc.h"

namespace tlc_internal {

struct ProfRec {
    const char* name;
    hipEvent_t a, b;
};
inline std::mutex g_prof_mu;
inline bool g_prof_on = false;
inline char g_prof_only[48] = {0};  // when set, only this kernel is bracketed
inline std::vector<ProfRec> g_prof;

template <typename Launch>
int launch(const char* name, hipStream_t st, Launch&& fn) {
    hipEvent_t a = nullptr, b = nullptr;
    bool prof;
    {
        std::lock_guard<std::mutex> lk(g_prof_mu);
        prof = g_prof_on && (!g_prof_only[0] || strcmp(g_prof_only, name) == 0);
    }
    if (prof) {
        if (hipEventCreate(&a) != hipSuccess || hipEventCreate(&b) != hipSuccess) return TLC_ERR_HIP;
        if (hipEventRecord(a, st) != hipSuccess) return TLC_ERR_HIP;
    }
    fn();
    if (hipGetLastError() != hipSuccess) return TLC_ERR_HIP;
    if (prof) {
        if (hipEventRecord(b, st) != hipSuccess) return TLC_ERR_HIP;
        std::lock_guard<std::mutex> lk(g_prof_mu);
        g_prof.push_back({name, a, b});
    }
    return TLC_OK;
}

// The same for `blocks` blocks of `threads` threads that may be too many for
// one launch: HIP refuses 2^32 threads, and past them runs what is left modulo
// 2^32 without an error.  Calls fn(first block, blocks of this launch).
template <typename Launch>
int launch_blocks(const char* name, hipStream_t st, uint64_t blocks, uint32_t threads, Launch&& fn) {
    const uint64_t most = 0xFFFFFFFFull / threads;
    for (uint64_t first = 0; first < blocks; first += most) {
        const uint32_t here = (uint32_t)std::min(most, blocks - first);
        const int rc = launch(name, st, [&] { fn(first, here); });
        if (rc) return rc;
    }
    return TLC_OK;
}

}  // namespace tlc_internal

#endif  // TLC_LAUNCH_H
