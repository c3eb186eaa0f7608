// gg_host.hpp -- what the C entry points share: the thread's last error, the
// device check, launch reports (defined in gg_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cstdio>

#include "gg_internal.hpp"
#include "gg_moe.h"

namespace gg {

// Records the message for gg_last_error and returns s.
gg_status fail(gg_status s, const char* fmt, ...);
// Clears the message and returns GG_OK.
gg_status ok();
gg_status hip_fail(hipError_t e, const char* what);
// GG_OK if the current device is a gfx950 (cached per device ordinal).
gg_status check_device();
// GG_LOG set (to anything but "0"): every launch reports the kernel variant
// it chose, the workgroup tile and the grid on stderr, one line per call.
bool log_enabled();
void log_launch(const char* op, const LaunchInfo& i, const char* shape);

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }
inline bool is_out_dtype(gg_dtype d) { return d == GG_BF16 || d == GG_F16 || d == GG_F32; }
inline bool is_fp8(gg_dtype d) { return d == GG_F8E4M3 || d == GG_F8E5M2; }
inline size_t size_of(gg_dtype d) { return d == GG_F32 ? 4 : d == GG_BF16 || d == GG_F16 ? 2 : 1; }
inline bool off(const void* p, size_t align) { return ((uintptr_t)p & (align - 1)) != 0; }

inline gg_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace)
        return fail(GG_ERR_NULL, "workspace must be non-NULL");
    if (off(workspace, 256))
        return fail(GG_ERR_ALIGN, "workspace must be 256-byte aligned");
    if (bytes < need)
        return fail(GG_ERR_WORKSPACE, "workspace too small: %zu < %zu bytes", bytes, need);
    return GG_OK;
}

inline void report(const char* op, const LaunchInfo& info, int64_t rows, int64_t cols) {
    char shape[96];
    snprintf(shape, sizeof shape, "(%lld x %lld)", (long long)rows, (long long)cols);
    if (info.grid > 0)
        log_launch(op, info, shape);
}

// What every entry does last: the device check, the launch, the report (of two
// kernels, where the launcher names a second).
template <class Launch>
gg_status go(const char* op, int64_t rows, int64_t cols, Launch launch) {
    gg_status st = check_device();
    if (st != GG_OK)
        return st;
    LaunchInfo info[2]{};
    LaunchInfo* li = log_enabled() ? info : nullptr;
    const hipError_t e = launch(li);
    if (e != hipSuccess)
        return hip_fail(e, op);
    if (li)
        for (const LaunchInfo& i : info)
            report(op, i, rows, cols);
    return ok();
}

}  // namespace gg
