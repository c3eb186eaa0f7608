// gg_host.hpp -- what the C entry points share: the thread's last error, the
// device check, launch reports (defined in gg_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

}  // namespace gg
