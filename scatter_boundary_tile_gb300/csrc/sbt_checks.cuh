// Argument checks shared by the C ABI's files.
#pragma once

#include "sbt_internal.cuh"

#define SBT_TRY(call)                   \
    do {                                \
        const sbt_status st_ = (call);  \
        if (st_) return st_;            \
    } while (0)

namespace sbt_checks {

// Messages are put together only where a check fails.
inline std::string say(const char* what, const char* text) { return std::string(what) + text; }

inline sbt_status check_dtype(sbt_dtype dtype, const char* what) {
    const int es = sbt_dtype_size(dtype);
    if (es != 2 && es != 4) return sbt_fail(SBT_ERR_UNSUPPORTED, say(what, ": unsupported dtype"));
    return SBT_OK;
}

inline sbt_status check_workspace(const void* ws, size_t bytes, size_t need, const char* what) {
    if (!ws || bytes < need)
        return sbt_fail(SBT_ERR_ALIGNMENT, say(what, ": workspace smaller than its size query"));
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
        return sbt_fail(SBT_ERR_ALIGNMENT, say(what, ": workspace must be 256-byte aligned"));
    return SBT_OK;
}

}  // namespace sbt_checks
