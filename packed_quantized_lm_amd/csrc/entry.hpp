// entry.hpp -- what the entry points of operators on tensors check alike (host code).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "api_internal.hpp"
#include "archead.h"

namespace archead {

inline bool bad_type(int t) { return t != ARCHEAD_F32 && t != ARCHEAD_BF16; }
inline int64_t size_of(int t) { return t == ARCHEAD_F32 ? 4 : t == ARCHEAD_BF16 ? 2 : 1; }
inline bool misaligned(const void *p, int64_t bytes) { return (uintptr_t)p % (uintptr_t)bytes != 0; }

// whether everything that `what` launched was taken
inline archead_status launched(const char *what)
{
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return api_fail(ARCHEAD_EHIP, std::string(what) + ": " + hipGetErrorString(e));
    return ARCHEAD_OK;
}

} // namespace archead
