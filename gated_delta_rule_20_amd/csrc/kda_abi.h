// kda_abi.h -- what the C entry points share: the calling thread's last error
// and the argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda.h"

namespace kda_abi {

extern thread_local char g_err[512];

// Records the message for kda_last_error_message and returns st.
kda_status_t fail(kda_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));

inline kda_status_t ok()
{
    g_err[0] = 0;
    return KDA_SUCCESS;
}

inline kda_status_t hip_fail(hipError_t e, const char *what)
{
    return fail(KDA_ERROR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace kda_abi
