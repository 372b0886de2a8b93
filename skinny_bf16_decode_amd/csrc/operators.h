// What the host sides of the operators share: errors and element types.
#pragma once

#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdio.h>

#include "skinny_internal.h"

namespace skinny {

inline skinny_status bad(skinny_status s, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
inline skinny_status bad(skinny_status s, const char *fmt, ...)
{
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_error("%s", buf);
    return s;
}

inline skinny_status hip_bad(hipError_t e, const char *what)
{
    return bad(e == hipErrorOutOfMemory ? SKINNY_ERR_NOMEM : SKINNY_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

inline bool is_type(int t) { return t == SKINNY_TYPE_BF16 || t == SKINNY_TYPE_F32 || t == SKINNY_TYPE_F16; }
inline int type_bytes(int t) { return t == SKINNY_TYPE_F32 ? 4 : 2; }

}  // namespace skinny
