// errors.hpp -- the thread-local error message behind gdnq_last_error and
// the checks that every C entry point shares (internal).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "gdnq.h"

namespace gdnq {

int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();                       // clears the message
int launched(hipError_t e);     // ok(), or GDNQ_ELAUNCH with the runtime's message

struct Span {
    const void *p;
    size_t n;
    const char *name;
};

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline bool overlap(const Span &a, const Span &b)
{
    if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.n && b0 < a0 + a.n;
}

}  // namespace gdnq
