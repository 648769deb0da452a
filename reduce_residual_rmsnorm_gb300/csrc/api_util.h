// Host-side argument checks shared by the translation units of the C ABI:
// the calling thread's error detail, alignment, and overlap of buffers.
#pragma once

#include <cstdint>

namespace tsfn {

constexpr int64_t kMaxRows = 0x7FFFFFFFLL;

// Record the reason of a failed call for ts_last_error_detail(); returns status.
int fail(int status, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clear the reason; returns TS_OK.
int ok();
const char *last_detail();

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi)
    const char *name = "";
};

inline Span span(const void *p, int64_t bytes, const char *name)
{
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + (uintptr_t)(bytes > 0 ? bytes : 0);
    s.name = name;
    return s;
}

inline bool overlap(const Span &a, const Span &b)
{
    if (a.lo == a.hi || b.lo == b.hi)
        return false;
    return a.lo < b.hi && b.lo < a.hi;
}

}  // namespace tsfn
