// Argument checks and error reporting shared by the C-ABI sources.
#pragma once

#include "xpress.h"

#include <hip/hip_runtime.h>

namespace xpress {

// Records the calling thread's message (xpress_last_error) and returns `st`.
xpress_status fail(xpress_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
xpress_status hip_check(hipError_t e, const char* what);

inline bool aligned_to(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

xpress_status check_ptr(const void* p, const char* name);  // not NULL, 16-byte aligned

}  // namespace xpress

#define XP_TRY(expr, what)                                   \
  do {                                                       \
    xpress_status st_ = xpress::hip_check((expr), (what));   \
    if (st_ != XPRESS_OK) return st_;                        \
  } while (0)

#define XP_PTR(p)                                        \
  do {                                                   \
    xpress_status st_ = xpress::check_ptr((p), #p);      \
    if (st_ != XPRESS_OK) return st_;                    \
  } while (0)
