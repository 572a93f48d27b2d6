// What the C-ABI host files share: the calling thread's error text and the
// checks every call makes.  Defined in zero_abi.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

namespace zero {

// Store the calling thread's error text; returns code.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int ok();  // clears the error text; returns ZERO_OK
int hip_fail(hipError_t e, const char* where);

inline bool aligned(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

inline bool finite_f(float x) { return isfinite(x) != 0; }

// [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + static_cast<uintptr_t>(nb) &&
           y < x + static_cast<uintptr_t>(na);
}

}  // namespace zero
