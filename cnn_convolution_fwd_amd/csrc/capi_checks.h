// Checks of arguments that the C entry points share.
#pragma once

#include "internal.h"

namespace cfwd {

// No exception leaves the library: what is left to throw is the allocation of an error text.
template <typename F>
cfwd_status guarded(F f) {
    try {
        return f();
    } catch (...) {
        return CFWD_ERR_HIP;
    }
}

inline cfwd_status invalid(const char* why) { return set_error(CFWD_ERR_INVALID_ARG, why); }

inline bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
inline size_t float_size(cfwd_dtype t) { return t == CFWD_F32 ? 4 : t == CFWD_BF16 ? 2 : 0; }

struct Span {
    const void* p;
    unsigned long long bytes;
};

inline bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

}  // namespace cfwd
