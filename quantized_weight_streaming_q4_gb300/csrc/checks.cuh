// checks.cuh -- host-side argument checks that the entry points' files share.
#pragma once

#include "common.cuh"

namespace muser {

// A 16-byte aligned pointer that must not be null.
int check_f32(const char* fn, const char* name, const void* p);

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace muser
