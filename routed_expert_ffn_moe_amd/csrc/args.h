// Checks of arguments that the entry points of the operators share.
#pragma once

#include <cstdint>

#include "../../include/moe.h"
#include "kernels.h"

namespace moe {

inline bool aligned(const void *p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool overlap(const void *a, int64_t na, const void *b, int64_t nb)
{
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

inline int bad(const char *what) { return api_fail(MOE_EINVAL, what); }

}  // namespace moe
