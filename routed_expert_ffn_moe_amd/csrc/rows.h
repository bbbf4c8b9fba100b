// Row tiles of grouped rows, which the grouped products share.
#pragma once

#include "common.h"

namespace moe {

// A value of read-only memory at a uniform address: a scalar load, whose wait
// does not touch the copies in flight.
template <class T>
__device__ __forceinline__ T uniform_load(const T *p)
{
    return *(const __attribute__((address_space(4))) T *)(uintptr_t)p;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Buffer of the bytes from p on; an offset of DROP is out of its range: loads give 0,
// stores do nothing.
constexpr int DROP = (int)0x80000000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_from(const void *p)
{
    return __builtin_amdgcn_make_buffer_rsrc((void *)p, 0, 0x7FFFFFFF, 0x00027000);
}

// A tile: rows [row0, row0 + nrows) of group g (g = -1: none), columns from n0.
struct Where {
    int g, row0, nrows, n0, q;
};

// Row tile mt of grouped rows.  The tiles of group g take the numbers from
// offsets[g] / BM + g on, at most offsets[g + 1] / BM + g: a number's group is
// found by bisection without a sum over the groups before it (the numbers that
// a group leaves over are empty tiles).  Offsets outside 0..M are cut off.
template <int BM>
__device__ __forceinline__ Where find_rows(const int32_t *offsets, int G, int M, int mt)
{
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int first = min(max(uniform_load(offsets + mid), 0), M) / BM + mid;
        if (first <= mt)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int a = min(max(uniform_load(offsets + lo), 0), M);
    const int b = min(uniform_load(offsets + lo + 1), M);
    const int m = mt - (a / BM + lo), row0 = a + m * BM;
    if (m < 0 || row0 >= b)
        return Where{-1, 0, 0, 0, 0};
    return Where{lo, row0, min(BM, b - row0), 0, 0};
}

}  // namespace moe
