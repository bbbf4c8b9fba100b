// Tiles of the grouped bf16 products: what a tile number stands for.
#pragma once

#include "common.h"
#include "kernels.h"
#include "rows.h"

namespace moe {

// What a tile multiplies (kernels.h says what P, Q and c are): np rows of P against nq of Q,
// over nc of c, all from where p and q point.
struct Mm16Job {
    const uint16_t *p, *q;
    int64_t out;      // element of the tile's first row
    int np, nq, nc;
    bool there;
    int next;         // where the workgroup goes on
};

// Rows t of a group against column tile tq (y, dx); the weights' c are adjacent in y.
template <int WAY, int BQ>
__device__ __forceinline__ Mm16Job mm16_row_job(const Mm16Args &a, Where t, int tq)
{
    Mm16Job j{};
    const int q0 = tq * BQ;
    j.there = t.g >= 0;
    j.np = t.nrows;
    j.nq = min(BQ, a.Q - q0);
    j.nc = a.C;
    j.p = a.p + (int64_t)t.row0 * a.ldp;
    j.q = a.q + (int64_t)t.g * a.qstride + (WAY == MM_DX ? (int64_t)q0 : (int64_t)q0 * a.ldq);
    j.out = (int64_t)t.row0 * a.ldo + q0;
    return j;
}

// Tile (tp, tq) of the matrices dw, whose row tiles are numbered on from group to group.
template <int BP, int BQ>
__device__ __forceinline__ Mm16Job mm16_dw_job(const Mm16Args &a, int tp, int tq)
{
    Mm16Job j{};
    const int ntp = (a.P + BP - 1) / BP, g = tp / ntp, p0 = (tp - g * ntp) * BP, q0 = tq * BQ;
    int lo = 0, hi = a.M;
    if (a.offsets) {
        lo = min(max(uniform_load(a.offsets + g), 0), a.M);
        hi = min(uniform_load(a.offsets + g + 1), a.M);
    }
    j.there = true;
    j.np = min(BP, a.P - p0);
    j.nq = min(BQ, a.Q - q0);
    j.nc = max(hi - lo, 0);
    j.p = a.p + (int64_t)lo * a.ldp + p0;
    j.q = a.q + (int64_t)lo * a.ldq + q0;
    j.out = (int64_t)g * a.ostride + (int64_t)p0 * a.ldo + q0;
    return j;
}

// Tiles of bp x bq, an upper bound where the groups have their own (rows.h).
inline int64_t mm16_tile_count(const Mm16Args &a, int bp, int bq)
{
    const int64_t ntq = ((int64_t)a.Q + bq - 1) / bq;
    if (a.way == MM_DW)
        return a.G * (((int64_t)a.P + bp - 1) / bp) * ntq;
    return (a.G > 1 ? a.M / bp + a.G : ((int64_t)a.M + bp - 1) / bp) * ntq;
}

}  // namespace moe
