// Tiles of the grouped bf16 products: what a tile number stands for.
#pragma once

#include "common.h"
#include "kernels.h"
#include "rows.h"

namespace moe {

// What a tile multiplies (kernels.h says what P, Q and c are): P rows p0 .. p0 + np - 1 against Q rows from q0, over c.
struct Mm16Job {
    const uint16_t *p, *q;
    int64_t out;      // element of the tile's first row
    int np, nq, nc, p0, q0;
    bool there;
    int next;         // where the workgroup goes on
};

// Tile `id`; the tiles of neighbouring numbers share their group.
template <int WAY, int BP, int BQ>
__device__ __forceinline__ Mm16Job find_job(const Mm16Args &a, int id)
{
    Mm16Job j{};
    const int ntq = (a.Q + BQ - 1) / BQ, tp = id / ntq, q0 = (id - tp * ntq) * BQ;
    j.q0 = q0;
    j.nq = min(BQ, a.Q - q0);
    if constexpr (WAY == MM_DW) {
        const int ntp = (a.P + BP - 1) / BP, g = tp / ntp;
        int lo = 0, hi = a.M;
        if (a.offsets) {
            lo = min(max(uniform_load(a.offsets + g), 0), a.M);
            hi = min(uniform_load(a.offsets + g + 1), a.M);
        }
        j.p0 = (tp - g * ntp) * BP;
        j.np = min(BP, a.P - j.p0);
        j.nc = max(hi - lo, 0);
        j.p = a.p + (int64_t)lo * a.ldp + j.p0;
        j.q = a.q + (int64_t)lo * a.ldq + q0;
        j.out = (int64_t)g * a.ostride + (int64_t)j.p0 * a.ldo + q0;
        j.there = true;
    } else {
        Where t{0, tp * BP, min(BP, a.M - tp * BP), 0, 0};
        if (a.offsets)
            t = find_rows<BP>(a.offsets, a.G, a.M, tp);
        j.there = t.g >= 0;
        j.p0 = t.row0;
        j.np = t.nrows;
        j.nc = a.C;
        j.p = a.p + (int64_t)t.row0 * a.ldp;
        j.q = a.q + (int64_t)t.g * a.qstride + (WAY == MM_DX ? (int64_t)q0 : (int64_t)q0 * a.ldq);
        j.out = (int64_t)t.row0 * a.ldo + q0;
    }
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
