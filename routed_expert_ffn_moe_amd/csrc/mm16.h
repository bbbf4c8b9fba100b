// Tiles of the grouped bf16 products: what a tile number stands for, and how an
// operand lies in LDS.
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

constexpr int STEP = 64;  // depth of a stage

// Tiles of the kernel for whole pieces of 16 bytes (matmul_bf16_tile.h, where the fields
// are explained), from the largest to the smallest.
struct Mm16Shape {
    int bp, bq, wp, wq, st, ex, wk;
};
constexpr Mm16Shape MM16_Y[] = {{256, 256, 2, 4, 2, 1, 1}, {128, 256, 2, 4, 3, 0, 1}, {64, 128, 2, 2, 3, 0, 1},
                                {64, 64, 2, 2, 3, 0, 2}, {16, 64, 1, 2, 3, 0, 4}, {16, 16, 1, 1, 4, 0, 4}};
constexpr Mm16Shape MM16_DX[] = {{256, 256, 2, 4, 2, 1, 1}, {128, 256, 2, 4, 3, 0, 1}, {64, 256, 2, 4, 3, 0, 1},
                                 {64, 128, 2, 2, 3, 0, 1}, {64, 64, 2, 2, 3, 0, 2}, {16, 64, 1, 2, 3, 0, 4}};
constexpr Mm16Shape MM16_DW[] = {{256, 256, 2, 4, 2, 1, 1}, {128, 128, 2, 2, 2, 1, 1}, {64, 64, 2, 2, 3, 0, 1},
                                 {64, 64, 2, 2, 3, 0, 2}, {32, 32, 1, 1, 4, 0, 4}};
constexpr int MM16_NY = sizeof MM16_Y / sizeof *MM16_Y, MM16_NDX = sizeof MM16_DX / sizeof *MM16_DX,
              MM16_NDW = sizeof MM16_DW / sizeof *MM16_DW;

// The element that row r of block b of 16 holds where the two are not alike: pairs
// of blocks share 32 elements such that a lane's results of a pair are 8 adjacent
// ones, and the rows of a block read both halves of the pieces of 8 elements (so
// that a transposing read falls on all banks).
__device__ __forceinline__ int paired(int b, int r)
{
    return (b >> 1) * 32 + (r >> 2) * 8 + (((b ^ (r >> 2)) & 1) << 2) + (r & 3);
}

// One operand's tile of XN elements by 64 c in LDS, in blocks of 16 elements whose
// order is that of paired() where PAIR says so (always where the read transposes).
template <int XN, bool ADJ, bool PAIR>
struct Operand {
    static constexpr int BYTES = XN * STEP * 2, COPIES = BYTES / 1024;
    static constexpr int ROW = ADJ ? 128 : XN * 2;     // bytes of a row in LDS
    static constexpr int PER = 1024 / ROW;             // rows of a copy
    static_assert(XN % (PAIR ? 32 : 16) == 0 && (ADJ || PAIR), "whole blocks");

    // What the pieces of a row are rotated by.
    __device__ static __forceinline__ int key(int row)
    {
        if (ADJ)
            return (row >> 1) & 7;
        const int half = (row >> 3) & 1;
        return XN >= 128 ? (row & 3) << 2 | half : XN >= 64 ? (row & 2) << 1 | half : (row & 2) | half;
    }
    // Copy i of the tile: the lane's element and c.
    struct Piece {
        int x, c;
    };
    __device__ static __forceinline__ Piece piece(int i, int lane)
    {
        const int row = i * PER + lane / (64 / PER), at = (lane % (64 / PER)) ^ key(row);
        if (!ADJ)
            return Piece{at * 8, row};
        return Piece{PAIR ? paired(row >> 4, row & 15) : row, at * 8};
    }
    // Byte offset in LDS of the lane's fragment of block b: 8 c of one element, c
    // from 8 * (lane / 16) on.
    __device__ static __forceinline__ int where(int b, int lane)
    {
        const int l16 = lane & 15, lg = lane >> 4;
        if (ADJ)
            return b * 2048 + l16 * 128 + ((lg ^ key(l16)) << 4);
        // 16 lanes read 4 c of 16 elements, 4 elements a lane, and get 4 c of one
        const int row = lg * 8 + (l16 >> 2), e = (b >> 1) * 32 + (l16 & 3) * 8;
        return row * ROW + (((e >> 3) ^ key(row)) << 4) + (((b ^ l16) & 1) << 3);
    }
    // The fragment of the 32 c of half h of the step.
    __device__ static __forceinline__ bf16x8 read(const uint8_t *tile, int at, int h)
    {
        if (ADJ)
            return *(const bf16x8 *)(tile + (at ^ (h << 6)));
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) bf16x4 *Ptr;
        const auto p = (__attribute__((address_space(3))) const uint8_t *)tile + at + h * (32 * ROW);
        const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Ptr)p);
        const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Ptr)(p + 4 * ROW));
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    }
};

}  // namespace moe
