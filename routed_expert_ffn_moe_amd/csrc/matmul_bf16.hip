// Grouped products of bf16 rows with row-major bf16 weights, forward and
// backward, in one form:
//
//   out[p, q] = sum over c of P[p, c] Q[q, c]   (+ add[p, q])
//
//   y  = x w^T     p a row of the group, q of N, c over K: both operands have c
//                  adjacent in memory
//   dx = dy w      p a row of the group, q of K, c over N: w has q adjacent
//   dw = dy^T x    p of N, q of K, c over the group's rows: both have p, q adjacent
//
// Sums in fp32, the addend joined in fp32, rounded once.
#include <algorithm>
#include <cmath>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "mm16.h"
#include "quant_fp8.h"

namespace moe {

namespace {

template <bool F32>
__device__ __forceinline__ void put(const Mm16Args &a, int64_t at, float v)
{
    if constexpr (F32) {
        if (a.add)
            v += ((const float *)a.add)[at];
        ((float *)a.out)[at] = v;
    } else {
        if (a.add)
            v += bf2f(((const uint16_t *)a.add)[at]);
        ((uint16_t *)a.out)[at] = (uint16_t)cvt_bf2(v, 0.0f);
    }
}

// ---- any strides and alignment ----------------------------------------------

// 64 x 64 tiles, 32 deep, through registers to LDS, where both operands lie with
// c adjacent.  Elements outside the operands are 0.
constexpr int ANY_T = 64, ANY_C = 32, ANY_LD = ANY_C + 8;

// Eight elements of an operand: along c of row `r` (c adjacent), or along the
// rows from `r` at depth c.
template <bool ADJ>
__device__ __forceinline__ u16x8 any_load(const uint16_t *base, int64_t ld, int r, int c, int nr, int nc)
{
    u16x8 v{0, 0, 0, 0, 0, 0, 0, 0};
    const int lim = ADJ ? nc - c : nr - r;
    if (ADJ ? r >= nr : c >= nc)
        return v;
    const uint16_t *s = base + (ADJ ? (int64_t)r * ld + c : (int64_t)c * ld + r);
    if (lim >= 8) {
        const words4 w = *(const words4 *)s;
        return __builtin_bit_cast(u16x8, w);
    }
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < lim)
            v[i] = s[i];
    return v;
}

template <bool ADJ>
__device__ __forceinline__ void any_store(uint16_t *s, int r, int c, u16x8 v)
{
    if constexpr (ADJ) {
        *(u16x8 *)(s + r * ANY_LD + c) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[(r + i) * ANY_LD + c] = v[i];
    }
}

template <int WAY, bool F32>
__global__ __launch_bounds__(256) void mm16_any(Mm16Args a, int tiles)
{
    constexpr bool PA = WAY != MM_DW, QA = WAY == MM_Y;
    __shared__ __attribute__((aligned(16))) uint16_t sp[ANY_T * ANY_LD], sq[ANY_T * ANY_LD];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4, w = tid >> 6;
    const int wp = (w & 1) * 32, wq = (w >> 1) * 32;
    // the thread's eight elements of each operand's step
    const int pr = PA ? tid >> 2 : (tid & 7) * 8, pc = PA ? (tid & 3) * 8 : tid >> 3;
    const int qr = QA ? tid >> 2 : (tid & 7) * 8, qc = QA ? (tid & 3) * 8 : tid >> 3;
    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
        const int ntq = (a.Q + ANY_T - 1) / ANY_T, tp = id / ntq, tq = id - tp * ntq;
        Mm16Job j;
        if constexpr (WAY == MM_DW) {
            j = mm16_dw_job<ANY_T, ANY_T>(a, tp, tq);
        } else {
            Where t{0, tp * ANY_T, min(ANY_T, a.M - tp * ANY_T), 0, 0};
            if (a.offsets)
                t = find_rows<ANY_T>(a.offsets, a.G, a.M, tp);
            j = mm16_row_job<WAY, ANY_T>(a, t, tq);
        }
        if (!j.there)
            continue;
        floatx4 acc[2][2] = {};
        u16x8 vp = any_load<PA>(j.p, a.ldp, pr, pc, j.np, j.nc);
        u16x8 vq = any_load<QA>(j.q, a.ldq, qr, qc, j.nq, j.nc);
        for (int c = 0; c < j.nc; c += ANY_C) {
            __syncthreads();
            any_store<PA>(sp, pr, pc, vp);
            any_store<QA>(sq, qr, qc, vq);
            __syncthreads();
            if (c + ANY_C < j.nc) {
                vp = any_load<PA>(j.p, a.ldp, pr, c + ANY_C + pc, j.np, j.nc);
                vq = any_load<QA>(j.q, a.ldq, qr, c + ANY_C + qc, j.nq, j.nc);
            }
            bf16x8 fp[2], fq[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                fp[i] = *(const bf16x8 *)(sp + (wp + i * 16 + l16) * ANY_LD + lg * 8);
                fq[i] = *(const bf16x8 *)(sq + (wq + i * 16 + l16) * ANY_LD + lg * 8);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    acc[i][k] = mfma16(fq[k], fp[i], acc[i][k]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int p = wp + i * 16 + l16, q = wq + k * 16 + lg * 4 + r;
                    if (p < j.np && q < j.nq)
                        put<F32>(a, j.out + (int64_t)p * a.ldo + q, acc[i][k][r]);
                }
    }
}

template <int WAY>
void launch_any(const Mm16Args &a, hipStream_t st)
{
    const int64_t tiles = mm16_tile_count(a, ANY_T, ANY_T);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1 << 20);
    if (a.out_f32)
        mm16_any<WAY, true><<<grid, 256, 0, st>>>(a, (int)tiles);
    else
        mm16_any<WAY, false><<<grid, 256, 0, st>>>(a, (int)tiles);
}

}  // namespace

namespace {

// Tiles of the variants for whole pieces of 16 bytes (matmul_bf16_tile.h), with what
// 64 of c cost in us: a tile alone, and on all CUs each of 256 tiles (several small
// ones share a CU).
struct Shape {
    int bp, bq;
    double alone, busy, end;
};

// Fitted to 56 products of each way, of 1 to 65536 rows in 1 to 256 groups, N and K
// from 72 to 4096, each with all tiles: the pick's time is on average 4% (y), 5% (dx)
// and 2% (dw) above the best tile's.  In us, largest against smallest tiles of that
// list: 8192 x 4096 x 4096 201 against 1456 (y), 48 rows of 256 groups, N=768, K=2048
// 138 against 59.  dx has no tiles of 16 columns, whose rows of c would be 32 bytes;
// of dw, whose depth is the group's rows, the small tiles' outputs cost most (`end`):
// 256 groups of 64 rows 236 against 388.
constexpr Shape SHAPES_Y[] = {{256, 256, 1.4, 1.9, 0}, {128, 256, 1.0, 1.08, 0}, {64, 256, 0.89, 0.8, 0},
                              {64, 128, 0.64, 0.44, 0}, {64, 64, 0.40, 0.34, 0}, {16, 64, 0.29, 0.21, 0},
                              {16, 16, 0.166, 0.08, 0}};
constexpr Shape SHAPES_DX[] = {{256, 256, 1.6, 1.95, 0}, {128, 256, 1.1, 1.15, 0}, {64, 256, 0.95, 0.87, 0},
                               {64, 128, 0.73, 0.48, 0}, {64, 64, 0.50, 0.41, 0}, {16, 64, 0.44, 0.28, 0}};
constexpr Shape SHAPES_DW[] = {{256, 256, 1.19, 1.69, 5.7}, {128, 128, 0.84, 0.57, 1.8}, {64, 64, 0.51, 0.275, 0.66}};

// The shape that takes least time.  Groups whose balanced rows (1.4 standard
// deviations above the mean) fit into a tile have one, larger ones leave half a tile
// empty.
template <int N>
int mm16_shape(const Mm16Args &a, const Shape (&shapes)[N])
{
    int best = 0;
    double least = 1e300;
    const double per = (double)a.M / a.G;
    for (int i = 0; i < N; ++i) {
        const Shape &s = shapes[i];
        const double tq = (double)((a.Q + s.bq - 1) / s.bq);
        double tiles, steps;
        if (a.way == MM_DW) {
            tiles = a.G * tq * ((a.P + s.bp - 1) / s.bp);
            steps = std::max(1.0, std::ceil(per / 64));
        } else {
            tiles = tq * (a.G == 1                                ? (double)((a.M + s.bp - 1) / s.bp)
                          : per + 1.4 * std::sqrt(per) <= s.bp ? (double)std::min(a.M, a.G)
                                                                  : (double)a.M / s.bp + 0.5 * a.G);
            steps = std::ceil(a.C / 64.0);
        }
        const double t = steps * std::max(s.alone, s.busy * tiles / 256) + s.end * std::max(1.0, tiles / 256);
        if (t < least) {
            least = t;
            best = i;
        }
    }
    return best;
}

// Whole pieces of 16 bytes along every row, and offsets inside a tile that fit 31
// bits.
bool whole_pieces(const Mm16Args &a)
{
    auto on16 = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
    const int esz = a.out_f32 ? 4 : 2;
    const bool sizes = a.Q % 8 == 0 && (a.way == MM_DW ? a.P % 8 == 0 : a.C % 8 == 0);
    return sizes && a.ldp % 8 == 0 && a.ldq % 8 == 0 && a.ldo * esz % 16 == 0 &&
           std::max({a.ldp, a.ldq, a.ldo}) < 1 << 20 && on16(a.p) && on16(a.q) && on16(a.out) && on16(a.add);
}

}  // namespace

int64_t mm16_most_tiles(const Mm16Args &a) { return mm16_tile_count(a, 16, 16); }

void launch_mm16(const Mm16Args &a, hipStream_t st)
{
    const bool whole = whole_pieces(a);
    if (a.way == MM_Y)
        whole ? launch_mm16_y(a, mm16_shape(a, SHAPES_Y), st) : launch_any<MM_Y>(a, st);
    else if (a.way == MM_DX)
        whole ? launch_mm16_dx(a, mm16_shape(a, SHAPES_DX), st) : launch_any<MM_DX>(a, st);
    else
        whole ? launch_mm16_dw(a, mm16_shape(a, SHAPES_DW), st) : launch_any<MM_DW>(a, st);
}

}  // namespace moe
