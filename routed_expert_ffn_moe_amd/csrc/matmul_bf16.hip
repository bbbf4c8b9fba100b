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
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "mm16.h"
#include "quant_fp8.h"

namespace moe {

namespace {

// ---- any strides and alignment ----------------------------------------------

// The tiles of mm16.h, staged through registers a step ahead: pieces of 8 elements
// are read at any element's address, and one by one where they end outside the
// operand (0 there).  Two stages in LDS, so that a step has one barrier.
// Bound by what a step waits for, one round of register loads: 6900 x 577 x 937 (dw) 56 us
// with warm caches, 75 cold, where its bytes take 4.7.  Reads two steps ahead made no difference.

// Elements of a piece: along c of element x (c adjacent), or elements from x on at c.
template <bool ADJ>
__device__ __forceinline__ words4 fetch(const uint16_t *base, int64_t ld, int x, int c, int nx, int nc)
{
    words4 v{0, 0, 0, 0};
    const int lim = ADJ ? nc - c : nx - x;
    if (lim <= 0 || (ADJ ? x >= nx : c >= nc))
        return v;
    const uint16_t *s = base + (ADJ ? (int64_t)x * ld + c : (int64_t)c * ld + x);
    if (lim >= 8)
        return *(const words4 *)s;
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < lim)
            v[i >> 1] |= (uint32_t)s[i] << (i & 1) * 16;
    return v;
}

// 8 adjacent results, `left` of them inside the output.  (load8 and store8 in its place
// cost the tiles of 128 x 128 a third of their rate: 5000 x 1001 x 777 with an addend 50 us, so 34.)
template <bool F32>
__device__ __forceinline__ void put8(const Mm16Args &a, int64_t at, float (&v)[8], int left)
{
    if (left >= 8) {
        if (a.add) {
            float d[8];
            load8<!F32, true>(d, a.add, at, 0, 8);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] += d[i];
        }
        if constexpr (F32) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
                *(words4 *)((float *)a.out + at + 4 * q) =
                    words4{__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                           __float_as_uint(v[4 * q + 3])};
        } else {
            *(words4 *)((uint16_t *)a.out + at) =
                words4{cvt_bf2(v[0], v[1]), cvt_bf2(v[2], v[3]), cvt_bf2(v[4], v[5]), cvt_bf2(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 7; ++i) {
        if (i >= left)
            continue;
        if constexpr (F32)
            ((float *)a.out)[at + i] = v[i] + (a.add ? ((const float *)a.add)[at + i] : 0.0f);
        else
            ((uint16_t *)a.out)[at + i] =
                (uint16_t)cvt_bf2(v[i] + (a.add ? bf2f(((const uint16_t *)a.add)[at + i]) : 0.0f), 0.0f);
    }
}

// WP x WQ waves a tile, and WK groups of them that take every WK-th 64 of c.
template <int WAY, bool F32, int BP, int BQ, int WP, int WQ, int WK>
__global__ __launch_bounds__(64 * WP * WQ * WK) void mm16_any(Mm16Args a, int tiles)
{
    constexpr bool PA = WAY != MM_DW, QA = WAY == MM_Y;
    constexpr int NW = WP * WQ, MB = BP / 16 / WP, NB = BQ / 16 / WQ;
    using P = Operand<BP, PA, !PA>;
    using Q = Operand<BQ, QA, true>;
    constexpr int PI = P::COPIES / NW, QI = Q::COPIES / NW, STAGE = P::BYTES + Q::BYTES;
    static_assert(P::COPIES % NW == 0 && Q::COPIES % NW == 0 && NB % 2 == 0 && (PA || MB % 2 == 0), "whole shares");
    static_assert((WK - 1) * BP * BQ * 4 <= 2 * WK * STAGE, "the sums fit the stages");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * WK * STAGE];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave % NW, kg = wave / NW;
    const int wq = w % WQ, wp = w / WQ;
    uint8_t *const ring = smem + kg * 2 * STAGE;
    for (int id = blockIdx.x; id < tiles; id += gridDim.x) {
        const int ntq = (a.Q + BQ - 1) / BQ, tp = id / ntq, tq = id - tp * ntq;
        Mm16Job j;
        if constexpr (WAY == MM_DW) {
            j = mm16_dw_job<BP, BQ>(a, tp, tq);
        } else {
            Where t{0, tp * BP, min(BP, a.M - tp * BP), 0, 0};
            if (a.offsets)
                t = find_rows<BP>(a.offsets, a.G, a.M, tp);
            j = mm16_row_job<WAY, BQ>(a, t, tq);
        }
        if (!j.there)
            continue;
        floatx4 acc[NB][MB];
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                acc[c][m] = floatx4{0, 0, 0, 0};
        words4 vp[PI], vq[QI];
        auto load = [&](int c0) {
#pragma unroll
            for (int i = 0; i < PI; ++i) {
                const auto s = P::piece(w * PI + i, lane);
                vp[i] = fetch<PA>(j.p, a.ldp, s.x, c0 + s.c, j.np, j.nc);
            }
#pragma unroll
            for (int i = 0; i < QI; ++i) {
                const auto s = Q::piece(w * QI + i, lane);
                vq[i] = fetch<QA>(j.q, a.ldq, s.x, c0 + s.c, j.nq, j.nc);
            }
        };
        const int n = (j.nc + WK * STEP - 1) / (WK * STEP);
        __syncthreads();  // the tile before is done with LDS
        if (n > 0)
            load(kg * STEP);
        for (int s = 0; s < n; ++s) {
            uint8_t *const st = ring + (s & 1) * STAGE;
#pragma unroll
            for (int i = 0; i < PI; ++i)
                *(u32v<1> *)(st + (w * PI + i) * 1024 + lane * 16) = u32v<1>{vp[i][0], vp[i][1], vp[i][2], vp[i][3]};
#pragma unroll
            for (int i = 0; i < QI; ++i)
                *(u32v<1> *)(st + P::BYTES + (w * QI + i) * 1024 + lane * 16) =
                    u32v<1>{vq[i][0], vq[i][1], vq[i][2], vq[i][3]};
            __syncthreads();
            if (s + 1 < n)
                load(((s + 1) * WK + kg) * STEP);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                bf16x8 qf[NB];
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    qf[c] = Q::read(st + P::BYTES, Q::where(wq * NB + c, lane), h);
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const bf16x8 pf = P::read(st, P::where(wp * MB + m, lane), h);
#pragma unroll
                    for (int c = 0; c < NB; ++c)
                        acc[c][m] = mfma16(qf[c], pf, acc[c][m]);
                }
            }
        }
        if constexpr (WK > 1) {  // the groups' sums, joined in their order by the first one
            __syncthreads();
            floatx4 *sum = (floatx4 *)smem + w * (NB * MB * 64) + lane;
            if (kg > 0)
#pragma unroll
                for (int c = 0; c < NB; ++c)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        sum[((kg - 1) * NW * NB * MB + c * MB + m) * 64] = acc[c][m];
            __syncthreads();
            if (kg > 0)
                continue;
#pragma unroll
            for (int g = 0; g < WK - 1; ++g)
#pragma unroll
                for (int c = 0; c < NB; ++c)
#pragma unroll
                    for (int m = 0; m < MB; ++m)
                        acc[c][m] += sum[(g * NW * NB * MB + c * MB + m) * 64];
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int p = wp * (16 * MB) + (PA ? m * 16 + l16 : paired(m, l16));
#pragma unroll
            for (int c = 0; c < NB / 2; ++c) {
                const int q = wq * (16 * NB) + c * 32 + lg * 8;
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = acc[2 * c][m][i], y = acc[2 * c + 1][m][i];
                    v[i] = lg & 1 ? y : x;
                    v[4 + i] = lg & 1 ? x : y;
                }
                if (p < j.np && q < j.nq)
                    put8<F32>(a, j.out + (int64_t)p * a.ldo + q, v, j.nq - q);
            }
        }
    }
}

// Tiles of 128 x 128 where they give every CU one (5000 x 1001 x 777 (y) 33 us, 40 with
// 64 x 64), else of 64 x 64 by two groups of waves, or by four where the tiles leave CUs
// without one and c is long: 3000 x 333 x 501 (dw, fp32) 62 us by two, 43 by four, 101 x 333 x
// 2050 (y) 15.3 and 13.3, but 73 x 204 x 141 (dw) 5.8 and 6.8; at c of 500 the two are alike
// (101 x 333 x 501 8.2 and 8.4).  Warm caches.
Mm16Pick any_pick(const Mm16Args &a)
{
    if (mm16_tile_count(a, 128, 128) >= 256)
        return Mm16Pick{128, 128, 1, 0, false};
    const bool few = mm16_tile_count(a, 64, 64) <= 256 && (a.way == MM_DW ? a.C / a.G : a.C) >= 512;
    return Mm16Pick{64, 64, few ? 4 : 2, 0, false};
}

template <int WAY>
void launch_any(const Mm16Args &a, Mm16Pick t, hipStream_t st)
{
    const int64_t tiles = mm16_tile_count(a, t.rows, t.cols);
    const unsigned grid = (unsigned)std::min<int64_t>(tiles, 1 << 20);
    auto run = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value;
        if (t.groups == 1)
            mm16_any<WAY, F32, 128, 128, 2, 2, 1><<<grid, 256, 0, st>>>(a, (int)tiles);
        else if (t.groups == 2)
            mm16_any<WAY, F32, 64, 64, 2, 2, 2><<<grid, 512, 0, st>>>(a, (int)tiles);
        else
            mm16_any<WAY, F32, 64, 64, 2, 2, 4><<<grid, 1024, 0, st>>>(a, (int)tiles);
    };
    a.out_f32 ? run(std::true_type{}) : run(std::false_type{});
}

}  // namespace

namespace {

// What a step of 64 of c (dw: of 64 for each group of waves) costs in us with the tiles
// of mm16.h: a tile alone, and on all CUs each of 256 tiles (several small ones share a CU).
struct Cost {
    double alone, busy, end;
};

// `end` is what a tile's sums and output cost, also once a round of tiles.
//
// Fitted to products of 1 to 65536 rows in 1 to 256 groups, N and K from 8 to 4096, each with
// all tiles.  70 others of each way, drawn as they come, take on average 3% (y), 2% (dx)
// and 3.5% (dw) more than with the best tile (warm caches; 33%, 15% and 48% at most).  In us, warm
// / cold caches, largest against smallest tiles of the list: 8192 x 4096 x 4096 198 / 193
// against 1405 / 1433 (y), 48 rows of 256 groups, N=768, K=2048 120 / 138 against 26 / 54; of
// K=8 16384 rows of 256 groups, N=2048 56 / 56 against 759 / 758 (64 x 128 37 / 38).
// dx has no tiles of 16 columns, whose rows of c would be 32 bytes.  Its 64 x 256 costs more
// than the first fit's 0.69 for a step: in 46 products where the two choose apart the tiles
// that 0.78 takes are 13% faster on average (8% cold), in 44 faster, 7% slower at most; 16384 rows of
// 256 groups 180 against 190 (Zipf), 163 against 163 (equal).
// Of dw, whose depth is the group's rows, the small tiles' outputs cost most (`end`): 256
// groups of 64 rows, N=768, K=2048 227 against 376 with 64 x 64.  Few tiles of dw are bound by
// what a CU reads.  There two groups of waves take 64 of c each: 28 / 46 against 37 / 55 for
// 8192 rows, N=256, K=2048 (128 tiles), but 63 / 87 against 60 / 79 for 4096 x 2048 x 2048
// (1024 tiles); and where 32 x 32 gives no more tiles than CUs, each reads half as much: 12 /
// 18 against 16 / 24 for 4096 x 512 x 512, but 43 / 59 against 28 / 46 for the 512 tiles of 8192 x 256 x 2048.
constexpr Cost COST_Y[MM16_NY] = {{1.3, 1.5, 7.8}, {1.1, 0.84, 5.9}, {0.49, 0.44, 1.4},
                                  {0.29, 0.48, 1.5}, {0.19, 0.27, 1.4}, {0.036, 0.06, 1.4}};
constexpr Cost COST_DX[MM16_NDX] = {{1.2, 2.2, 10}, {0.96, 1.1, 5.3}, {0.93, 0.78, 3.6},
                                    {0.75, 0.48, 1.6}, {0.52, 0.59, 1.6}, {0.4, 0.5, 1.5}};
constexpr Cost COST_DW[MM16_NDW] = {{1.19, 1.69, 5.7}, {0.84, 0.57, 1.8}, {0.51, 0.275, 0.66},
                                    {0.73, 0.72, 1.1}, {1.05, 0.88, 1.2}};

// The shape that takes least time.  Groups whose balanced rows (1.4 standard
// deviations above the mean) fit into a tile have one, larger ones leave half a tile
// empty.
//
// Groups of a few rows read their weights once, from memory, and tiles of 16 columns
// keep more of it busy than those of 64, unless c is so short that the tiles' ends
// count.  In us, warm / cold: 48 rows of 256 groups with N=768, K=2048 26 / 54 against 30 /
// 65, 1024 rows 143 / 183 against 149 / 189, but 48 rows with N=2048, K=768 44 / 57 against
// 30 / 57.  Over 60 products of at most 11 rows a group, N from 256 and c from 1024 on, this
// choice is on average 4% / 3% above the best of three tiles (27% / 20% at most: Zipf rows, or c of
// little more than 1024), the costs alone 12% / 15%, 16 x 64 always 10% / 16%.
template <int N>
int mm16_shape(const Mm16Args &a, const Mm16Shape (&shapes)[N], const Cost (&costs)[N])
{
    int best = 0;
    double least = 1e300;
    const double per = (double)a.M / a.G;
    if (a.way == MM_Y && a.G > 1 && a.C >= 1024 && per + 1.4 * std::sqrt(per) <= shapes[N - 1].bp)
        return N - 1;
    for (int i = 0; i < N; ++i) {
        const Mm16Shape &s = shapes[i];
        const double tq = (double)((a.Q + s.bq - 1) / s.bq);
        double tiles, steps;
        if (a.way == MM_DW) {
            tiles = a.G * tq * ((a.P + s.bp - 1) / s.bp);
            steps = std::max(1.0, std::ceil(per / (STEP * s.wk)));
        } else {
            tiles = tq * (a.G == 1                                ? (double)((a.M + s.bp - 1) / s.bp)
                          : per + 1.4 * std::sqrt(per) <= s.bp ? (double)std::min(a.M, a.G)
                                                                  : (double)a.M / s.bp + 0.5 * a.G);
            steps = std::ceil(a.C / (double)STEP);
        }
        const Cost &c = costs[i];
        const double t = steps * std::max(c.alone, c.busy * tiles / 256) + c.end * std::max(1.0, tiles / 256);
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

Mm16Pick mm16_pick(const Mm16Args &a)
{
    if (!whole_pieces(a))
        return any_pick(a);
    const int n = a.way == MM_Y ? mm16_shape(a, MM16_Y, COST_Y) : a.way == MM_DX ? mm16_shape(a, MM16_DX, COST_DX)
                                                                : mm16_shape(a, MM16_DW, COST_DW);
    const Mm16Shape &s = (a.way == MM_Y ? MM16_Y : a.way == MM_DX ? MM16_DX : MM16_DW)[n];
    return Mm16Pick{s.bp, s.bq, s.wk, n, true};
}

void launch_mm16(const Mm16Args &a, hipStream_t st)
{
    const Mm16Pick t = mm16_pick(a);
    if (a.way == MM_Y)
        t.whole ? launch_mm16_y(a, t.shape, st) : launch_any<MM_Y>(a, t, st);
    else if (a.way == MM_DX)
        t.whole ? launch_mm16_dx(a, t.shape, st) : launch_any<MM_DX>(a, t, st);
    else
        t.whole ? launch_mm16_dw(a, t.shape, st) : launch_any<MM_DW>(a, t, st);
}

}  // namespace moe
