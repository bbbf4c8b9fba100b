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
        const Mm16Job j = find_job<WAY, ANY_T, ANY_T>(a, id);
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

int64_t mm16_most_tiles(const Mm16Args &a) { return mm16_tile_count(a, 16, 16); }

void launch_mm16(const Mm16Args &a, hipStream_t st)
{
    if (mm16_tiles_ok(a))
        return launch_mm16_tiles(a, st);
    if (a.way == MM_Y)
        launch_any<MM_Y>(a, st);
    else if (a.way == MM_DX)
        launch_any<MM_DX>(a, st);
    else
        launch_any<MM_DW>(a, st);
}

}  // namespace moe
