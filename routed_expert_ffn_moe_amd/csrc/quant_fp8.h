// Quantising rows of bf16 or fp32 values to E4M3 codes in blocks of 1 x 128.
#pragma once

#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

// 16 bytes at any element's address (full speed where they are aligned)
typedef uint32_t words4 __attribute__((ext_vector_type(4), aligned(2)));

// The 8 elements at column c of a row, 0 behind K.  VEC: K is a multiple of 8,
// so they are all inside or all behind.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(float (&v)[8], const void *x, int64_t row, int c, int K)
{
    if constexpr (VEC) {
        if (c >= K) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = 0.0f;
        } else if constexpr (BF16) {
            const words4 r = *(const words4 *)((const uint16_t *)x + row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(r[i] << 16);
                v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
            }
        } else {
            const words4 p = *(const words4 *)((const float *)x + row + c);
            const words4 q = *(const words4 *)((const float *)x + row + c + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i] = __uint_as_float(p[i]);
                v[4 + i] = __uint_as_float(q[i]);
            }
        }
    } else if (c + 8 <= K) {  // at any element's address
        load8<BF16, true>(v, (const char *)x + row * (BF16 ? 2 : 4), 0, c, K);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t at = row + c + i;
            v[i] = c + i >= K ? 0.0f : BF16 ? bf2f(((const uint16_t *)x)[at]) : ((const float *)x)[at];
        }
    }
}

__device__ __forceinline__ float amax8(const float (&v)[8])
{
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        m = fmaxf(m, fabsf(v[i]));
    return m;
}

// The blocks b, b + step, ... of 1 x 128: a block per 16 lanes, 8 elements a lane.
template <bool BF16, bool VEC>
__device__ __forceinline__ void quant_row_blocks(const QuantArgs &a, int64_t b, int64_t step)
{
    const int64_t n = (int64_t)a.R * a.KB;
    const int sub = threadIdx.x & 15;
    for (; b < n; b += step) {
        const int64_t r = b / a.KB;
        const int c = (int)(b - r * a.KB) * FP8_BLOCK + sub * 8;
        float v[8];
        load8<BF16, VEC>(v, a.x, r * a.ld, c, a.K);
        const Fp8Block q = fp8_block(row16_max(amax8(v)));
        *(uint2 *)(a.codes + b * FP8_BLOCK + sub * 8) =
            uint2{fp8x4(v[0], v[1], v[2], v[3], q), fp8x4(v[4], v[5], v[6], v[7], q)};
        if (sub == 0)
            a.scales[b] = q.scale;
    }
}

}  // namespace moe
