// SwiGLU between a caller's own products, with gate and up kept in 8 bits for
// the backward pass.
//
//   s = 1 / (1 + exp(-g)),  h = g s u
//   dg = dh u s (1 + g (1 - s)),  du = dh g s
//
// The checkpoint holds g and u as E4M3 codes with a scale for each 1 x 128 block
// (the definition of moe_quant_fp8): half of what bf16 rows take.  The backward
// pass decodes them in registers and gives h again, which the gradient of the
// next matrix needs, so that h need not be kept at all.
//
// s and 1 - s come from e = exp(-|g|) and r = 1 / (1 + e), as r and e r, or e r and r of a
// negative gate: both to 2^-21 of themselves (the exponential and the hardware's reciprocal
// are off by an ulp each), where a difference from 1 would lose 1 - s of large gates
// (dg 2^-20 off at g = 17) and 1 / (1 + exp(-g)) what is left of s below the normal numbers
// (h was 0 from g = -87.4 on; now from -104 on, where e is).  16 lanes a block of 128
// columns, as the codes' scales need them.
//
// Bound by memory: 16384 x 768 with the checkpoint 19 to 21 us (101 MB, 4.8 to 5.4 TB/s);
// the gradient of 48169 x 2048 from codes 169 (993 MB, 5.9 TB/s: more than a copy's 4.9, with
// three parts in five of it written).
#include <algorithm>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "quant_fp8.h"

namespace moe {

namespace {

// Blocks of 1 x 128: 16 lanes each, 8 columns a lane.
struct Block {
    int64_t row;
    int kb, c;  // number of the block in its row, the lane's first column
};

// Rows in use: all, or as many as the count in memory says.
__device__ __forceinline__ int64_t rows_used(const SwigluArgs &a)
{
    return a.used ? min(max(*a.used, 0), a.R) : a.R;
}

// Quotient by the blocks of a row (host: div_magic).
__device__ __forceinline__ Block block_at(const SwigluArgs &a, uint32_t b)
{
    Block r;
    r.row = (int64_t)(((uint64_t)b * a.magic) >> a.magic_shift);
    r.kb = (int)(b - (uint32_t)r.row * (uint32_t)a.KB);
    r.c = r.kb * FP8_BLOCK + (int)(threadIdx.x & 15) * 8;
    return r;
}

// The lane's 8 codes, and the block's scale from its first lane.
__device__ __forceinline__ void keep8(const float (&v)[8], uint8_t *codes, float *scale)
{
    const Fp8Block q = fp8_block(row16_max(amax8(v)));
    *(uint2 *)codes = uint2{fp8x4(v[0], v[1], v[2], v[3], q), fp8x4(v[4], v[5], v[6], v[7], q)};
    if ((threadIdx.x & 15) == 0)
        *scale = q.scale;
}

// s and 1 - s of a gate.
struct Sigmoid {
    float s, rest;
};

__device__ __forceinline__ Sigmoid sigmoid(float z)
{
    const float e = expf(-fabsf(z)), r = __builtin_amdgcn_rcpf(1.0f + e);
    return z < 0.0f ? Sigmoid{e * r, r} : Sigmoid{r, e * r};
}

template <bool BF16, bool KEEP>
__global__ __launch_bounds__(256) void swiglu_rows(SwigluArgs a)
{
    const uint32_t n = (uint32_t)(rows_used(a) * a.KB), step = gridDim.x * 16;
    for (uint32_t b = blockIdx.x * 16 + (threadIdx.x >> 4); b < n; b += step) {
        const Block k = block_at(a, b);
        float g[8], u[8], h[8];
        load8<BF16, false>(g, a.gate, k.row * a.ld, k.c, a.I);
        load8<BF16, false>(u, a.up, k.row * a.ld, k.c, a.I);
        if constexpr (KEEP) {
            const int64_t at = k.row * 2 * a.KB + k.kb;
            const int sub = (threadIdx.x & 15) * 8;
            keep8(g, a.codes + at * FP8_BLOCK + sub, a.scales + at);
            keep8(u, a.codes + (at + a.KB) * FP8_BLOCK + sub, a.scales + at + a.KB);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = g[i] * sigmoid(g[i]).s * u[i];
        store8<BF16>(h, a.h, k.row * a.ldh + k.c, a.I - k.c);
    }
}

template <bool BF16, bool KEPT>
__global__ __launch_bounds__(256) void swiglu_rows_grad(SwigluArgs a)
{
    const uint32_t n = (uint32_t)(rows_used(a) * a.KB), step = gridDim.x * 16;
    for (uint32_t b = blockIdx.x * 16 + (threadIdx.x >> 4); b < n; b += step) {
        const Block k = block_at(a, b);
        if (k.c >= a.I)
            continue;
        float g[8], u[8], d[8];
        load8<BF16, false>(d, a.dh, k.row * a.ldh, k.c, a.I);
        if constexpr (KEPT) {
            const int64_t at = k.row * 2 * a.KB + k.kb;
            const int sub = (threadIdx.x & 15) * 8;
            decode8(g, a.codes + at * FP8_BLOCK + sub, a.scales[at]);
            decode8(u, a.codes + (at + a.KB) * FP8_BLOCK + sub, a.scales[at + a.KB]);
        } else {
            load8<BF16, false>(g, a.gate, k.row * a.ld, k.c, a.I);
            load8<BF16, false>(u, a.up, k.row * a.ld, k.c, a.I);
        }
        float h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Sigmoid s = sigmoid(g[i]);
            const float z = g[i] * s.s;
            h[i] = z * u[i];
            const float slope = fmaf(z, s.rest, s.s);  // s (1 + g (1 - s))
            g[i] = d[i] * u[i] * slope;
            u[i] = d[i] * z;
        }
        const int left = a.I - k.c;
        store8<BF16>(g, a.dgate, k.row * a.ld + k.c, left);
        store8<BF16>(u, a.dup, k.row * a.ld + k.c, left);
        if (a.h)
            store8<BF16>(h, a.h, k.row * a.ldh + k.c, left);
    }
}

// b / d as (b * magic) >> shift, exact for b < 2^31: with 2^s the power of two not
// below d, magic = ceil(2^(31 + s) / d) is off by less than 2^s / d in units of
// 2^(31 + s) / d, which b < 2^31 leaves below 1.
void div_magic(SwigluArgs &a)
{
    int s = 0;
    while ((1ll << s) < a.KB)
        ++s;
    a.magic = (uint32_t)(((1ull << (31 + s)) + a.KB - 1) / a.KB);
    a.magic_shift = 31 + s;
}

unsigned swiglu_grid(const SwigluArgs &a)
{
    return (unsigned)std::min<int64_t>(((int64_t)a.R * a.KB + 15) / 16, 1 << 16);
}

}  // namespace

void launch_swiglu(SwigluArgs a, hipStream_t st)
{
    div_magic(a);
    const unsigned grid = swiglu_grid(a);
    if (a.bf16)
        a.codes ? swiglu_rows<true, true><<<grid, 256, 0, st>>>(a) : swiglu_rows<true, false><<<grid, 256, 0, st>>>(a);
    else
        a.codes ? swiglu_rows<false, true><<<grid, 256, 0, st>>>(a) : swiglu_rows<false, false><<<grid, 256, 0, st>>>(a);
}

void launch_swiglu_grad(SwigluArgs a, hipStream_t st)
{
    div_magic(a);
    const unsigned grid = swiglu_grid(a);
    if (a.bf16)
        a.codes ? swiglu_rows_grad<true, true><<<grid, 256, 0, st>>>(a)
                : swiglu_rows_grad<true, false><<<grid, 256, 0, st>>>(a);
    else
        a.codes ? swiglu_rows_grad<false, true><<<grid, 256, 0, st>>>(a)
                : swiglu_rows_grad<false, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace moe
