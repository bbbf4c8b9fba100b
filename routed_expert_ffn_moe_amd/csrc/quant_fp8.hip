// Rows to E4M3 codes with fp32 block scales.
//
//   top = max(max |x| over the block, 2^-100),  scale = top / 448,
//   code = round-to-nearest-even E4M3 of 448 x / top
//
// over blocks of 1 x 128 (activations) or 128 x 128 (weights).  Code rows are
// K rounded up to a multiple of 128 wide; the columns behind K get zero codes,
// so that products over them need no mask.  The maximum passes over NaN; a
// NaN element gets the NaN code, and all of a block with an infinity does.
//
// Bound by memory: 8192 x 4000 fp32 in 128 x 128 blocks 33 us, 5.0 TB/s (a copy
// reaches 4.8); 2048 x 2048 bf16 in 1 x 128 blocks 4.3 us, a launch's latency.
#include <type_traits>

#include "quant_fp8.h"

namespace moe {

namespace {

template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void quant_rows(QuantArgs a)
{
    quant_row_blocks<BF16, VEC>(a, (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4), (int64_t)gridDim.x * 16);
}

// One 128 x 128 block per workgroup: 16 rows a pass, the values kept in
// registers between the maximum and the codes.
template <bool BF16, bool VEC>
__global__ __launch_bounds__(256) void quant_blocks(QuantArgs a)
{
    __shared__ float s_max[16];
    const int sub = threadIdx.x & 15, rr = threadIdx.x >> 4;
    const int rb = blockIdx.x / a.KB, kb = blockIdx.x - rb * a.KB;
    const int c = kb * FP8_BLOCK + sub * 8;
    float v[8][8];
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = rb * FP8_BLOCK + p * 16 + rr;
        load8<BF16, VEC>(v[p], a.x, (int64_t)min(r, a.R - 1) * a.ld, c, a.K);
        if (r < a.R)
            m = fmaxf(m, amax8(v[p]));
    }
    m = row16_max(m);
    if (sub == 0)
        s_max[rr] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        m = fmaxf(m, s_max[i]);
    const Fp8Block q = fp8_block(m);
#pragma unroll
    for (int p = 0; p < 8; ++p) {
        const int r = rb * FP8_BLOCK + p * 16 + rr;
        if (r < a.R)
            *(uint2 *)(a.codes + ((int64_t)r * a.KB + kb) * FP8_BLOCK + sub * 8) =
                uint2{fp8x4(v[p][0], v[p][1], v[p][2], v[p][3], q),
                      fp8x4(v[p][4], v[p][5], v[p][6], v[p][7], q)};
    }
    if (threadIdx.x == 0)
        a.scales[blockIdx.x] = q.scale;
}

template <bool BF16, bool VEC>
void launch_typed(const QuantArgs &a, hipStream_t st)
{
    if (a.block_rows == 1) {
        const int64_t n = (int64_t)a.R * a.KB;
        const unsigned wgs = (unsigned)std::min<int64_t>((n + 15) / 16, 4096);
        quant_rows<BF16, VEC><<<wgs, 256, 0, st>>>(a);
    } else {
        const unsigned wgs = (unsigned)((a.R + FP8_BLOCK - 1) / FP8_BLOCK * a.KB);
        quant_blocks<BF16, VEC><<<wgs, 256, 0, st>>>(a);
    }
}

}  // namespace

void launch_quant_fp8(const QuantArgs &a, hipStream_t st)
{
    if (a.R == 0)
        return;
    const bool vec = a.K % 8 == 0;
    if (a.bf16)
        vec ? launch_typed<true, true>(a, st) : launch_typed<true, false>(a, st);
    else
        vec ? launch_typed<false, true>(a, st) : launch_typed<false, false>(a, st);
}

}  // namespace moe
