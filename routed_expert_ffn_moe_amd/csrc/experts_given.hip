// The combine of experts run with given routing: y_t = sum_j w[t, j] *
// stage[row of (t, j)] in j order, fp32 sum, rounded once, as in moe_forward;
// an empty slot (row_of < 0) adds nothing whatever its weight, and a token
// with empty slots only gets zeros.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

// 16 bytes of one output row per thread, the rows' pieces loaded together.
template <int KM, bool BF16>
__global__ __launch_bounds__(256) void combine_given(const void *__restrict__ stage,
                                                     const int32_t *__restrict__ row_of,
                                                     const float *__restrict__ topk_w,
                                                     void *__restrict__ y, int T, int H, int k)
{
    constexpr int W = BF16 ? 8 : 4;  // columns of a thread
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int per_row = H / W;
    if (i >= (int64_t)T * per_row)
        return;
    const int64_t t = i / per_row;
    const int c = (int)(i - t * per_row) * W;
    int row[KM];
    float w[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        row[j] = j < k ? row_of[t * k + j] : -1;
        w[j] = j < k ? topk_w[t * k + j] : 0.0f;
    }
    uint4 v[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (row[j] >= 0)
            v[j] = *(const uint4 *)((const char *)stage + ((int64_t)row[j] * H + c) * (BF16 ? 2 : 4));
    float acc[W];
#pragma unroll
    for (int q = 0; q < W; ++q)
        acc[q] = 0.0f;
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        if (row[j] < 0)
            continue;
        const uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if constexpr (BF16) {
                acc[2 * q] = fmaf(w[j], __uint_as_float(u[q] << 16), acc[2 * q]);
                acc[2 * q + 1] = fmaf(w[j], __uint_as_float(u[q] & 0xFFFF0000u), acc[2 * q + 1]);
            } else {
                acc[q] = fmaf(w[j], __uint_as_float(u[q]), acc[q]);
            }
        }
    }
    if constexpr (BF16)
        *(uint4 *)((uint16_t *)y + t * H + c) = uint4{pack_bf2(acc[0], acc[1]), pack_bf2(acc[2], acc[3]),
                                                      pack_bf2(acc[4], acc[5]), pack_bf2(acc[6], acc[7])};
    else
        *(float4 *)((float *)y + t * H + c) = float4{acc[0], acc[1], acc[2], acc[3]};
}

template <bool BF16>
void launch_typed(const CombineArgs &a, hipStream_t st)
{
    const int64_t n = (int64_t)a.T * (a.H / (BF16 ? 8 : 4));
    const unsigned wgs = (unsigned)((n + 255) / 256);
    if (a.k <= 4)
        combine_given<4, BF16><<<wgs, 256, 0, st>>>(a.stage, a.row_of, a.topk_w, a.y, a.T, a.H, a.k);
    else if (a.k <= 8)
        combine_given<8, BF16><<<wgs, 256, 0, st>>>(a.stage, a.row_of, a.topk_w, a.y, a.T, a.H, a.k);
    else
        combine_given<16, BF16><<<wgs, 256, 0, st>>>(a.stage, a.row_of, a.topk_w, a.y, a.T, a.H, a.k);
}

}  // namespace

void launch_combine_given(const CombineArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return;
    if (a.act == ACT_BF16)
        launch_typed<true>(a, st);
    else
        launch_typed<false>(a, st);
}

}  // namespace moe
