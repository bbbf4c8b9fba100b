// The combine of experts run with given routing: y_t = sum_j w[t, j] *
// stage[row of (t, j)] in j order, fp32 sum, rounded once, as in moe_forward;
// an empty slot (row_of < 0) adds nothing whatever its weight, and a token
// with empty slots only gets zeros.  Rows of the FP8 experts are half values
// under an exponent for each 8 columns (fp8.h).  Bound by reading the staging
// rows: T=8192, H=4096, k=6 90 us, 5.5 TB/s with y.
#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

namespace {

enum { ROWS_F32 = 0, ROWS_BF16 = 1, ROWS_FP8 = 2 };

// 16 bytes of one output row per thread, the rows' pieces loaded together.
template <int KM, int ROWS>
__global__ __launch_bounds__(256) void combine_given(const void *__restrict__ stage,
                                                     const int32_t *__restrict__ row_of,
                                                     const float *__restrict__ topk_w,
                                                     const uint8_t *__restrict__ exps,
                                                     void *__restrict__ y, int T, int H, int k)
{
    constexpr int W = ROWS == ROWS_F32 ? 4 : 8;  // columns of a thread
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
    uint32_t ex[KM];
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (row[j] >= 0) {
            v[j] = *(const uint4 *)((const char *)stage + ((int64_t)row[j] * H + c) * (16 / W));
            if constexpr (ROWS == ROWS_FP8)
                ex[j] = exps[((int64_t)row[j] * H + c) >> 3];
        }
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
            if constexpr (ROWS == ROWS_FP8) {
                typedef _Float16 half2 __attribute__((ext_vector_type(2)));
                const half2 hv = __builtin_bit_cast(half2, u[q]);
                const float f = stage_unpack(ex[j]);
                acc[2 * q] = fmaf(w[j], (float)hv[0] * f, acc[2 * q]);
                acc[2 * q + 1] = fmaf(w[j], (float)hv[1] * f, acc[2 * q + 1]);
            } else if constexpr (ROWS == ROWS_BF16) {
                acc[2 * q] = fmaf(w[j], __uint_as_float(u[q] << 16), acc[2 * q]);
                acc[2 * q + 1] = fmaf(w[j], __uint_as_float(u[q] & 0xFFFF0000u), acc[2 * q + 1]);
            } else {
                acc[q] = fmaf(w[j], __uint_as_float(u[q]), acc[q]);
            }
        }
    }
    if constexpr (ROWS == ROWS_FP8)
        *(uint4 *)((uint16_t *)y + t * H + c) = uint4{cvt_bf2(acc[0], acc[1]), cvt_bf2(acc[2], acc[3]),
                                                      cvt_bf2(acc[4], acc[5]), cvt_bf2(acc[6], acc[7])};
    else if constexpr (ROWS == ROWS_BF16)
        *(uint4 *)((uint16_t *)y + t * H + c) = uint4{pack_bf2(acc[0], acc[1]), pack_bf2(acc[2], acc[3]),
                                                      pack_bf2(acc[4], acc[5]), pack_bf2(acc[6], acc[7])};
    else
        *(float4 *)((float *)y + t * H + c) = float4{acc[0], acc[1], acc[2], acc[3]};
}

template <int ROWS>
void launch_typed(const CombineArgs &a, hipStream_t st)
{
    const int64_t n = (int64_t)a.T * (a.H / (ROWS == ROWS_F32 ? 4 : 8));
    const unsigned wgs = (unsigned)((n + 255) / 256);
    auto run = [&](auto km) {
        combine_given<decltype(km)::value, ROWS>
            <<<wgs, 256, 0, st>>>(a.stage, a.row_of, a.topk_w, a.exps, a.y, a.T, a.H, a.k);
    };
    if (a.k <= 4)
        run(std::integral_constant<int, 4>{});
    else if (a.k <= 8)
        run(std::integral_constant<int, 8>{});
    else
        run(std::integral_constant<int, 16>{});
}

}  // namespace

void launch_combine_given(const CombineArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return;
    if (a.exps)
        launch_typed<ROWS_FP8>(a, st);
    else if (a.act == ACT_BF16)
        launch_typed<ROWS_BF16>(a, st);
    else
        launch_typed<ROWS_F32>(a, st);
}

}  // namespace moe
