// Gradient of moe_select's weights, and of a sum of scores, to the logits.
//
// With d_j the gradient of weight j, k slots with experts e_j, scale c:
//   renormalised   p_j = s_j / sum of the selected s,
//                  a_j = c p_j sum over i of p_i (d_j - d_i), and softmax
//                  dl[e_j] += a_j, sigmoid dl[e_j] += a_j (1 - s_j)
//   as they are    a gradient c d_j of score e_j, with the scores' below
//   scores         g_e of score e (the caller's dscore and the line above):
//                  softmax dl_e += s_e (g_e - sum over i of s_i g_i), sigmoid
//                  dl_e += g_e s_e (1 - s_e)
//
// Differences are taken before they are weighted: sum_i p_i (d_j - d_i) in place
// of d_j - sum_i p_i d_i, and g_e less the g of the largest score, so that a score
// near 1, whose gradient is the small rest, keeps its digits.  The ratios p come
// from the logarithms of the scores less the largest selected one, and neither
// over- nor underflow.
//
// One wave per token, its row of logits in registers; slots are passed round by
// readlane (LDS shuffles in their place: T=8192 14.4 us).
//
// Bound by its instructions, as they stand: every slot is compared with every register of
// the row under a branch of its own, and what a slot needs is computed by a wave of which
// only k lanes live.  On the GPU, warm: T=8192, E=384, k=6, sigmoid with a balance gradient 12.2
// us, without one 10.1 (its 25 MB take 5.2), T=2048, E=256, k=8, softmax over bf16 logits 4.6, from
// Python 5.9, the host's call.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "topk.h"

namespace moe {

namespace {

constexpr float LARGEST = 3.4028234e38f;
// Logits whose 64-bit score is 0: selected ones have weight 0 and no gradient.
constexpr float SIGMOID_ZERO = -709.78f, SOFTMAX_ZERO = -745.14f;

// Sum and maximum over the wave, in every lane.
__device__ __forceinline__ float wave_sum(float v)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lanes_sum(v, 6)), 63));
}

__device__ __forceinline__ float wave_max(float v) { return key_value(wave_max_u32(order_key(v))); }

// The value of lane i (the same i in every lane).
__device__ __forceinline__ float from_lane(float v, int i)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}

// Lane l's experts are l, l + 64, ...
template <int PER, bool BF16, bool OUT_F32>
__global__ __launch_bounds__(256) void select_grad_rows(SelectGradArgs a)
{
    const int lane = threadIdx.x & 63;
    for (int64_t t = blockIdx.x * 4ll + (threadIdx.x >> 6); t < a.T; t += gridDim.x * 4ll) {
        float l[PER], top = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int64_t at = t * a.ld + min(lane + 64 * i, a.E - 1);  // without a branch: all reads together
            const float v = BF16 ? bf2f(((const uint16_t *)a.logits)[at]) : ((const float *)a.logits)[at];
            l[i] = v > -INFINITY && lane + 64 * i < a.E ? fminf(v, LARGEST) : -INFINITY;  // NaN: masked
            top = fmaxf(top, l[i]);
        }
        // lane j < k: slot j, its expert's logit, masked if it or the bias is
        int e = -1;
        float d = 0.0f, z = -INFINITY;
        if (lane < a.k) {
            e = a.idx[t * a.k + lane];
            e = (unsigned)e < (unsigned)a.E ? e : -1;
            if (e >= 0) {
                d = a.dw[t * a.k + lane];
                const float v = BF16 ? bf2f(((const uint16_t *)a.logits)[t * a.ld + e])
                                     : ((const float *)a.logits)[t * a.ld + e];
                const float b = a.bias ? a.bias[e] : 0.0f;
                z = v > -INFINITY && b > -INFINITY ? fminf(v, LARGEST) : -INFINITY;
            }
        }
        if (a.softmax) {
            top = wave_max(top);
            if (z - top < SOFTMAX_ZERO)
                z = -INFINITY;
        } else if (z < SIGMOID_ZERO) {
            z = -INFINITY;
        }
        const bool live = z > -INFINITY;
        float slot = d * a.scale;  // what a slot adds: to its logit if renormalised, else to its score's gradient
        if (a.renorm) {
            // logarithm of the score (of a softmax, up to the token's constant)
            const float ls = !live || a.softmax ? z : fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
            const float most = wave_max(ls);  // every lane takes part
            const float q = live ? expf(ls - most) : 0.0f;
            float total = 0.0f, sum = 0.0f;
            for (int i = 0; i < a.k; ++i) {
                const float qi = from_lane(q, i), di = from_lane(d, i);
                total += qi;
                sum += qi > 0.0f ? qi * (d - di) : 0.0f;
            }
            slot = live ? a.scale * (q / total) * (sum / total) : 0.0f;
            if (!a.softmax && live)
                slot *= z > 0.0f ? expf(-z) / (1.0f + expf(-z)) : 1.0f / (1.0f + expf(z));
        }
        if (!live)
            e = -1;
        float g[PER], out[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i)
            g[i] = out[i] = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int ej = __builtin_amdgcn_readlane(e, j);
            const float v = from_lane(slot, j);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (ej == lane + 64 * i) {
                    if (a.renorm)
                        out[i] += v;
                    else
                        g[i] += v;
                }
        }
        if (a.dscore || !a.renorm) {  // uniform
            if (a.dscore)
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int x = min(lane + 64 * i, a.E - 1);
                    const float d = a.dscore[x], b = a.bias ? a.bias[x] : 0.0f;
                    g[i] += l[i] > -INFINITY && b > -INFINITY ? d : 0.0f;
                }
            if (a.softmax) {
                float s[PER], sum = 0.0f, mean = 0.0f, ref = 0.0f;
                bool at_top = false;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    s[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.0f;
                    sum += s[i];
                    if (l[i] == top && !at_top) {
                        at_top = true;
                        ref = g[i];
                    }
                }
                const uint64_t who = __ballot(at_top);  // never empty unless all are NaN
                ref = from_lane(ref, who ? __ffsll((unsigned long long)who) - 1 : 0);
                sum = wave_sum(sum);
                const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    s[i] *= inv;
                    g[i] -= ref;
                    mean += s[i] > 0.0f ? s[i] * g[i] : 0.0f;
                }
                mean = wave_sum(mean);
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    out[i] += s[i] > 0.0f ? s[i] * (g[i] - mean) : 0.0f;
            } else {
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const float x = expf(-fabsf(l[i])), y = __builtin_amdgcn_rcpf(1.0f + x);  // masked: 0
                    out[i] += x > 0.0f ? g[i] * (x * y * y) : 0.0f;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int x = lane + 64 * i;
            if (x < a.E) {
                if constexpr (OUT_F32)
                    ((float *)a.dlogits)[t * a.E + x] = out[i];
                else
                    ((uint16_t *)a.dlogits)[t * a.E + x] = (uint16_t)cvt_bf2(out[i], 0.0f);
            }
        }
    }
}

template <int PER>
void launch_per(const SelectGradArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)std::min<int64_t>(((int64_t)a.T + 3) / 4, 1 << 20);
    if (a.bf16)
        a.out_f32 ? select_grad_rows<PER, true, true><<<grid, 256, 0, st>>>(a)
                  : select_grad_rows<PER, true, false><<<grid, 256, 0, st>>>(a);
    else
        a.out_f32 ? select_grad_rows<PER, false, true><<<grid, 256, 0, st>>>(a)
                  : select_grad_rows<PER, false, false><<<grid, 256, 0, st>>>(a);
}

}  // namespace

void launch_select_grad(const SelectGradArgs &a, hipStream_t st)
{
    const int per = (a.E + 63) / 64;
    if (per <= 1)
        launch_per<1>(a, st);
    else if (per <= 2)
        launch_per<2>(a, st);
    else if (per <= 4)
        launch_per<4>(a, st);
    else if (per <= 6)
        launch_per<6>(a, st);
    else if (per <= 8)
        launch_per<8>(a, st);
    else
        launch_per<16>(a, st);
}

}  // namespace moe
