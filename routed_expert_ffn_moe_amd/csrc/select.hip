// Routing of tokens to experts from given logits: softmax or sigmoid scores,
// a bias that counts in the selection only, expert groups, top-k,
// renormalised and scaled weights.
//
//   s_e = softmax(l)_e or 1 / (1 + exp(-l_e)),  key_e = s_e + b_e
//   groups of E / n_group consecutive experts are valued by their largest
//   key or by the sum of their two largest; the topk_group best stay open
//   the k open experts with the largest keys, equal keys to the lower index
//   w = s of the selected (/ their sum) * scale
//
// The order is that of the keys in 64 bits: 256 experts a token leave gaps
// between neighbouring keys that fp32 rounding (6e-8 near 1) closes for about
// one token in ten thousand, and another expert would run.
//
// An expert whose logit is -inf or NaN, or whose bias is -inf or NaN, is
// masked: it ranks behind every other one (among masked ones by index) and
// its weight is 0; a masked logit has no share of the softmax.  +inf counts
// as the largest finite value.  Where the selected scores sum to 0 all
// weights are 0.
//
// One wave per token.
#include "common.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int SEL_WAVES = 4;  // tokens per workgroup

__device__ __forceinline__ double wave_max_f64(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v = fmax(v, __shfl_xor(v, d));
    return v;
}

__device__ __forceinline__ double wave_sum_f64(double v)
{
#pragma unroll
    for (int d = 32; d; d >>= 1)
        v += __shfl_xor(v, d);
    return v;
}

// Best (key, index) pair of the wave, in every lane: the larger key, equal
// keys to the lower index.
__device__ __forceinline__ void wave_best(double &key, int &e)
{
#pragma unroll
    for (int d = 32; d; d >>= 1) {
        const double ok = __shfl_xor(key, d);
        const int oe = __shfl_xor(e, d);
        if (ok > key || (ok == key && oe < e)) {
            key = ok;
            e = oe;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ float logit_at(const void *l, int64_t i)
{
    return BF16 ? bf2f(((const uint16_t *)l)[i]) : ((const float *)l)[i];
}

template <int PER, bool BF16>
__global__ __launch_bounds__(64 * SEL_WAVES) void select_kernel(SelectArgs a)
{
    extern __shared__ double s_key[];  // [waves][E], grouped selection only
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t = blockIdx.x * SEL_WAVES + wv;
    if (t >= a.T)  // uniform in the wave; no workgroup barrier below
        return;
    double key[PER], sc[PER];
    float l[PER];
    bool masked[PER];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < a.E ? logit_at<BF16>(a.logits, (int64_t)t * a.ld + e) : -INFINITY;
        masked[i] = !(l[i] > -INFINITY);
        l[i] = fminf(l[i], 3.4028234e38f);
        if (!masked[i])
            mx = fmaxf(mx, l[i]);
    }
    if (a.softmax) {
        mx = (float)wave_max_f64(mx);
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            sc[i] = masked[i] ? 0.0 : exp((double)l[i] - (double)mx);
            z += sc[i];
        }
        z = wave_sum_f64(z);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sc[i] = z > 0.0 ? sc[i] / z : 0.0;
    } else {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            sc[i] = masked[i] ? 0.0 : 1.0 / (1.0 + exp(-(double)l[i]));
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        const float b = a.bias && e < a.E ? a.bias[e] : 0.0f;
        masked[i] |= !(b > -INFINITY);
        key[i] = masked[i] ? -INFINITY : sc[i] + (double)fminf(b, 3.4028234e38f);
        sc[i] = masked[i] ? 0.0 : sc[i];
    }
    uint32_t taken = 0;  // slots of this lane that cannot be selected
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lane + 64 * i >= a.E)
            taken |= 1u << i;
    if (a.n_group > 1) {
        double *row = s_key + (int64_t)wv * a.E;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < a.E)
                row[lane + 64 * i] = key[i];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
        const int gs = a.E / a.n_group;
        double val = -INFINITY;
        if (lane < a.n_group) {
            double m1 = -INFINITY, m2 = -INFINITY;
            for (int i = 0; i < gs; ++i) {
                const double v = row[lane * gs + i];
                m2 = fmax(m2, fmin(m1, v));
                m1 = fmax(m1, v);
            }
            val = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
        }
        uint64_t open = 0;
        bool gone = lane >= a.n_group;
        for (int r = 0; r < a.topk_group; ++r) {
            double k = gone ? -INFINITY : val;
            int g = gone ? 1 << 30 : lane;
            wave_best(k, g);
            open |= 1ull << g;
            gone |= lane == g;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (!((open >> ((lane + 64 * i) / gs & 63)) & 1))
                taken |= 1u << i;
    }
    int my_e = 0;
    double my_s = 0.0, sum = 0.0;
    for (int r = 0; r < a.k; ++r) {
        double k = -INFINITY;
        int e = 1 << 30;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (!((taken >> i) & 1) && (key[i] > k || e == 1 << 30)) {
                k = key[i];
                e = lane + 64 * i;
            }
        wave_best(k, e);
        const int slot = e >> 6;
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i == slot) {
                s = sc[i];
                if (lane == (e & 63))
                    taken |= 1u << i;
            }
        s = __shfl(s, e & 63);
        sum += s;
        if (lane == r) {
            my_e = e;
            my_s = s;
        }
    }
    if (lane < a.k) {
        const double d = a.renorm ? (sum > 0.0 ? my_s / sum : 0.0) : my_s;
        a.idx[(int64_t)t * a.k + lane] = my_e;
        if (a.w)
            a.w[(int64_t)t * a.k + lane] = (float)(d * (double)a.scale);
    }
}

template <int PER>
void launch_per(const SelectArgs &a, hipStream_t st)
{
    const unsigned nb = (unsigned)((a.T + SEL_WAVES - 1) / SEL_WAVES);
    const size_t lds = a.n_group > 1 ? (size_t)SEL_WAVES * a.E * sizeof(double) : 0;
    if (a.bf16)
        select_kernel<PER, true><<<nb, 64 * SEL_WAVES, lds, st>>>(a);
    else
        select_kernel<PER, false><<<nb, 64 * SEL_WAVES, lds, st>>>(a);
}

}  // namespace

void launch_select(const SelectArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return;
    const int per = (a.E + 63) / 64;
    if (per <= 1)
        launch_per<1>(a, st);
    else if (per <= 2)
        launch_per<2>(a, st);
    else if (per <= 4)
        launch_per<4>(a, st);
    else if (per <= 8)
        launch_per<8>(a, st);
    else
        launch_per<16>(a, st);
}

}  // namespace moe
