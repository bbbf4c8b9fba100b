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
// one token in ten thousand, and another expert would run.  So a token is
// routed in fp32 and the gaps that its selection rests on are checked against
// the bound of the fp32 keys' errors; where one is too small (1 token in 1000
// with sigmoid and a bias, 1 in 100 with softmax and a bias, none without a
// bias unless the scores saturate) the experts in question are ordered in 64
// bits, or, where those are many, the doubt is between groups or the selected
// scores are too small for fp32, the token is routed again in 64 bits.  The
// weights of the others are computed in fp32: 6e-8 off, the size of their own
// rounding to fp32 (3e-8).
//
// An expert whose logit is -inf or NaN, or whose bias is -inf or NaN, is
// masked: it ranks behind every other one (among masked ones by index) and
// its weight is 0; a masked logit has no share of the softmax.  +inf counts
// as the largest finite value.  Where the selected scores sum to 0 all
// weights are 0.
//
// One wave per token.  Bound by its instructions, of which the k + 1 selection
// rounds, a wave maximum each, are the most: T=8192, E=384, k=6, sigmoid and bias
// 12.9 us for 694 vector instructions a token (9 us of issue on 1024 SIMDs; its
// bytes take 2), all in 64 bits 25 us.  T=2048, E=256, k=8, softmax over bf16 logits,
// which often tie on the last place, 6.8 us, T=1 with 4 of 8 groups 6.0.
#include <algorithm>

#include "common.h"
#include "kernels.h"
#include "topk.h"

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

__device__ __forceinline__ void wave_lds_sync()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
}

constexpr float LARGEST = 3.4028234e38f;

// Token t in 64 bits: lane r < k ends with the expert of rank r and its weight.
template <int PER, bool BF16>
__device__ __forceinline__ void select_exact(const SelectArgs &a, int t, double *row, int &my_e, float &my_w)
{
    const int lane = threadIdx.x & 63;
    double key[PER], sc[PER];
    float l[PER];
    bool masked[PER];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        l[i] = e < a.E ? logit_at<BF16>(a.logits, (int64_t)t * a.ld + e) : -INFINITY;
        masked[i] = !(l[i] > -INFINITY);
        l[i] = fminf(l[i], LARGEST);
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
        key[i] = masked[i] ? -INFINITY : sc[i] + (double)fminf(b, LARGEST);
        sc[i] = masked[i] ? 0.0 : sc[i];
    }
    uint32_t taken = 0;  // slots of this lane that cannot be selected
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (lane + 64 * i >= a.E)
            taken |= 1u << i;
    if (a.n_group > 1) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < a.E)
                row[lane + 64 * i] = key[i];
        wave_lds_sync();
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
    my_e = 0;
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
    const double d = a.renorm ? (sum > 0.0 ? my_s / sum : 0.0) : my_s;
    my_w = (float)(d * (double)a.scale);
}

// Twice the bound of a fp32 key's error, in units of 2^-24.  Sigmoid: the
// exponential's argument is off by |l| (s (1 - s) |l| <= 0.23 in the score), the
// exponential by 2 (s (1 - s) <= 0.25), the reciprocal by 2, the key's own sum by
// 1: below 4.  Softmax: difference and argument 2 |l - m| (p |l - m| <= 0.37),
// the exponential 2, the products 2, and the sum over the experts: their own
// errors weighted by p (2 |l - m| averages to 2 ln 1024 = 14 at most, and 2) and
// at most 23 additions: below 64 with the key's sum.
__device__ __forceinline__ float key_slack(float k, int softmax)
{
    return (softmax ? 0x1p-17f : 0x1p-21f) * fmaxf(1.0f, fabsf(k));
}

// Whether the keys in 64 bits of two logits l > m (no bias) are sure to differ:
// their ratio is 1 + (l - m) (1 - s) at least, s = 0 for softmax, against 2^-52
// roundings, and neither may underflow.  `top`: the largest logit, for softmax.
__device__ __forceinline__ bool logits_apart(float l, float m, float top, bool softmax)
{
    const float d = l - m;
    return softmax ? d > 1e-13f && m - top > -600.0f : d * __expf(-fmaxf(l, 0.0f)) > 1e-13f && m > -600.0f;
}

// The order of the few experts (c <= 64) that may be among the k best, in 64
// bits: lane j < c takes one of them (cand[j]) and its rank by counting.
template <int PER, bool BF16>
__device__ __forceinline__ void select_refine(const SelectArgs &a, int t, const float (&l)[PER], float top,
                                              int *cand, int c, int &my_e)
{
    const int lane = threadIdx.x & 63;
    double z = 1.0;
    if (a.softmax) {
        z = 0.0;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            z += l[i] > -INFINITY ? exp((double)l[i] - (double)top) : 0.0;
        z = wave_sum_f64(z);
    }
    const int e = cand[min(lane, c - 1)];
    const double v = (double)fminf(logit_at<BF16>(a.logits, (int64_t)t * a.ld + e), LARGEST);
    double key = a.softmax ? exp(v - (double)top) / z : 1.0 / (1.0 + exp(-v));
    if (a.bias)
        key += (double)fminf(a.bias[e], LARGEST);
    int rank = 0;
    for (int j = 0; j < c; ++j) {
        const double o = __shfl(key, j);
        const int oe = __shfl(e, j);
        rank += o > key || (o == key && oe < e) ? 1 : 0;
    }
    wave_lds_sync();
    if (lane < c && rank < a.k)
        cand[rank] = e;
    wave_lds_sync();
    my_e = cand[min(lane, a.k - 1)];
}

// Token t in fp32, and where a gap is too small to be sure of the order, in 64
// bits among the experts in question; false if they are too many, if the doubt is
// between groups, or if the selected scores are too small for fp32.
template <int PER, bool BF16>
__device__ __forceinline__ bool select_fast(const SelectArgs &a, int t, float *row, int &my_e, float &my_w)
{
    const int lane = threadIdx.x & 63;
    const bool bias = a.bias != nullptr;
    const bool grouped = a.n_group > 1;
    float l[PER], key[PER];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        const float v = e < a.E ? logit_at<BF16>(a.logits, (int64_t)t * a.ld + e) : -INFINITY;
        l[i] = v > -INFINITY ? fminf(v, LARGEST) : -INFINITY;
        top = fmaxf(top, l[i]);
    }
    float inv_z = 0.0f;
    auto sum_scores = [&]() {
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            z += l[i] > -INFINITY ? __expf(l[i] - top) : 0.0f;
#pragma unroll
        for (int d = 32; d; d >>= 1)
            z += __shfl_xor(z, d);
        inv_z = z > 0.0f ? 1.0f / z : 0.0f;
    };
    if (a.softmax) {
        top = key_value(wave_max_u32(order_key(top)));
        // not needed for an order of logits with renormalised weights
        if (bias || !a.renorm || (grouped && a.group_top2))
            sum_scores();
    }
    auto score = [&](float v) {
        return a.softmax ? __expf(v - top) * inv_z : __builtin_amdgcn_rcpf(1.0f + __expf(-v));
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = lane + 64 * i;
        key[i] = l[i];
        if (bias) {
            const float b = e < a.E ? a.bias[e] : 0.0f;
            key[i] = l[i] > -INFINITY && b > -INFINITY ? score(l[i]) + fminf(b, LARGEST) : -INFINITY;
        }
    }
    bool sure = true;
    uint64_t open = ~0ull;
    const int gs = a.E / a.n_group;
    if (grouped) {
        // a group's two largest keys: `per` lanes a group, then their halves joined
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (lane + 64 * i < a.E)
                row[lane + 64 * i] = key[i];
        wave_lds_sync();
        const int sh = 31 - __clz(64 / a.n_group), per = 1 << sh;
        const int g = lane >> sh;
        float m1 = -INFINITY, m2 = -INFINITY;
        if (g < a.n_group)
            for (int i = lane & (per - 1); i < gs; i += per) {
                const float v = row[g * gs + i];
                m2 = fmaxf(m2, fminf(m1, v));
                m1 = fmaxf(m1, v);
            }
        for (int d = 1; d < per; d <<= 1) {
            const float o1 = __shfl_xor(m1, d), o2 = __shfl_xor(m2, d);
            m2 = fmaxf(fminf(m1, o1), fmaxf(m2, o2));
            m1 = fmaxf(m1, o1);
        }
        float val = m1;
        if (a.group_top2) {
            if (!bias && m1 > -INFINITY)
                val = score(m1);
            if (m2 > -INFINITY)
                val += bias ? m2 : score(m2);
        }
        // Bound of the value's error: 7/8 of a slack a key (half, and 3 units of 2^-24
        // for the roundings of the sum and of the bound added to it), all of the larger
        // key's size, which the sum need not have (keys of opposite signs).
        float err = 0.0f;
        if (bias || a.group_top2) {
            const float size = !bias ? 1.0f : fmaxf(m1 > -INFINITY ? fabsf(m1) : 0.0f,
                                                    a.group_top2 && m2 > -INFINITY ? fabsf(m2) : 0.0f);
            err = (a.group_top2 ? 1.75f : 0.875f) * key_slack(size, a.softmax);
        }
        wave_lds_sync();
        if (g < a.n_group && (lane & (per - 1)) == 0) {
            row[g] = val;
            row[a.n_group + g] = err;
        }
        wave_lds_sync();
        // rank by counting; lane g < n_group for group g
        const float mine = lane < a.n_group ? row[lane] : -INFINITY;
        int rank = 0;
        for (int j = 0; j < a.n_group; ++j) {
            const float o = row[j];
            rank += o > mine || (o == mine && j < lane) ? 1 : 0;
        }
        const bool in = lane < a.n_group && rank < a.topk_group;
        open = __ballot(in);
        // the gap between the open and the closed groups: the least that an open
        // one's value may be, against the most that a closed one's may
        const float off = lane < a.n_group ? row[a.n_group + lane] : 0.0f;
        const float lo = -key_value(wave_max_u32(order_key(in ? off - mine : -INFINITY)));
        const float hi = key_value(wave_max_u32(order_key(lane < a.n_group && !in ? mine + off : -INFINITY)));
        if (hi > -INFINITY)  // (groups of masked experts only are in order)
            sure = bias || a.group_top2 ? lo > hi : logits_apart(lo, hi, top, a.softmax);
    }
    auto may = [&](int e) { return e < a.E && (!grouped || (open >> (e / gs & 63)) & 1); };
    uint32_t ok[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        ok[i] = may(lane + 64 * i) ? order_key(key[i]) : 0u;
    // one more than k: the gap behind the last one
    uint32_t my_k;
    wave_topk_keys<PER>(ok, min(a.k + 1, a.E), my_e, my_k);
    const bool have = my_k != 0u;
    const float kv = have ? key_value(my_k) : -INFINITY;
    float lv = kv, bv = 0.0f;
    if (bias && lane <= a.k && have) {
        lv = logit_at<BF16>(a.logits, (int64_t)t * a.ld + my_e);
        lv = lv > -INFINITY ? fminf(lv, LARGEST) : -INFINITY;
        bv = a.bias[my_e];
    }
    const float nk = __shfl_down(kv, 1), nl = __shfl_down(lv, 1), nb = __shfl_down(bv, 1);
    bool fine = true;
    if (lane < a.k && nk > -INFINITY)
        fine = (lv == nl && bv == nb) ||
               (bias ? kv - nk > key_slack(kv, a.softmax) : logits_apart(kv, nk, top, a.softmax));
    // The last one selected and the one behind it may be equal, logit and bias:
    // then it is the next different key that must be apart (it may be larger in 64
    // bits, or equal there, with a lower index).
    if (__any(lane == a.k - 1 && nk > -INFINITY && lv == nl && bv == nb)) {
        const float kl = __shfl(kv, a.k - 1), ll = __shfl(lv, a.k - 1), bl = __shfl(bv, a.k - 1);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = lane + 64 * i;
            if (!may(e) || !(key[i] > -INFINITY) || key[i] > kl)
                continue;
            const bool same = l[i] == ll && (!bias || a.bias[e] == bl);
            fine &= same || (bias ? kl - key[i] > key_slack(kl, a.softmax)
                                  : logits_apart(kl, key[i], top, a.softmax));
        }
    }
    if (!sure)
        return false;
    if (!__all(fine)) {
        // every expert whose key is not surely below the k-th one's; where no
        // bias was added the keys are the scores now, not the logits
        if (a.softmax && inv_z == 0.0f)
            sum_scores();
        const float last = __shfl(bias ? kv : score(kv), a.k - 1);
        if (!(last > -INFINITY))
            return false;
        const float least = last - key_slack(last, a.softmax);
        int *cand = (int *)row;
        int c = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = may(lane + 64 * i) && key[i] > -INFINITY &&
                            (bias ? key[i] : score(key[i])) >= least;
            const uint64_t m = __ballot(in);
            if (in && c + __popcll(m & ((1ull << lane) - 1)) < 64)
                cand[c + __popcll(m & ((1ull << lane) - 1))] = lane + 64 * i;
            c += __popcll(m);
        }
        if (c > 64 || c < a.k)
            return false;
        wave_lds_sync();
        select_refine<PER, BF16>(a, t, l, top, cand, c, my_e);
        lv = -INFINITY;
        if (lane < a.k)
            lv = fminf(logit_at<BF16>(a.logits, (int64_t)t * a.ld + my_e), LARGEST);
    }
    // weights; a masked expert (key -inf) has none
    const bool live = lane < a.k && lv > -INFINITY && kv > -INFINITY;
    // sigmoid scores that fp32 does not hold (from e^-88 on): their ratios are weights all the same
    if (!a.softmax && __any(live && lv < -80.0f))
        return false;
    float s;
    if (a.softmax) {
        const float base = a.renorm ? key_value(wave_max_u32(order_key(live ? lv : -INFINITY))) : top;
        s = live ? expf(lv - base) * (a.renorm ? 1.0f : inv_z) : 0.0f;
    } else {
        s = live ? 1.0f / (1.0f + expf(-lv)) : 0.0f;
    }
    if (a.renorm) {
        float sum = s;
#pragma unroll
        for (int d = 1; d < 16; d <<= 1)
            sum += __shfl_xor(sum, d);
        s = sum > 0.0f ? s / sum : 0.0f;
    }
    my_w = s * a.scale;
    return sure;
}

template <int PER, bool BF16>
__global__ __launch_bounds__(64 * SEL_WAVES) void select_kernel(SelectArgs a)
{
    extern __shared__ double s_key[];  // [waves][max(E, 32)]
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int t = blockIdx.x * SEL_WAVES + wv;
    if (t >= a.T)  // uniform in the wave; no workgroup barrier below
        return;
    double *row = s_key + wv * max(a.E, 32);
    int my_e;
    float my_w;
    if (!select_fast<PER, BF16>(a, t, (float *)row, my_e, my_w))  // uniform
        select_exact<PER, BF16>(a, t, row, my_e, my_w);
    if (lane < a.k) {
        a.idx[(int64_t)t * a.k + lane] = my_e;
        if (a.w)
            a.w[(int64_t)t * a.k + lane] = my_w;
    }
}

// Tokens of a launch: 2^30 threads.  A grid of 2^32 threads and more is launched
// short, without an error.
constexpr int LAUNCH_TOKENS = 1 << 24;

template <int PER>
void launch_per(const SelectArgs &all, hipStream_t st)
{
    const size_t lds = (size_t)SEL_WAVES * std::max(all.E, 32) * sizeof(double);
    for (int64_t t0 = 0; t0 < all.T; t0 += LAUNCH_TOKENS) {
        SelectArgs a = all;
        a.T = (int)std::min<int64_t>(all.T - t0, LAUNCH_TOKENS);
        a.logits = (const char *)all.logits + t0 * all.ld * (all.bf16 ? 2 : 4);
        a.idx = all.idx + t0 * all.k;
        a.w = all.w ? all.w + t0 * all.k : nullptr;
        const unsigned nb = (unsigned)((a.T + SEL_WAVES - 1) / SEL_WAVES);
        if (a.bf16)
            select_kernel<PER, true><<<nb, 64 * SEL_WAVES, lds, st>>>(a);
        else
            select_kernel<PER, false><<<nb, 64 * SEL_WAVES, lds, st>>>(a);
    }
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
    else if (per <= 6)
        launch_per<6>(a, st);
    else if (per <= 8)
        launch_per<8>(a, st);
    else
        launch_per<16>(a, st);
}

}  // namespace moe
