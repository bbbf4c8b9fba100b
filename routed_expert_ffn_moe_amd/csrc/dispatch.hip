// Tokens sorted by expert and back: the order, the rows in it, the weighted
// sum of a token's rows and its gradient.
//
//   row_of[t, j]  place of pair (t, j) in the stable order by expert (t, then j,
//                 within one), -1 for an empty slot; row_src is its inverse
//   gather        rows[row_of[t, j]] = x[t]
//   combine       y[t] = sum over j of w[t, j] rows[row_of[t, j]], in j order
//   its gradient  drows[row_of[t, j]] = w[t, j] dy[t],
//                 dw[t, j] = sum over columns of dy[t] rows[row_of[t, j]]
//
// Combine with weights of 1 is the gradient of gather, so the pair of them is
// closed under differentiation.
//
// Sums over a token's slots in j order and over its columns by a fixed tree, in fp32:
// no atomics but integer counts, the same bits in every call.  16 to 256 threads a
// token, 8 columns each: rows are read token by token, so that x, y and dy move once,
// and a token's rows are in flight together.
//
// Bound by memory.  T=8192, H=4096, k=6: dispatch 104 us, of which the copy of 67 MB to
// 395 is 94 (4.9 TB/s, a large copy's rate) and the order 10; combine's gradient 177 (856
// MB, 4.8 TB/s).  T=2048, H=2048, k=8: combine 13.4 us (75 MB, partly from the infinity
// cache).  One token's dispatch 3.8 us on the GPU, 7.1 from Python: the host's call; 17, 128
// and 512 tokens, k=8, H=2048 7.5, 8.3 and 10.9 (9.9 to 11 from Python), of which the order takes
// 4.0 to 5.2 in a launch of its own.  The gradient
// of 7 tokens, k=10, H=980: 8.4 us, 17.8 while a tail went element by element and the sums
// through LDS.
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "place.h"
#include "quant_fp8.h"

namespace moe {

namespace {

// ---- the order --------------------------------------------------------------

// Passes of at most this many pairs are sorted by comparing all pairs in every
// workgroup of the launch that also copies the rows.
constexpr int TINY_PAIRS = 128;
// Most blocks of pairs that each placing workgroup counts by itself, and whose
// histograms it sums by itself; that work grows with the square of their number.  The
// order alone on the GPU, with 4 blocks counted against 16: 136 pairs 4.0 us and 4.9,
// 4096 5.2 and 6.0, 5120 6.4 (in two launches) and 6.2, 8192 6.4 and 6.7, 16384 6.7 and 8.1.
constexpr int COUNT_BLOCKS = 4, SUM_BLOCKS = 64;

// Pairs of a block: whole tokens, at most 1024.
int block_pairs(int k) { return 1024 / k * k; }

// Pairs of each block and expert: blk[b, e].
__global__ __launch_bounds__(1024) void sort_hist(SortArgs a, int n, int per)
{
    __shared__ int32_t s_cnt[1024];
    s_cnt[threadIdx.x] = 0;
    __syncthreads();
    const int p = (int)blockIdx.x * per + threadIdx.x;
    const int e = (int)threadIdx.x < per ? pair_expert(a.idx, p, n, a.E) : -1;
    if (e >= 0)
        atomicAdd(&s_cnt[e], 1);  // integer counts: order-free
    __syncthreads();
    if ((int)threadIdx.x < a.E)
        a.blk[(int64_t)blockIdx.x * a.E + threadIdx.x] = s_cnt[threadIdx.x];
}

// blk[b, e] becomes the pairs of expert e in the blocks before b, and the row
// behind the last block the experts' totals.  64 experts a workgroup, whose 16
// waves take a share of the blocks each.
__global__ __launch_bounds__(1024) void sort_prefix(SortArgs a, int nblk)
{
    __shared__ int32_t s_sum[16][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int e = (int)blockIdx.x * 64 + lane;
    const int share = (nblk + 15) / 16, b0 = wv * share, b1 = min(nblk, b0 + share);
    int sum = 0;
    if (e < a.E)
        for (int b = b0; b < b1; ++b)
            sum += a.blk[(int64_t)b * a.E + e];
    s_sum[wv][lane] = sum;
    __syncthreads();
    int run = 0;
    for (int w = 0; w < wv; ++w)
        run += s_sum[w][lane];
    if (e >= a.E)
        return;
    for (int b = b0; b < b1; ++b) {
        const int c = a.blk[(int64_t)b * a.E + e];
        a.blk[(int64_t)b * a.E + e] = run;
        run += c;
    }
    if (wv == 15)
        a.blk[(int64_t)nblk * a.E + e] = run;
}

// Places one block's pairs (place.h), and the experts' offsets.
template <int FROM>
__global__ __launch_bounds__(1024) void sort_place(SortArgs a, int n, int per, int nblk)
{
    const int tid = threadIdx.x, b = blockIdx.x, p = b * per + tid;
    const Placed r = place_pair<FROM, COUNT_BLOCKS>(a.idx, a.blk, nblk, b, per, n, a.E);
    if (b == 0) {
        if (tid < a.E)
            a.offsets[tid] = r.first;
        if (tid == a.E - 1)
            a.offsets[a.E] = r.first + r.total;
    }
    if (tid >= per || p >= n)
        return;
    if (r.at >= 0 && a.row_src)
        a.row_src[r.at] = p;
    a.row_of[p] = r.at;
}

// ---- rows -------------------------------------------------------------------

// Columns c .. c + 7 of a row as they are stored, 16 bytes at any element's
// address.
template <bool F32>
struct Raw8 {
    words4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw8<F32> load_raw(const void *p, int64_t at)
{
    Raw8<F32> r;
    const char *s = (const char *)p + at * (F32 ? 4 : 2);
    r.w[0] = *(const words4 *)s;
    if constexpr (F32)
        r.w[1] = *(const words4 *)(s + 16);
    return r;
}

template <bool F32>
__device__ __forceinline__ void store_raw(const Raw8<F32> &r, void *p, int64_t at)
{
    char *d = (char *)p + at * (F32 ? 4 : 2);
    *(words4 *)d = r.w[0];
    if constexpr (F32)
        *(words4 *)(d + 16) = r.w[1];
}

template <bool F32>
__device__ __forceinline__ float elem(const Raw8<F32> &r, int i)
{
    if constexpr (F32)
        return __uint_as_float(r.w[i >> 2][i & 3]);
    const uint32_t u = r.w[0][i >> 1];
    return __uint_as_float(i & 1 ? u & 0xFFFF0000u : u << 16);
}

template <bool F32>
__device__ __forceinline__ Raw8<F32> make_raw(const float (&v)[8])
{
    Raw8<F32> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (F32) {
            r.w[0][i] = __float_as_uint(v[i]);
            r.w[1][i] = __float_as_uint(v[4 + i]);
        } else {
            r.w[0][i] = cvt_bf2(v[2 * i], v[2 * i + 1]);
        }
    }
    return r;
}

template <bool F32>
__device__ __forceinline__ float load_one(const void *p, int64_t at)
{
    return F32 ? ((const float *)p)[at] : bf2f(((const uint16_t *)p)[at]);
}

template <bool F32>
__device__ __forceinline__ void store_one(float v, void *p, int64_t at)
{
    if constexpr (F32)
        ((float *)p)[at] = v;
    else
        ((uint16_t *)p)[at] = (uint16_t)cvt_bf2(v, 0.0f);
}

// First column of the 8 from c on, moved back to where 8 are inside the row (there
// are 8 at least): those in front of c are handled twice, with the same results.
__device__ __forceinline__ int inside(int c, int H) { return min(c, H - 8); }

// Columns c .. c + 7 of token t of x to the rows place(0) .. place(k - 1), those
// of them that are rows.
template <int SRC, bool F32, class Place>
__device__ __forceinline__ void gather_columns(const GatherArgs &a, int64_t t, int c, Place place)
{
    Raw8<F32> v;
    int left = a.H - c;
    if constexpr (SRC == GATHER_FP8) {
        float x[8];  // whole blocks: no tail
        decode8(x, (const uint8_t *)a.x + t * a.ldx + c,
                a.sx[t * ((a.H + FP8_BLOCK - 1) / FP8_BLOCK) + c / FP8_BLOCK]);
        v = make_raw<F32>(x);
    } else if (a.H >= 8) {
        c = inside(c, a.H);
        left = 8;
        v = load_raw<F32>(a.x, t * a.ldx + c);
    } else {  // the bits of what there is
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (F32) {
                v.w[i >> 2][i & 3] = i < left ? ((const uint32_t *)a.x)[t * a.ldx + c + i] : 0;
            } else {
                const uint32_t u = i < left ? ((const uint16_t *)a.x)[t * a.ldx + c + i] : 0;
                v.w[0][i >> 1] = i & 1 ? v.w[0][i >> 1] | u << 16 : u;
            }
        }
    }
    for (int j = 0; j < a.k; ++j) {
        const int r = place(j);
        if ((unsigned)r >= (unsigned)a.R)
            continue;
        if (left >= 8) {
            store_raw<F32>(v, a.rows, (int64_t)r * a.ldr + c);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < left) {
                    if constexpr (F32)
                        ((uint32_t *)a.rows)[(int64_t)r * a.ldr + c + i] = v.w[i >> 2][i & 3];
                    else
                        ((uint16_t *)a.rows)[(int64_t)r * a.ldr + c + i] = (uint16_t)(v.w[0][i >> 1] >> (i & 1) * 16);
                }
        }
    }
}

// Few pairs: order and rows in one launch.  Every workgroup finds the places of
// all pairs by comparing them with each other, and copies its share of columns.
template <int SRC, bool F32>
__global__ __launch_bounds__(256) void dispatch_tiny(SortArgs s, GatherArgs a)
{
    __shared__ __attribute__((aligned(16))) int s_e[TINY_PAIRS];
    __shared__ int s_at[TINY_PAIRS];
    const int n = s.T * s.k, n4 = (n + 3) & ~3, tid = threadIdx.x;
    for (int p = tid; p < n4; p += 256) {
        const int e = pair_expert(s.idx, p, n, s.E);
        s_e[p] = e < 0 ? s.E : e;  // empty slots (and what fills up a word) behind all others
    }
    __syncthreads();
    for (int p = tid; p < n; p += 256) {
        const int e = s_e[p];
        int at = 0;
#pragma unroll 8
        for (int q = 0; q < n4; q += 4) {
            const int4 o = *(const int4 *)(s_e + q);
            at += (o.x < e || (o.x == e && q < p)) + (o.y < e || (o.y == e && q + 1 < p)) +
                  (o.z < e || (o.z == e && q + 2 < p)) + (o.w < e || (o.w == e && q + 3 < p));
        }
        s_at[p] = at = e < s.E ? at : -1;
        if (blockIdx.x == 0) {
            s.row_of[p] = at;
            if (s.row_src && at >= 0)
                s.row_src[at] = p;
        }
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= s.E; e += 256) {
            int before = 0;
#pragma unroll 8
            for (int q = 0; q < n4; q += 4) {
                const int4 o = *(const int4 *)(s_e + q);
                before += (o.x < e) + (o.y < e) + (o.z < e) + (o.w < e);
            }
            s.offsets[e] = before;
        }
    if (!a.x)
        return;
    __syncthreads();
    const int per_row = (a.H + 7) / 8;
    for (int64_t i = (int64_t)blockIdx.x * 256 + tid; i < (int64_t)s.T * per_row; i += (int64_t)gridDim.x * 256) {
        const int t = (int)(i / per_row);
        gather_columns<SRC, F32>(a, t, (int)(i - (int64_t)t * per_row) * 8, [&](int j) { return s_at[t * s.k + j]; });
    }
}

// 1 << shift threads a token.
template <int SRC, bool F32>
__global__ __launch_bounds__(256) void gather_rows(GatherArgs a, int shift)
{
    const int sub = threadIdx.x & ((1 << shift) - 1);
    const int64_t per = 256 >> shift;
    for (int64_t t = blockIdx.x * per + (threadIdx.x >> shift); t < a.T; t += gridDim.x * per) {
        const int32_t *row = a.row_of + t * a.k;
        for (int c = sub * 8; c < a.H; c += 8 << shift)
            gather_columns<SRC, F32>(a, t, c, [&](int j) { return row[j]; });
    }
}

// Rows and weights of token t's slots; a slot without a row: -1.
template <int KM>
__device__ __forceinline__ void load_slots(const CombineRowsArgs &a, int64_t t, int (&row)[KM], float (&w)[KM])
{
#pragma unroll
    for (int j = 0; j < KM; ++j) {
        row[j] = j < a.k ? a.row_of[t * a.k + j] : -1;
        w[j] = j < a.k && a.w ? a.w[t * a.k + j] : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < KM; ++j)
        row[j] = (unsigned)row[j] < (unsigned)a.R ? row[j] : -1;
}

// Columns c .. c + 7 of the slots' rows, all reads in flight together: an empty
// slot reads the first row, which is not used (R > 0).
template <int KM, bool F32>
__device__ __forceinline__ void load_rows(const CombineRowsArgs &a, const int (&row)[KM], int c, Raw8<F32> (&v)[KM])
{
#pragma unroll
    for (int j = 0; j < KM; ++j)
        if (j < a.k)
            v[j] = load_raw<F32>(a.rows, (int64_t)max(row[j], 0) * a.ldr + c);
}

template <int KM, bool F32>
__global__ __launch_bounds__(256) void combine_rows(CombineRowsArgs a, int shift)
{
    const int sub = threadIdx.x & ((1 << shift) - 1);
    const int64_t per = 256 >> shift;
    for (int64_t t = blockIdx.x * per + (threadIdx.x >> shift); t < a.T; t += gridDim.x * per) {
        int row[KM];
        float w[KM];
        load_slots<KM>(a, t, row, w);
        for (int c0 = sub * 8; c0 < a.H; c0 += 8 << shift) {
            float acc[8] = {};
            if (a.H >= 8) {
                const int c = inside(c0, a.H);
                if (a.R > 0) {
                    Raw8<F32> v[KM];
                    load_rows<KM, F32>(a, row, c, v);
#pragma unroll
                    for (int j = 0; j < KM; ++j)
                        if (j < a.k && row[j] >= 0)
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                acc[i] = fmaf(w[j], elem(v[j], i), acc[i]);
                }
                store_raw(make_raw<F32>(acc), a.y, t * a.ldy + c);
            } else {
                for (int i = 0; i < a.H; ++i) {
                    float s = 0.0f;
#pragma unroll
                    for (int j = 0; j < KM; ++j)
                        if (row[j] >= 0)
                            s = fmaf(w[j], load_one<F32>(a.rows, (int64_t)row[j] * a.ldr + i), s);
                    store_one<F32>(s, a.y, t * a.ldy + i);
                }
            }
        }
    }
}

template <int KM, bool F32>
__global__ __launch_bounds__(256) void combine_rows_grad(CombineRowsArgs a, int shift)
{
    __shared__ float s_dot[4][KM];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int sub = tid & ((1 << shift) - 1);
    const int64_t per = 256 >> shift;
    for (int64_t t0 = blockIdx.x * per; t0 < a.T; t0 += gridDim.x * per) {  // uniform in the workgroup
        const int64_t t = t0 + (tid >> shift);
        const bool there = t < a.T;
        int row[KM];
        float w[KM], dot[KM] = {};
        if (there) {
            load_slots<KM>(a, t, row, w);
            for (int c0 = sub * 8; c0 < a.H; c0 += 8 << shift) {
                if (a.H >= 8) {
                    const int c = inside(c0, a.H);
                    const Raw8<F32> d = load_raw<F32>(a.dy, t * a.ldy + c);
                    if (a.dw && a.R > 0) {
                        Raw8<F32> v[KM];
                        load_rows<KM, F32>(a, row, c, v);
#pragma unroll
                        for (int j = 0; j < KM; ++j)
                            if (j < a.k && row[j] >= 0)
#pragma unroll
                                for (int i = 0; i < 8; ++i)  // those in front of c0 are another thread's
                                    dot[j] = c + i < c0 ? dot[j] : fmaf(elem(d, i), elem(v[j], i), dot[j]);
                    }
                    if (a.drows)
#pragma unroll
                        for (int j = 0; j < KM; ++j)
                            if (j < a.k && row[j] >= 0) {
                                float f[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    f[i] = w[j] * elem(d, i);
                                store_raw(make_raw<F32>(f), a.drows, (int64_t)row[j] * a.ldr + c);
                            }
                } else {
                    for (int i = 0; i < a.H; ++i) {
                        const float d = load_one<F32>(a.dy, t * a.ldy + i);
#pragma unroll
                        for (int j = 0; j < KM; ++j)
                            if (row[j] >= 0) {
                                const int64_t at = (int64_t)row[j] * a.ldr + i;
                                if (a.dw)
                                    dot[j] = fmaf(d, load_one<F32>(a.rows, at), dot[j]);
                                if (a.drows)
                                    store_one<F32>(w[j] * d, a.drows, at);
                            }
                    }
                }
            }
        }
        if (!a.dw)
            continue;
#pragma unroll
        for (int j = 0; j < KM; ++j)
            if (j < a.k)
                dot[j] = lanes_sum(dot[j], shift);
        if (shift > 6) {  // a token over several waves
            if (lane == 63)
#pragma unroll
                for (int j = 0; j < KM; ++j)
                    s_dot[wv][j] = dot[j];
            __syncthreads();
            if (sub < a.k && there) {
                float s = 0.0f;
                for (int i = 0; i < 1 << (shift - 6); ++i)
                    s += s_dot[wv + i][sub];
                a.dw[t * a.k + sub] = s;
            }
            __syncthreads();
        } else if (there && sub == (1 << shift) - 1) {
#pragma unroll
            for (int j = 0; j < KM; ++j)
                if (j < a.k)
                    a.dw[t * a.k + j] = dot[j];
        }
    }
}

// log2 of the threads of a token: 8 columns each, 16 to 256 threads.
int token_shift(int H)
{
    int s = 4;
    while (s < 8 && (8 << s) < H)
        ++s;
    return s;
}

unsigned token_grid(int64_t T, int shift)
{
    const int64_t per = 256 >> shift;
    return (unsigned)std::min<int64_t>((T + per - 1) / per, 1 << 20);
}

template <class Run>
void with_source(const GatherArgs &a, Run run)
{
    if (a.src == GATHER_F32)
        run(std::integral_constant<int, GATHER_F32>{}, std::true_type{});
    else if (a.src == GATHER_BF16)
        run(std::integral_constant<int, GATHER_BF16>{}, std::false_type{});
    else if (a.out_f32)
        run(std::integral_constant<int, GATHER_FP8>{}, std::true_type{});
    else
        run(std::integral_constant<int, GATHER_FP8>{}, std::false_type{});
}

template <class Run>
void with_slots(const CombineRowsArgs &a, Run run)
{
    auto typed = [&](auto km) { a.f32 ? run(km, std::true_type{}) : run(km, std::false_type{}); };
    if (a.k <= 2)
        typed(std::integral_constant<int, 2>{});
    else if (a.k <= 4)
        typed(std::integral_constant<int, 4>{});
    else if (a.k <= 6)
        typed(std::integral_constant<int, 6>{});
    else if (a.k <= 8)
        typed(std::integral_constant<int, 8>{});
    else if (a.k <= 12)
        typed(std::integral_constant<int, 12>{});
    else
        typed(std::integral_constant<int, 16>{});
}

}  // namespace

size_t sort_blk_bytes(int T, int E, int k)
{
    const int64_t per = block_pairs(k), nblk = ((int64_t)T * k + per - 1) / per;
    return nblk <= COUNT_BLOCKS ? 0 : (size_t)(nblk + 1) * E * 4;
}

void launch_gather(const GatherArgs &a, hipStream_t st)
{
    if (a.T == 0)
        return;
    const int shift = token_shift(a.H);
    with_source(a, [&](auto src, auto f32) {
        gather_rows<decltype(src)::value, decltype(f32)::value><<<token_grid(a.T, shift), 256, 0, st>>>(a, shift);
    });
}

void launch_dispatch(const SortArgs &s, const GatherArgs &a, hipStream_t st)
{
    const int n = s.T * s.k;
    if (n <= TINY_PAIRS) {
        const int64_t items = a.x ? (int64_t)s.T * ((a.H + 7) / 8) : 1;
        const unsigned wgs = (unsigned)std::min<int64_t>(std::max<int64_t>((items + 255) / 256, 1), 512);
        with_source(a, [&](auto src, auto f32) {
            dispatch_tiny<decltype(src)::value, decltype(f32)::value><<<wgs, 256, 0, st>>>(s, a);
        });
        return;
    }
    const int per = block_pairs(s.k), nblk = (n + per - 1) / per;
    if (nblk <= COUNT_BLOCKS) {
        sort_place<PLACE_COUNT><<<nblk, 1024, 0, st>>>(s, n, per, nblk);
    } else {
        sort_hist<<<nblk, 1024, 0, st>>>(s, n, per);
        if (nblk <= SUM_BLOCKS) {
            sort_place<PLACE_SUM><<<nblk, 1024, 0, st>>>(s, n, per, nblk);
        } else {
            sort_prefix<<<(s.E + 63) / 64, 1024, 0, st>>>(s, nblk);
            sort_place<PLACE_PREFIX><<<nblk, 1024, 0, st>>>(s, n, per, nblk);
        }
    }
    if (a.x)
        launch_gather(a, st);
}

void launch_combine_rows(const CombineRowsArgs &a, hipStream_t st)
{
    const int shift = token_shift(a.H);
    with_slots(a, [&](auto km, auto f32) {
        combine_rows<decltype(km)::value, decltype(f32)::value><<<token_grid(a.T, shift), 256, 0, st>>>(a, shift);
    });
}

void launch_combine_rows_grad(const CombineRowsArgs &a, hipStream_t st)
{
    const int shift = token_shift(a.H);
    with_slots(a, [&](auto km, auto f32) {
        combine_rows_grad<decltype(km)::value, decltype(f32)::value><<<token_grid(a.T, shift), 256, 0, st>>>(a, shift);
    });
}

}  // namespace moe
