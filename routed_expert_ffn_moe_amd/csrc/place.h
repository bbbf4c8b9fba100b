// Places of (t, j) pairs in the stable order by expert (t, then j within one),
// which the layer's permutation and the dispatch operator share.
#pragma once

#include "common.h"

namespace moe {

// Expert of pair p, or -1 if its slot is empty (an index outside 0..E-1: given
// routing may leave slots empty) or p is behind the last pair.
__device__ __forceinline__ int pair_expert(const int32_t *__restrict__ idx, int p, int n_pairs, int E)
{
    const int e = p < n_pairs ? idx[p] : -1;
    return (unsigned)e < (unsigned)E ? e : -1;
}

// Where the experts' totals and their pairs in the blocks before come from: counted
// from all pairs (of MOST blocks at most: that work grows with the square of their
// number, and a thread holds a pair of each), summed over the blocks' histograms
// blk [nblk, E], or read from prefixes of them, with the totals in a row behind.
enum { PLACE_COUNT = 0, PLACE_SUM = 1, PLACE_PREFIX = 2 };

struct Placed {
    int at;            // place of the thread's pair, -1 for an empty slot
    int first, total;  // first place of expert threadIdx.x, and its pairs
};

// Places one block's pairs, a pair a thread (1024 threads, blocks of `per` pairs,
// at most 1024; E <= 1024).  A block's first place with an expert is the expert's
// offset (prefix over the experts' totals) plus the expert's pairs in earlier
// blocks; inside the block the waves follow in order, and a wave's lanes of one
// expert are ranked by a mask that ballots on the expert's bits build.
template <int FROM, int MOST = 1>
__device__ __forceinline__ Placed place_pair(const int32_t *__restrict__ idx, const int32_t *__restrict__ blk,
                                             int nblk, int b, int per, int n_pairs, int E)
{
    __shared__ int32_t s_start[1024];
    __shared__ uint16_t s_wave[16][1024];  // pairs of a wave and expert, then those of the waves before
    __shared__ int32_t s_wsum[16];
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int e = tid < per ? pair_expert(idx, b * per + tid, n_pairs, E) : -1;
    int total = 0, before = 0;
    if constexpr (FROM == PLACE_COUNT) {
        __shared__ int32_t s_before[1024], s_rest[1024];
        s_before[tid] = s_rest[tid] = 0;
        __syncthreads();
        int ev[MOST];  // all reads in flight together
#pragma unroll
        for (int i = 0; i < MOST; ++i)
            ev[i] = tid < per ? pair_expert(idx, i * per + tid, n_pairs, E) : -1;
#pragma unroll
        for (int i = 0; i < MOST; ++i)
            if (ev[i] >= 0)
                atomicAdd(i < b ? &s_before[ev[i]] : &s_rest[ev[i]], 1);  // integer counts: order-free
        __syncthreads();
        before = s_before[tid];
        total = before + s_rest[tid];
    } else if (tid < E) {
        if constexpr (FROM == PLACE_SUM) {
            constexpr int AT = 16;
            for (int b0 = 0; b0 < nblk; b0 += AT) {
                int c[AT];
#pragma unroll
                for (int i = 0; i < AT; ++i)  // all reads in flight together
                    c[i] = b0 + i < nblk ? blk[(int64_t)(b0 + i) * E + tid] : 0;
#pragma unroll
                for (int i = 0; i < AT; ++i) {
                    total += c[i];
                    before += b0 + i < b ? c[i] : 0;
                }
            }
        } else {
            total = blk[(int64_t)nblk * E + tid];
            before = blk[(int64_t)b * E + tid];
        }
    }
#pragma unroll
    for (int w = 0; w < 16; ++w)
        s_wave[w][tid] = 0;
    // exclusive prefix of the experts' totals
    const int inc = wave_scan_add(total);
    if (lane == 63)
        s_wsum[wv] = inc;
    __syncthreads();
    int first = inc - total;
#pragma unroll
    for (int w = 0; w < 16; ++w)
        first += w < wv ? s_wsum[w] : 0;
    if (tid < E)
        s_start[tid] = first + before;
    // rank among this wave's earlier pairs of the same expert
    uint64_t same = __ballot(e >= 0);
    for (int bit = 0; bit < 10; ++bit) {
        const bool on = (e >> bit) & 1;
        const uint64_t ones = __ballot(e >= 0 && on);
        same &= on ? ones : ~ones;
    }
    const int rank = __popcll(same & (lane == 0 ? 0ull : ~0ull >> (64 - lane)));
    if (e >= 0 && rank == 0)  // one writer per wave and expert
        s_wave[wv][e] = (uint16_t)__popcll(same);
    __syncthreads();
    if (tid < E) {
        int run = 0;
#pragma unroll
        for (int w = 0; w < 16; ++w) {
            const int c = s_wave[w][tid];
            s_wave[w][tid] = (uint16_t)run;
            run += c;
        }
    }
    __syncthreads();
    return Placed{e >= 0 ? s_start[e] + s_wave[wv][e] + rank : -1, first, total};
}

}  // namespace moe
