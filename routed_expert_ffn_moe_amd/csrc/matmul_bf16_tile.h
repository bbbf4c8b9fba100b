// The grouped bf16 products where both operands can be copied to LDS in pieces
// of 16 bytes (the form of the products is in matmul_bf16.hip).
//
// A workgroup of WP x WQ waves owns BP x BQ outputs and steps through c 64 at a
// time, with ST stages of both operands in LDS, filled by asynchronous copies.  Of
// WK groups of such waves each takes every WK-th 64 of c; their sums are joined.
// An operand with c adjacent lies there in rows of 64 c, one with p or q adjacent
// as it comes, 64 rows of c, and is transposed by the LDS read itself
// (ds_read_b64_tr_b16: 16 lanes read 4 rows of 16 elements and get columns of 4).
// Pieces of 16 bytes are rotated (XOR) by their row so that the lanes of one read
// fall on distinct banks: 2.3 cycles for a wave's 512 bytes transposed (15.8
// unrotated), 4.1 for its 1024 bytes in rows.
//
// Bound by the matrix cores, at the clock that they leave, where there are many rows:
// 8192 x 4096 x 4096 193 to 211 us (boxes differ; 1.30 to 1.42 PFLOP/s), MFMAs in 75% of
// the cycles at 1.7 to 1.8 GHz, where the products below run at 2.1 to 2.3.  Hence the
// largest tiles that registers and LDS hold.  MFMAs of 32 x 32 x 16 in place of 16 x 16 x 32
// are slower (dx 212 us against 197, dw 212 against 205); four waves of 128 x 128 in place of
// eight (y 215 to 223 against 212 to 229) and raised priority around the MFMAs (dx 202
// against 197, dw 204 against 205) make no difference beyond the runs' own.
// Bound by memory where groups have few rows, N=768, K=2048: 48 rows of 256 groups 29 to 32
// us with inputs that change from call to call (26 warm, 54 cold), 4.7 to 5.2 TB/s; 16384
// rows (Zipf) of 256 groups back to dx 181 us (180 warm, 212 cold), 5.0 TB/s; their dw with an
// fp32 addend 668 us, 5.0 TB/s.
// Bound by the CUs that take part where there are few tiles and c is long, since c is split
// over the waves of a workgroup only: 8192 x 256 x 2048 (dw) 28 us warm, where its bytes take
// 8; 512 x 4096 x 4096 (y) 26 warm, where its flops take 11.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"
#include "mm16.h"

namespace moe {

namespace {

// The words of buffer_from(p), for the copies.
__device__ __forceinline__ intx4 buffer_words(const void *p)
{
    const uint64_t b = (uint64_t)(uintptr_t)p;
    return intx4{(int)b, (int)(b >> 32) & 0xFFFF, 0x7FFFFFFF, 0x00027000};
}

// As dma16 (fp8.h), through a buffer: an offset of DROP writes zeros to LDS.
__device__ __forceinline__ void dma16_buffer(intx4 rsrc, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(off),
                 "s"(rsrc)
                 : "memory", "m0");
}

template <int I>
using Int = std::integral_constant<int, I>;

// f(Int<B>) .. f(Int<E - 1>)
template <int B, int E, class F>
__device__ __forceinline__ void each(F &&f)
{
    if constexpr (B < E) {
        f(Int<B>{});
        each<B + 1, E>(f);
    }
}

// Waits until at most N copies and stores of this wave are outstanding and its LDS
// reads are done, then, unless each wave has stages of its own, for the workgroup.
template <int N, bool ALONE>
__device__ __forceinline__ void stage_wait()
{
    if constexpr (ALONE)
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    else
        dma_wait_barrier<N>();
}

constexpr int TAB_GROUPS = 512;  // groups that the table has room for
constexpr int TAB_BYTES = 2 * 4 * TAB_GROUPS + 64;

template <int WAY, bool F32, int BP, int BQ, int WP, int WQ, int ST, int EX, int WK>
struct Tiling {
    static constexpr int NW = WP * WQ, MB = BP / 16 / WP, NB = BQ / 16 / WQ;
    using P = Operand<BP, WAY != MM_DW, WAY == MM_DW>;
    using Q = Operand<BQ, WAY == MM_Y, (NB > 1)>;
    static constexpr int PI = (P::COPIES + NW - 1) / NW, QI = (Q::COPIES + NW - 1) / NW, L = PI + QI;
    static constexpr int O_Q = (ST + EX) * P::BYTES, RING = O_Q + ST * Q::BYTES;  // of a group
    static constexpr int O_SUM = WK * RING, O_TAB = O_SUM + (WK - 1) * BP * BQ * 4;
    // Row tiles by group, where there is room: a number for each of them, none for
    // empty groups, and found in LDS.
    static constexpr bool TAB = WAY != MM_DW && O_TAB + TAB_BYTES <= 163840;
    static constexpr int LDS = O_TAB + (TAB ? TAB_BYTES : 0);
    static_assert(LDS <= 163840, "LDS of one workgroup");
    static constexpr int OCC = 163840 / LDS;
    static constexpr int NS = MB * (NB > 1 ? NB / 2 * (F32 ? 2 : 1) : 1);  // stores of a wave and tile
    static_assert(MB * WP * 16 == BP && NB * WQ * 16 == BQ && (NB % 2 == 0 || NB == 1), "whole blocks");
    static_assert(WAY != MM_DW || MB % 2 == 0, "whole pairs");
    static_assert((ST - 1) * L + EX * PI < 64 && (ST - 2) * L + EX * PI + NS < 64, "the counter of outstanding operations holds 63");
};

// Persistent workgroups: the copies run on into the next tile while the results of
// this one are stored.
template <int WAY, bool F32, int BP, int BQ, int WP, int WQ, int ST, int EX, int WK>
__global__ __launch_bounds__(64 * WP * WQ * WK) void mm16_tile(Mm16Args a, int mtiles)
{
    using C = Tiling<WAY, F32, BP, BQ, WP, WQ, ST, EX, WK>;
    using P = typename C::P;
    using Q = typename C::Q;
    constexpr int MB = C::MB, NB = C::NB, L = C::L, NS = C::NS;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave % C::NW, kg = wave / C::NW;
    const int wq = w % WQ, wp = w / WQ;
    uint8_t *const ring = smem + kg * C::RING;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(ring));
    constexpr int DEEP = WK * STEP;  // depth of a step of all groups

    // ---- tiles: contiguous runs per XCD, dealt in turn to its workgroups ----
    // Panels of 4 row tiles by all column tiles, so that what an XCD works on at
    // a time is about square.
    const int ntq = (a.Q + BQ - 1) / BQ;
    int *const tab = (int *)(smem + C::O_TAB), *const start = tab + TAB_GROUPS;  // first tile and row of each group
    const bool listed = C::TAB && a.offsets && a.G <= TAB_GROUPS;
    if (listed) {
        int *const part = start + TAB_GROUPS;  // of each wave
        constexpr int NT = 64 * C::NW * WK;
        int run = 0;
        for (int g0 = 0; g0 < a.G; g0 += NT) {
            const int g = g0 + tid;
            int lo = 0, hi = 0;
            if (g < a.G) {
                lo = min(max(a.offsets[g], 0), a.M);
                hi = max(lo, min(a.offsets[g + 1], a.M));
            }
            const int n = (hi - lo + BP - 1) / BP, inc = wave_scan_add(n);
            if (lane == 63)
                part[wave] = inc;
            __syncthreads();
            int before = run;
            for (int i = 0; i < C::NW * WK; ++i) {
                before += i < wave ? part[i] : 0;
                run += part[i];
            }
            if (g < a.G) {
                tab[g] = before + inc - n;
                start[g] = lo;
            }
            __syncthreads();
        }
        mtiles = __builtin_amdgcn_readfirstlane(run);
    }
    // Row tile mt of the table: its group is the last one that does not begin behind it.
    auto listed_rows = [&](int mt) {
        int lo = 0, hi = a.G - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (__builtin_amdgcn_readfirstlane(tab[mid]) <= mt)
                lo = mid;
            else
                hi = mid - 1;
        }
        const int row = __builtin_amdgcn_readfirstlane(start[lo]);
        const int row0 = row + (mt - __builtin_amdgcn_readfirstlane(tab[lo])) * BP;
        const int end = min(uniform_load(a.offsets + lo + 1), a.M);
        if (row0 < row || row0 >= end)  // not with offsets that do not decrease
            return Where{-1, 0, 0, 0, 0};
        return Where{lo, row0, min(BP, end - row0), 0, 0};
    };
    const int total = mtiles * ntq, per = (total + 7) / 8;
    const int first = ((int)blockIdx.x & 7) * per, step_q = (int)gridDim.x >> 3;
    auto find = [&](int q) {
        for (; q < per && first + q < total; q += step_q) {
            const int id = first + q, panel = id / (4 * ntq), in = id - panel * 4 * ntq;
            const int rows = min(4, mtiles - panel * 4), tq = in / rows, tp = panel * 4 + (in - tq * rows);
            Mm16Job j;
            if constexpr (WAY == MM_DW)
                j = mm16_dw_job<BP, BQ>(a, tp, tq);
            else if (listed)
                j = mm16_row_job<WAY, BQ>(a, listed_rows(tp), tq);
            else if (a.offsets)
                j = mm16_row_job<WAY, BQ>(a, find_rows<BP>(a.offsets, a.G, a.M, tp), tq);
            else
                j = mm16_row_job<WAY, BQ>(a, Where{0, tp * BP, min(BP, a.M - tp * BP), 0, 0}, tq);
            j.next = q + step_q;
            if (j.there)
                return j;
        }
        return Mm16Job{};
    };

    // ---- copies, on into the next tiles: ST stages of Q and EX more of P ----
    // Each stage of Q is copied behind the same one of P, and so finds the tile
    // that it belongs to as that of P.  Behind the last tile the copies go on with
    // offsets outside the buffer, which write zeros into free stages and read
    // nothing: every step issues the same copies, without a branch.
    uint32_t poff[C::PI], qoff[C::QI];
    const uint16_t *gp = a.p, *gq = a.q, *gq_first = a.q;
    int pleft = 0, qleft = 0, nc = 0, nq = 0;  // c not yet copied; c and columns of P's tile
    uint32_t pst = 0, qst = 0;                 // byte of the next stage
    int pnext = (int)blockIdx.x >> 3;
    // The next stage of P: its tile, zeros behind the last c.
    auto next_p = [&]() {
        if (pleft >= DEEP)
            return;
        int ln = lane;  // hidden from the compiler, which would keep what depends on it in registers
        asm volatile("" : "+v"(ln));
        if (pleft <= 0) {
            Mm16Job j;
            do {
                j = find(pnext);
                pnext = j.next;
            } while (j.there && j.nc == 0);
            if (j.there) {
                gp = j.p + (WAY == MM_DW ? (int64_t)(kg * STEP) * a.ldp : kg * STEP);
                gq_first = j.q + (WAY != MM_Y ? (int64_t)(kg * STEP) * a.ldq : kg * STEP);
            }
            nc = j.there ? j.nc : 1 << 30;
            nq = j.nq;
            pleft = nc;
#pragma unroll
            for (int i = 0; i < C::PI; ++i) {
                const auto s = P::piece((w * C::PI + i) % P::COPIES, ln);
                const uint32_t at = WAY == MM_DW ? s.c * (uint32_t)a.ldp + s.x : s.x * (uint32_t)a.ldp + s.c;
                poff[i] = s.x < j.np ? at * 2 : (uint32_t)DROP;
            }
        }
        if (pleft < DEEP)
#pragma unroll
            for (int i = 0; i < C::PI; ++i)
                if (P::piece((w * C::PI + i) % P::COPIES, ln).c >= pleft - kg * STEP)
                    poff[i] = (uint32_t)DROP;
    };
    auto next_q = [&]() {
        if (qleft >= DEEP)
            return;
        int ln = lane;
        asm volatile("" : "+v"(ln));
        if (qleft <= 0) {
            gq = gq_first;
            qleft = nc;
#pragma unroll
            for (int i = 0; i < C::QI; ++i) {
                const auto s = Q::piece((w * C::QI + i) % Q::COPIES, ln);
                const uint32_t at = WAY != MM_Y ? s.c * (uint32_t)a.ldq + s.x : s.x * (uint32_t)a.ldq + s.c;
                qoff[i] = s.x < nq ? at * 2 : (uint32_t)DROP;
            }
        }
        if (qleft < DEEP)
#pragma unroll
            for (int i = 0; i < C::QI; ++i)
                if (Q::piece((w * C::QI + i) % Q::COPIES, ln).c >= qleft - kg * STEP)
                    qoff[i] = (uint32_t)DROP;
    };
    // part J of N of a stage's copies
    auto issue_p = [&](auto part, auto parts) {
        constexpr int J = decltype(part)::value, N = decltype(parts)::value;
        if constexpr (J == 0)
            next_p();
#pragma unroll
        for (int i = 0; i < C::PI; ++i)
            if (i * N / C::PI == J)
                dma16_buffer(buffer_words(gp), poff[i], lds + pst + (uint32_t)((w * C::PI + i) % P::COPIES) * 1024u);
        if constexpr (J == N - 1) {
            gp += WAY == MM_DW ? (int64_t)DEEP * a.ldp : DEEP;
            pleft -= DEEP;
            pst = pst + P::BYTES == C::O_Q ? 0 : pst + P::BYTES;
        }
    };
    auto issue_q = [&](auto part, auto parts) {
        constexpr int J = decltype(part)::value, N = decltype(parts)::value;
        if constexpr (J == 0)
            next_q();
#pragma unroll
        for (int i = 0; i < C::QI; ++i)
            if (i * N / C::QI == J)
                dma16_buffer(buffer_words(gq), qoff[i],
                             lds + C::O_Q + qst + (uint32_t)((w * C::QI + i) % Q::COPIES) * 1024u);
        if constexpr (J == N - 1) {
            gq += WAY != MM_Y ? (int64_t)DEEP * a.ldq : DEEP;
            qleft -= DEEP;
            qst = qst + Q::BYTES == ST * Q::BYTES ? 0 : qst + Q::BYTES;
        }
    };
    constexpr Int<0> all{};
    constexpr Int<1> once{};

    Mm16Job cur = find((int)blockIdx.x >> 3);
    if (!cur.there)
        return;
    // up to where a step's first copies go on
    for (int s = 0; s < ST; ++s) {
        issue_p(all, once);
        if (EX || s + 1 < ST)
            issue_q(all, once);
    }
    int pat[MB], qat[NB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
        pat[m] = P::where(wp * MB + m, lane);
#pragma unroll
    for (int c = 0; c < NB; ++c)
        qat[c] = C::O_Q + Q::where(wq * NB + c, lane);

    // A step is U units: the 16 rows of block u % MB against all columns over half
    // u / MB of the 64 c.  A unit's rows are read D units before, the columns of the
    // second half during the first.  Once the last rows of a stage are read, D units
    // before the step's end, the workgroup turns to the next stage: it is there for
    // every wave, this one's buffer falls free, and the first fragments of the next
    // stage are under way while the last units are multiplied.
    constexpr int U = 2 * MB, D = MB >= 4 ? 3 : 1;
    static_assert(U % (D + 1) == 0 && D <= MB && (EX || ST >= 3), "the ring of rows goes on from step to step");
    bf16x8 qf[2][NB], pf[D + 1];
    uint32_t pc = 0, qc = 0;  // byte of the stage that is multiplied
    auto load_q = [&](int c, int h) { qf[h & 1][c] = Q::read(ring + qc, qat[c], h); };
    auto load_p = [&](auto unit) {  // unit U + u: of the next stage, which is the one multiplied by then
        constexpr int u = decltype(unit)::value;
        pf[u % (D + 1)] = P::read(ring + pc, pat[u % MB], u / MB % 2);
    };
    stage_wait<EX ? (ST - 1) * L : (ST - 2) * L + C::PI, C::NW == 1>();
#pragma unroll
    for (int c = 0; c < NB; ++c)
        load_q(c, 0);
    each<0, D>(load_p);

    // Copies hold up what the wave issues behind them while the memory system is
    // busy, so they are spread: the operand whose stage is needed first over the
    // units behind the barrier that frees its buffer, the other one over the next
    // step's units.
    auto copies = [&](auto unit) {
        constexpr int u = decltype(unit)::value;
        if constexpr (u >= U - D) {
            if constexpr (EX)
                issue_q(Int<u - (U - D)>{}, Int<D>{});
            else
                issue_p(Int<u - (U - D)>{}, Int<D>{});
        } else {
            if constexpr (EX)
                issue_p(Int<u>{}, Int<U - D>{});
            else
                issue_q(Int<u>{}, Int<U - D>{});
        }
    };

    bool stored = false;  // NS stores were issued behind the copies of this tile's first ST - 1 stages
    for (;;) {
        floatx4 acc[NB][MB];
#pragma unroll
        for (int c = 0; c < NB; ++c)
#pragma unroll
            for (int m = 0; m < MB; ++m)
                acc[c][m] = floatx4{0, 0, 0, 0};
        const int n = (cur.nc + DEEP - 1) / DEEP;
        for (int s = 0; s < n; ++s) {
            each<0, U>([&](auto unit) {
                constexpr int u = decltype(unit)::value;
                if constexpr (u < MB) {  // the columns of the second half
#pragma unroll
                    for (int c = 0; c < NB; ++c)
                        if (c * std::min(MB, 4) / NB == u)
                            load_q(c, 1);
                }
                if constexpr (u == U - D) {
                    // older than what may be under way: the next stage
                    if (s + 2 - EX < ST && stored)
                        stage_wait<(ST - 2) * L + EX * C::PI + NS, C::NW == 1>();
                    else
                        stage_wait<(ST - 2) * L + EX * C::PI, C::NW == 1>();
                    pc = pc + P::BYTES == C::O_Q ? 0 : pc + P::BYTES;
                    qc = qc + Q::BYTES == ST * Q::BYTES ? 0 : qc + Q::BYTES;
                }
                if constexpr (u >= U - D) {
#pragma unroll
                    for (int c = 0; c < NB; ++c)
                        if (c * D / NB == u - (U - D))
                            load_q(c, 0);
                }
                load_p(Int<u + D>{});
                copies(unit);
#pragma unroll
                for (int c = 0; c < NB; ++c)
                    acc[c][u % MB] = mfma16(qf[u / MB][c], pf[u % (D + 1)], acc[c][u % MB]);
                __builtin_amdgcn_sched_barrier(0);
            });
        }
        mfma_acc_drain();
        if constexpr (WK > 1) {
            // the groups' sums, joined in their order by the first one
            if (n > 0) {
                if (C::NW == 1)
                    lds_barrier();  // the first group has read the tile before
                floatx4 *sum = (floatx4 *)(smem + C::O_SUM) + w * (NB * MB * 64) + lane;
                if (kg > 0)
#pragma unroll
                    for (int c = 0; c < NB; ++c)
#pragma unroll
                        for (int m = 0; m < MB; ++m)
                            sum[((kg - 1) * C::NW * NB * MB + c * MB + m) * 64] = acc[c][m];
                lds_barrier();
                if (kg == 0)
#pragma unroll
                    for (int g = 0; g < WK - 1; ++g)
#pragma unroll
                        for (int c = 0; c < NB; ++c)
#pragma unroll
                            for (int m = 0; m < MB; ++m)
                                acc[c][m] += sum[(g * C::NW * NB * MB + c * MB + m) * 64];
            }
        }
        const Mm16Job next = find(cur.next);
        __builtin_amdgcn_sched_barrier(0);

        // ---- results: 8 adjacent columns of a row from a pair of blocks.  Lanes
        // outside the output store out of the buffer's range, so that every wave issues
        // the same number of stores and the waits above can count them.
        int e16 = lane & 15, eg = lane >> 4;  // hidden as in next_p()
        asm volatile("" : "+v"(e16), "+v"(eg));
        constexpr int esz = F32 ? 4 : 2, V = F32 ? 2 : 1;  // 16-byte stores of a pair
        const auto ro = buffer_from((const char *)a.out + cur.out * esz);
        const auto ra = buffer_from((const char *)(a.add ? a.add : a.out) + cur.out * esz);
        const int pitch = (int)a.ldo * esz;
        if constexpr (NB == 1) {  // 4 adjacent columns of a row
            if (kg == 0)
#pragma unroll
                for (int m = 0; m < MB; ++m) {
                    const int p = wp * (16 * MB) + m * 16 + e16, q = wq * 16 + eg * 4;
                    const int at = p < cur.np && q < cur.nq ? p * pitch + q * esz : DROP;
                    floatx4 v = acc[0][m];
                    if constexpr (F32) {
                        if (a.add)
                            v += __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(ra, at, 0, 0));
                        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), ro, at, 0, 0);
                    } else {
                        if (a.add) {
                            const u32x2 d = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(ra, at, 0, 0));
                            v += floatx4{__uint_as_float(d[0] << 16), __uint_as_float(d[0] & 0xFFFF0000u),
                                         __uint_as_float(d[1] << 16), __uint_as_float(d[1] & 0xFFFF0000u)};
                        }
                        __builtin_amdgcn_raw_buffer_store_b64(u32x2{cvt_bf2(v[0], v[1]), cvt_bf2(v[2], v[3])}, ro, at,
                                                              0, 0);
                    }
                }
        } else if (kg == 0)
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int p = wp * (16 * MB) + (WAY == MM_DW ? paired(m, e16) : m * 16 + e16);
            int at[(NB + 1) / 2];
            u32x4 add[(NB + 1) / 2][V];
#pragma unroll
            for (int c = 0; c < NB / 2; ++c) {
                const int q = wq * (16 * NB) + c * 32 + eg * 8;
                at[c] = p < cur.np && q < cur.nq ? p * pitch + q * esz : DROP;
                if (a.add)
#pragma unroll
                    for (int i = 0; i < V; ++i)
                        add[c][i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(ra, at[c], 16 * i, 0));
            }
#pragma unroll
            for (int c = 0; c < NB / 2; ++c) {
                float v[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x = acc[2 * c][m][i], y = acc[2 * c + 1][m][i];
                    v[i] = eg & 1 ? y : x;
                    v[4 + i] = eg & 1 ? x : y;
                }
                if (a.add)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        v[i] += F32 ? __uint_as_float(add[c][F32 ? i >> 2 : 0][i & 3])
                                    : __uint_as_float(i & 1 ? add[c][0][i >> 1] & 0xFFFF0000u : add[c][0][i >> 1] << 16);
                if constexpr (F32) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]),
                                  __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])},
                            ro, at[c], 16 * i, 0);
                } else {
                    __builtin_amdgcn_raw_buffer_store_b128(
                        u32x4{cvt_bf2(v[0], v[1]), cvt_bf2(v[2], v[3]), cvt_bf2(v[4], v[5]), cvt_bf2(v[6], v[7])},
                        ro, at[c], 0, 0);
                }
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!next.there) {
            stage_wait<0, true>();  // no copy outlives the workgroup
            break;
        }
        cur = next;
        stored = kg == 0;
    }
}

template <int WAY, bool F32, int BP, int BQ, int WP, int WQ, int ST, int EX, int WK>
void launch_tiling(const Mm16Args &a, hipStream_t st)
{
    using C = Tiling<WAY, F32, BP, BQ, WP, WQ, ST, EX, WK>;
    const int64_t tiles = mm16_tile_count(a, BP, BQ);
    const int ntq = (a.Q + BQ - 1) / BQ;
    const unsigned grid = (unsigned)(std::min<int64_t>(tiles, 256 * C::OCC) + 7) / 8 * 8;
    mm16_tile<WAY, F32, BP, BQ, WP, WQ, ST, EX, WK><<<grid, 64 * C::NW * WK, 0, st>>>(a, (int)(tiles / ntq));
}

}  // namespace

// The tiles of the lists in mm16.h by their number.
template <int WAY, bool F32, int I = 0>
void launch_shape(const Mm16Args &a, int shape, hipStream_t st)
{
    constexpr int N = WAY == MM_Y ? MM16_NY : WAY == MM_DX ? MM16_NDX : MM16_NDW;
    if constexpr (I < N) {
        constexpr Mm16Shape S = WAY == MM_Y ? MM16_Y[I < MM16_NY ? I : 0]
                                : WAY == MM_DX ? MM16_DX[I < MM16_NDX ? I : 0] : MM16_DW[I < MM16_NDW ? I : 0];
        if (shape == I || I + 1 == N)
            launch_tiling<WAY, F32, S.bp, S.bq, S.wp, S.wq, S.st, S.ex, S.wk>(a, st);
        else
            launch_shape<WAY, F32, I + 1>(a, shape, st);
    }
}

}  // namespace moe
