// Products of E4M3 codes with block scales on the matrix cores: a dense or
// grouped matrix product, and the two products of the FP8 experts (gate and
// up with SwiGLU and the quantisation of h, and down).
//
//   y[m, n] = sum over blocks q of 128 K of
//             sa[m, q] * sb[n / 128, q] * sum_{k in q} a[m, k] b[n, k]
//
// One scaled-format MFMA of 16 x 16 x 128 covers exactly one scale block, so
// the sum inside a block stays in the matrix core and the blocks are joined
// by one fp32 FMA per output and block, with the product of the two scales
// (fp32 results and the sums of gate and up multiply the codes as bf16, four
// MFMAs per block: fp8.h).
// The weights are the MFMA's A operand and the rows of `a` its B operand: a
// lane then holds one row of y, whose scale is one register, and adjacent
// columns, which it stores as whole words.
//
// A workgroup of WN x WM waves owns BR = 16 * NBW * WN weight rows and BM rows of
// a.  Both operands go to LDS by asynchronous copies (row-major rows of 128
// bytes are whole cache lines, so the weights need no packing; the pattern
// alone streams 6.1 TB/s), ST stages of 128 K deep.  In LDS the 16-byte pieces
// of a row are rotated (XOR) by the row, so that the 16 rows a fragment read
// touches fall on distinct banks (tiles of 144 rows count no conflicts, those of 96
// rows cycles that are 1% of the time of a CU), and the weight rows lie in the order
// in which a lane's results come out adjacent.  The rows'
// scales are copied a few blocks of K at a time: one 4-byte copy per row and
// block fetched as many cache lines as the weights themselves.
//
// Bound by memory where groups have few rows: 16 rows a group read their weights
// at 5.7 TB/s, 64 rows at K=2048 at 4.9, 128 rows (384 experts of H=4096, I=2048,
// down 825 us) at 4.2, where the copies alone take 85% of the time.  Gate+up of those
// experts, whose products are bf16's, takes 1.8 to 2.0 ms (2.2 in single calls) and
// is bound by its instructions: MFMAs run in 47% of the cycles and other vector
// instructions, half of them the codes' conversion (once a stage for the weights,
// once a row block for the rows), in 44%, at a clock that this load brings down to
// 1.7 GHz.  Bound by the MFMAs and the FMAs beside them
// for one matrix of many rows: 8192 x 4096 x 4096 in 140 us, 2.0 PFLOP/s (the two
// alone reach 2.5 in registers; 44% and 27% of the cycles).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int MAX_KB = FP8_MAX_K / FP8_BLOCK;  // scale blocks along K whose weight scales fit LDS

// Results as they are, h = silu(gate) * up as codes, or staging rows (fp8.h).
enum { EPI_PLAIN = 0, EPI_SWIGLU = 1, EPI_STAGE = 2 };

// A value of read-only memory at a uniform address: a scalar load, whose wait
// does not touch the copies in flight.
template <class T>
__device__ __forceinline__ T uniform_load(const T *p)
{
    return *(const __attribute__((address_space(4))) T *)(uintptr_t)p;
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// Buffer of the bytes from p on; an offset of DROP is out of its range, where
// stores do nothing.
constexpr int DROP = (int)0x80000000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_rsrc(void *p)
{
    return __builtin_amdgcn_make_buffer_rsrc(p, 0, 0x7FFFFFFF, 0x00027000);
}

// A tile: rows [row0, row0 + nrows) of group g (g = -1: none), columns from n0.
struct Where {
    int g, row0, nrows, n0, q;
};

// Row tile mt of grouped rows.  The tiles of group g take the numbers from
// offsets[g] / BM + g on, at most offsets[g + 1] / BM + g: a number's group is
// found by bisection without a sum over the groups before it (the numbers that
// a group leaves over are empty tiles).  Offsets outside 0..M are cut off.
template <int BM>
__device__ __forceinline__ Where find_rows(const int32_t *offsets, int G, int M, int mt)
{
    int lo = 0, hi = G - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        const int first = min(max(uniform_load(offsets + mid), 0), M) / BM + mid;
        if (first <= mt)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int a = min(max(uniform_load(offsets + lo), 0), M);
    const int b = min(uniform_load(offsets + lo + 1), M);
    const int m = mt - (a / BM + lo), row0 = a + m * BM;
    if (m < 0 || row0 >= b)
        return Where{-1, 0, 0, 0, 0};
    return Where{lo, row0, min(BM, b - row0), 0, 0};
}

template <int NBW, int BM_, int WN, int WM, int ST, int EPI>
struct Cfg {
    static constexpr int NW = WN * WM, BR = 16 * NBW * WN, BM = BM_;
    static constexpr int MB = (BM / 16 + WM - 1) / WM;            // row blocks of a wave
    static constexpr int COLS = EPI == EPI_SWIGLU ? BR / 2 : BR;  // output columns of a tile
    static constexpr int WI = BR / 8 / NW;                        // weight copies of a wave and stage
    static constexpr int TI = (BM / 8 + NW - 1) / NW;             // row copies (some twice)
    static constexpr int L = WI + TI;                             // both
    static constexpr int STAGE = (BR + BM) * FP8_BLOCK;
    // Scales of the rows: CH blocks of K at a time, three such chunks
    static constexpr int CH = BM > 128 && ST > 2 ? 2 : 4;
    static constexpr int CP = (BM * CH + 63) / 64;                // copies of a chunk
    static constexpr int CI = (CP + NW - 1) / NW;                 // those of a wave (some twice)
    static constexpr int CHUNK = CP * 256;
    // Scales of the weights, of two tiles
    static constexpr int NSB = EPI == EPI_SWIGLU ? 2 : (BR + 127) / 128;  // rows of them
    static constexpr int SIDE = EPI == EPI_SWIGLU ? WN * BM * 4 : 0;      // block maxima / next rows
    static constexpr int O_CHUNK = ST * STAGE, O_W = O_CHUNK + 3 * CHUNK,
                         O_SIDE = O_W + 2 * NSB * MAX_KB * 4, LDS = O_SIDE + SIDE;
    static constexpr int OCC = 163840 / LDS;                      // workgroups of a CU
    // Stores of a wave and tile (EPI_PLAIN: bf16 in whole words; more otherwise)
    static constexpr int NS = EPI == EPI_SWIGLU ? 2 * MB : EPI == EPI_STAGE ? 3 * MB : MB * (NBW / 2);
    // Stages the copies are ahead of the one that is multiplied.  A copy that the
    // memory system is not ready for holds up the wave's MFMAs behind it, so with
    // three stages a stage's copies are spread over the row blocks of a step
    // (into the buffer that the step before has left); with two that would leave
    // them too little time, and with four the tiles are small and wait for memory
    // anyway: there all copies of a stage are made when its buffer falls free.
    // (T=8192 over 384 experts: down 825 us spread, 860 at once.)
    static constexpr bool SPREAD = ST == 3 && NW == 8;
    static constexpr int LEAD = SPREAD ? ST - 1 : ST;
    // The next tile's row numbers (EPI_SWIGLU) are copied behind the first LEAD
    // stages and the stores of the tile before, and read when the next tile's
    // copies begin, before step kb - LEAD.  Whether a wait has covered that copy by
    // then: the wave's operations since it (`newer`), counted as the loop issues
    // them, are no fewer than the wait leaves outstanding.  A wait that leaves NS
    // stores out does not cover it, since the stores are older than the copy.
    static constexpr bool rows_arrive(int kb)
    {
        int newer = 0;
        for (int s = 0; s < kb - LEAD; ++s) {
            const int copies = L + ((s + LEAD) % CH == 0 ? CI : 0);
            if (SPREAD)
                newer += copies;
            const int left = (ST - 2) * L + (s < LEAD - 1 ? NS : ST == 3 && (s + 2) % CH == 0 ? CI : 0);
            if (newer >= left)
                return true;
            if (!SPREAD)
                newer += copies;
        }
        return false;
    }
    // Depth from which a tile's last stages are multiplied while the next
    // tile's first ones are copied.  With row numbers to wait for, the step before
    // has to be behind the first LEAD - 1, whose waits leave stores out.
    static constexpr int DEEP = std::max(ST + LEAD - 1, EPI == EPI_SWIGLU ? 2 * LEAD : 0);
    static_assert(EPI != EPI_SWIGLU || (rows_arrive(DEEP) && rows_arrive(DEEP + 1) && rows_arrive(DEEP + 2) &&
                                        rows_arrive(DEEP + 3)), "the next rows are there when they are read");
    static_assert(BR / 8 % NW == 0, "weight copies divide among the waves");
    static_assert(EPI != EPI_SWIGLU || (COLS == 128 && NBW % 2 == 0), "a tile of h is one scale block wide");
    static_assert(LDS <= 163840, "LDS of one workgroup");
    static_assert(ST >= 2 && ST <= 4, "chunks of scales in use or under way: three");
    static_assert((LEAD - 1) * L + NS < 64 && NBW % 2 == 0, "the counter of outstanding operations holds 63");
};

// Persistent workgroups.  The consumer multiplies stage after stage of its
// tile; the producer (the same waves) is LEAD stages ahead and goes on to the
// next tile, so that a tile's epilogue and its first latency overlap with
// copies.
template <int NBW, int BM, int WN, int WM, int ST, int EPI, bool EXACT>
__global__ __launch_bounds__(64 * WN * WM) void fp8_tile(Fp8Args p)
{
    using C = Cfg<NBW, BM, WN, WM, ST, EPI>;
    constexpr int MB = C::MB;
    constexpr bool GATHER = EPI == EPI_SWIGLU;  // rows of a through row_tok
    __shared__ __attribute__((aligned(256))) uint8_t smem[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = w % WN, wm = w / WN;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));
    const int KB = p.KB;

    // ---- tiles: contiguous runs per XCD, dealt in turn to its workgroups ----
    const int ntn = (p.N + C::COLS - 1) / C::COLS;
    const int mtiles = p.tiles ? min(p.mtiles, uniform_load(p.ntiles)) : p.mtiles;
    const int total = mtiles * ntn, per = (total + 7) / 8;
    const int first = ((int)blockIdx.x & 7) * per, step_q = (int)gridDim.x >> 3;
    auto find = [&](int q) {
        for (; q < per && first + q < total; q += step_q) {
            const int id = first + q, mt = id / ntn, nt = id - mt * ntn;
            Where t;
            if (p.tiles) {
                const int g = uniform_load(&p.tiles[mt].g), row0 = uniform_load(&p.tiles[mt].row0);
                t = Where{g, row0, min(C::BM, uniform_load(p.offsets + g + 1) - row0), 0, 0};
            } else if (p.offsets) {
                t = find_rows<C::BM>(p.offsets, p.G, p.M, mt);
            } else {
                t = Where{0, mt * C::BM, min(C::BM, p.M - mt * C::BM), 0, 0};
            }
            t.n0 = nt * C::COLS;
            t.q = q;
            if (t.g >= 0)
                return t;
        }
        return Where{-1, 0, 0, 0, q};
    };

    // ---- producer: uniform bases that advance along K, lane offsets ---------
    uint32_t woff[C::WI], toff[C::TI], soff[C::CI];
    const uint8_t *ga, *gw0, *gw1;
    const float *gsa;
    int pk = 0, pq = 0, pc = 0, pt = 0;  // next stage of the tile; stages, chunks and tiles begun
    auto aim = [&](const Where &t, bool rows_in_lds) {
        int ln = lane;  // hidden from the compiler: kept over the loops, what depends on it would
        asm volatile("" : "+v"(ln));  // take fifty registers
        const int sub = ln >> 3, slot = ln & 7;
        const int64_t gb = (int64_t)t.g * p.bstride;
        gw0 = p.b0 + gb;
        gw1 = EPI == EPI_SWIGLU ? p.b1 + gb : nullptr;
        ga = p.a + (GATHER ? 0 : (int64_t)t.row0 * p.lda);
        gsa = p.sa + (GATHER ? 0 : (int64_t)t.row0 * KB);
        auto row_of = [&](int rr) -> int64_t {
            const int at = min(rr, t.nrows - 1);
            if (!GATHER)
                return at;
            return rows_in_lds ? ((const int *)(smem + C::O_SIDE))[at] : p.row_tok[t.row0 + at];
        };
#pragma unroll
        for (int i = 0; i < C::WI; ++i) {
            const int rr = (w * C::WI + i) * 8 + sub, m = rr & 15, c = rr >> 4;
            const int own = c / NBW, cb = c - own * NBW;
            constexpr int HB = EPI == EPI_SWIGLU ? NBW / 2 : NBW;
            const int n = t.n0 + own * (HB * 16) + (m >> 2) * (4 * HB) + (cb % HB) * 4 + (m & 3);
            woff[i] = (uint32_t)((int64_t)min(n, p.N - 1) * p.ldb) + ((slot ^ (m >> 1)) << 4);
        }
#pragma unroll
        for (int i = 0; i < C::TI; ++i) {
            const int rr = ((w * C::TI + i) % (C::BM / 8)) * 8 + sub;
            toff[i] = (uint32_t)(row_of(rr) * p.lda) + ((slot ^ ((rr >> 1) & 7)) << 4);
        }
#pragma unroll
        for (int i = 0; i < C::CI; ++i) {
            const int rr = ((w * C::CI + i) % C::CP) * (64 / C::CH) + ln / C::CH;
            soff[i] = (uint32_t)(row_of(rr) * KB);
        }
        // the tile's weight scales
        const int64_t gs = (int64_t)t.g * p.sstride;
        const int np = (KB + 63) / 64;  // pieces of 64 blocks
        for (int i = w; i < C::NSB * np; i += C::NW) {
            const int q = i / np, at = (i - q * np) * 64;
            const float *src = EPI == EPI_SWIGLU && q ? p.s1 : p.s0;
            const int nb = EPI == EPI_SWIGLU ? t.n0 >> 7 : min((t.n0 >> 7) + q, ((p.N + 127) >> 7) - 1);
            dma4(src + gs + (int64_t)nb * KB, (uint32_t)min(at + ln, KB - 1) * 4,
                 lds + C::O_W + (uint32_t)(((pt & 1) * C::NSB + q) * MAX_KB + at) * 4);
        }
        ++pt;
        pk = 0;
    };
    // part J of N of the next stage's copies
    auto issue = [&](auto part, auto parts) {
        constexpr int J = decltype(part)::value, N = decltype(parts)::value;
        const uint32_t st = lds + (uint32_t)(pq % ST) * C::STAGE;
        const int64_t k = (int64_t)pk * FP8_BLOCK;
        if (J == 0 && pk % C::CH == 0) {  // the scales of this stage and the CH - 1 behind it
            const int kb = min(pk + lane % C::CH, KB - 1);
#pragma unroll
            for (int i = 0; i < C::CI; ++i)
                dma4(gsa, (soff[i] + kb) * 4,
                     lds + C::O_CHUNK + (uint32_t)(pc % 3) * C::CHUNK +
                         (uint32_t)((w * C::CI + i) % C::CP) * 256u);
            ++pc;
        }
#pragma unroll
        for (int i = 0; i < C::L; ++i) {
            if (i * N / C::L != J)
                continue;
            if (i < C::WI) {
                const uint8_t *base = gw0;
                if (EPI == EPI_SWIGLU && ((((w * C::WI + i) * 8) >> 4) % NBW) >= NBW / 2)
                    base = gw1;
                dma16(base + k, woff[i], st + (uint32_t)(w * C::WI + i) * 1024u);
            } else {
                dma16(ga + k, toff[i - C::WI],
                      st + C::BR * 128u + (uint32_t)((w * C::TI + i - C::WI) % (C::BM / 8)) * 1024u);
            }
        }
        if (J == N - 1) {
            ++pk;
            ++pq;
        }
    };
    constexpr std::integral_constant<int, 0> all{};
    constexpr std::integral_constant<int, 1> once{};

    Where cur = find((int)blockIdx.x >> 3);
    if (cur.g < 0)
        return;
    const bool deep = KB >= C::DEEP;  // uniform in the grid
    const int o0 = l16 * 128 + ((lg ^ (l16 >> 1)) << 4), o1 = o0 ^ 64;
    const int nsb = EPI == EPI_SWIGLU ? 0 : (wn * NBW * 16) >> 7;
    aim(cur, false);
    for (int s = 0; s < C::LEAD && s < KB; ++s)
        issue(all, once);

    int cq = 0, cc = 0, ct = 0;  // consumer: stages, chunks and tiles done
    bool stored = false;  // NS stores (at least) were issued behind this tile's first LEAD stages
    for (;;) {
    const Where next = find(cur.q + step_q);
    const bool go_on = next.g >= 0, ahead = go_on && deep;
    const int row0 = cur.row0, nrows = cur.nrows, n0 = cur.n0;
    // the next tile's rows, for the producer: behind this tile's first stages
    if (GATHER && ahead) {
        constexpr int RI = (C::BM + 63) / 64;
        if (w < RI)
            dma4(p.row_tok + next.row0, (uint32_t)min(w * 64 + lane, next.nrows - 1) * 4,
                 lds + C::O_SIDE + (uint32_t)w * 256u);
    }

    floatx4 acc[NBW][MB];
#pragma unroll
    for (int c = 0; c < NBW; ++c)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            acc[c][m] = floatx4{0, 0, 0, 0};

    // Fragments and scales of stage s of this tile.  (The copies that a wave
    // waits for include scales now and then: counting as if there were none
    // only waits for a few copies more.)
    struct Weights {
        Fp8Raw v[NBW];
        float s0, s1;
    };
    struct Block {
        Fp8Raw v;
        float s;
    };
    const float *s_w = (const float *)(smem + C::O_W) + ((ct & 1) * C::NSB + nsb) * MAX_KB;
    auto load_weights = [&](Weights &a, int s) {
        const uint8_t *wt = smem + ((cq + s) % ST) * C::STAGE + wn * (NBW * 2048);
#pragma unroll
        for (int c = 0; c < NBW; ++c)
            a.v[c] = fp8_raw(*(const uint4 *)(wt + c * 2048 + o0), *(const uint4 *)(wt + c * 2048 + o1));
        a.s0 = s_w[s];
        a.s1 = EPI == EPI_SWIGLU ? s_w[MAX_KB + s] : 0.0f;
    };
    auto load_block = [&](Block &b, int s, int m) {
        const uint8_t *st = smem + ((cq + s) % ST) * C::STAGE + C::BR * 128;
        const uint8_t *tt = st + (m * WM + wm) * 2048;
        b.v = fp8_raw(*(const uint4 *)(tt + o0), *(const uint4 *)(tt + o1));
        b.s = ((const float *)(smem + C::O_CHUNK + ((cc + s / C::CH) % 3) * C::CHUNK))[
            ((m * WM + wm) * 16 + l16) * C::CH + s % C::CH];
    };

    // The K loop over the first NM of the wave's MB row blocks (the others hold
    // no rows of this tile).  A block's fragment is read while the one before
    // it is multiplied.  Behind the MFMAs of a stage's last block, while they
    // run, the workgroup turns to the next stage: everything of it has arrived
    // for every wave, every wave is done reading this one (whose buffer is free
    // for the stage that is ST further), and the next weights and first block
    // are read.  The sums of a block are scaled and added while the next block's
    // MFMAs run (LAG), where there are registers for it.  The copies stand before
    // a block's MFMAs: behind them, their branch stood between the MFMAs and the
    // first use of the sums, and the wait states before that were missing on one
    // of its paths (a wrong last sum).
    constexpr bool LAG = MB < 8;
    auto kloop = [&](auto nm) {
        constexpr int NM = decltype(nm)::value;
        Weights wf;
        Block bf[2];
        floatx4 t[NBW];  // the last block's sums, not yet scaled
        float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
        for (int c = 0; c < NBW; ++c)
            t[c] = floatx4{0, 0, 0, 0};
        auto join = [&](int m) {
#pragma unroll
            for (int c = 0; c < NBW; ++c) {
                const float f = EPI == EPI_SWIGLU && c >= NBW / 2 ? t1 : t0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][m][i] = fmaf(t[c][i], f, acc[c][m][i]);
                // here, not behind the next branch, up to which every sum of
                // the stage would stay in a register
                asm volatile("" : "+v"(acc[c][m]));
            }
        };
        // MORE: 2 = the copies made in stage s are the tile's own, 1 = the next
        // tile's (if `ahead`), 0 = as 1, in the tile's last stage
        auto part = [&](int m) {  // (m is a constant in every call)
            constexpr std::integral_constant<int, NM> n{};
            if (m == 0) issue(std::integral_constant<int, 0>{}, n);
            if (m == 1) issue(std::integral_constant<int, 1>{}, n);
            if (m == 2) issue(std::integral_constant<int, 2>{}, n);
            if (m == 3) issue(std::integral_constant<int, 3>{}, n);
            if (m == 4) issue(std::integral_constant<int, 4>{}, n);
            if (m == 5) issue(std::integral_constant<int, 5>{}, n);
            if (m == 6) issue(std::integral_constant<int, 6>{}, n);
            if (m == 7) issue(std::integral_constant<int, 7>{}, n);
        };
        auto step = [&](int s, auto more) {
            constexpr int MORE = decltype(more)::value;
#pragma unroll
            for (int m = 0; m < NM; ++m) {
                if (m + 1 < NM)
                    load_block(bf[(m + 1) & 1], s, m + 1);
                if (C::SPREAD && (MORE == 2 || ahead))
                    part(m);
                const Fp8Frag<EXACT> B(bf[m & 1].v);
                floatx4 n[NBW];
#pragma unroll
                for (int c = 0; c < NBW; ++c)
                    n[c] = mfma_fp8(Fp8Frag<EXACT>(wf.v[c]), B);
                const float f0 = bf[m & 1].s * wf.s0, f1 = bf[m & 1].s * wf.s1;
                if (m + 1 == NM && MORE) {
                    __builtin_amdgcn_sched_barrier(0);
                    if (MORE != 2 && !ahead)
                        dma_wait_barrier<0>();
                    else if (s < C::LEAD - 1 && stored)  // the stores of the tile before are newer
                        dma_wait_barrier<(ST - 2) * C::L + C::NS>();
                    else if (ST == 3 && (s + 2 < KB ? s + 2 : s + 2 - KB) % C::CH == 0)
                        dma_wait_barrier<(ST - 2) * C::L + C::CI>();  // stage s + 2 holds scales
                    else
                        dma_wait_barrier<(ST - 2) * C::L>();
                    load_weights(wf, s + 1);
                    load_block(bf[0], s + 1, 0);
                    if (!C::SPREAD && (MORE == 2 || ahead))
                        issue(all, once);
                }
                if (LAG)
                    join(m ? m - 1 : NM - 1);
#pragma unroll
                for (int c = 0; c < NBW; ++c)
                    t[c] = n[c];
                t0 = f0;
                t1 = f1;
                if (!LAG)
                    join(m);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        if (stored)
            dma_wait_barrier<(C::LEAD - 1) * C::L + C::NS>();
        else if (KB >= C::LEAD)
            dma_wait_barrier<(C::LEAD - 1) * C::L>();
        else
            dma_wait_barrier<0>();
        load_weights(wf, 0);
        load_block(bf[0], 0, 0);
        int s = 0;
        for (; s + C::LEAD < KB; ++s)
            step(s, std::integral_constant<int, 2>{});
        if (ahead)
            aim(next, true);
        for (; s + 1 < KB; ++s)
            step(s, std::integral_constant<int, 1>{});
        step(s, std::integral_constant<int, 0>{});
        if (LAG)
            join(NM - 1);
    };
    const int act = ((nrows + 15) / 16 - wm + WM - 1) / WM;  // the wave's row blocks with rows
    constexpr int HALF = (MB + 1) / 2;
    if (act > HALF) {
        if (MB > 4 && act < MB)  // a tile of 16 * MB * WM - 16 rows, or as many
            kloop(std::integral_constant<int, MB - 1>{});
        else
            kloop(std::integral_constant<int, MB>{});
    } else {
        kloop(std::integral_constant<int, HALF>{});
    }
    lds_barrier();  // every wave is done with this tile's last stage
    if (!C::SPREAD && ahead)
        issue(all, once);

    __builtin_amdgcn_sched_barrier(0);
    int e16 = l16, eg = lg;  // hidden as in aim()
    asm volatile("" : "+v"(e16), "+v"(eg));
    // Stores go through a buffer descriptor of the tile's rows: lanes without a
    // row (or columns) store out of its range, which drops them, so that each
    // wave issues the same number of stores and the waits above can count them.
    if constexpr (EPI == EPI_PLAIN) {
        const int n = n0 + wn * (NBW * 16) + eg * (4 * NBW);
        const int esz = p.out_f32 ? 4 : 2;
        const int pitch = (int)p.ldy * esz;  // checked by the host where p.vec
        const auto rsrc = tile_rsrc((char *)p.y + (int64_t)row0 * p.ldy * esz);
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int rr = (m * WM + wm) * 16 + e16;
            if (p.vec) {
                const int at = rr < nrows && n < p.N ? rr * pitch + n * esz : DROP;
                if (p.out_f32) {
#pragma unroll
                    for (int c = 0; c < NBW; ++c)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            __builtin_bit_cast(u32x4, acc[c][m]), rsrc, at, 16 * c, 0);
                } else {
                    uint32_t v[2 * NBW];
#pragma unroll
                    for (int c = 0; c < NBW; ++c) {
                        v[2 * c] = cvt_bf2(acc[c][m][0], acc[c][m][1]);
                        v[2 * c + 1] = cvt_bf2(acc[c][m][2], acc[c][m][3]);
                    }
#pragma unroll
                    for (int c = 0; c < NBW; c += 2)
                        __builtin_amdgcn_raw_buffer_store_b128(
                            u32x4{v[2 * c], v[2 * c + 1], v[2 * c + 2], v[2 * c + 3]}, rsrc, at, 8 * c, 0);
                }
            } else if (rr < nrows && n + 4 * NBW <= p.N) {
                // 16-byte stores at any element's address: the hardware takes
                // them, if not at full speed
                char *at = (char *)p.y + ((int64_t)(row0 + rr) * p.ldy + n) * esz;
                if (p.out_f32) {
#pragma unroll
                    for (int c = 0; c < NBW; ++c)
                        *(u32x4_any *)(at + 16 * c) = __builtin_bit_cast(u32x4, acc[c][m]);
                } else {
#pragma unroll
                    for (int c = 0; c < NBW; c += 2)
                        *(u32x4_any *)(at + 8 * c) =
                            u32x4{cvt_bf2(acc[c][m][0], acc[c][m][1]), cvt_bf2(acc[c][m][2], acc[c][m][3]),
                                  cvt_bf2(acc[c + 1][m][0], acc[c + 1][m][1]),
                                  cvt_bf2(acc[c + 1][m][2], acc[c + 1][m][3])};
                }
            } else if (rr < nrows) {
                const int64_t at = (int64_t)(row0 + rr) * p.ldy + n;
#pragma unroll
                for (int c = 0; c < NBW; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (n + 4 * c + i >= p.N)
                            continue;
                        if (p.out_f32)
                            ((float *)p.y)[at + 4 * c + i] = acc[c][m][i];
                        else
                            ((uint16_t *)p.y)[at + 4 * c + i] = (uint16_t)cvt_bf2(acc[c][m][i], 0.0f);
                    }
            }
        }
    } else if constexpr (EPI == EPI_STAGE) {
        static_assert(NBW == 4, "a lane holds the columns under two exponents");
        const int n = n0 + wn * 64 + eg * 16;
        const auto rsrc = tile_rsrc((uint16_t *)p.y + (int64_t)row0 * p.N);
        const auto rexp = tile_rsrc(p.exps + (int64_t)row0 * (p.N / 8));
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int rr = (m * WM + wm) * 16 + e16;
            uint32_t ex[2], v[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ex[h] = STAGE_MIN_EXP;
#pragma unroll
                for (int c = 2 * h; c < 2 * h + 2; ++c)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        ex[h] = max(ex[h], stage_exponent(acc[c][m][i]));
                const float f = stage_pack(ex[h]);
#pragma unroll
                for (int c = 2 * h; c < 2 * h + 2; ++c) {
                    v[2 * c] = cvt_half2(acc[c][m][0] * f, acc[c][m][1] * f);
                    v[2 * c + 1] = cvt_half2(acc[c][m][2] * f, acc[c][m][3] * f);
                }
            }
            const bool in = rr < nrows && n < p.N;
            const int at = in ? (rr * p.N + n) * 2 : DROP;
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[0], v[1], v[2], v[3]}, rsrc, at, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[4], v[5], v[6], v[7]}, rsrc, at, 16, 0);
            __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(ex[0] | ex[1] << 8), rexp,
                                                  in ? (rr * p.N + n) / 8 : DROP, 0, 0);
        }
    } else {
        // h = silu(gate) * up, its block maximum over the tile's 128 columns
        // (4 lanes of a wave, then the waves), and its codes.  (silu's hardware
        // reciprocal is 1 ulp off, less than the sums are, and moves a code as rarely.)
        constexpr int HB = NBW / 2;
        float *s_max = (float *)(smem + C::O_SIDE);  // [WN][BM] (the next rows have been read)
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            if ((m * WM + wm) * 16 >= BM)  // uniform: a block that the tile does not have
                continue;
            float mx = 0.0f;
#pragma unroll
            for (int c = 0; c < HB; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = acc[c][m][i];
                    const float h = silu(z) * acc[c + HB][m][i];
                    acc[c][m][i] = h;
                    mx = fmaxf(mx, fabsf(h));
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            if (eg == 0)
                s_max[wn * BM + (m * WM + wm) * 16 + e16] = mx;
        }
        lds_barrier();
        const auto rh = tile_rsrc(p.hq + (int64_t)row0 * p.N);
        const auto rs = tile_rsrc(p.hs + (int64_t)row0 * (p.N >> 7));
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int rr = (m * WM + wm) * 16 + e16, at = min(rr, BM - 1);
            float mx = s_max[at];
#pragma unroll
            for (int i = 1; i < WN; ++i)
                mx = fmaxf(mx, s_max[i * BM + at]);
            const Fp8Block q = fp8_block(mx);
            static_assert(HB == 2, "a lane holds 8 columns of h");
            __builtin_amdgcn_raw_buffer_store_b64(
                u32x2{fp8x4(acc[0][m][0], acc[0][m][1], acc[0][m][2], acc[0][m][3], q),
                      fp8x4(acc[1][m][0], acc[1][m][1], acc[1][m][2], acc[1][m][3], q)},
                rh, rr < nrows ? rr * p.N + n0 + wn * (HB * 16) + eg * (4 * HB) : DROP, 0, 0);
            __builtin_amdgcn_raw_buffer_store_b32(
                __float_as_uint(q.scale), rs,
                rr < nrows && wn == 0 && eg == 0 ? (rr * (p.N >> 7) + (n0 >> 7)) * 4 : DROP, 0, 0);
        }
        lds_barrier();  // s_max is free again
    }

    __builtin_amdgcn_sched_barrier(0);
    if (!go_on)
        break;
    cq += KB;
    cc += (KB + C::CH - 1) / C::CH;
    ++ct;
    cur = next;
    stored = deep && (EPI != EPI_PLAIN || p.vec);
    if (!deep) {  // few stages: no copies under way between tiles
        aim(cur, false);
        for (int s = 0; s < C::LEAD && s < KB; ++s)
            issue(all, once);
    }
    }
}

template <int NBW, int BM, int WN, int WM, int ST, int EPI>
void launch_cfg(const Fp8Args &p, hipStream_t st)
{
    using C = Cfg<NBW, BM, WN, WM, ST, EPI>;
    const int64_t tiles = (int64_t)p.mtiles * ((p.N + C::COLS - 1) / C::COLS);
    const unsigned grid = (unsigned)(std::min<int64_t>(tiles, 256 * C::OCC) + 7) / 8 * 8;
    if constexpr (EPI == EPI_SWIGLU) {
        fp8_tile<NBW, BM, WN, WM, ST, EPI, true><<<grid, 64 * C::NW, 0, st>>>(p);
    } else {
        if constexpr (EPI == EPI_PLAIN && BM < 256) {  // fp8_size
            if (p.out_f32)
                return fp8_tile<NBW, BM, WN, WM, ST, EPI, true><<<grid, 64 * C::NW, 0, st>>>(p);
        }
        fp8_tile<NBW, BM, WN, WM, ST, EPI, false><<<grid, 64 * C::NW, 0, st>>>(p);
    }
}

}  // namespace

// Size of a tile.  The time is that of the rounds in which the CUs take their
// tiles, times a round's.  A step of 128 of K costs a CU about 0.33 us plus 6 ns
// for each row of the tile (measured with one tile a CU and K = 2048, in units of
// 5.5 ns: 32 rows 95, 64 rows 130, 96 rows 160, 128 rows 195, 144 rows 210, 256
// rows 345), 64 x 64 tiles 90 up to two of them a CU, then 72 for each 256.
// Groups whose balanced rows (1.4 standard deviations above the mean) fit into a
// tile have one; larger ones leave half a tile empty.  So groups are covered by
// one tile where that is possible, which then streams their weights once (T=8192
// over 384 experts, 128 rows each: a whole call 2850 us with gate+up tiles of 144
// rows, 3280 with 128), long matrices take the largest tiles (8192 x 4096 x 4096: 144 us with
// 256 rows, 163 with 128) and short ones tiles that give every CU one (8 groups of
// 347 rows, N=1664, K=2048: 18 us with 96 rows, 33 with 256; 4 groups of 217 rows,
// N=1024, K=640: 7.3 us with 64 x 64, 14.7 with 256 rows).  Products by bf16
// (`exact`) would need more registers than there are in the largest tiles (71 us
// against 33 in the first of these), so they go without them.  Their steps cost more
// than the ones these times are of, alike for all sizes: over eight expert passes of
// 32 to 2048 rows an expert, gate+up by any one size was at best 4% faster.
Fp8Tile fp8_size(int64_t rows, int groups, int64_t N, bool swiglu, bool exact, bool narrow)
{
    const double per = (double)rows / groups;
    Fp8Tile best{16, 256};
    double least = 1e300;
    const auto take = [&](int bm, int cols, double first, double round, double cus) {
        double tiles = groups == 1                       ? (double)((rows + bm - 1) / bm)
                       : per + 1.4 * std::sqrt(per) <= bm ? (double)std::min<int64_t>(rows, groups)
                                                          : (double)rows / bm + 0.5 * groups;
        tiles *= (double)((N + cols - 1) / cols);
        const double t = tiles <= cus ? first : groups == 1 ? std::ceil(tiles / 256) * round
                                                            : (tiles / 256 + 0.5) * round;
        if (t < least) {
            least = t;
            best = Fp8Tile{bm, cols};
        }
    };
    for (int bm : {16, 32, 64, 96, 128, 144, 256}) {
        const double t = std::max(92.0, 60 + 1.1 * bm);
        if (bm != 256 || !exact)
            take(bm, swiglu ? 128 : 256, t, t, 256);
    }
    if (narrow)
        take(64, 64, 90, 72, 512);
    return best;
}

int64_t fp8_row_tiles(int64_t rows, int groups, int bm)
{
    return groups > 1 ? rows / bm + groups : (rows + bm - 1) / bm;
}

namespace {

template <int EPI>
void launch_rows(const Fp8Args &p, int bm, hipStream_t st)
{
    switch (bm) {
    case 16: launch_cfg<4, 16, 4, 1, 4, EPI>(p, st); break;
    case 32: launch_cfg<4, 32, 4, 2, 4, EPI>(p, st); break;
    case 64: launch_cfg<4, 64, 4, 2, 3, EPI>(p, st); break;
    case 96: launch_cfg<4, 96, 4, 2, 3, EPI>(p, st); break;
    case 128: launch_cfg<4, 128, 4, 2, 3, EPI>(p, st); break;
    case 256:
        if constexpr (EPI != EPI_SWIGLU) {  // fp8_size
            launch_cfg<4, 256, 4, 2, 2, EPI>(p, st);
            break;
        }
        [[fallthrough]];
    default: launch_cfg<4, 144, 4, 2, 3, EPI>(p, st); break;
    }
}

}  // namespace

void launch_fp8_matmul(const Fp8Args &p, Fp8Tile t, hipStream_t st)
{
    if (p.exps)
        launch_rows<EPI_STAGE>(p, t.rows, st);
    else if (fp8_split_ok(p))
        launch_fp8_split(p, st);
    else if (t.cols == 64)
        launch_cfg<2, 64, 2, 2, 3, EPI_PLAIN>(p, st);
    else
        launch_rows<EPI_PLAIN>(p, t.rows, st);
}
void launch_fp8_gate_up(const Fp8Args &p, int bm, hipStream_t st) { launch_rows<EPI_SWIGLU>(p, bm, st); }

}  // namespace moe
