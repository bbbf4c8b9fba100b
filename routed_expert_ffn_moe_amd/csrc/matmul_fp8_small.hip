// The FP8 products of few rows, where there are too few tiles for the kernel
// in matmul_fp8.hip to fill the chip and a call is a matter of latency: K is
// split over the waves of a workgroup, which read their fragments straight
// from memory and meet once in LDS.
//
//  fp8_split        one matrix of few tiles: wave sums over every KS-th block of
//                   K, joined in wave order.  M=1, N=K=4096: 5.2 us, where its
//                   16.8 MB take 2.8 and a launch with one wait for memory 3.
//  fp8_pair_gate_up decode rows of the experts (T <= 8): one workgroup per
//                   (token, slot) pair and 16 columns of h, no permutation;
//                   the pair's x is quantised on the way.  The codes are
//                   multiplied as bf16, as in the tiles (fp8.h).
//  fp8_token_down   their down projections and the combine: one workgroup per
//                   token and 16 columns of y, h quantised on the way.
// T=1, H=2048, k=8, I=768: 8.3 + 9.6 us, 16.2 a call in a run of them (38 MB take
// 6.2): each is a chain of indices, weights, MFMA, LDS and the sums of the blocks in
// their order.
//
// The decode kernels pass the sums of single blocks of K through LDS and join
// them in K order with the same FMAs as the tile kernel, and round each
// slot's row as its staging row would be: y has the same bits whichever path
// a pass takes.
#include <algorithm>

#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

namespace {

// Fragment of a 16-row block at block kb of K: lane (l16, lg) holds pieces lg
// and lg + 4 of its row's 128 bytes, as in the tile kernel.
__device__ __forceinline__ Fp8Raw frag_at(const uint8_t *row, int kb, int lg)
{
    const uint8_t *p = row + (int64_t)kb * FP8_BLOCK + lg * 16;
    return fp8_raw(*(const uint4 *)p, *(const uint4 *)(p + 64));
}

// NB weight and MB row blocks a wave; KS waves along K, 8 / KS along the columns.
template <int NB, int MB, int KS, bool EXACT>
__global__ __launch_bounds__(512) void fp8_split(Fp8Args p)
{
    constexpr int WN = 8 / KS, BN = 16 * NB * WN, BM = 16 * MB, LD = BN + 1;
    __shared__ float s_acc[KS][BM * LD];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6), ks = w % KS, wn = w / KS;
    const int ntn = (p.N + BN - 1) / BN;
    const int mt = blockIdx.x / ntn, n0 = (blockIdx.x - mt * ntn) * BN, row0 = mt * BM;
    const int nw = n0 + wn * NB * 16;  // the wave's first column

    const uint8_t *wr[NB], *ar[MB];
    const float *sr[MB];
#pragma unroll
    for (int c = 0; c < NB; ++c)
        wr[c] = p.b0 + (int64_t)min(nw + c * 16 + l16, p.N - 1) * p.ldb;
#pragma unroll
    for (int m = 0; m < MB; ++m) {
        const int64_t r = min(row0 + m * 16 + l16, p.M - 1);
        ar[m] = p.a + r * p.lda;
        sr[m] = p.sa + r * p.KB;
    }
    const float *sw = p.s0 + (int64_t)min(nw >> 7, ((p.N + 127) >> 7) - 1) * p.KB;
    floatx4 acc[NB][MB];
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            acc[c][m] = floatx4{0, 0, 0, 0};
    // U blocks of K in flight
    constexpr int U = NB * MB <= 1 ? 4 : NB * MB <= 4 ? 2 : 1;
    for (int k0 = ks; k0 < p.KB; k0 += KS * U) {
        Fp8Raw A[U][NB], B[U][MB];
        float fw[U], fr[U][MB];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(k0 + u * KS, p.KB - 1);
#pragma unroll
            for (int c = 0; c < NB; ++c)
                A[u][c] = frag_at(wr[c], kb, lg);
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                B[u][m] = frag_at(ar[m], kb, lg);
                fr[u][m] = sr[m][kb];
            }
            // a block behind the last one is the last one again, with a scale
            // of 0 (no branch, behind which its loads would be moved)
            fw[u] = sw[kb];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
            for (int m = 0; m < MB; ++m) {
                const Fp8Frag<EXACT> b(B[u][m]);
                const float f = k0 + u * KS < p.KB ? fr[u][m] * fw[u] : 0.0f;
#pragma unroll
                for (int c = 0; c < NB; ++c) {
                    const floatx4 t = mfma_fp8(Fp8Frag<EXACT>(A[u][c]), b);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[c][m][i] = fmaf(t[i], f, acc[c][m][i]);
                }
            }
        }
    }
#pragma unroll
    for (int c = 0; c < NB; ++c)
#pragma unroll
        for (int m = 0; m < MB; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_acc[ks][(m * 16 + l16) * LD + (wn * NB + c) * 16 + lg * 4 + i] = acc[c][m][i];
    __syncthreads();
    const int rows = min(BM, p.M - row0), cols = min(BN, p.N - n0);
    for (int i = tid; i < rows * BN; i += 512) {
        const int r = i / BN, c = i - r * BN;
        if (c >= cols)
            continue;
        float v = s_acc[0][r * LD + c];
#pragma unroll
        for (int k = 1; k < KS; ++k)
            v += s_acc[k][r * LD + c];
        const int64_t at = (int64_t)(row0 + r) * p.ldy + n0 + c;
        if (p.out_f32)
            ((float *)p.y)[at] = v;
        else
            ((uint16_t *)p.y)[at] = (uint16_t)cvt_bf2(v, 0.0f);
    }
}

template <int NB, int MB, int KS>
void launch_split(const Fp8Args &p, hipStream_t st)
{
    constexpr int BN = 16 * NB * (8 / KS), BM = 16 * MB;
    const unsigned grid = (unsigned)(((p.M + BM - 1) / BM) * ((p.N + BN - 1) / BN));
    if (p.out_f32)
        fp8_split<NB, MB, KS, true><<<grid, 512, 0, st>>>(p);
    else
        fp8_split<NB, MB, KS, false><<<grid, 512, 0, st>>>(p);
}

// ---- decode rows of the experts ------------------------------------------------

// The codes of 128 values, two a lane, as the fragment of a one-row operand:
// the row in column 0 of the MFMA, zeros elsewhere.  `buf`: 128 bytes of LDS of
// this wave's own.
__device__ __forceinline__ Fp8Raw one_row_frag(float x0, float x1, uint8_t *buf, int lane, float &scale)
{
    float m = row16_max(fmaxf(fabsf(x0), fabsf(x1)));
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const Fp8Block q = fp8_block(m);
    scale = q.scale;
    ((uint16_t *)buf)[lane] =
        (uint16_t)__builtin_amdgcn_cvt_pk_fp8_f32(fp8_quot(x0, q), fp8_quot(x1, q), 0, false);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup");
    const int lg = lane >> 4;
    Fp8Raw f = fp8_raw(*(const uint4 *)(buf + lg * 16), *(const uint4 *)(buf + 64 + lg * 16));
    if (lane & 15)
        f = Fp8Raw{0, 0, 0, 0, 0, 0, 0, 0};
    return f;
}

// One output from the sums of its KB blocks (N apart) and their scales, in K order.
template <int N>
__device__ __forceinline__ float chain(const float *t, const float *f, int KB)
{
    float acc = 0.0f;
    int kb = 0;
    for (; kb + 8 <= KB; kb += 8) {
        float tv[8], fv[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // the reads in flight together
            tv[i] = t[(kb + i) * N];
            fv[i] = f[kb + i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            acc = fmaf(tv[i], fv[i], acc);
    }
    for (; kb < KB; ++kb)
        acc = fmaf(t[kb * N], f[kb], acc);
    return acc;
}

constexpr int GW = 8;  // waves of fp8_pair_gate_up

__global__ __launch_bounds__(64 * GW) void fp8_pair_gate_up(Fp8Decode p)
{
    extern __shared__ float s_t[];  // [2][KB][16] sums of blocks, then [2][KB] their scales
    __shared__ __attribute__((aligned(16))) uint8_t s_code[GW][FP8_BLOCK];
    const int pair = blockIdx.x / (p.I / 16), n0 = (blockIdx.x - pair * (p.I / 16)) * 16;
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KB = p.H / FP8_BLOCK;
    const uint16_t *x = p.x + (int64_t)(pair / p.k) * p.H;
    constexpr int U = 2;  // blocks of K in flight
    uint32_t xv[U];       // under way with the expert's number
#pragma unroll
    for (int u = 0; u < U; ++u)
        xv[u] = *(const uint32_t *)(x + min(w + u * GW, KB - 1) * FP8_BLOCK + lane * 2);
    const int e = p.idx[pair];
    if ((unsigned)e >= (unsigned)p.E)  // uniform: an empty slot
        return;
    float *s_f = s_t + 2 * KB * 16;
    const int64_t sc = ((int64_t)e * (p.I >> 7) + (n0 >> 7)) * KB;
    const int64_t mat = (int64_t)e * p.I * p.H + (int64_t)(n0 + l16) * p.H;
    for (int k0 = w; k0 < KB; k0 += GW * U) {
        Fp8Raw G[U], V[U];
        float fg[U], fv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = min(k0 + u * GW, KB - 1);
            G[u] = frag_at(p.w_gate + mat, kb, lg);
            V[u] = frag_at(p.w_up + mat, kb, lg);
            fg[u] = p.s_gate[sc + kb];
            fv[u] = p.s_up[sc + kb];
        }
        // x into codes while the weights are on their way
        Fp8Raw B[U];
        float sx[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            B[u] = one_row_frag(__uint_as_float(xv[u] << 16), __uint_as_float(xv[u] & 0xFFFF0000u),
                                s_code[w], lane, sx[u]);
            xv[u] = *(const uint32_t *)(x + min(k0 + (U + u) * GW, KB - 1) * FP8_BLOCK + lane * 2);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int kb = k0 + u * GW;
            const Fp8Frag<true> b(B[u]);  // the exact sums that codes of h need (fp8.h)
            const floatx4 g = mfma_fp8(Fp8Frag<true>(G[u]), b);
            const floatx4 v = mfma_fp8(Fp8Frag<true>(V[u]), b);
            if (kb < KB && l16 == 0) {
                *(floatx4 *)(s_t + kb * 16 + lg * 4) = g;
                *(floatx4 *)(s_t + (KB + kb) * 16 + lg * 4) = v;
                if (lane == 0) {
                    s_f[kb] = sx[u] * fg[u];
                    s_f[KB + kb] = sx[u] * fv[u];
                }
            }
        }
    }
    __syncthreads();
    if (w)
        return;
    // lanes 0..15: gate, 16..31: up
    const int m = (lane >> 4) & 1;
    const float acc = chain<16>(s_t + m * KB * 16 + l16, s_f + m * KB, KB);
    const float up = __shfl(acc, l16 + 16);
    if (lane < 16)
        p.h[(int64_t)pair * p.I + n0 + lane] = silu(acc) * up;
}

constexpr int DN = 16;  // columns of y of a workgroup

// DW waves, no fewer than a token's slots
template <int DW>
__global__ __launch_bounds__(64 * DW) void fp8_token_down(Fp8Decode p)
{
    extern __shared__ float s_t[];  // [k][KB][DN] sums of blocks, then [k][KB] their scales
    __shared__ __attribute__((aligned(16))) uint8_t s_code[DW][FP8_BLOCK];
    __shared__ float s_o[DW][DN], s_w[DW];
    __shared__ int s_live[DW];
    const int t = blockIdx.x / (p.H / DN), n0 = (blockIdx.x - t * (p.H / DN)) * DN;
    const int lane = threadIdx.x & 63, l16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KB = p.I / FP8_BLOCK, units = p.k * KB;
    float *s_f = s_t + units * DN;
    // this wave's slot of the combine, loaded early
    const int my_e = w < p.k ? p.idx[t * p.k + w] : -1;
    const float my_w = w < p.k ? p.topk_w[t * p.k + w] : 0.0f;
    const float *h = p.h + (int64_t)t * p.k * p.I + lane * 2;
    constexpr int U = 4;  // units in flight
    for (int u0 = w; u0 < units; u0 += DW * U) {
        Fp8Raw W[U];
        float2 hv[U];
        int e[U];
        float fw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = min(u0 + u * DW, units - 1), j = q / KB;
            e[u] = p.idx[t * p.k + j];
            hv[u] = *(const float2 *)(h + (int64_t)j * p.I + (q - j * KB) * FP8_BLOCK);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = min(u0 + u * DW, units - 1), kb = q - q / KB * KB;
            // an empty slot reads expert 0, and nobody its results
            const int64_t ev = (unsigned)e[u] < (unsigned)p.E ? e[u] : 0;
            W[u] = frag_at(p.w_down + (ev * p.H + n0 + l16) * p.I, kb, lg);
            fw[u] = p.s_down[(ev * (p.H >> 7) + (n0 >> 7)) * KB + kb];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int q = u0 + u * DW;
            float sh;
            const Fp8Frag<false> B(one_row_frag(hv[u].x, hv[u].y, s_code[w], lane, sh));
            const floatx4 o = mfma_fp8(Fp8Frag<false>(W[u]), B);
            if (q < units && l16 == 0)
                *(floatx4 *)(s_t + q * DN + lg * 4) = o;
            if (q < units && lane == 0)
                s_f[q] = sh * fw[u];
        }
    }
    __syncthreads();
    // wave j: slot j's outputs, rounded as a staging row is
    const bool mine = (unsigned)my_e < (unsigned)p.E;
    if (mine) {
        const float acc = chain<DN>(s_t + w * KB * DN + l16, s_f + w * KB, KB);
        uint32_t ex = stage_exponent(acc);
#pragma unroll
        for (int d = 1; d < 8; d <<= 1)
            ex = max(ex, (uint32_t)__shfl_xor((int)ex, d));
        ex = max(ex, STAGE_MIN_EXP);
        if (lane < DN)
            s_o[w][lane] = (float)(_Float16)(acc * stage_pack(ex)) * stage_unpack(ex);
    }
    if (lane == 0) {
        s_live[w] = mine;
        s_w[w] = my_w;
    }
    __syncthreads();
    if (threadIdx.x < DN) {
        float y = 0.0f;
        for (int j = 0; j < p.k; ++j)
            if (s_live[j])
                y = fmaf(s_w[j], s_o[j][threadIdx.x], y);
        p.y[(int64_t)t * p.H + n0 + threadIdx.x] = (uint16_t)cvt_bf2(y, 0.0f);
    }
}

}  // namespace

// One matrix of few rows.  (A wave's fragment reads fetch 38 bytes a
// nanosecond per CU from the caches, copies to LDS 130, so rows that many
// columns share are better copied: 601 x 2050 x 776 took 15 us this way.)
bool fp8_split_ok(const Fp8Args &p)
{
    return !p.tiles && !p.offsets && p.M <= 32 && (p.N + 255) / 256 < 256;
}

void launch_fp8_split(const Fp8Args &p, hipStream_t st)
{
    if (p.M <= 16)
        launch_split<1, 1, 8>(p, st);
    else
        launch_split<2, 2, 8>(p, st);
}

// Decode rows: LDS holds a block sum for each unit of work.  Pairs read their
// weights one by one, so more tokens than 8 are faster as tiles where they share
// experts (H=2688, I=256, k=7 of 8 experts: T=8 33.5 us as pairs, 33.4 as tiles
// with a permutation; T=12 45 and 34), and below it pairs are (T=4 21 and 34).
bool fp8_decode_ok(int T, int H, int k, int I)
{
    return T <= 8 && H / FP8_BLOCK <= 256 && (int64_t)k * (I / FP8_BLOCK) <= 512;
}

void launch_fp8_decode(const Fp8Decode &p, hipStream_t st)
{
    const int kb = p.H / FP8_BLOCK, units = p.k * (p.I / FP8_BLOCK);
    fp8_pair_gate_up<<<(unsigned)(p.T * p.k * (p.I / 16)), 64 * GW, (size_t)kb * 34 * 4, st>>>(p);
    // Eight waves where the slots allow it, which start sooner and share a CU with
    // another group's: where their 32 units in flight are all there are (T=1,
    // H=1536, I=512, k=8 11.7 us for both products, 13.7 with sixteen waves) or the
    // groups are more than the 256 CUs take at once (H=2048, I=768, k=8: T=3 28.8 us
    // and 30.7, T=4 33.0 and 35.2).  Else sixteen (the same, T=1 16.2 us, 17.0 with
    // eight, T=2, 256 groups, 19.6 and 20.9; T=1, H=4096 22.5 and 23.7).
    const unsigned grid = (unsigned)(p.T * (p.H / DN));
    const size_t lds = (size_t)units * (DN + 1) * 4;
    if (p.k <= 8 && (units <= 32 || grid > 256))
        fp8_token_down<8><<<grid, 64 * 8, lds, st>>>(p);
    else
        fp8_token_down<16><<<grid, 64 * 16, lds, st>>>(p);
}

}  // namespace moe
