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
// (fp32 results multiply the codes as bf16, four MFMAs per block: fp8.h).
// The weights are the MFMA's A operand and the rows of `a` its B operand: a
// lane then holds one row of y, whose scale is one register, and adjacent
// columns, which it stores as whole words.
//
// A workgroup of WN x WM waves owns BR = 16 * NBW * WN weight rows and BM = 16 *
// MB * WM rows of a.  Both operands go to LDS by asynchronous copies (row-major
// rows of 128 bytes are whole cache lines, so the weights need no packing),
// ST stages deep; a stage also holds the rows' scales.  In LDS the 16-byte
// pieces of a row are rotated (XOR) by the row, so that the 16 rows a fragment
// read touches fall on distinct banks, and the weight rows lie in the order
// in which a lane's results come out adjacent.
#include <type_traits>

#include "common.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {

namespace {

constexpr int MAX_KB = FP8_MAX_K / FP8_BLOCK;  // scale blocks along K whose weight scales fit LDS

enum { EPI_PLAIN = 0, EPI_SWIGLU = 1 };

// The tile of index mt along the rows: its group and rows [row0, end).
struct Rows {
    int g, row0, end;
};

// Row tile mt of grouped rows: groups' tiles follow each other.  Every wave
// finds it from the offsets, 64 groups a step; offsets outside 0..M or out of
// order are cut to the rows that exist.  g = -1 behind the last tile.
template <int BM>
__device__ __forceinline__ Rows find_rows(const int32_t *__restrict__ offsets, int G, int M, int mt)
{
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int g0 = 0; g0 < G; g0 += 64) {
        const int g = g0 + lane;
        int lo = 0, n = 0;
        if (g < G) {
            lo = min(max(offsets[g], 0), M);
            n = max(min(offsets[g + 1], M) - lo, 0);
        }
        const int nt = (n + BM - 1) / BM;
        const int inc = wave_scan_add(nt);
        const uint64_t hit = __ballot(base + inc > mt);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            const int before = base + __builtin_amdgcn_readlane(inc, l) - __builtin_amdgcn_readlane(nt, l);
            const int glo = __builtin_amdgcn_readlane(lo, l);
            return Rows{g0 + l, glo + (mt - before) * BM, glo + __builtin_amdgcn_readlane(n, l)};
        }
        base += __builtin_amdgcn_readlane(inc, 63);
    }
    return Rows{-1, 0, 0};
}

template <int NBW, int MB, int WN, int WM, int ST, int EPI>
struct Cfg {
    static constexpr int NW = WN * WM, BR = 16 * NBW * WN, BM = 16 * MB * WM;
    static constexpr int COLS = EPI == EPI_SWIGLU ? BR / 2 : BR;  // output columns of a tile
    static constexpr int WI = BR / 8 / NW;                        // weight copies of a wave and stage
    static constexpr int TI = BM / 8 < NW ? 1 : BM / 8 / NW;      // row copies
    static constexpr int L = WI + TI + 1;                         // all, with the scales
    static constexpr int SROWS = BM < 64 ? 64 : BM;
    static constexpr int STAGE = (BR + BM) * FP8_BLOCK + SROWS * 4;
    static constexpr int NSB = EPI == EPI_SWIGLU ? 2 : (BR + 127) / 128;  // weight scale rows of a tile
    static constexpr int LDS = ST * STAGE + NSB * MAX_KB * 4;
    static_assert(BR / 8 % NW == 0 && (BM / 8 < NW || BM / 8 % NW == 0), "copies divide among the waves");
    static_assert(EPI != EPI_SWIGLU || (COLS == 128 && NBW % 2 == 0), "a tile of h is one scale block wide");
    static_assert(LDS <= 163840, "LDS of one workgroup");
    static_assert(WN * BM * 4 <= ST * STAGE, "the block maxima reuse the stages");
};

template <int NBW, int MB, int WN, int WM, int ST, int EPI, bool EXACT>
__global__ __launch_bounds__(64 * WN * WM) void fp8_tile(Fp8Args p)
{
    using C = Cfg<NBW, MB, WN, WM, ST, EPI>;
    __shared__ __attribute__((aligned(256))) uint8_t smem[C::LDS];
    const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, lg = lane >> 4;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wn = w % WN, wm = w / WN;

    // ---- this workgroup's tile, dealt out in contiguous runs per XCD ------
    const int ntn = (p.N + C::COLS - 1) / C::COLS;
    int mtiles = p.mtiles;
    if (p.tiles)
        mtiles = min(mtiles, *p.ntiles);
    const int total = mtiles * ntn, per = (total + 7) / 8;
    const int id = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
    if (((int)blockIdx.x >> 3) >= per || id >= total)
        return;
    const int mt = id / ntn, n0 = (id - mt * ntn) * C::COLS;
    Rows r;
    if (p.tiles) {
        const Tile t = p.tiles[mt];
        r = Rows{t.g, t.row0, p.offsets[t.g + 1]};
    } else if (p.offsets) {
        r = find_rows<C::BM>(p.offsets, p.G, p.M, mt);
        if (r.g < 0)
            return;
    } else {
        r = Rows{0, mt * C::BM, p.M};
    }
    const int g = __builtin_amdgcn_readfirstlane(r.g), row0 = __builtin_amdgcn_readfirstlane(r.row0);
    const int nrows = min(C::BM, __builtin_amdgcn_readfirstlane(r.end) - row0);

    // ---- copy addresses: uniform bases that advance along K, lane offsets --
    const int sub = lane >> 3, slot = lane & 7;
    const int64_t gb = (int64_t)g * p.bstride, gs = (int64_t)g * p.sstride;
    uint32_t woff[C::WI], toff[C::TI], soff;
#pragma unroll
    for (int i = 0; i < C::WI; ++i) {
        const int rr = (w * C::WI + i) * 8 + sub, m = rr & 15, c = rr >> 4;
        const int own = c / NBW, cb = c - own * NBW;
        constexpr int HB = EPI == EPI_SWIGLU ? NBW / 2 : NBW;
        const int n = n0 + own * (HB * 16) + (m >> 2) * (4 * HB) + (cb % HB) * 4 + (m & 3);
        woff[i] = (uint32_t)((int64_t)min(n, p.N - 1) * p.ldb) + ((slot ^ (m >> 1)) << 4);
    }
#pragma unroll
    for (int i = 0; i < C::TI; ++i) {
        const int rr = ((w * C::TI + i) % (C::BM / 8)) * 8 + sub;
        const int at = min(rr, nrows - 1);
        const int64_t row = p.row_tok ? p.row_tok[row0 + at] : at;
        toff[i] = (uint32_t)(row * p.lda) + ((slot ^ ((rr >> 1) & 7)) << 4);
    }
    constexpr int SW = C::SROWS / 64;  // waves whose copies fill the scales
    {
        const int at = min((w % SW) * 64 + lane, nrows - 1);
        const int64_t row = p.row_tok ? p.row_tok[row0 + at] : at;
        soff = (uint32_t)(row * p.KB * 4);
    }
    const uint8_t *ga = p.a + (p.row_tok ? 0 : (int64_t)row0 * p.lda);
    const float *gsa = p.sa + (p.row_tok ? 0 : (int64_t)row0 * p.KB);
    const uint8_t *gw0 = p.b0 + gb, *gw1 = EPI == EPI_SWIGLU ? p.b1 + gb : nullptr;
    const uint32_t lds = __builtin_amdgcn_readfirstlane(lds_addr(smem));

    auto issue = [&](int s) {
        const uint32_t st = lds + (uint32_t)(s % ST) * C::STAGE;
        const int64_t k = (int64_t)s * FP8_BLOCK;
#pragma unroll
        for (int i = 0; i < C::WI; ++i) {
            const uint8_t *base = gw0;
            if (EPI == EPI_SWIGLU && ((((w * C::WI + i) * 8) >> 4) % NBW) >= NBW / 2)
                base = gw1;
            dma16(base + k, woff[i], st + (uint32_t)(w * C::WI + i) * 1024u);
        }
#pragma unroll
        for (int i = 0; i < C::TI; ++i)
            dma16(ga + k, toff[i],
                  st + C::BR * 128u + (uint32_t)((w * C::TI + i) % (C::BM / 8)) * 1024u);
        dma4(gsa + s, soff, st + (C::BR + C::BM) * 128u + (uint32_t)(w % SW) * 256u);
    };

    const int KB = p.KB;
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
        if (s < KB)
            issue(s);

    // ---- the tile's weight scales -----------------------------------------
    float *s_w = (float *)(smem + ST * C::STAGE);
    const int nb0 = n0 >> 7;
    for (int i = tid; i < C::NSB * KB; i += 64 * C::NW) {
        const int q = i / KB, k = i - q * KB;
        if constexpr (EPI == EPI_SWIGLU)
            s_w[q * MAX_KB + k] = (q ? p.s1 : p.s0)[gs + (int64_t)nb0 * KB + k];
        else
            s_w[q * MAX_KB + k] = p.s0[gs + (int64_t)min(nb0 + q, ((p.N + 127) >> 7) - 1) * KB + k];
    }

    floatx4 acc[NBW][MB];
#pragma unroll
    for (int c = 0; c < NBW; ++c)
#pragma unroll
        for (int m = 0; m < MB; ++m)
            acc[c][m] = floatx4{0, 0, 0, 0};

    const int o0 = l16 * 128 + ((lg ^ (l16 >> 1)) << 4), o1 = o0 ^ 64;
    const int nsb = EPI == EPI_SWIGLU ? 0 : (wn * NBW * 16) >> 7;
    for (int s = 0; s < KB; ++s) {
        // stage s has arrived for every wave, and every wave is done with the
        // stage that the next copies overwrite
        if (s + ST - 2 < KB)
            dma_wait_barrier<(ST - 2) * C::L>();
        else
            dma_wait_barrier<0>();
        if (s + ST - 1 < KB)
            issue(s + ST - 1);
        const uint8_t *st = smem + (s % ST) * C::STAGE;
        const uint8_t *wt = st + wn * (NBW * 2048), *tt = st + C::BR * 128 + wm * (MB * 2048);
        const float *ts = (const float *)(st + (C::BR + C::BM) * 128) + wm * (MB * 16);
        Fp8Frag<EXACT> A[NBW];
#pragma unroll
        for (int c = 0; c < NBW; ++c)
            A[c].set(*(const uint4 *)(wt + c * 2048 + o0), *(const uint4 *)(wt + c * 2048 + o1));
        const float sw0 = s_w[nsb * MAX_KB + s], sw1 = EPI == EPI_SWIGLU ? s_w[MAX_KB + s] : 0.0f;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            Fp8Frag<EXACT> B;
            B.set(*(const uint4 *)(tt + m * 2048 + o0), *(const uint4 *)(tt + m * 2048 + o1));
            const float sr = ts[m * 16 + l16];
            const float f0 = sr * sw0, f1 = sr * sw1;
#pragma unroll
            for (int c = 0; c < NBW; ++c) {
                const floatx4 t = mfma_fp8(A[c], B);
                const float f = EPI == EPI_SWIGLU && c >= NBW / 2 ? f1 : f0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[c][m][i] = fmaf(t[i], f, acc[c][m][i]);
            }
        }
    }

    if constexpr (EPI == EPI_PLAIN) {
        const int n = n0 + wn * (NBW * 16) + lg * (4 * NBW);
        const bool whole = p.vec && n + 4 * NBW <= p.N;
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int rr = (wm * MB + m) * 16 + l16;
            if (rr >= nrows)
                continue;
            const int64_t at = (int64_t)(row0 + rr) * p.ldy + n;
            if (p.out_f32) {
                float *y = (float *)p.y + at;
#pragma unroll
                for (int c = 0; c < NBW; ++c) {
                    if (whole)
                        *(floatx4 *)(y + 4 * c) = acc[c][m];
                    else
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (n + 4 * c + i < p.N)
                                y[4 * c + i] = acc[c][m][i];
                }
            } else {
                uint16_t *y = (uint16_t *)p.y + at;
                uint32_t v[2 * NBW];
#pragma unroll
                for (int c = 0; c < NBW; ++c) {
                    v[2 * c] = pack_bf2(acc[c][m][0], acc[c][m][1]);
                    v[2 * c + 1] = pack_bf2(acc[c][m][2], acc[c][m][3]);
                }
                if (whole) {
                    if constexpr (NBW % 2 == 0) {
#pragma unroll
                        for (int c = 0; c < NBW; c += 2)
                            *(uint4 *)(y + 4 * c) = uint4{v[2 * c], v[2 * c + 1], v[2 * c + 2], v[2 * c + 3]};
                    } else {
#pragma unroll
                        for (int c = 0; c < NBW; ++c)
                            *(uint2 *)(y + 4 * c) = uint2{v[2 * c], v[2 * c + 1]};
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4 * NBW; ++i)
                        if (n + i < p.N)
                            y[i] = (uint16_t)(v[i >> 1] >> (16 * (i & 1)));
                }
            }
        }
    } else {
        // h = silu(gate) * up, its block maximum over the tile's 128 columns
        // (4 lanes of a wave, then the waves), and its codes
        constexpr int HB = NBW / 2;
        float *s_max = (float *)smem;  // [WN][BM]
        __syncthreads();               // every wave is done with the last stage
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            float mx = 0.0f;
#pragma unroll
            for (int c = 0; c < HB; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float z = acc[c][m][i];
                    const float h = z / (1.0f + expf(-z)) * acc[c + HB][m][i];
                    acc[c][m][i] = h;
                    mx = fmaxf(mx, fabsf(h));
                }
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            if (lg == 0)
                s_max[wn * C::BM + (wm * MB + m) * 16 + l16] = mx;
        }
        __syncthreads();
#pragma unroll
        for (int m = 0; m < MB; ++m) {
            const int rr = (wm * MB + m) * 16 + l16;
            float mx = s_max[rr];
#pragma unroll
            for (int i = 1; i < WN; ++i)
                mx = fmaxf(mx, s_max[i * C::BM + rr]);
            if (rr >= nrows)
                continue;
            const Fp8Block q = fp8_block(mx);
            uint8_t *h = p.hq + (int64_t)(row0 + rr) * p.N + n0 + wn * (HB * 16) + lg * (4 * HB);
#pragma unroll
            for (int c = 0; c < HB; ++c)
                *(uint32_t *)(h + 4 * c) = fp8x4(acc[c][m][0], acc[c][m][1], acc[c][m][2], acc[c][m][3], q);
            if (wn == 0 && lg == 0)
                p.hs[(int64_t)(row0 + rr) * (p.N >> 7) + (n0 >> 7)] = q.scale;
        }
    }
}

template <int NBW, int MB, int WN, int WM, int ST, int EPI>
void launch_cfg(const Fp8Args &p, hipStream_t st)
{
    using C = Cfg<NBW, MB, WN, WM, ST, EPI>;
    const int64_t ntn = (p.N + C::COLS - 1) / C::COLS;
    const unsigned grid = (unsigned)((p.mtiles * ntn + 7) / 8 * 8);
    if (EPI == EPI_PLAIN && p.out_f32)
        fp8_tile<NBW, MB, WN, WM, ST, EPI, EPI == EPI_PLAIN><<<grid, 64 * C::NW, 0, st>>>(p);
    else
        fp8_tile<NBW, MB, WN, WM, ST, EPI, false><<<grid, 64 * C::NW, 0, st>>>(p);
}

}  // namespace

int fp8_bm(int64_t rows, int groups)
{
    const int64_t per = rows / (groups > 0 ? groups : 1);
    return per <= 16 ? 16 : per <= 48 ? 32 : per <= 96 ? 64 : 128;
}

int64_t fp8_row_tiles(int64_t rows, int groups, int bm)
{
    return (rows + bm - 1) / bm + (groups > 1 ? std::min<int64_t>(groups, rows) : 0);
}

void launch_fp8_matmul(const Fp8Args &p, int bm, hipStream_t st)
{
    switch (bm) {
    case 16: launch_cfg<2, 1, 4, 1, 4, EPI_PLAIN>(p, st); break;
    case 32: launch_cfg<4, 2, 4, 1, 3, EPI_PLAIN>(p, st); break;
    case 64: launch_cfg<4, 4, 4, 1, 3, EPI_PLAIN>(p, st); break;
    default: launch_cfg<4, 8, 4, 1, 3, EPI_PLAIN>(p, st); break;
    }
}

void launch_fp8_gate_up(const Fp8Args &p, int bm, hipStream_t st)
{
    switch (bm) {
    case 16: launch_cfg<4, 1, 4, 1, 4, EPI_SWIGLU>(p, st); break;
    case 32: launch_cfg<4, 2, 4, 1, 3, EPI_SWIGLU>(p, st); break;
    case 64: launch_cfg<4, 4, 4, 1, 3, EPI_SWIGLU>(p, st); break;
    default: launch_cfg<4, 8, 4, 1, 3, EPI_SWIGLU>(p, st); break;
    }
}

}  // namespace moe
