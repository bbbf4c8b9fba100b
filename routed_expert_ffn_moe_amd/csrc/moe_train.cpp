// C ABI of the operators between the router and a caller's own step through the
// experts, and of their gradients: argument checks and launches, all asynchronous
// on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>

#include "../../include/moe.h"
#include "args.h"
#include "kernels.h"

using moe::aligned;
using moe::bad;
using moe::cdiv;
using moe::overlap;

namespace {

// Largest stride, number of pairs, number of rows and size of a row: every offset in
// bytes then stays below 2^63, and every count of columns that a kernel rounds up
// below 2^31.
constexpr int64_t MAX_LD = (int64_t)1 << 31, MAX_PAIRS = (int64_t)1 << 30;
constexpr int32_t MAX_COLS = 1 << 30, MAX_ROWS = 1 << 30;

bool float_type(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }

int64_t size_of(int dt) { return dt == MOE_F32 ? 4 : 2; }

bool stride_ok(int64_t ld, int64_t cols) { return ld == 0 || (ld >= cols && ld <= MAX_LD); }

// Bytes from the first to the last element of a matrix.
int64_t span(int64_t rows, int64_t cols, int64_t ld, int64_t esz)
{
    return rows > 0 ? ((rows - 1) * ld + cols) * esz : 0;
}

// Stretches of memory of one call; an output may overlap none of the others.
struct Stretch {
    const void *p;
    int64_t bytes;
    bool out;
};

template <int N>
bool collide(const Stretch (&s)[N])
{
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < i; ++j)
            if ((s[i].out || s[j].out) && s[i].p && s[j].p && s[i].bytes && s[j].bytes &&
                overlap(s[i].p, s[i].bytes, s[j].p, s[j].bytes))
                return true;
    return false;
}

// nullptr, or what is wrong with the sizes.
const char *dispatch_sizes(const moe_dispatch_t *s)
{
    if (!s)
        return "dispatch is NULL";
    if (s->T < 0 || s->H < 1 || s->H > MAX_COLS)
        return "T >= 0 and H in 1..2^30";
    if (s->E < 1 || s->E > 1024)
        return "E must be in 1..1024";
    if (s->top_k < 1 || s->top_k > 16)
        return "top_k must be in 1..16";
    if ((int64_t)s->T * s->top_k > MAX_PAIRS)
        return "more than 2^30 pairs";
    if (s->x_dtype != MOE_F32 && s->x_dtype != MOE_BF16 && s->x_dtype != MOE_FP8)
        return "x_dtype must be MOE_F32, MOE_BF16 or MOE_FP8";
    if (s->x_dtype == MOE_FP8 ? !float_type(s->row_dtype) : s->row_dtype != s->x_dtype)
        return "row_dtype must be x_dtype, and MOE_F32 or MOE_BF16 where x is codes";
    const int64_t width = s->x_dtype == MOE_FP8 ? cdiv(s->H, moe::FP8_K) * moe::FP8_K : s->H;
    if (!stride_ok(s->ldx, width) || (s->x_dtype == MOE_FP8 && s->ldx % 16))
        return "ldx must be 0 or at least a row (codes: a multiple of 16), and at most 2^31";
    if (!stride_ok(s->ldr, s->H))
        return "ldr must be 0 or at least H, and at most 2^31";
    return nullptr;
}

struct Rows {
    moe::GatherArgs a;
    int64_t x, sx, rows;  // bytes
};

Rows gather_args(const moe_dispatch_t *s, const void *x, const float *sx, void *rows, const int32_t *row_of)
{
    Rows r{};
    const int64_t kb = cdiv(s->H, moe::FP8_K);
    const bool fp8 = s->x_dtype == MOE_FP8;
    r.a.x = x;
    r.a.sx = fp8 ? sx : nullptr;
    r.a.rows = rows;
    r.a.row_of = row_of;
    r.a.ldx = s->ldx ? s->ldx : fp8 ? kb * moe::FP8_K : s->H;
    r.a.ldr = s->ldr ? s->ldr : s->H;
    r.a.T = s->T;
    r.a.H = s->H;
    r.a.k = s->top_k;
    r.a.R = s->T * s->top_k;
    r.a.src = fp8 ? moe::GATHER_FP8 : s->x_dtype == MOE_F32 ? moe::GATHER_F32 : moe::GATHER_BF16;
    r.a.out_f32 = s->row_dtype == MOE_F32;
    r.x = fp8 ? span(s->T, kb * moe::FP8_K, r.a.ldx, 1) : span(s->T, s->H, r.a.ldx, size_of(s->x_dtype));
    r.sx = fp8 ? s->T * kb * 4 : 0;
    r.rows = span(r.a.R, s->H, r.a.ldr, size_of(s->row_dtype));
    return r;
}

// The same for the rows' pointers.
const char *gather_pointers(const moe_dispatch_t *s, const void *x, const float *sx, const void *rows)
{
    if (!x || !rows || (s->x_dtype == MOE_FP8 && !sx))
        return "NULL pointer";
    if (!aligned(x, s->x_dtype == MOE_FP8 ? 16 : size_of(s->x_dtype)) || !aligned(sx, 4) ||
        !aligned(rows, size_of(s->row_dtype)))
        return "codes not 16-byte, or another pointer not element aligned";
    return nullptr;
}

int fail(const char *entry, const char *what)
{
    static thread_local char text[256];
    snprintf(text, sizeof text, "%s: %s", entry, what);
    return bad(text);
}

const char *combine_sizes(const moe_combine_t *s)
{
    if (!s)
        return "combine is NULL";
    if (s->T < 0 || s->R < 0 || s->R > MAX_ROWS || s->H < 1 || s->H > MAX_COLS)
        return "T >= 0, R in 0..2^30 and H in 1..2^30";
    if (s->top_k < 1 || s->top_k > 16)
        return "top_k must be in 1..16";
    if ((int64_t)s->T * s->top_k > MAX_PAIRS)
        return "more than 2^30 pairs";
    if (!float_type(s->dtype))
        return "dtype must be MOE_F32 or MOE_BF16";
    if (!stride_ok(s->ldr, s->H) || !stride_ok(s->ldy, s->H))
        return "ldr and ldy must be 0 or at least H, and at most 2^31";
    return nullptr;
}

moe::CombineRowsArgs combine_args(const moe_combine_t *s, const int32_t *row_of, const float *w)
{
    moe::CombineRowsArgs a{};
    a.row_of = row_of;
    a.w = w;
    a.ldr = s->ldr ? s->ldr : s->H;
    a.ldy = s->ldy ? s->ldy : s->H;
    a.T = s->T;
    a.H = s->H;
    a.k = s->top_k;
    a.R = s->R;
    a.f32 = s->dtype == MOE_F32;
    return a;
}

const char *swiglu_sizes(const moe_swiglu_t *s)
{
    if (!s)
        return "swiglu is NULL";
    if (s->R < 0 || s->R > MAX_ROWS || s->I < 1 || s->I > MAX_COLS)
        return "R in 0..2^30 and I in 1..2^30";
    if (!float_type(s->dtype))
        return "dtype must be MOE_F32 or MOE_BF16";
    if (!stride_ok(s->ld, s->I) || !stride_ok(s->ldh, s->I))
        return "ld and ldh must be 0 or at least I, and at most 2^31";
    if (s->R * cdiv(s->I, moe::FP8_K) >= (int64_t)1 << 31)
        return "2^31 blocks of 1 x 128 or more";
    return nullptr;
}

moe::SwigluArgs swiglu_args(const moe_swiglu_t *s, const int32_t *used)
{
    moe::SwigluArgs a{};
    a.used = used;
    a.ld = s->ld ? s->ld : s->I;
    a.ldh = s->ldh ? s->ldh : s->I;
    a.R = s->R;
    a.I = s->I;
    a.KB = (int)cdiv(s->I, moe::FP8_K);
    a.bf16 = s->dtype == MOE_BF16;
    return a;
}

// nullptr and the sizes of a product, or what is wrong with them.
struct Product {
    moe::Mm16Args a;
    int64_t np, nq, no;  // elements from the first to the last of p, q and the output
};

const char *matmul_args(const moe_matmul_bf16_t *s, int way, bool grouped, Product &r)
{
    if (!s)
        return "matmul is NULL";
    if (s->M < 0 || s->M > MAX_ROWS || s->N < 1 || s->N > MAX_COLS || s->K < 1 || s->K > MAX_COLS || s->G < 1 ||
        s->G > 65535)
        return "M in 0..2^30, N and K in 1..2^30 and G in 1..65535";
    if (!float_type(s->out_dtype))
        return "out_dtype must be MOE_F32 or MOE_BF16";
    if (!stride_ok(s->ldx, s->K) || !stride_ok(s->ldw, s->K) || !stride_ok(s->ldy, s->N))
        return "ldx and ldw must be 0 or at least K, ldy 0 or at least N, and at most 2^31";
    if (s->G > 1 && !grouped)
        return "G > 1 needs offsets";
    const int64_t ldx = s->ldx ? s->ldx : s->K, ldw = s->ldw ? s->ldw : s->K, ldy = s->ldy ? s->ldy : s->N;
    if ((double)s->G * s->N * (double)ldw >= 1e18)
        return "the matrices w take more than 10^18 elements";
    moe::Mm16Args &a = r.a;
    a = {};
    a.M = s->M;
    a.G = s->G;
    a.way = way;
    a.out_f32 = s->out_dtype == MOE_F32;
    const int64_t nx = span(s->M, s->K, ldx, 1), nw = span((int64_t)s->G * s->N, s->K, ldw, 1),
                  ny = span(s->M, s->N, ldy, 1);
    if (way == moe::MM_Y) {
        a.P = s->M, a.Q = s->N, a.C = s->K;
        a.ldp = ldx, a.ldq = ldw, a.ldo = ldy;
        r.np = nx, r.nq = nw, r.no = ny;
    } else if (way == moe::MM_DX) {
        a.P = s->M, a.Q = s->K, a.C = s->N;
        a.ldp = ldy, a.ldq = ldw, a.ldo = ldx;
        r.np = ny, r.nq = nw, r.no = nx;
    } else {
        a.P = s->N, a.Q = s->K, a.C = s->M;
        a.ldp = ldy, a.ldq = ldx, a.ldo = ldw;
        r.np = ny, r.nq = nx, r.no = nw;
    }
    a.qstride = a.ostride = s->N * ldw;
    if (moe::mm16_most_tiles(a) >= (int64_t)1 << 31)
        return "too many tiles of 16 x 16";
    return nullptr;
}

int matmul_bf16(const char *entry, int way, const moe_matmul_bf16_t *s, const void *p, const void *q,
                const int32_t *offsets, const void *add, void *out, void *stream)
{
    Product r;
    if (const char *what = matmul_args(s, way, offsets, r))
        return fail(entry, what);
    moe::Mm16Args &a = r.a;
    a.p = (const uint16_t *)p;
    a.q = (const uint16_t *)q;
    a.offsets = offsets;
    a.add = add;
    a.out = out;
    const int64_t esz = size_of(s->out_dtype), np = r.np, nq = r.nq, no = r.no;
    if (s->M == 0 && way != moe::MM_DW)
        return MOE_OK;
    if (!out || (s->M > 0 && (!p || !q)))
        return fail(entry, "NULL pointer");
    if (!aligned(p, 2) || !aligned(q, 2) || !aligned(out, esz) || !aligned(add, esz) || !aligned(offsets, 4))
        return fail(entry, "pointer not aligned to its elements");
    const Stretch mem[] = {{out, no * esz, true}, {p, np * 2, false}, {q, nq * 2, false},
                           {offsets, (s->G + (int64_t)1) * 4, false},
                           {add == out ? nullptr : add, no * esz, false}};
    if (collide(mem))
        return fail(entry, "the output overlaps an operand, or add without being the same");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::launch_mm16(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

}  // namespace

extern "C" {

size_t moe_dispatch_workspace_bytes(const moe_dispatch_t *s)
{
    if (dispatch_sizes(s))
        return 0;
    return std::max<size_t>(256, moe::sort_blk_bytes(s->T, s->E, s->top_k));
}

int moe_dispatch(const moe_dispatch_t *s, const int32_t *topk_idx, const void *x, const float *sx, void *rows,
                 int32_t *offsets, int32_t *row_src, int32_t *row_of, void *ws, size_t ws_bytes, void *stream)
{
    const char *entry = "moe_dispatch";
    if (const char *what = dispatch_sizes(s))
        return fail(entry, what);
    const int64_t pairs = (int64_t)s->T * s->top_k;
    if (!offsets || (pairs && (!topk_idx || !row_of)))
        return fail(entry, "topk_idx, offsets or row_of is NULL");
    if (!aligned(topk_idx, 4) || !aligned(offsets, 4) || !aligned(row_src, 4) || !aligned(row_of, 4))
        return fail(entry, "pointer not aligned to its elements");
    if ((x || rows) && pairs)
        if (const char *what = gather_pointers(s, x, sx, rows))
            return fail(entry, what);
    const size_t need = moe::sort_blk_bytes(s->T, s->E, s->top_k);
    if (need && (!ws || !aligned(ws, 256)))
        return fail(entry, "ws is NULL or not 256-byte aligned");
    if (ws_bytes < need)
        return moe::api_fail(MOE_EWORKSPACE, "moe_dispatch: ws_bytes below moe_dispatch_workspace_bytes");
    Rows r = gather_args(s, x, sx, rows, row_of);
    const Stretch mem[] = {{topk_idx, pairs * 4, false}, {x, r.x, false}, {r.a.sx, r.sx, false}, {rows, r.rows, true},
                           {offsets, (s->E + 1) * 4, true}, {row_src, pairs * 4, true}, {row_of, pairs * 4, true},
                           {need ? ws : nullptr, (int64_t)need, true}};
    if (collide(mem))
        return fail(entry, "outputs or workspace overlap an input or each other");
    if (const int rc = moe::api_check_device())
        return rc;
    if (!pairs)
        r.a.x = nullptr;
    const moe::SortArgs a{topk_idx, offsets, row_src, row_of, (int32_t *)ws, s->T, s->E, s->top_k};
    moe::launch_dispatch(a, r.a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_gather(const moe_dispatch_t *s, const int32_t *row_of, const void *x, const float *sx, void *rows,
               void *stream)
{
    const char *entry = "moe_gather";
    if (const char *what = dispatch_sizes(s))
        return fail(entry, what);
    if (s->T == 0)
        return MOE_OK;
    if (!row_of || !aligned(row_of, 4))
        return fail(entry, "row_of is NULL or not aligned to its elements");
    if (const char *what = gather_pointers(s, x, sx, rows))
        return fail(entry, what);
    const Rows r = gather_args(s, x, sx, rows, row_of);
    const Stretch mem[] = {{rows, r.rows, true}, {x, r.x, false}, {r.a.sx, r.sx, false},
                           {row_of, (int64_t)r.a.R * 4, false}};
    if (collide(mem))
        return fail(entry, "rows overlap an input");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::launch_gather(r.a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_combine(const moe_combine_t *s, const void *rows, const int32_t *row_of, const float *topk_w, void *y,
                void *stream)
{
    const char *entry = "moe_combine";
    if (const char *what = combine_sizes(s))
        return fail(entry, what);
    if (s->T == 0)
        return MOE_OK;
    const int64_t esz = size_of(s->dtype), pairs = (int64_t)s->T * s->top_k;
    if ((!rows && s->R) || !row_of || !y)
        return fail(entry, "NULL pointer");
    if (!aligned(rows, esz) || !aligned(y, esz) || !aligned(row_of, 4) || !aligned(topk_w, 4))
        return fail(entry, "pointer not aligned to its elements");
    moe::CombineRowsArgs a = combine_args(s, row_of, topk_w);
    const Stretch mem[] = {{y, span(s->T, s->H, a.ldy, esz), true}, {rows, span(s->R, s->H, a.ldr, esz), false},
                           {row_of, pairs * 4, false}, {topk_w, pairs * 4, false}};
    if (collide(mem))
        return fail(entry, "y overlaps an input");
    if (const int rc = moe::api_check_device())
        return rc;
    a.rows = rows;
    a.y = y;
    moe::launch_combine_rows(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_combine_grad(const moe_combine_t *s, const void *dy, const void *rows, const int32_t *row_of,
                     const float *topk_w, void *drows, float *dtopk_w, void *stream)
{
    const char *entry = "moe_combine_grad";
    if (const char *what = combine_sizes(s))
        return fail(entry, what);
    if (s->T == 0 || (!drows && !dtopk_w))
        return MOE_OK;
    const int64_t esz = size_of(s->dtype), pairs = (int64_t)s->T * s->top_k;
    if (!dy || !row_of || (dtopk_w && !rows && s->R))
        return fail(entry, "NULL pointer");
    if (!aligned(dy, esz) || !aligned(rows, esz) || !aligned(drows, esz) || !aligned(row_of, 4) ||
        !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
        return fail(entry, "pointer not aligned to its elements");
    moe::CombineRowsArgs a = combine_args(s, row_of, topk_w);
    const int64_t nr = span(s->R, s->H, a.ldr, esz);
    const Stretch mem[] = {{drows, nr, true}, {dtopk_w, pairs * 4, true}, {dy, span(s->T, s->H, a.ldy, esz), false},
                           {dtopk_w ? rows : nullptr, nr, false}, {row_of, pairs * 4, false},
                           {topk_w, pairs * 4, false}};
    if (collide(mem))
        return fail(entry, "outputs overlap an input or each other");
    if (const int rc = moe::api_check_device())
        return rc;
    a.rows = rows;
    a.dy = dy;
    a.drows = drows;
    a.dw = dtopk_w;
    moe::launch_combine_rows_grad(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_swiglu(const moe_swiglu_t *s, const void *gate, const void *up, const int32_t *used, void *h, void *codes,
               float *scales, void *stream)
{
    const char *entry = "moe_swiglu";
    if (const char *what = swiglu_sizes(s))
        return fail(entry, what);
    if (!codes != !scales)
        return fail(entry, "codes and scales come together");
    if (s->R == 0)
        return MOE_OK;
    if (!gate || !up || !h)
        return fail(entry, "NULL pointer");
    const int64_t esz = size_of(s->dtype);
    if (!aligned(gate, esz) || !aligned(up, esz) || !aligned(h, esz) || !aligned(used, 4) || !aligned(codes, 16) ||
        !aligned(scales, 4))
        return fail(entry, "codes not 16-byte, or another pointer not element aligned");
    moe::SwigluArgs a = swiglu_args(s, used);
    const int64_t blocks = 2ll * s->R * a.KB, in = span(s->R, s->I, a.ld, esz);
    const Stretch mem[] = {{h, span(s->R, s->I, a.ldh, esz), true}, {codes, blocks * moe::FP8_K, true},
                           {scales, blocks * 4, true}, {gate, in, false}, {up, in, false}, {used, 4, false}};
    if (collide(mem))
        return fail(entry, "outputs overlap an input or each other");
    if (const int rc = moe::api_check_device())
        return rc;
    a.gate = gate;
    a.up = up;
    a.h = h;
    a.codes = (uint8_t *)codes;
    a.scales = scales;
    moe::launch_swiglu(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_swiglu_grad(const moe_swiglu_t *s, const void *gate, const void *up, const void *codes, const float *scales,
                    const void *dh, const int32_t *used, void *dgate, void *dup, void *h, void *stream)
{
    const char *entry = "moe_swiglu_grad";
    if (const char *what = swiglu_sizes(s))
        return fail(entry, what);
    if (!codes != !scales)
        return fail(entry, "codes and scales come together");
    if (s->R == 0)
        return MOE_OK;
    if ((!codes && (!gate || !up)) || !dh || !dgate || !dup)
        return fail(entry, "NULL pointer");
    const int64_t esz = size_of(s->dtype);
    if (!aligned(gate, esz) || !aligned(up, esz) || !aligned(dh, esz) || !aligned(dgate, esz) ||
        !aligned(dup, esz) || !aligned(h, esz) || !aligned(used, 4) || !aligned(codes, 16) || !aligned(scales, 4))
        return fail(entry, "codes not 16-byte, or another pointer not element aligned");
    moe::SwigluArgs a = swiglu_args(s, used);
    const int64_t blocks = 2ll * s->R * a.KB, in = span(s->R, s->I, a.ld, esz), hb = span(s->R, s->I, a.ldh, esz);
    // gate | up, and dgate | dup, may be the columns of one matrix: rows between rows
    const bool side = dgate != dup && a.ld >= 2 * (int64_t)s->I &&
                      std::abs((const char *)dup - (const char *)dgate) % (a.ld * esz) >= s->I * esz &&
                      std::abs((const char *)dup - (const char *)dgate) % (a.ld * esz) <= (a.ld - s->I) * esz;
    if (!side && overlap(dgate, in, dup, in))
        return fail(entry, "dgate and dup overlap");
    for (const void *out : {(const void *)dgate, (const void *)dup}) {
        const Stretch mem[] = {{out, in, true}, {h, hb, true}, {codes, blocks * moe::FP8_K, false},
                               {scales, blocks * 4, false}, {codes ? nullptr : gate, in, false},
                               {codes ? nullptr : up, in, false}, {dh, hb, false}, {used, 4, false}};
        if (collide(mem))
            return fail(entry, "outputs overlap an input or each other");
    }
    if (const int rc = moe::api_check_device())
        return rc;
    a.gate = gate;
    a.up = up;
    a.dh = dh;
    a.dgate = dgate;
    a.dup = dup;
    a.h = h;
    a.codes = (uint8_t *)codes;
    a.scales = (float *)scales;
    moe::launch_swiglu_grad(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_select_grad(const moe_select_t *s, const void *logits, const float *bias, const int32_t *topk_idx,
                    const float *dtopk_w, const float *dscore, void *dlogits, int dlogit_dtype, void *stream)
{
    const char *entry = "moe_select_grad";
    if (!s)
        return fail(entry, "select is NULL");
    if (s->T < 0 || s->T > MAX_ROWS)
        return fail(entry, "T must be in 0..2^30");
    if (s->E < 1 || s->E > 1024)
        return fail(entry, "E must be in 1..1024");
    if (s->top_k < 1 || s->top_k > s->E || s->top_k > 16)
        return fail(entry, "top_k must be in 1..min(E, 16)");
    if (s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID)
        return fail(entry, "unknown score");
    if (!float_type(s->logit_dtype) || !float_type(dlogit_dtype))
        return fail(entry, "logit_dtype and dlogit_dtype must be MOE_F32 or MOE_BF16");
    if (!stride_ok(s->ld, s->E))
        return fail(entry, "ld must be 0 or at least E, and at most 2^31");
    if (s->T == 0)
        return MOE_OK;
    if (!logits || !topk_idx || !dtopk_w || !dlogits)
        return fail(entry, "NULL pointer");
    const int64_t esz = size_of(s->logit_dtype), osz = size_of(dlogit_dtype), pairs = (int64_t)s->T * s->top_k;
    if (!aligned(logits, esz) || !aligned(dlogits, osz) || !aligned(bias, 4) || !aligned(topk_idx, 4) ||
        !aligned(dtopk_w, 4) || !aligned(dscore, 4))
        return fail(entry, "pointer not aligned to its elements");
    moe::SelectGradArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.idx = topk_idx;
    a.dw = dtopk_w;
    a.dscore = dscore;
    a.dlogits = dlogits;
    a.ld = s->ld ? s->ld : s->E;
    a.T = s->T;
    a.E = s->E;
    a.k = s->top_k;
    a.softmax = s->score == MOE_SCORE_SOFTMAX;
    a.renorm = s->renorm != 0;
    a.bf16 = s->logit_dtype == MOE_BF16;
    a.out_f32 = dlogit_dtype == MOE_F32;
    a.scale = s->scale;
    const Stretch mem[] = {{dlogits, (int64_t)s->T * s->E * osz, true}, {logits, span(s->T, s->E, a.ld, esz), false},
                           {bias, s->E * 4, false}, {topk_idx, pairs * 4, false}, {dtopk_w, pairs * 4, false},
                           {dscore, s->E * 4, false}};
    if (collide(mem))
        return fail(entry, "dlogits overlap an input");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::launch_select_grad(a, (hipStream_t)stream);
    return moe::api_launched(entry);
}

int moe_matmul_bf16(const moe_matmul_bf16_t *matmul, const void *x, const void *w, const int32_t *offsets,
                    const void *add, void *y, void *stream)
{
    return matmul_bf16("moe_matmul_bf16", moe::MM_Y, matmul, x, w, offsets, add, y, stream);
}

int moe_matmul_bf16_tile(const moe_matmul_bf16_t *matmul, int way, int off16, int32_t *tile)
{
    const char *entry = "moe_matmul_bf16_tile";
    if (way < moe::MM_Y || way > moe::MM_DW || !tile)
        return fail(entry, "way must be 0, 1 or 2 and tile not NULL");
    Product r;
    if (const char *what = matmul_args(matmul, way, true, r))
        return fail(entry, what);
    r.a.p = (const uint16_t *)(uintptr_t)(off16 ? 2 : 0);
    const moe::Mm16Pick t = moe::mm16_pick(r.a);
    const int32_t v[] = {t.rows, t.cols, t.groups, t.whole};
    std::copy(v, v + 4, tile);
    return MOE_OK;
}

int moe_matmul_bf16_dx(const moe_matmul_bf16_t *matmul, const void *dy, const void *w, const int32_t *offsets,
                       const void *add, void *dx, void *stream)
{
    return matmul_bf16("moe_matmul_bf16_dx", moe::MM_DX, matmul, dy, w, offsets, add, dx, stream);
}

int moe_matmul_bf16_dw(const moe_matmul_bf16_t *matmul, const void *dy, const void *x, const int32_t *offsets,
                       const void *add, void *dw, void *stream)
{
    return matmul_bf16("moe_matmul_bf16_dw", moe::MM_DW, matmul, dy, x, offsets, add, dw, stream);
}

}  // extern "C"
