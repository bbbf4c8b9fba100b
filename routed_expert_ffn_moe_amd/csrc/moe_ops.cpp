// C ABI of the routing and FP8 operators: argument checks and launches, all
// asynchronous on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/moe.h"
#include "args.h"
#include "kernels.h"

using moe::aligned;
using moe::bad;
using moe::cdiv;
using moe::overlap;

extern "C" {

int moe_select(const moe_select_t *s, const void *logits, const float *bias, int32_t *topk_idx,
               float *topk_w, void *stream)
{
    if (!s)
        return bad("moe_select: select is NULL");
    if (s->T < 0)
        return bad("moe_select: T < 0");
    if (s->E < 1 || s->E > 1024)
        return bad("moe_select: E must be in 1..1024");
    if (s->top_k < 1 || s->top_k > s->E || s->top_k > 16)
        return bad("moe_select: top_k must be in 1..min(E, 16)");
    if (s->score != MOE_SCORE_SOFTMAX && s->score != MOE_SCORE_SIGMOID)
        return bad("moe_select: unknown score");
    if (s->group_score != MOE_GROUP_MAX && s->group_score != MOE_GROUP_TOP2)
        return bad("moe_select: unknown group_score");
    if (s->logit_dtype != MOE_F32 && s->logit_dtype != MOE_BF16)
        return bad("moe_select: logit_dtype must be MOE_F32 or MOE_BF16");
    if (s->n_group < 1 || s->n_group > 64 || s->E % s->n_group)
        return bad("moe_select: n_group must be in 1..64 and divide E");
    if (s->topk_group < 1 || s->topk_group > s->n_group)
        return bad("moe_select: topk_group must be in 1..n_group");
    if ((int64_t)s->topk_group * (s->E / s->n_group) < s->top_k)
        return bad("moe_select: the open groups hold fewer than top_k experts");
    if (s->ld != 0 && s->ld < s->E)
        return bad("moe_select: ld must be 0 or at least E");
    if (s->T == 0)
        return MOE_OK;
    if (!logits || !topk_idx)
        return bad("moe_select: logits or topk_idx is NULL");
    if (!aligned(logits, s->logit_dtype == MOE_F32 ? 4 : 2) || !aligned(bias, 4) ||
        !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return bad("moe_select: pointer not aligned to its elements");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::SelectArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.idx = topk_idx;
    a.w = topk_w;
    a.ld = s->ld ? s->ld : s->E;
    a.T = s->T;
    a.E = s->E;
    a.k = s->top_k;
    // all groups open: the same selection without them
    a.n_group = s->topk_group < s->n_group ? s->n_group : 1;
    a.topk_group = s->topk_group;
    a.softmax = s->score == MOE_SCORE_SOFTMAX;
    a.group_top2 = s->group_score == MOE_GROUP_TOP2;
    a.renorm = s->renorm != 0;
    a.bf16 = s->logit_dtype == MOE_BF16;
    a.scale = s->scale;
    moe::launch_select(a, (hipStream_t)stream);
    return moe::api_launched("moe_select");
}

int moe_quant_fp8(const moe_quant_t *s, const void *x, void *codes, float *scales, void *stream)
{
    if (!s)
        return bad("moe_quant_fp8: quant is NULL");
    if (s->R < 0 || s->K < 1)
        return bad("moe_quant_fp8: R >= 0 and K >= 1");
    if (s->block_rows != 1 && s->block_rows != moe::FP8_K)
        return bad("moe_quant_fp8: block_rows must be 1 or 128");
    if (s->src_dtype != MOE_F32 && s->src_dtype != MOE_BF16)
        return bad("moe_quant_fp8: src_dtype must be MOE_F32 or MOE_BF16");
    if (s->ld != 0 && s->ld < s->K)
        return bad("moe_quant_fp8: ld must be 0 or at least K");
    const int64_t KB = cdiv(s->K, moe::FP8_K);
    // blocks of 128 x 128: a workgroup of 256 threads each, below 2^32 threads
    const int64_t blocks = cdiv(s->R, s->block_rows) * KB;
    if (blocks >= (int64_t)1 << (s->block_rows == 1 ? 31 : 24))
        return bad("moe_quant_fp8: 2^31 blocks of 1 x 128, or 2^24 of 128 x 128, or more");
    if (s->R == 0)
        return MOE_OK;
    if (!x || !codes || !scales)
        return bad("moe_quant_fp8: NULL pointer");
    const int esz = s->src_dtype == MOE_F32 ? 4 : 2;
    if (!aligned(x, esz) || !aligned(codes, 16) || !aligned(scales, 4))
        return bad("moe_quant_fp8: codes not 16-byte, or x or scales not element aligned");
    const int64_t ld = s->ld ? s->ld : s->K;
    const int64_t xb = ((s->R - 1) * ld + s->K) * esz, cb = s->R * KB * moe::FP8_K;
    const int64_t sb = cdiv(s->R, s->block_rows) * KB * 4;
    if (overlap(x, xb, codes, cb) || overlap(x, xb, scales, sb) || overlap(codes, cb, scales, sb))
        return bad("moe_quant_fp8: outputs overlap the input or each other");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::QuantArgs a{};
    a.x = x;
    a.codes = (uint8_t *)codes;
    a.scales = scales;
    a.ld = ld;
    a.R = s->R;
    a.K = s->K;
    a.KB = (int)KB;
    a.block_rows = s->block_rows;
    a.bf16 = s->src_dtype == MOE_BF16;
    moe::launch_quant_fp8(a, (hipStream_t)stream);
    return moe::api_launched("moe_quant_fp8");
}

int moe_matmul_fp8(const moe_matmul_t *s, const void *a, const float *sa, const void *b,
                   const float *sb, const int32_t *offsets, void *y, void *stream)
{
    if (!s)
        return bad("moe_matmul_fp8: matmul is NULL");
    if (s->M < 0 || s->N < 1 || s->K < 1 || s->G < 1)
        return bad("moe_matmul_fp8: M >= 0 and N, K, G >= 1");
    if (s->out_dtype != MOE_F32 && s->out_dtype != MOE_BF16)
        return bad("moe_matmul_fp8: out_dtype must be MOE_F32 or MOE_BF16");
    if (s->K > moe::FP8_MAX_K)
        return moe::api_fail(MOE_EUNSUPPORTED, "moe_matmul_fp8: K up to 32768");
    const int64_t KB = cdiv(s->K, moe::FP8_K), Kp = KB * moe::FP8_K;
    const int64_t lda = s->lda ? s->lda : Kp, ldb = s->ldb ? s->ldb : Kp, ldy = s->ldy ? s->ldy : s->N;
    if (lda < Kp || lda % 16 || ldb < Kp || ldb % 16)
        return bad("moe_matmul_fp8: lda and ldb must be 0, or multiples of 16 that hold K rounded up "
                   "to a multiple of 128");
    if (ldy < s->N)
        return bad("moe_matmul_fp8: ldy must be 0 or at least N");
    if (s->N * ldb >= (int64_t)1 << 32 || 256 * lda >= (int64_t)1 << 32)
        return bad("moe_matmul_fp8: a matrix b or 256 rows of a reach 2^32 bytes");
    if (s->G > 1 && !offsets)
        return bad("moe_matmul_fp8: G > 1 needs offsets");
    const moe::Fp8Tile t = moe::fp8_size(s->M, s->G, s->N, false, s->out_dtype == MOE_F32, true);
    const int64_t mtiles = moe::fp8_row_tiles(s->M, s->G, t.rows);
    if (mtiles * cdiv(s->N, 32) >= (int64_t)1 << 31 || s->G > 65535)
        return bad("moe_matmul_fp8: too many tiles or groups");
    if (s->M == 0)
        return MOE_OK;
    if (!a || !sa || !b || !sb || !y)
        return bad("moe_matmul_fp8: NULL pointer");
    const int esz = s->out_dtype == MOE_F32 ? 4 : 2;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
        !aligned(offsets, 4) || !aligned(y, esz))
        return bad("moe_matmul_fp8: a or b not 16-byte, or another pointer not element aligned");
    const int64_t yb = ((s->M - 1) * ldy + s->N) * esz;
    const int64_t bb = (s->G * (int64_t)s->N - 1) * ldb + Kp, sbb = s->G * cdiv(s->N, moe::FP8_K) * KB * 4;
    if (overlap(y, yb, a, (s->M - 1) * lda + Kp) || overlap(y, yb, sa, s->M * KB * 4) ||
        overlap(y, yb, b, bb) || overlap(y, yb, sb, sbb) ||
        (offsets && overlap(y, yb, offsets, (s->G + (int64_t)1) * 4)))
        return bad("moe_matmul_fp8: y overlaps an operand");
    if (const int rc = moe::api_check_device())
        return rc;
    moe::Fp8Args p{};
    p.a = (const uint8_t *)a;
    p.sa = sa;
    p.b0 = (const uint8_t *)b;
    p.s0 = sb;
    p.offsets = offsets;
    p.y = y;
    p.lda = lda;
    p.ldb = ldb;
    p.ldy = ldy;
    p.bstride = s->N * ldb;
    p.sstride = cdiv(s->N, moe::FP8_K) * KB;
    p.M = s->M;
    p.N = s->N;
    p.KB = (int)KB;
    p.G = s->G;
    p.mtiles = (int)mtiles;
    p.out_f32 = s->out_dtype == MOE_F32;
    // whole words, with 32-bit offsets inside a tile of up to 256 rows
    p.vec = aligned(y, 16) && ldy * esz % 16 == 0 && s->N % 16 == 0 && 256 * ldy * esz < (int64_t)1 << 31;
    moe::launch_fp8_matmul(p, t, (hipStream_t)stream);
    return moe::api_launched("moe_matmul_fp8");
}

}  // extern "C"
