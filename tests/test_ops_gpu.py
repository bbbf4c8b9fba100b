"""The routing and FP8 operators on the GPU against their 64-bit definitions
(tests/ops_ref.py), alone and together: indices and codes equal, sums within
the bounds that counting roundings gives."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import ops_ref as ref  # noqa: E402
import routed_expert_ffn_moe_amd as moe  # noqa: E402

F8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


def within(got, want, bound, what=""):
    """|got - want| <= bound everywhere (want float64 on the CPU); NaN fails."""
    d = (got.double().cpu() - want).abs()
    over = ~(d <= bound)
    say("[%s] largest error %.3g of its bound" % (what, float((d / bound.clamp(min=1e-300)).max()) if d.numel() else 0))
    assert not bool(over.any()), (what, int(over.sum()), float(d.max()))


# ---- select -----------------------------------------------------------------

def run_select(logits, bias, k, want_w=True, ld=0, E=None, **kw):
    T = logits.shape[0]
    E = logits.shape[1] if E is None else E
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    s = moe.make_select(T, E, k, logits="bf16" if logits.dtype == torch.bfloat16 else "f32", ld=ld, **kw)
    moe.moe_select(s, logits, bias, idx, w if want_w else None)
    torch.cuda.synchronize()
    assert (idx[T] == -7).all() and (w[T] == -7).all()  # nothing behind the last token
    return idx[:T].cpu(), w[:T].cpu()


# weights: the exponential's argument is off by 2^-24 of |l - max| <= 16 (2^-20 of the value), the
# exponential, sum, quotient and factor by a few 2^-24 more: 2^-19 in all, of a largest weight <= scale
W_TOL = 2.0 ** -19


def check_select(logits, bias, k, what="", **kw):
    idx, w = run_select(logits.cuda(), None if bias is None else bias.cuda(), k, **kw)
    ridx, rw = ref.select(logits, bias, k, **kw)
    assert torch.equal(idx, ridx), (what, (idx != ridx).nonzero()[:4].tolist())
    within(w, rw, torch.full_like(rw, W_TOL * kw.get("scale", 1.0)), "select " + what)


SELECT = [
    # T, E, k, score, bias, n_group, topk_group, group_score, renorm, scale, type
    (1, 1, 1, "softmax", False, 1, 1, "max", True, 1.0, "f32"),
    (3, 7, 7, "sigmoid", True, 1, 1, "max", False, 1.0, "f32"),
    (5, 16, 4, "softmax", True, 4, 2, "top2", True, 1.0, "bf16"),
    (33, 64, 8, "softmax", False, 8, 3, "max", False, 16.0, "f32"),
    (2, 65, 3, "sigmoid", True, 5, 2, "top2", True, 2.5, "f32"),
    (9, 160, 6, "softmax", False, 8, 3, "max", True, 1.0, "f32"),
    (6, 192, 16, "sigmoid", True, 64, 8, "top2", True, 1.0, "bf16"),
    (70, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, "f32"),
    (70, 256, 8, "sigmoid", True, 8, 4, "top2", True, 2.5, "bf16"),
    (130, 256, 8, "softmax", False, 1, 1, "max", True, 1.0, "bf16"),
    (130, 384, 6, "sigmoid", True, 1, 1, "max", True, 1.0, "f32"),
    (4, 400, 10, "softmax", True, 4, 1, "max", True, 1.0, "f32"),
    (4, 1000, 16, "sigmoid", False, 8, 7, "top2", True, 1.0, "bf16"),
    (17, 1024, 16, "softmax", True, 16, 16, "top2", False, 1.0, "f32"),
    (64, 8, 2, "softmax", False, 1, 1, "max", True, 1.0, "f32"),
    (4, 12, 3, "sigmoid", True, 12, 3, "top2", True, 1.0, "f32"),
]


@pytest.mark.parametrize("T,E,k,score,bias,ng,tg,gsc,renorm,scale,dt", SELECT)
def test_select(T, E, k, score, bias, ng, tg, gsc, renorm, scale, dt):
    g = gen(T * 1000 + E)
    check_select(randn(g, T, E, dtype=DT[dt]), randn(g, E) * 0.1 if bias else None, k,
                 "T%d E%d k%d" % (T, E, k), score=score, n_group=ng, topk_group=tg, group_score=gsc,
                 renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
def test_select_equal_scores_go_to_the_lower_index(score, bias):
    """Logits from four values, so most scores are equal, and equal biases."""
    g = gen(11)
    l = torch.randint(-2, 2, (40, 96), generator=g).float()
    check_select(l, torch.full((96,), 0.25) if bias else None, 8, score=score)
    check_select(l, torch.full((96,), 0.25) if bias else None, 8, score=score, n_group=6, topk_group=3,
                 group_score="top2")


@pytest.mark.parametrize("ng", [1, 8])
def test_select_orders_keys_that_fp32_cannot_tell_apart(ng):
    """Keys whose neighbours differ by 1e-9 to 1e-8 relative: all within one
    fp32 rounding, distinct in 64 bits."""
    g = gen(5)
    T, E = 24, 128
    base = torch.linspace(-1, 1, E).double()
    s = 1 / (1 + torch.exp(-base))
    bias = (0.75 - s).float()  # s + bias = 0.75 up to the bias's own rounding (3e-8)
    perm = torch.randperm(E, generator=g)
    l = base.float()[perm].repeat(T, 1)
    l += torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -24
    check_select(l, bias[perm], 8, score="sigmoid", n_group=ng, topk_group=3 if ng > 1 else 1,
                 group_score="top2")
    check_select(l, bias[perm], 8, score="softmax", n_group=ng, topk_group=3 if ng > 1 else 1)


@pytest.mark.parametrize("ng", [1, 8])
def test_select_orders_softmax_keys_that_fp32_cannot_tell_apart(ng):
    """As above with softmax scores: bias = 0.05 - p of the row without its noise."""
    g = gen(6)
    T, E = 24, 128
    base = torch.linspace(-1, 1, E).float()[torch.randperm(E, generator=g)]
    p = torch.softmax(base.double(), 0)
    l = base.repeat(T, 1) + torch.randint(-2, 3, (T, E), generator=g) * 2.0 ** -24
    check_select(l, (0.05 - p).float(), 8, score="softmax", n_group=ng, topk_group=3 if ng > 1 else 1,
                 group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("ng", [1, 4])
def test_select_masked_experts(score, ng):
    """-inf and NaN logits and biases: some, all but a few, all of a group, all of a row."""
    g = gen(3)
    T, E, k = 12, 64, 6
    l, b = randn(g, T, E), randn(g, E) * 0.1
    l[0, ::2] = -math.inf
    l[1, 3:] = -math.inf
    l[2, :] = -math.inf
    l[3, 5] = math.nan
    l[4, :] = math.nan
    l[5, 16:32] = -math.inf
    l[6, 1:] = -math.inf
    l[7, 10] = math.inf
    l[8, 10] = l[8, 40] = math.inf
    l[9, :] = torch.finfo(torch.float32).min
    l[10, 20:] = torch.finfo(torch.float32).min
    b[7], b[8], b[9] = -math.inf, math.nan, 1e30
    kw = dict(score=score, n_group=ng, topk_group=2 if ng > 1 else 1, group_score="top2")
    check_select(l, None, k, **kw)
    check_select(l, b, k, **kw)
    check_select(l, b, k, renorm=False, **kw)


def test_select_wide_range_of_logits():
    g = gen(8)
    for sigma in (1e-6, 30.0, 1e4):
        l = randn(g, 20, 256) * sigma
        check_select(l, None, 8, score="sigmoid")
        check_select(l, randn(g, 256) * 0.01, 8, score="sigmoid")
        check_select(l, None, 8, score="softmax", n_group=8, topk_group=4, group_score="top2")


def test_select_strided_logits_and_no_weights():
    g = gen(4)
    whole = randn(g, 20, 300, dtype=torch.bfloat16)
    part = whole[:, 7:167]
    ridx, _ = ref.select(part, None, 4, score="sigmoid")
    dev = whole.cuda()
    idx, w = run_select(dev[:, 7:167], None, 4, want_w=False, ld=300, score="sigmoid")
    assert torch.equal(idx, ridx) and (w == -7).all()


# ---- quant ------------------------------------------------------------------

def run_quant(x, K, rows, ld=0):
    R = x.shape[0]
    Kp = ref.padded(K)
    n_s = -(-R // rows) * (Kp // 128)
    codes = torch.full((R + 1, Kp), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((n_s + 4,), -7.0, device="cuda")
    q = moe.make_quant(R, K, "bf16" if x.dtype == torch.bfloat16 else "f32", rows, ld)
    moe.moe_quant_fp8(q, x, codes, scales)
    torch.cuda.synchronize()
    assert (codes[R] == 0x55).all() and (scales[n_s:] == -7).all()
    return codes[:R].view(F8), scales[:n_s].view(-1, Kp // 128)


def check_quant(x, rows, what=""):
    codes, scales = run_quant(x.cuda(), x.shape[1], rows)
    rq, rs, v = ref.quant(x, rows)
    within(scales, rs, rs * 2 * ref.U32, "scales " + what)
    got = codes.cpu().double()
    if x.dtype == torch.bfloat16:
        # quotients of bf16 values are midpoints or at least 2^-13 away from them
        assert torch.equal(got, rq), what
    else:
        # two roundings of the quotient may cross a midpoint that is as near
        _, step, off = ref.e4m3_grid(v)
        near = off <= 4 * ref.U32 * v.abs()
        assert bool(((got == rq) | (near & ((got - rq).abs() <= step))).all()), what
    assert not got[:, x.shape[1]:].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 128), (3, 130), (5, 776), (130, 200), (257, 384), (64, 2048)])
def test_quant(R, K, rows, dt):
    g = gen(R + K)
    x = randn(g, R, K) * torch.exp(2 * randn(g, 1, K))
    check_quant(x.to(DT[dt]), rows, "%dx%d" % (R, K))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 128])
def test_quant_extreme_blocks(rows, dt):
    """Zero blocks, values below the smallest maximum, subnormals, the largest values."""
    g = gen(2)
    x = randn(g, 6, 1024)
    x[:, :128] = 0
    x[:, 128:256] *= 2.0 ** -110
    x[:, 256:384] *= 2.0 ** -132
    x[:, 384:512] *= 2.0 ** 100
    x[:, 512:640] *= 2.0 ** 124
    x[:, 640] = 3e38
    x[:, 768:896] *= 2.0 ** -9
    x[:, 800] = 448.0
    check_quant(x.to(DT[dt]), rows)


@pytest.mark.parametrize("rows", [1, 128])
def test_quant_nan_and_infinity(rows):
    x = randn(gen(6), 2, 384)
    x[0, 5] = math.nan
    x[0, 130] = math.inf
    codes, scales = run_quant(x.cuda(), 384, rows)
    c = codes.float().cpu()
    clean = x.clone()
    clean[0, 5] = 0
    rq, rs, _ = ref.quant(clean, rows)
    assert math.isnan(c[0, 5]) and not c[0, :5].isnan().any() and not c[0, 6:128].isnan().any()
    assert torch.equal(c[0, 6:128].double(), rq[0, 6:128])
    assert math.isinf(scales[0, 1])
    assert (c[0:rows, 128:256].isnan()).all()
    assert torch.equal(c[:, 256:].double(), rq[:, 256:])


def test_quant_strided_rows_and_helper():
    g = gen(9)
    for dt in (torch.bfloat16, torch.float32):
        whole = randn(g, 40, 301, dtype=dt)
        for lo, K in ((0, 256), (3, 251), (8, 128)):
            rq, rs, _ = ref.quant(whole[:, lo:lo + K])
            dev = whole.cuda()
            codes, _ = run_quant(dev[:, lo:lo + K], K, 1, ld=301)
            if dt == torch.bfloat16:
                assert torch.equal(codes.cpu().double(), rq)
            c2, s2 = moe.quant_fp8(dev[:, lo:lo + K])
            assert torch.equal(c2.view(torch.uint8), codes.view(torch.uint8))
    w = randn(g, 3, 256, 200, dtype=torch.bfloat16)
    codes, scales = moe.quant_fp8(w.cuda(), block_rows=128)
    assert codes.shape == (3, 256, 256) and scales.shape == (3, 2, 2)
    for e in range(3):
        rq, rs, _ = ref.quant(w[e], 128)
        assert torch.equal(codes[e].cpu().double(), rq)


def test_quant_helper_copies_on_the_stream_it_runs_on():
    """x transposed, so that the helper copies it first, on a stream that has
    work before it."""
    g = gen(10)
    x = randn(g, 4096, 2048, dtype=torch.bfloat16).cuda()
    want = moe.quant_fp8(x.t().contiguous())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for s in (st, st.cuda_stream):
        junk = torch.empty(2048, 4096, dtype=torch.bfloat16, device="cuda").fill_(math.nan)
        del junk  # its block would be taken for a copy made on the current stream
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            for _ in range(20):
                x.add_(0)
        got = moe.quant_fp8(x.t(), stream=s)
        st.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---- matmul -----------------------------------------------------------------

def codes_of(g, *shape):
    return (randn(g, *shape) * 120).clamp(-448, 448).to(F8)


def operands(g, M, N, K, G=1):
    Kp = ref.padded(K)
    a, b = codes_of(g, M, Kp), codes_of(g, G, N, Kp)
    a.view(torch.uint8)[:, K:] = 0
    b.view(torch.uint8)[:, :, K:] = 0
    sa = torch.rand(M, Kp // 128, generator=g) + 0.1
    sb = torch.rand(G, -(-N // 128), Kp // 128, generator=g) * 0.01 + 1e-4
    return a, sa, b, sb


def check_matmul(M, N, K, out, ldy=None, off=None, G=1, what=""):
    g = gen(M * 7 + N * 3 + K + G)
    a, sa, b, sb = operands(g, M, N, K, G)
    ld = N if ldy is None else ldy
    y = torch.full((M + 1, ld), -7.0, dtype=DT[out], device="cuda")
    mm = moe.make_matmul(M, N, K, G=G, out=out, ldy=0 if ldy is None else ldy)
    moe.moe_matmul_fp8(mm, a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), y,
                       None if off is None else torch.tensor(off, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    av = ref.rows_value(a, sa)
    got, done = y.cpu(), torch.zeros(M + 1, dtype=torch.bool)
    for i in range(G):
        lo, hi = (0, M) if off is None else (min(max(off[i], 0), M), min(off[i + 1], M))
        if hi <= lo:
            continue
        want, tol = ref.product(av[lo:hi], ref.matrix_value(b[i], sb[i]), narrow=out == "bf16")
        if out == "bf16":
            tol = tol + ref.UBF * (want.abs() + tol)
        within(got[lo:hi, :N], want, tol + 1e-30, "matmul %dx%dx%d group %d %s" % (M, N, K, i, what))
        done[lo:hi] = True
    assert (got[~done] == -7).all() and (got[:, N:] == -7).all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 16, 128), (1, 4096, 2048), (2, 130, 200), (7, 48, 384),
                                   (15, 257, 776), (16, 256, 256), (17, 100, 512), (33, 96, 128),
                                   (64, 512, 896), (65, 300, 640), (129, 770, 1024), (300, 129, 2048),
                                   (1, 33, 8192), (700, 260, 300)])
def test_matmul(M, N, K, out):
    check_matmul(M, N, K, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,ldy", [(3, 263), (40, 272), (150, 264)])
def test_matmul_strided_rows_of_y(M, ldy, out):
    check_matmul(M, 260, 384, out, ldy=ldy)


@pytest.mark.parametrize("M", [1, 20, 140])
def test_matmul_strided_operands(M):
    g = gen(M)
    N, K = 96, 256
    a, sa, b, sb = operands(g, M, N, K)
    wa, wb = codes_of(g, M, 432).cuda(), codes_of(g, N, 304).cuda()
    wa.view(torch.uint8)[:, 16:16 + K] = a.cuda().view(torch.uint8)
    wb.view(torch.uint8)[:, :K] = b[0].cuda().view(torch.uint8)
    y = torch.empty(M, N, device="cuda")
    moe.moe_matmul_fp8(moe.make_matmul(M, N, K, out="f32", lda=432, ldb=304), wa[:, 16:16 + K], sa.cuda(),
                       wb, sb.cuda(), y)
    want, tol = ref.product(ref.rows_value(a, sa), ref.matrix_value(b[0], sb[0]))
    within(y, want, tol, "strided operands")


GROUPS = {
    "even": (96, [0, 32, 64, 96]),
    "empty and one": (90, [0, 0, 1, 90, 90]),
    "rows before and behind": (100, [10, 40, 40, 77]),
    "one group": (50, [5, 45]),
    "none": (20, [0, 0, 0]),
    "past the end": (40, [0, 30, 60, 80]),
    "before the start": (40, [-5, 10, 20]),
    "tile edges": (400, [0, 16, 48, 112, 240, 241, 400]),
}


@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_matmul_groups(name, out):
    M, off = GROUPS[name]
    check_matmul(M, 200, 256, out, off=off, G=len(off) - 1, what=name)


@pytest.mark.parametrize("M,G", [(300, 65), (2000, 130), (5000, 1000), (70, 300)])
def test_matmul_many_groups(M, G):
    g = gen(G)
    cuts = torch.randint(0, M + 1, (G - 1,), generator=g).sort().values.tolist()
    check_matmul(M, 128, 128, "bf16", off=[0] + cuts + [M], G=G)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(1000, 4200, 260), (2000, 4200, 1100), (4000, 4100, 130), (4000, 4100, 900)])
def test_matmul_more_tiles_than_workgroups(M, N, K, out):
    """One matrix of more tiles than CUs: a workgroup takes several, the copies of
    the next begin while the last steps of one still run (or, in few steps of K,
    after them)."""
    check_matmul(M, N, K, out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("K", [100, 384, 640, 1152])
@pytest.mark.parametrize("per", [10, 20, 45, 70, 100, 150, 220])
def test_matmul_groups_of_every_tile_height(per, K, out):
    """Uneven groups of `per` rows on average, over 300 tiles in all: tiles of
    16, 32, 64, 96, 144, 128 and 256 rows, one to nine steps of K."""
    G, N = 9, 8008
    g = gen(per + K)
    cuts = (torch.arange(1, G) * per + torch.randint(-(per // 2), per // 2, (G - 1,), generator=g)).tolist()
    check_matmul(G * per, N, K, out, off=[0] + cuts + [G * per], G=G, what="%d rows a group" % per)


@pytest.mark.parametrize("M", [4, 40, 200])
def test_matmul_nan_stays_in_its_row_and_column(M):
    g = gen(1)
    a, sa, b, sb = operands(g, M, 160, 384)
    a.view(torch.uint8)[2, 200] = 0x7F
    sb[0, 1, 0] = math.inf
    b.view(torch.uint8)[0, 40, 300] = 0xFF
    y = torch.empty(M, 160, device="cuda")
    moe.moe_matmul_fp8(moe.make_matmul(M, 160, 384, out="f32"), a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), y)
    bad = ~torch.isfinite(y).cpu()
    want = torch.zeros(M, 160, dtype=torch.bool)
    want[2], want[:, 40], want[:, 128:] = True, True, True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M", [3, 20, 40])
def test_matmul_infinite_scale_of_a_row(M, out):
    """The last block's scale of a row infinite: y there is infinite with the
    sign of that block's sum, in whatever way K is divided."""
    g = gen(M)
    a, sa, b, sb = operands(g, M, 96, 384)
    sa[1, 2] = math.inf
    y = torch.empty(M, 96, dtype=DT[out], device="cuda")
    moe.moe_matmul_fp8(moe.make_matmul(M, 96, 384, out=out), a.cuda(), sa.cuda(), b.cuda(), sb.cuda(), y)
    t = a[1, 256:].double() @ b[0, :, 256:].double().t()
    # sums far from what the FP8 instruction may lose of them (2^-10 of the products)
    sure = t.abs() > 2.0 ** -9 * (a[1, 256:].double().abs() @ b[0, :, 256:].double().abs().t())
    got = y[1].cpu().double()
    assert int(sure.sum()) > 60 and torch.equal(got[sure], torch.sign(t[sure]) * math.inf)
    assert torch.isfinite(y[0]).all() and torch.isfinite(y[2:]).all()


# ---- experts ----------------------------------------------------------------

class Experts:
    def __init__(self, E, H, I, seed=0):
        g = gen(seed)
        self.E, self.H, self.I = E, H, I
        self.mats = {}
        for n, r, c in (("gate", I, H), ("up", I, H), ("down", H, I)):
            self.mats["w_" + n] = codes_of(g, E, r, c)
            self.mats["s_" + n] = (torch.rand(E, r // 128, c // 128, generator=g) + 0.5) / (120 * math.sqrt(c))
        self.dev = {n: t.cuda() for n, t in self.mats.items()}
        self.router = randn(g, E, H, dtype=torch.bfloat16)
        self.router_dev = (self.router / math.sqrt(H)).to(torch.bfloat16).cuda()
        self.weights = moe.make_weights(self.router_dev, **{n: self.dev[n] for n in self.dev})

    def shape(self, T, k, chunk_T=0):
        return moe.make_shape(T, self.H, self.E, k, self.I, chunk_T=chunk_T, act="bf16", w="fp8")

    def run(self, x, idx, w, chunk_T=0, stream=None, ws=None, y=None):
        T, k = idx.shape
        sh = self.shape(T, k, chunk_T)
        n = moe.moe_workspace_bytes(sh)
        if ws is None:
            ws = torch.full((max(n, 1),), 0xFF, dtype=torch.uint8, device="cuda")
        if y is None:
            y = torch.full((T, self.H), math.nan, dtype=torch.bfloat16, device="cuda")
        moe.moe_experts(sh, self.weights, x, idx, w, y, ws, n, stream=stream)
        return y

    def ref(self, x, idx, w):
        m = self.mats
        return ref.experts(x, m["w_gate"], m["s_gate"], m["w_up"], m["s_up"], m["w_down"], m["s_down"], idx, w)


def routing(g, T, E, k, skew=0.0):
    lean = -skew * torch.log(1.0 + torch.arange(E))
    z = lean - torch.log(-torch.log(torch.rand(T, E, generator=g).clamp(1e-9, 1 - 1e-7)))
    w, idx = z.topk(k, 1)
    return idx.to(torch.int32), torch.softmax(w, 1)


EXPERTS = [(1, 4, 2, 256, 128), (1, 64, 8, 512, 384), (6, 16, 4, 384, 256), (9, 8, 8, 256, 128),
           (17, 8, 2, 128, 256), (130, 8, 2, 640, 128), (64, 3, 1, 256, 384), (200, 2, 2, 256, 256),
           (400, 1, 1, 256, 128), (70, 64, 6, 256, 128), (1100, 5, 3, 128, 128)]


@pytest.mark.parametrize("T,E,k,H,I", EXPERTS)
def test_experts(T, E, k, H, I):
    g = gen(T + E)
    L = Experts(E, H, I, T)
    x = randn(g, T, H, dtype=torch.bfloat16)
    idx, w = routing(g, T, E, k, 1.1 if T > 64 else 0.0)
    y = L.run(x.cuda(), idx.cuda(), w.cuda())
    want, tol = L.ref(x, idx, w)
    within(y, want, tol + 1e-30, "experts T%d E%d k%d" % (T, E, k))
    say("bound over y: %.3g" % float(tol.norm() / want.norm()))


@pytest.mark.parametrize("T,E,k,H,I", [(1, 64, 8, 512, 1024), (1, 16, 2, 128, 128), (3, 20, 16, 384, 256),
                                       (8, 32, 12, 2176, 128), (8, 8, 8, 640, 640), (2, 16, 3, 4096, 256),
                                       (1, 4, 4, 256, 16384)])
def test_experts_decode_rows_have_the_bits_of_long_passes(T, E, k, H, I):
    """Few rows in the kernels of their own, and as the first rows of a longer pass."""
    g = gen(T + k)
    L = Experts(E, H, I, T)
    x = randn(g, 20, H, dtype=torch.bfloat16)
    idx, w = routing(g, 20, E, k)
    y = L.run(x[:T].contiguous().cuda(), idx[:T].contiguous().cuda(), w[:T].contiguous().cuda())
    want, tol = L.ref(x[:T], idx[:T], w[:T])
    within(y, want, tol + 1e-30, "decode rows T%d k%d H%d I%d" % (T, k, H, I))
    assert torch.equal(y, L.run(x.cuda(), idx.cuda(), w.cuda())[:T])


@pytest.mark.parametrize("per", [10, 20, 45, 70, 100, 150, 220])
def test_experts_of_every_tile_height(per):
    """Every tile height, in more tiles than there are CUs."""
    E, H, I = 20, 768, 2048
    g = gen(per)
    L = Experts(E, H, I, per)
    x = randn(g, E * per, H, dtype=torch.bfloat16)
    idx, w = routing(g, E * per, E, 1, 0.2)
    y = L.run(x.cuda(), idx.cuda(), w.cuda())
    want, tol = L.ref(x, idx, w)
    within(y, want, tol + 1e-30, "%d rows an expert" % per)


@pytest.mark.parametrize("T", [1, 5, 40, 300])
def test_experts_empty_slots_and_repeated_experts(T):
    g = gen(T)
    L = Experts(6, 256, 128, 1)
    x = randn(g, T, 256, dtype=torch.bfloat16)
    idx, w = routing(g, T, 6, 3)
    idx[::2, 1] = -1
    idx[1::5, 0] = 6          # outside: empty too
    idx[2::7, 2] = 1 << 30
    idx[3::4, 1] = idx[3::4, 2]  # the same expert twice
    idx[0] = -1               # a token with empty slots only
    w[idx < 0] = math.nan     # an empty slot's weight does not matter
    y = L.run(x.cuda(), idx.cuda(), w.cuda())
    live = (idx >= 0) & (idx < 6)
    want, tol = L.ref(x, torch.where(live, idx, torch.full_like(idx, -1)),
                      torch.where(live, w, torch.zeros_like(w)))
    assert (y[0] == 0).all()
    within(y, want, tol + 1e-30, "experts with empty slots T%d" % T)


@pytest.mark.parametrize("T", [1, 12, 200])
def test_experts_nothing_routed(T):
    L = Experts(4, 256, 128)
    x = randn(gen(0), T, 256, dtype=torch.bfloat16).cuda()
    idx = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
    assert (L.run(x, idx, torch.ones(T, 2, device="cuda")) == 0).all()


def test_experts_chunks_and_repeats_give_the_same_bits():
    g = gen(21)
    L = Experts(16, 512, 256, 3)
    x = randn(g, 150, 512, dtype=torch.bfloat16).cuda()
    idx, w = (t.cuda() for t in routing(g, 150, 16, 4, 1.1))
    y = L.run(x, idx, w)
    assert torch.equal(y, L.run(x, idx, w))
    for c in (1, 7, 64, 149, 150):
        assert torch.equal(y, L.run(x, idx, w, chunk_T=c)), c


@pytest.mark.parametrize("T", [1, 8, 9, 130, 600])
def test_forward_with_fp8_experts_matches_its_parts(T):
    """moe_forward (and its allocation-free form) against moe_logits, moe_select
    and moe_experts: the same routing, and y the same bit for bit."""
    g = gen(T)
    L = Experts(16, 512, 256, 5)
    x = randn(g, T, 512, dtype=torch.bfloat16).cuda()
    sh = L.shape(T, 4)
    ws = torch.full((moe.moe_workspace_bytes(sh),), 0xFF, dtype=torch.uint8, device="cuda")
    out = []
    for noalloc in (False, True):
        y = torch.full((T, 512), math.nan, dtype=torch.bfloat16, device="cuda")
        idx = torch.full((T, 4), -1, dtype=torch.int32, device="cuda")
        w = torch.full((T, 4), math.nan, device="cuda")
        if noalloc:
            moe.moe_forward_noalloc(sh, L.weights, x, y, idx, w)
        else:
            moe.moe_forward(sh, L.weights, x, y, idx, w, ws)
        out.append((y, idx, w))
    y, idx, w = out[0]
    assert all(torch.equal(a, b) for a, b in zip(*out))
    assert torch.equal(y, L.run(x, idx, w))
    want, tol = L.ref(x.cpu(), idx.cpu(), w.cpu())
    within(y, want, tol, "forward fp8 T%d" % T)


@pytest.mark.parametrize("score,ng,tg", [("sigmoid", 4, 2), ("softmax", 1, 1)])
@pytest.mark.parametrize("T", [1, 7, 150])
def test_logits_select_experts_together(T, score, ng, tg):
    """The layer in its three calls, each checked on what the one before it gave."""
    g = gen(T)
    L = Experts(32, 512, 256, 7)
    x = randn(g, T, 512, dtype=torch.bfloat16).cuda()
    bias = (randn(g, 32) * 0.05).cuda()
    sh = L.shape(T, 4)
    logits = torch.full((T, 32), math.nan, device="cuda")
    moe.moe_logits(sh, L.weights, x, logits)
    want = x.cpu().double() @ L.router_dev.cpu().double().t()
    # K products of bf16 values (exact in fp32) and as many additions
    mag = x.cpu().double().abs() @ L.router_dev.cpu().double().abs().t()
    within(logits, want, 2 * 512 * ref.U32 * mag, "logits")
    idx, w = run_select(logits, bias, 4, score=score, n_group=ng, topk_group=tg, group_score="top2", scale=2.5)
    ridx, rw = ref.select(logits, bias, 4, score=score, n_group=ng, topk_group=tg, group_score="top2", scale=2.5)
    assert torch.equal(idx, ridx)
    y = L.run(x, idx.cuda(), w.cuda())
    want, tol = L.ref(x.cpu(), idx, w)
    within(y, want, tol, "layer in three calls")


@pytest.mark.parametrize("wt,T", [("bf16", 1), ("bf16", 70), ("bf16", 600), ("mxfp4", 4), ("mxfp4", 60),
                                  ("mxfp4", 600), ("f32", 20)])
def test_experts_of_the_other_weight_types(wt, T):
    """Given the routing that moe_forward chose, moe_experts gives its y; with
    slots emptied, what the remaining slots give."""
    import moe_inputs as mi
    import harness as hx
    H, I, E, k = 512, 512, 16, 4
    c = dict(mi.cfg({"bf16": "c1", "mxfp4": "c4_t6", "f32": "c0"}[wt]), T=T, H=H, E=E, top_k=k, I=I)
    lay = mi.make_layer(c, "cuda")
    G = hx.GpuLayer(c, lay)
    x = hx.act_torch(hx.mi.make_x(c), c["act"], "cuda")
    y, idx, w = G.forward(x)
    sh = G.shape(T)
    ws = torch.full((moe.moe_workspace_bytes(sh),), 0xFF, dtype=torch.uint8, device="cuda")
    y2 = torch.full_like(y, math.nan)
    moe.moe_experts(sh, G.weights, x, idx, w, y2, ws)
    if wt == "mxfp4" and T <= 8:  # decode rows take other kernels; both are held to this bar against the oracle
        assert float((y.double() - y2.double()).abs().max() / y.double().abs().max()) <= 2 * hx.TIGHT[wt]
    else:
        assert torch.equal(y, y2)
    # half of the slots emptied: as if their weights were 0
    idx3 = idx.clone()
    idx3[:, 1::2] = -1
    w0 = w.clone()
    w0[:, 1::2] = 0
    y3, y4 = torch.full_like(y, math.nan), torch.full_like(y, math.nan)
    moe.moe_experts(sh, G.weights, x, idx3, w, y3, ws)
    moe.moe_experts(sh, G.weights, x, idx, w0, y4, ws)
    assert torch.equal(y3, y4)


# ---- streams, graphs ----------------------------------------------------------

def test_operators_on_another_stream():
    g = gen(31)
    L = Experts(8, 256, 128, 2)
    x = randn(g, 50, 256, dtype=torch.bfloat16).cuda()
    logits = randn(g, 50, 8).cuda()
    idx0, w0 = run_select(logits, None, 2)
    y0 = L.run(x, idx0.cuda(), w0.cuda())
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    idx = torch.empty(50, 2, dtype=torch.int32, device="cuda")
    w = torch.empty(50, 2, device="cuda")
    n = moe.moe_workspace_bytes(L.shape(50, 2))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    y = torch.empty(50, 256, dtype=torch.bfloat16, device="cuda")
    moe.moe_select(moe.make_select(50, 8, 2), logits, None, idx, w, stream=st)
    L.run(x, idx, w, stream=st, ws=ws, y=y)
    st.synchronize()
    assert torch.equal(idx.cpu(), idx0) and torch.equal(y, y0)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_layer_in_a_graph_replayed(T):
    """logits, select, experts and a product in one captured graph, replayed on
    new inputs with eager calls between the replays."""
    g = gen(17)
    L = Experts(16, 256, 128, 4)
    sh = L.shape(T, 4)
    n = moe.moe_workspace_bytes(sh)
    x = torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
    bias = (randn(g, 16) * 0.05).cuda()
    sel = moe.make_select(T, 16, 4, score="sigmoid", n_group=4, topk_group=2, group_score="top2")
    mm = moe.make_matmul(T, 256, 256, out="bf16")
    qn = moe.make_quant(T, 256)
    _, _, b, sb = operands(g, 1, 256, 256)
    b, sb = b.cuda(), sb.cuda()

    def bufs():
        return dict(logits=torch.empty(T, 16, device="cuda"), w=torch.empty(T, 4, device="cuda"),
                    idx=torch.empty(T, 4, dtype=torch.int32, device="cuda"),
                    y=torch.empty(T, 256, dtype=torch.bfloat16, device="cuda"),
                    c=torch.empty(T, 256, dtype=F8, device="cuda"), s=torch.empty(T, 2, device="cuda"),
                    z=torch.empty(T, 256, dtype=torch.bfloat16, device="cuda"),
                    ws=torch.empty(n, dtype=torch.uint8, device="cuda"))

    def step(o):
        moe.moe_logits(sh, L.weights, x, o["logits"])
        moe.moe_select(sel, o["logits"], bias, o["idx"], o["w"])
        moe.moe_experts(sh, L.weights, x, o["idx"], o["w"], o["y"], o["ws"])
        moe.moe_quant_fp8(qn, o["y"], o["c"], o["s"])
        moe.moe_matmul_fp8(mm, o["c"], o["s"], b, sb, o["z"])

    eager, held = bufs(), bufs()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step(held)
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step(held)
    for i in range(5):
        x.copy_(randn(g, T, 256, dtype=torch.bfloat16))
        step(eager)
        torch.cuda.synchronize()
        for t in ("y", "z", "idx"):
            held[t].fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        for t in ("idx", "w", "y", "c", "s", "z"):
            assert torch.equal(held[t].view(torch.uint8), eager[t].view(torch.uint8)), (i, t)
