"""The training operators on the GPU against their 64-bit definitions
(tests/train_ref.py), alone and together.  Sums of small whole numbers are exact
in fp32 whatever their order, so the products are checked for equality; other
bounds count roundings and are derived where they stand."""
import math
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import ops_ref  # noqa: E402
import routed_expert_ffn_moe_amd as moe  # noqa: E402
import train_ref as ref  # noqa: E402

F8 = torch.float8_e4m3fn
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U32 = ref.U32
TINY = 2.0 ** -120  # results this small may be flushed


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g).to(dtype)


def ints(g, *shape, top=8, dtype=torch.float32):
    return torch.randint(-top, top + 1, shape, generator=g).to(dtype)


def within(got, want, bound, what=""):
    """|got - want| <= bound everywhere (want float64 on the CPU); NaN fails."""
    d = (got.double().cpu() - want).abs()
    over = ~(d <= bound)
    print("[%s] largest error %.3g of its bound" %
          (what, float((d / bound.clamp(min=1e-300)).max()) if d.numel() else 0), file=sys.stderr, flush=True)
    assert not bool(over.any()), (what, int(over.sum()), float(d.max()))


def strided(t, ld, fill=0.0):
    """A copy of a matrix whose rows lie ld elements apart, the rest filled."""
    wide = torch.full((t.shape[0], ld), fill, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]], wide


def routing(g, T, E, k, empty=0.0):
    idx = torch.rand(T, E, generator=g).topk(min(k, E), dim=1).indices.to(torch.int32)
    if k > E:
        idx = torch.cat([idx] * -(-k // E), 1)[:, :k].contiguous()
    return torch.where(torch.rand(T, k, generator=g) < empty, -1, idx).contiguous()


# ---- dispatch -------------------------------------------------------------------

def run_dispatch(idx, x, E, H, kind="bf16", sx=None, out=None, ldx=0, ldr=0, src=True, stream=None):
    T, k = idx.shape
    d = moe.make_dispatch(T, H, E, k, x=kind, rows=out, ldx=ldx, ldr=ldr)
    dt = DT[out or ("bf16" if kind == "fp8" else kind)]
    wide = torch.full((T * k + 1, ldr or H), -77.0, dtype=dt, device="cuda")
    rows = wide[:T * k, :H]
    offsets = torch.full((E + 2,), -5, dtype=torch.int32, device="cuda")
    row_src = torch.full((T * k + 1,), -5, dtype=torch.int32, device="cuda")
    row_of = torch.full((T + 1, k), -5, dtype=torch.int32, device="cuda")
    need = moe.moe_dispatch_workspace_bytes(d)
    ws = torch.full((need + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    moe.moe_dispatch(d, idx.cuda(), x, sx, rows if x is not None else None, offsets[:E + 1],
                     row_src[:T * k] if src else None, row_of[:T], ws, ws_bytes=need, stream=stream)
    torch.cuda.synchronize()
    assert (ws[need:] == 0xA5).all() and int(offsets[E + 1]) == -5 and int(row_src[T * k]) == -5
    assert (row_of[T] == -5).all() and (wide[T * k] == -77).all() and (wide[:, H:] == -77).all()
    return rows, offsets[:E + 1].cpu(), row_src[:T * k].cpu(), row_of[:T].cpu()


def check_dispatch(idx, x, E, kind="bf16", sx=None, values=None, out=None, ldx=0, ldr=0):
    """values: the rows' exact bits where x is codes."""
    T, k = idx.shape
    H = (x if values is None else values).shape[1]
    rows, offsets, src, of = run_dispatch(idx, x, E, H, kind, sx, out, ldx, ldr)
    woff, wsrc, wof = ref.sort(idx, E)
    n = int(woff[-1])
    assert torch.equal(offsets, woff) and torch.equal(of, wof)
    assert torch.equal(src[:n], wsrc) and (src[n:] == -5).all()
    want = (x if values is None else values).cpu()[(wsrc // k).long()]
    bits = torch.int16 if want.dtype == torch.bfloat16 else torch.int32
    assert torch.equal(rows[:n].cpu().contiguous().view(bits), want.contiguous().view(bits))
    assert (rows[n:] == -77).all()
    return offsets, of


DISPATCH = [(1, 1, 1, 1), (1, 256, 8, 2048), (2, 4, 2, 7), (5, 3, 3, 100), (6, 256, 8, 2048), (16, 1024, 8, 264),
            (8, 16, 16, 65), (9, 16, 16, 64), (43, 7, 3, 130), (300, 5, 3, 72), (333, 64, 16, 40),
            (600, 1024, 8, 17), (1000, 384, 6, 256), (2048, 256, 8, 33), (3000, 8, 7, 24), (2731, 1000, 6, 10),
            (20000, 384, 6, 8), (16400, 1, 1, 8), (70000, 130, 4, 8)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,H", DISPATCH)
def test_dispatch(T, E, k, H, kind):
    g = gen(T + E)
    check_dispatch(routing(g, T, E, k, 0.1 if T % 2 else 0.0), randn(g, T, H, dtype=DT[kind]).cuda(), E, kind)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,H", [(1, 8, 2, 128), (3, 16, 4, 200), (40, 16, 4, 1000), (500, 64, 8, 130), (9, 4, 1, 5)])
def test_dispatch_from_codes(T, E, k, H, out):
    g = gen(H)
    x = randn(g, T, H).cuda()
    codes, scales = moe.quant_fp8(x)
    values = (codes.float() * scales.repeat_interleave(128, 1))[:, :H].to(DT[out])  # fp32 product, one rounding
    check_dispatch(routing(g, T, E, k, 0.2), codes, E, "fp8", scales, values, out)
    wide = torch.zeros(T, codes.shape[1] + 48, dtype=F8, device="cuda")
    wide[:, :codes.shape[1]] = codes
    check_dispatch(routing(g, T, E, k, 0.2), wide[:, :codes.shape[1]], E, "fp8", scales, values, out,
                   ldx=codes.shape[1] + 48, ldr=H + 3)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 200])
@pytest.mark.parametrize("pad", [1, 8, 13])
def test_dispatch_strided_rows(T, pad, kind):
    g = gen(pad)
    H = 96 + pad % 2
    x, _ = strided(randn(g, T, H, dtype=DT[kind]), H + pad, math.nan)
    check_dispatch(routing(g, T, 9, 3, 0.1), x, 9, kind, ldx=H + pad, ldr=H + 2 * pad)


def test_dispatch_keeps_every_bit_of_x():
    x = torch.tensor([math.nan, math.inf, -math.inf, -0.0, 1e-40, 3e38, -1.0, 0.0] * 3)[None].repeat(4, 1)
    bits = torch.arange(4 * 24, dtype=torch.int16).view(4, 24) + 0x7F80  # every payload, signalling ones too
    check_dispatch(routing(gen(1), 4, 5, 2), x.cuda(), 5, "f32")
    check_dispatch(routing(gen(1), 4, 5, 2), bits.view(torch.bfloat16).cuda(), 5, "bf16")


@pytest.mark.parametrize("T", [1, 100, 5000])
def test_dispatch_empty_slots_only_and_one_expert(T):
    x = randn(gen(2), T, 32, dtype=torch.bfloat16).cuda()
    empty = torch.tensor([-1, 8, 1 << 30, -(1 << 31)], dtype=torch.int32).repeat(T, 1)
    offsets, of = check_dispatch(empty, x, 8)
    assert (offsets == 0).all() and (of == -1).all()
    check_dispatch(torch.full((T, 4), 7, dtype=torch.int32), x, 8)  # the same expert in every slot


def test_dispatch_no_tokens_and_order_alone():
    rows, offsets, _, _ = run_dispatch(torch.zeros(0, 2, dtype=torch.int32), torch.zeros(0, 8, device="cuda"), 5, 8, "f32")
    assert (offsets == 0).all()
    for T in (4, 300, 9000):
        idx = routing(gen(T), T, 12, 3, 0.1)
        _, offsets, src, of = run_dispatch(idx, None, 12, 8, src=False)
        woff, _, wof = ref.sort(idx, 12)
        assert torch.equal(offsets, woff) and torch.equal(of, wof) and (src == -5).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(1, 5), (7, 264), (600, 33)])
def test_gather(T, H, kind):
    g = gen(T)
    k, n = 3, 3 * T
    place = torch.randperm(n, generator=g).to(torch.int32).view(T, k)
    place[torch.rand(T, k, generator=g) < 0.3] = -1
    place[0, 0] = n  # not a row
    x = randn(g, T, H, dtype=DT[kind]).cuda()
    rows = torch.full((n + 1, H), -77.0, dtype=DT[kind], device="cuda")
    moe.moe_gather(moe.make_dispatch(T, H, 1, k, x=kind), place.cuda(), x, None, rows)
    want = torch.full((n + 1, H), -77.0, dtype=DT[kind])
    for t in range(T):
        for j in range(k):
            if 0 <= place[t, j] < n:
                want[place[t, j]] = x[t].cpu()
    assert torch.equal(rows.cpu(), want)


# ---- combine --------------------------------------------------------------------

COMBINE = [(1, 8, 2048, 8), (1, 1, 1, 1), (2, 2, 7, 5), (5, 3, 100, 20), (40, 8, 1000, 400), (17, 16, 2056, 300),
           (300, 5, 130, 1500), (9, 4, 4096, 36), (3, 6, 6000, 18)]


def combine_inputs(T, k, H, R, kind, weighted, whole=False):
    g = gen(T + H)
    make = ints if whole else randn
    rows, dy = make(g, R, H, dtype=DT[kind]), make(g, T, H, dtype=DT[kind])
    place = torch.randperm(max(R, T * k), generator=g)[:T * k].to(torch.int32).view(T, k)  # some behind R
    place[torch.rand(T, k, generator=g) < 0.15] = -1
    w = torch.rand(T, k, generator=g) if weighted else None
    if weighted:
        w[place < 0] = math.nan  # an empty slot's weight does not count
    if T > 2:
        place[1] = -1
    return rows, dy, place, w


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H,R", COMBINE)
def test_combine(T, k, H, R, kind, weighted):
    rows, _, place, w = combine_inputs(T, k, H, R, kind, weighted)
    for ldr, ldy in ((0, 0), (H + 5, H + 3), (-(-H // 8) * 8 + 8, -(-H // 8) * 8)):
        r, _ = strided(rows, ldr or H, math.nan)
        y, wide = strided(torch.full((T + 1, H), 7.0, dtype=DT[kind]), ldy or H, 7.0)
        moe.moe_combine(moe.make_combine(T, H, k, R, dtype=kind, ldr=ldr, ldy=ldy), r, place.cuda(),
                        None if w is None else w.cuda(), y)
        want, mag = ref.combine(rows, place, w)
        # k products and sums of fp32, one rounding to the output
        within(y[:T], want, mag * (k + 1) * U32 + want.abs() * ref.half_step(DT[kind]) * 1.01 + TINY, "combine")
        assert (wide[T] == 7).all() and (wide[:, H:] == 7).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,H,R", COMBINE)
def test_combine_grad(T, k, H, R, kind, weighted):
    """Whole numbers: dw is exact (sums below 2^24), drows rounded once or twice."""
    rows, dy, place, w = combine_inputs(T, k, H, R, kind, weighted, whole=True)
    want_r, want_w, mag, named = ref.combine_grad(dy, rows, place, w)
    assert float(mag.max()) < 2 ** 24
    for ldr, ldy in ((0, 0), (H + 5, H + 3)):
        r, _ = strided(rows, ldr or H, math.nan)
        d, _ = strided(dy, ldy or H, math.nan)
        c = moe.make_combine(T, H, k, R, dtype=kind, ldr=ldr, ldy=ldy)
        for parts in ("both", "rows", "weights"):
            dr, wide = strided(torch.full((R + 1, H), 7.0, dtype=DT[kind]), ldr or H, 7.0)
            dw = torch.full((T + 1, k), 7.0, device="cuda")
            moe.moe_combine_grad(c, d, r if parts != "rows" else None, place.cuda(), None if w is None else w.cuda(),
                                 dr if parts != "weights" else None, dw[:T] if parts != "rows" else None)
            if parts != "rows":
                assert torch.equal(dw[:T].cpu().double(), want_w) and (dw[T] == 7).all()
            if parts != "weights":
                bound = want_r.abs() * (U32 + ref.half_step(DT[kind]) * 1.01)
                within(dr[:R][named], want_r[named], bound[named], "drows")
                assert (dr[:R].cpu()[~named] == 7).all()
            assert (wide[R] == 7).all() and (wide[:, H:] == 7).all()


def test_combine_grad_of_ordinary_numbers():
    """fp32 sums of H products: each addend passes H / 128 + 9 roundings at most (a thread's chain and the tree)."""
    T, k, H, R = 50, 8, 2048, 400
    rows, dy, place, w = combine_inputs(T, k, H, R, "bf16", True)
    dw = torch.empty(T, k, device="cuda")
    moe.moe_combine_grad(moe.make_combine(T, H, k, R), dy.cuda(), rows.cuda(), place.cuda(), w.cuda(), None, dw)
    _, want, mag, _ = ref.combine_grad(dy, rows, place, w)
    within(dw, want, mag * (H / 128 + 9) * U32, "dw")


def test_combine_without_rows():
    c = moe.make_combine(3, 16, 2, 0)
    y = torch.full((3, 16), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((3, 2), 7.0, device="cuda")
    place = torch.tensor([[0, -1], [1, 5], [-1, -1]], dtype=torch.int32, device="cuda")
    moe.moe_combine(c, None, place, None, y)
    moe.moe_combine_grad(c, y, None, place, None, None, dw)
    assert (y == 0).all() and (dw == 0).all()


# ---- SwiGLU ---------------------------------------------------------------------

SWIGLU = [(1, 1), (1, 768), (3, 7), (5, 128), (17, 130), (64, 2048), (300, 250), (2, 4104), (1000, 72)]


def side_by_side(a, b):
    """Two matrices as the halves of one."""
    wide = torch.cat([a, b], 1).cuda()
    return wide[:, :a.shape[1]], wide[:, a.shape[1]:]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("R,I", SWIGLU)
def test_swiglu(R, I, kind):
    g = gen(R + I)
    gate, up = randn(g, R, I) * 3, randn(g, R, I)
    gate[0, 0] = -85.0
    gate, up = gate.to(DT[kind]), up.to(DT[kind])
    kb = -(-I // 128)
    want = ref.swiglu(gate, up)
    # exp within 2 ulp, 1 + e, reciprocal within 1 ulp, two products: 2^-20; then the output's rounding
    bound = want.abs() * (2.0 ** -20 + ref.half_step(DT[kind]) * 1.01) + TINY
    parts = [moe.quant_fp8(t.cuda()) for t in (gate, up)]
    codes_of, scales_of = (torch.cat(p, 1) for p in zip(*parts))
    if kind == "bf16":  # quotients of bf16 values are exact to the code
        for (c, _), t in zip(parts, (gate, up)):
            assert torch.equal(c.cpu().double(), ops_ref.quant(t)[0])
    for halves, used in ((False, None), (True, R), (True, R // 2)):
        a, b = side_by_side(gate, up) if halves else (gate.cuda(), up.cuda())
        ldh = I + 3 if halves else 0
        h, wide = strided(torch.full((R + 1, I), 7.0, dtype=DT[kind]), ldh or I, 7.0)
        codes = torch.full((R + 1, 256 * kb), 1.0, dtype=F8, device="cuda")
        scales = torch.full((R + 1, 2 * kb), 7.0, device="cuda")
        count = None if used is None else torch.tensor([99, used], dtype=torch.int32, device="cuda")[1:]
        s = moe.make_swiglu(R, I, dtype=kind, ld=2 * I if halves else 0, ldh=ldh)
        moe.moe_swiglu(s, a, b, h[:R], codes[:R], scales[:R], count)
        n = R if used is None else used
        within(h[:n], want[:n], bound[:n], "swiglu")
        assert torch.equal(codes[:n].float(), codes_of[:n].float()) and torch.equal(scales[:n], scales_of[:n])
        assert (wide[n:] == 7).all() and (wide[:, I:] == 7).all()
        assert (codes[n:].float() == 1).all() and (scales[n:] == 7).all()
        again = torch.empty(R, I, dtype=DT[kind], device="cuda")
        moe.moe_swiglu(moe.make_swiglu(R, I, dtype=kind, ld=s.ld), a, b, again, used=count)
        assert torch.equal(again[:n], h[:n])


@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("R,I", SWIGLU)
def test_swiglu_grad(R, I, kind, kept):
    g = gen(R + I)
    gate, up, dh = (randn(g, R, I) * 3).to(DT[kind]), randn(g, R, I, dtype=DT[kind]), randn(g, R, I, dtype=DT[kind])
    kb = -(-I // 128)
    codes = scales = None
    vg, vu = gate, up
    if kept:
        parts = [moe.quant_fp8(t.cuda()) for t in (gate, up)]
        codes, scales = (torch.cat(p, 1) for p in zip(*parts))
        # the values that the kernel multiplies: code times scale, rounded to fp32
        vg, vu = ((c.float() * s.repeat_interleave(128, 1))[:, :I].cpu() for c, s in parts)
    wg, wu, wh = ref.swiglu_grad(vg, vu, dh)
    sig, half = torch.sigmoid(vg.double()), ref.half_step(DT[kind]) * 1.01
    # s to 2^-21; 1 - s to 2^-21 of 1, so the slope to 2^-20 (s + |g| s); two more products
    bg = (dh.double() * vu.double()).abs() * 2.0 ** -19 * (sig + vg.double().abs() * sig) + wg.abs() * half + TINY
    for halves, used in ((False, None), (True, R // 2)):
        a, b = (None, None) if kept else side_by_side(gate, up) if halves else (gate.cuda(), up.cuda())
        both = torch.full((R + 1, 2 * I), 7.0, dtype=DT[kind], device="cuda")
        if halves:
            da, db = both[:R, :I], both[:R, I:]
        else:
            da, db = torch.full_like(both[:, :I], 7.0, memory_format=torch.contiguous_format)[:R], \
                torch.full_like(both[:, :I], 7.0, memory_format=torch.contiguous_format)[:R]
        h = torch.full((R + 1, I), 7.0, dtype=DT[kind], device="cuda")
        count = None if used is None else torch.tensor([used], dtype=torch.int32, device="cuda")
        s = moe.make_swiglu(R, I, dtype=kind, ld=2 * I if halves else 0)
        moe.moe_swiglu_grad(s, a, b, codes, scales, dh.cuda(), da, db, h[:R], count)
        n = R if used is None else used
        within(da[:n], wg[:n], bg[:n], "dgate")
        within(db[:n], wu[:n], wu[:n].abs() * (2.0 ** -20 + half) + TINY, "dup")
        within(h[:n], wh[:n], wh[:n].abs() * (2.0 ** -20 + half) + TINY, "h")
        assert (da[n:] == 7).all() and (db[n:] == 7).all() and (h[n:] == 7).all()
        d2, u2 = torch.empty_like(h[:R]), torch.empty_like(h[:R])
        moe.moe_swiglu_grad(moe.make_swiglu(R, I, dtype=kind), None if kept else gate.cuda(),
                            None if kept else up.cuda(), codes, scales, dh.cuda(), d2, u2, None, count)
        assert torch.equal(d2[:n], da[:n]) and torch.equal(u2[:n], db[:n])


@pytest.mark.parametrize("used", [-3, 0, 5, 99])
def test_swiglu_count_is_cut_off(used):
    g, u = (randn(gen(i), 5, 40, dtype=torch.bfloat16).cuda() for i in (1, 2))
    h = torch.full((6, 40), 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_swiglu(moe.make_swiglu(5, 40), g, u, h[:5], used=torch.tensor([used], dtype=torch.int32, device="cuda"))
    n = min(max(used, 0), 5)
    assert (h[n:] == 7).all() and not (h[:n] == 7).all(1).any()


# ---- selection ------------------------------------------------------------------

def check_select_grad(l, idx, dw, dscore, bias=None, out="f32", ld=0, **kw):
    T, E = l.shape
    k = idx.shape[1]
    dl = torch.full((T + 1, E), 7.0, dtype=DT[out], device="cuda")
    x, _ = strided(l, ld or E, 5.0)
    s = moe.make_select(T, E, k, logits="bf16" if l.dtype == torch.bfloat16 else "f32", ld=ld, **kw)
    moe.moe_select_grad(s, x, idx.cuda(), dw.cuda(), None if dscore is None else dscore.cuda(), dl[:T],
                        bias=None if bias is None else bias.cuda())
    want, mag = ref.select_grad(l, bias, idx, dw, dscore, **kw)
    # the exponentials' arguments, of up to 32, are off by 2^-24 of themselves: 2^-19 in a score, two scores in
    # a product, and sums of 16 slots or 1024 experts in trees: 2^-17 of the sums of magnitudes
    within(dl[:T], want, mag * 2.0 ** -17 + want.abs() * ref.half_step(DT[out]) * 1.01 + TINY, "select_grad")
    assert (dl[T] == 7).all()
    return dl[:T]


SELECT = [(1, 1, 1), (3, 7, 3), (5, 64, 8), (2, 65, 3), (9, 129, 16), (33, 256, 8), (4, 384, 6), (2, 513, 10), (3, 1024, 16)]


@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", SELECT)
def test_select_grad(T, E, k, score, renorm, balance):
    g = gen(T + E)
    l = randn(g, T, E) * 2
    idx = routing(g, T, E, k)
    dw, dscore = randn(g, T, k), randn(g, E) if balance else None
    for dt in ("f32", "bf16"):
        check_select_grad(l.to(DT[dt]), idx, dw, dscore, out=dt, score=score, renorm=renorm, scale=2.5)
    check_select_grad(l, idx, dw, dscore, ld=E + 3, out="bf16", score=score, renorm=renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_select_grad_masked_and_empty(score, renorm):
    g = gen(5)
    T, E, k = 6, 70, 4
    l, dw, dscore = randn(g, T, E), randn(g, T, k), randn(g, E)
    bias = torch.zeros(E)
    idx = routing(g, T, E, k)
    for t in range(T):
        l[t, idx[t, 0]] = [-math.inf, math.nan, math.inf, 0.0, 0.0, -math.inf][t]
    dw[0, 0] = dw[1, 0] = math.nan  # of a masked slot: not used
    bias[idx[3, 1]] = -math.inf
    dscore[idx[3, 1]] = math.nan  # of a masked expert
    idx[4] = torch.tensor([-1, E, 1 << 30, -5])
    l[5] = -math.inf
    got = check_select_grad(l, idx, dw, dscore, bias, score=score, renorm=renorm)
    assert (got[5] == 0).all()
    got = check_select_grad(l, idx, dw, None, bias, score=score, renorm=renorm)
    assert (got[4] == 0).all()


def test_select_grad_keeps_the_digits_of_saturated_scores():
    """One score near 1: its gradient, and the others', are small rests."""
    l = torch.tensor([[20.0, 0.0, 1.0, -3.0, 2.0], [60.0, 30.0, 29.0, 0.0, 1.0], [-100.0, -101.0, -99.0, -160.0, -600.0]])
    idx = torch.tensor([[0, 2], [0, 1], [2, 0]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 1.001], [3.0, -2.0], [1.0, 2.0]])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            if score == "softmax" or renorm:
                check_select_grad(l, idx, dw, None, score=score, renorm=renorm)
    check_select_grad(l, idx, dw, torch.tensor([1.0, 1.002, 0.999, 1.0, 1.0]), score="softmax")


def test_select_grad_where_scores_are_zero_in_64_bits():
    l = torch.tensor([[-800.0, -900.0, 5.0], [-800.0, 3.0, 5.0]])
    idx = torch.tensor([[0, 1], [0, 1]], dtype=torch.int32)
    dw = torch.tensor([[1.0, 2.0], [1.0, 2.0]])
    for score in ("softmax", "sigmoid"):
        got = check_select_grad(l, idx, dw, None, score=score)
        assert (got == 0).all()


@pytest.mark.parametrize("score,ng,tg", [("softmax", 1, 1), ("sigmoid", 4, 2)])
def test_select_grad_of_moe_select_by_differences(score, ng, tg):
    """Differences of moe_select's own weights: over 2h with h = 2^-6 they are off by h^2 / 6 of the third
    derivative (below 1 for these scores, times the sum of |dw|) and by the weights' 2^-19 / h."""
    g = gen(3)
    T, E, k, h = 4, 16, 4, 2.0 ** -6
    l, dw = torch.randperm(T * E, generator=g).view(T, E).float() / 8 - 4, randn(g, T, k)  # 1/8 apart: no h reorders
    s = moe.make_select(T, E, k, score=score, n_group=ng, topk_group=tg)
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")

    def loss(x):
        moe.moe_select(s, x.cuda(), None, idx, w)
        return (w.double().cpu() * dw.double()).sum(1)

    loss(l)
    dl = torch.empty(T, E, device="cuda")
    moe.moe_select_grad(s, l.cuda(), idx.clone(), dw.cuda(), None, dl)
    chosen = idx.clone()
    bound = dw.abs().sum(1).double() * (h * h / 6 + 2.0 ** -19 / h)
    for e in range(E):
        step = torch.zeros(E)
        step[e] = h
        up = loss(l + step)
        assert torch.equal(idx, chosen)
        want = (up - loss(l - step)) / (2 * h)
        assert ((dl[:, e].double().cpu() - want).abs() <= bound).all()


# ---- products -------------------------------------------------------------------

WAYS = ["y", "dx", "dw"]


def run_matmul(way, m, p, q, out, off=None, add=None, stream=None):
    f = {"y": moe.moe_matmul_bf16, "dx": moe.moe_matmul_bf16_dx, "dw": moe.moe_matmul_bf16_dw}[way]
    f(m, p, q, out, off, add, stream=stream)


def check_matmul(way, M, N, K, ends=None, out="f32", add=False, pad=(0, 0, 0), whole=True, at=0, poison=True):
    """pad: what the rows of x, w and y are longer; at: elements by which the operands are off a 16-byte address;
    whole numbers are exact in fp32, so equality is asked for.  Rows outside the groups hold NaN."""
    G = 1 if ends is None else len(ends) - 1
    g = gen(M + 3 * N + 7 * K + G)
    make = (lambda *s: ints(g, *s)) if whole else (lambda *s: randn(g, *s))
    ldx, ldw, ldy = K + pad[0], K + pad[1], N + pad[2]
    bounds = [0, M] if ends is None else [min(max(e, 0), M) for e in ends]
    used = torch.zeros(M, dtype=torch.bool)
    used[bounds[0]:max(bounds[0], bounds[-1])] = True

    def lay(t, ld, poisoned):
        """(CPU values, the tensor on the GPU): rows ld apart, `at` elements behind an aligned address."""
        t = t.to(torch.bfloat16)
        if poisoned and poison:
            t[~used] = math.nan
        n = t.shape[0] * ld
        flat = torch.full((n + 64,), math.nan, dtype=torch.bfloat16, device="cuda")
        v = flat[at:at + n].view(t.shape[0], ld)
        v[:, :t.shape[1]] = t.cuda()
        return t, v[:, :t.shape[1]]

    x, w, dy = lay(make(M, K), ldx, True), lay(make(G * N, K), ldw, False), lay(make(M, N), ldy, True)
    p, q = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    shape, ld = {"y": ((M, N), ldy), "dx": ((M, K), ldx), "dw": ((G * N, K), ldw)}[way]
    extra = ints(g, *shape).to(DT[out]) if add else None
    res, wide = strided(torch.full((shape[0] + 1, shape[1]), 7.0, dtype=DT[out]), ld, 7.0)
    av = None if extra is None else strided(extra, ld)[0]
    off = None if ends is None else torch.tensor(ends, dtype=torch.int32, device="cuda")
    m = moe.make_matmul_bf16(M, N, K, G=G, out=out, ldx=ldx, ldw=ldw, ldy=ldy)
    run_matmul(way, m, p[1], q[1], res[:shape[0]], off, av)
    cq = q[0].view(G, N, K) if way != "dw" else q[0]
    want, mag = ref.matmul(way, p[0], cq, bounds, None if extra is None else extra.view(G, N, K) if way == "dw" else extra,
                           (G, N, K) if way == "dw" else shape)
    want, mag = want.view(shape), mag.view(shape)
    rows = torch.ones(shape[0], dtype=torch.bool) if way == "dw" else used
    got = res[:shape[0]].cpu()
    if whole:
        assert float(mag[rows].max() if rows.any() else 0) < 2 ** 24
        assert torch.equal(got[rows], want[rows].to(DT[out])), (way, M, N, K, (got[rows] != want[rows].to(DT[out])).nonzero()[:5])
    else:
        # a sum of C products passes at most C roundings (of 2^-23: the matrix cores may cut) and the addend's
        C = {"y": K, "dx": N, "dw": M}[way]
        within(got[rows], want[rows], mag[rows] * (C + 1) * 2.0 ** -23 + want[rows].abs() * ref.half_step(DT[out]) * 1.01 + TINY,
               "matmul " + way)
    assert (got[~rows] == 7).all()
    assert (wide[shape[0]] == 7).all() and (wide[:, shape[1]:] == 7).all()
    if add:  # onto itself
        res[:shape[0]] = extra.cuda()
        run_matmul(way, m, p[1], q[1], res[:shape[0]], off, res[:shape[0]])
        assert torch.equal(res[:shape[0]].cpu()[rows], got[rows])


DENSE = [(1, 1, 1), (1, 16, 32), (1, 768, 2048), (3, 7, 5), (2, 130, 200), (7, 48, 384), (16, 256, 64), (17, 264, 72),
         (33, 64, 1000), (64, 64, 64), (65, 136, 136), (100, 250, 250), (128, 256, 512), (130, 520, 264), (256, 256, 256),
         (300, 1000, 328), (511, 768, 640), (1025, 264, 2056), (640, 2304, 768)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("M,N,K", DENSE)
def test_matmul(M, N, K, way, out):
    check_matmul(way, M, N, K, out=out)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("M,N,K", [(5, 40, 24), (70, 136, 264), (300, 512, 320)])
def test_matmul_add(M, N, K, way, out):
    check_matmul(way, M, N, K, out=out, add=True)
    check_matmul(way, M, N, K, [0, M // 3, M // 3, M], out=out, add=True)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("pad,at", [((8, 16, 24), 0), ((1, 0, 0), 0), ((0, 3, 0), 0), ((0, 0, 5), 0), ((0, 0, 0), 1),
                                    ((8, 8, 8), 4), ((8, 8, 8), 8)])
@pytest.mark.parametrize("M,N,K", [(9, 40, 48), (140, 264, 136)])
def test_matmul_strides_and_alignment(M, N, K, pad, at, way):
    for out in ("f32", "bf16"):
        check_matmul(way, M, N, K, out=out, pad=pad, at=at)
    check_matmul(way, M, N, K, [1, M // 2, M - 2], out="bf16", pad=pad, at=at)


GROUPS = {
    "one row each": list(range(0, 41)), "empty ends": [0, 0, 0, 5, 40, 40], "all empty": [20] * 9,
    "from behind the start": [7, 9, 30, 30, 33], "cut off": [-9, 3, 20, 99], "last only": [0, 0, 0, 0, 40],
    "one group": [3, 37], "reversed": [30, 10, 20, 5], "outside": [50, 60, 70],
}


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("name", sorted(GROUPS))
@pytest.mark.parametrize("N,K", [(72, 136), (50, 33)])
def test_matmul_groups(name, way, N, K):
    if name == "reversed":  # not allowed: nothing is read or written out of range
        m = moe.make_matmul_bf16(40, N, K, G=3, out="f32")
        shape = {"y": (40, N), "dx": (40, K), "dw": (3, N, K)}[way]
        p = torch.ones(40, K if way == "y" else N, dtype=torch.bfloat16, device="cuda")
        q = torch.ones((40, K) if way == "dw" else (3, N, K), dtype=torch.bfloat16, device="cuda")
        run_matmul(way, m, p, q, torch.zeros(shape, device="cuda"),
                   torch.tensor(GROUPS[name], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        return
    check_matmul(way, 40, N, K, GROUPS[name])
    check_matmul(way, 40, N, K, GROUPS[name], out="bf16", add=True)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("N,K,pad", [(768, 1024, 0), (64, 1032, 0), (256, 136, 0), (33, 72, 1)])
@pytest.mark.parametrize("copies", [1, 40, 200])
def test_matmul_offsets_that_decrease_stay_inside(way, N, K, pad, copies):
    """Groups of every tile height in an order that is not allowed (in the table of row tiles and without it):
    the rows that no offset reaches and what lies behind the last row stay as they were."""
    M, ends = 2000, [100, 1900, 300, 310, 120, 900, 100, 1800] * copies
    G = len(ends) - 1
    m = moe.make_matmul_bf16(M, N, K, G=G, ldx=K + pad, ldw=K, ldy=N + pad)
    cols = {"y": N + pad, "dx": K + pad, "dw": K}[way]
    rows = G * N if way == "dw" else M
    out = torch.full((rows + 300, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    x = torch.ones(M, K + pad, dtype=torch.bfloat16, device="cuda")[:, :K]
    dy = torch.ones(M, N + pad, dtype=torch.bfloat16, device="cuda")[:, :N]
    w = torch.ones(G, N, K, dtype=torch.bfloat16, device="cuda")
    p, q = {"y": (x, w), "dx": (dy, w), "dw": (dy, x)}[way]
    res = out[:rows] if way == "dw" else out[:rows, :cols - pad]
    run_matmul(way, m, p, q, res, torch.tensor(ends, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (out[rows:] == 7).all()
    if way != "dw":
        assert (out[:100] == 7).all() and (out[1900:] == 7).all() and (out[:, cols - pad:] == 7).all()


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("M,G,N,K", [(300, 65, 64, 128), (2000, 130, 136, 72), (1500, 5, 264, 520), (70, 300, 24, 40),
                                     (5000, 1000, 16, 8), (900, 8, 768, 256)])
def test_matmul_many_groups(M, G, N, K, way):
    g = gen(G)
    cuts = torch.randint(0, M - M // 50 + 1, (G - 1,), generator=g).sort().values.tolist()
    check_matmul(way, M, N, K, [0] + cuts + [M - M // 50], out="bf16")
    check_matmul(way, M, N, K, [0] + cuts + [M - M // 50], out="f32")


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("per", [5, 16, 20, 45, 70, 100, 128, 150, 220, 300])
def test_matmul_groups_of_every_tile_height(per, way):
    n = 9
    ends = [0]
    for i in range(n):
        ends.append(ends[-1] + max(0, per + (i * 7) % 11 - 5))
    check_matmul(way, ends[-1] + 3, 520, 328, ends, out="bf16")


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("M,N,K", [(2000, 4200, 264), (4100, 1032, 520), (520, 2056, 4096)])
def test_matmul_more_tiles_than_workgroups(M, N, K, way):
    check_matmul(way, M, N, K, out="bf16")


@pytest.mark.parametrize("way", WAYS)
def test_matmul_of_ordinary_numbers(way):
    for out in ("f32", "bf16"):
        check_matmul(way, 300, 520, 264, out=out, whole=False, add=True)
        check_matmul(way, 300, 520, 264, [0, 100, 101, 250], out=out, whole=False)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("M,N,K", [(20, 48, 64), (200, 264, 328)])
def test_matmul_nan_stays_in_its_row_and_column(M, N, K, way):
    """One NaN of p and one infinity of q: only the sums over them are not finite."""
    g = gen(1)
    p, q = {"y": ((M, K), (N, K)), "dx": ((M, N), (N, K)), "dw": ((M, N), (M, K))}[way]
    a, b = ints(g, *p, dtype=torch.bfloat16).cuda(), (ints(g, *q).abs() + 1).to(torch.bfloat16).cuda()
    a[p[0] // 2, p[1] // 3] = math.nan
    b[q[0] // 3, q[1] // 2] = math.inf
    shape = {"y": (M, N), "dx": (M, K), "dw": (1, N, K)}[way]
    out = torch.empty(shape, device="cuda")
    run_matmul(way, moe.make_matmul_bf16(M, N, K, out="f32"), a, b if way == "dw" else b[None], out)
    bad = torch.zeros(shape, dtype=torch.bool).view(shape[-2:])
    if way == "dw":
        bad[p[1] // 3] = True
        bad[:, q[1] // 2] = True
    else:
        bad[p[0] // 2] = True
        bad[:, q[0] // 3 if way == "y" else q[1] // 2] = True
    ok = torch.isfinite(out.view(shape[-2:])).cpu()
    assert ok[~bad].all()


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M", [0, 5])
def test_matmul_dw_of_no_rows(M, out):
    add = ints(gen(1), 3, 24, 40, dtype=DT[out]).cuda()
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    m = moe.make_matmul_bf16(M, 24, 40, G=3, out=out)
    dy, x = torch.empty(M, 24, dtype=torch.bfloat16, device="cuda"), torch.empty(M, 40, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((3, 24, 40), 7.0, dtype=DT[out], device="cuda")
    run_matmul("dw", m, dy if M else None, x if M else None, dw, off)
    assert (dw == 0).all()
    run_matmul("dw", m, dy if M else None, x if M else None, dw, off, add)
    assert torch.equal(dw, add)


# Products that the rule of the tile shapes (mm16_shape) gives to each of them, as one matrix and as groups:
# largest tiles first; the last sizes are the smallest tiles'.
SHAPED = {
    "y": [(2500, 4104, 136, 1), (2500, 4104, 136, 3), (9000, 1544, 200, 40), (1200, 4104, 136, 3), (2500, 2056, 1032, 1),
          (9000, 520, 264, 40), (2500, 1544, 200, 1), (2500, 1544, 200, 9), (9000, 200, 1544, 600), (700, 4104, 136, 1),
          (1200, 1544, 200, 3), (9000, 520, 264, 600), (500, 1544, 200, 1), (500, 2056, 1032, 3), (9000, 136, 72, 40),
          (1200, 200, 1544, 1), (2500, 136, 4104, 1), (5000, 136, 72, 600), (37, 4104, 136, 3), (37, 264, 4104, 3),
          (700, 200, 1544, 1), (37, 136, 72, 600)],
    "dx": [(5000, 136, 4104, 1), (5000, 264, 4104, 3), (9000, 200, 1544, 40), (2500, 264, 4104, 1), (1200, 136, 4104, 3),
           (5000, 200, 1544, 40), (1200, 264, 4104, 1), (700, 264, 4104, 9), (9000, 200, 1544, 600), (700, 136, 4104, 1),
           (500, 264, 4104, 3), (9000, 520, 264, 600), (500, 2056, 1032, 1), (200, 264, 4104, 3), (9000, 136, 72, 40),
           (1200, 4104, 136, 1), (37, 1544, 200, 3), (2500, 520, 264, 600)],
    "dw": [(500, 2056, 1032, 9), (9000, 200, 1544, 600), (300, 2056, 1032, 3), (5000, 136, 72, 600), (200, 264, 4104, 3),
           (9000, 136, 4104, 1), (37, 1544, 200, 3), (5000, 136, 72, 40), (1200, 1544, 200, 1)],
}


# The same for sums that are short, whose tiles' ends count.
SHAPED["y"] += [(9000, 1056, 64, 3), (5000, 2080, 64, 1), (9000, 1352, 64, 40), (5000, 1512, 72, 3), (4100, 2056, 520, 1),
                (200, 544, 72, 40), (1030, 1032, 8, 1), (1200, 160, 80, 40), (200, 1056, 64, 9), (200, 104, 64, 40),
                (330, 520, 16, 1), (200, 72, 64, 9), (200, 64, 120, 1), (200, 88, 200, 40)]
SHAPED["dx"] += [(9000, 64, 1472, 40), (9000, 80, 1448, 40), (5000, 64, 960, 40), (4100, 8, 2056, 1), (200, 72, 1992, 40),
                 (2060, 520, 2056, 1), (200, 72, 528, 40), (1030, 8, 1032, 1), (200, 72, 984, 9), (2500, 72, 88, 40),
                 (200, 64, 80, 9), (200, 96, 112, 3), (330, 16, 520, 1)]


@pytest.mark.parametrize("way,M,N,K,G", [(w,) + c for w in WAYS for c in SHAPED[w]])
def test_matmul_of_every_tile_shape(way, M, N, K, G):
    ends = None
    if G > 1:
        g = gen(M + G)
        ends = [1] + torch.randint(1, M - 7, (G - 1,), generator=g).sort().values.tolist() + [M - 7]
    check_matmul(way, M, N, K, ends, out="bf16")
    check_matmul(way, M, N, K, ends, out="f32", add=True)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("C", [1, 8, 16, 56, 63, 64, 65, 72, 120, 128, 129, 136, 184, 192, 200, 248, 256, 264, 320, 520, 1000])
def test_matmul_of_every_depth(C, way):
    """The depth's last stages, which the groups of waves share out: few rows, some, many."""
    for P, Q in ((9, 264), (70, 136), (330, 520), (1030, 1032)):
        M, N, K = {"y": (P, Q, C), "dx": (P, C, Q), "dw": (C, P, Q)}[way]
        check_matmul(way, M, N, K, out="f32")
    M, N, K = {"y": (40, 136, C), "dx": (40, C, 136), "dw": (3 * C, 72, 136)}[way]
    check_matmul(way, M, N, K, [0, M // 3, M // 3, 2 * (M // 3), M], out="f32")


@pytest.mark.parametrize("N,K", [(8, 8), (16, 40), (32, 32), (40, 64), (64, 200), (184, 192), (512, 512)])
@pytest.mark.parametrize("C", [192, 193, 255, 256, 257, 320, 321, 449, 512, 513, 577, 700, 1030, 2049])
def test_matmul_dw_of_smallest_tiles(C, N, K):
    """Four groups of waves share the depth of tiles of 32 x 32; rows outside the groups hold NaN."""
    check_matmul("dw", C, N, K, out="bf16", add=True)
    check_matmul("dw", C, N, K, out="f32", pad=(8, 0, 16))
    check_matmul("dw", 3 * C, N, K, [5, 5 + C, 5 + C, 7 + 2 * C, 3 * C - 4])


@pytest.mark.parametrize("way", ["y", "dx"])
@pytest.mark.parametrize("C", [8, 64, 72, 136, 200, 264])
def test_matmul_of_large_outputs_and_every_depth(C, way):
    for P, Q in ((2060, 2056), (4100, 2056), (4360, 4104)):
        check_matmul(way, P, *((Q, C) if way == "y" else (C, Q)), out="bf16")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("N,K", [(64, 64), (72, 136), (136, 264), (256, 520)])
@pytest.mark.parametrize("lengths", [[193], [256], [1001], [0, 1, 63, 64, 65, 127, 128, 129, 191, 192, 193, 3000, 0],
                                     [700, 0, 0, 650], [5, 1400, 64, 1]])
def test_matmul_dw_of_few_tiles_and_many_rows(lengths, N, K, out):
    """Groups whose rows are few tiles of dw: two groups of waves share the depth, of which the second may have none."""
    ends = [3]
    for n in lengths:
        ends.append(ends[-1] + n)
    check_matmul("dw", ends[-1] + 2, N, K, ends, out=out)
    check_matmul("dw", ends[-1] + 2, N, K, ends, out=out, add=True, pad=(8, 16, 24))
    if len(lengths) == 1:
        check_matmul("dw", lengths[0], N, K, out=out)


@pytest.mark.parametrize("way", WAYS)
@pytest.mark.parametrize("C", [511, 512, 513, 575, 639, 641, 705, 769, 1023, 1025, 1281, 2050])
def test_matmul_odd_sizes_of_few_tiles_and_long_sums(C, way):
    M, N, K = {"y": (37, 77, C), "dx": (37, C, 77), "dw": (C, 37, 77)}[way]
    check_matmul(way, M, N, K, out="bf16", pad=(1, 0, 3))
    check_matmul(way, M, N, K, add=True)
    cut = M // 3
    ends = [1, cut, cut, M - 1] if way != "dw" else [0, 1600 * C // 1601, C - 1, C]
    check_matmul(way, M, N, K, ends)


@pytest.mark.parametrize("way", WAYS)
def test_matmul_odd_sizes_of_many_tiles(way):
    check_matmul(way, 2111, 2049, 131, out="bf16")
    check_matmul(way, 1501, 1311, 77, [3, 3, 700, 1111, 1490], out="f32", add=True)


def test_matmul_beyond_32_bits():
    """Matrices of more than 2^32 bytes: the last groups' products, and nothing in front of them."""
    G, N, K, M = 300, 2048, 4096, 40
    w = torch.zeros(G, N, K, dtype=torch.bfloat16, device="cuda")
    g = gen(4)
    w[-1] = ints(g, N, K, dtype=torch.bfloat16).cuda()
    ends = torch.zeros(G + 1, dtype=torch.int32)
    ends[-1] = M
    off = ends.cuda()
    x, dy = ints(g, M, K, dtype=torch.bfloat16), ints(g, M, N, dtype=torch.bfloat16)
    m = moe.make_matmul_bf16(M, N, K, G=G, out="f32")
    y, dx = torch.empty(M, N, device="cuda"), torch.empty(M, K, device="cuda")
    moe.moe_matmul_bf16(m, x.cuda(), w, y, off)
    moe.moe_matmul_bf16_dx(m, dy.cuda(), w, dx, off)
    last = w[-1].cpu().double()
    assert torch.equal(y.cpu().double(), x.double() @ last.t()) and torch.equal(dx.cpu().double(), dy.double() @ last)
    moe.moe_matmul_bf16_dw(moe.make_matmul_bf16(M, N, K, G=G), dy.cuda(), x.cuda(), w, off)
    assert torch.equal(w[-1].cpu().double(), (dy.double().t() @ x.double()).to(torch.bfloat16).double())
    assert int(torch.count_nonzero(w[:-1].view(torch.int16).view(-1, 4096)[::64])) == 0


def test_rows_beyond_32_bits():
    """Rows past 2^32 bytes in moe_gather, moe_combine and its gradient, and in SwiGLU with its checkpoint."""
    H, k = 8192, 2
    T = 140_000
    R = T * k
    rows = torch.empty(R, H, dtype=torch.bfloat16, device="cuda")
    x = torch.arange(T, device="cuda", dtype=torch.float32).remainder_(251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    of = torch.arange(R, dtype=torch.int32, device="cuda").view(T, k)
    moe.moe_gather(moe.make_dispatch(T, H, 1, k), of, x, None, rows)
    for r in (0, R // 2, R - 1):
        assert (rows[r] == float((r // k) % 251)).all()
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    c = moe.make_combine(T, H, k, R)
    moe.moe_combine(c, rows, of, None, y)
    assert torch.equal(y[-3:], 2 * x[-3:]) and torch.equal(y[:3], 2 * x[:3])
    dw = torch.empty(T, k, device="cuda")
    drows = torch.empty_like(rows)
    moe.moe_combine_grad(c, x, rows, of, torch.full((T, k), 0.5, device="cuda"), drows, dw)
    assert torch.equal(drows[-2:], 0.5 * x[-1:].expand(2, H))
    v = float(x[-1, 0])
    assert float(dw[-1, 1]) == v * v * H
    s = moe.make_swiglu(R, H)
    codes = torch.empty(R, 2 * H, dtype=F8, device="cuda")
    scales = torch.empty(R, 2 * H // 128, device="cuda")
    h = torch.empty_like(rows)
    moe.moe_swiglu(s, rows, rows, h, codes, scales)
    want = ref.swiglu(rows[-1].cpu(), rows[-1].cpu())
    within(h[-1], want, want.abs() * (2.0 ** -20 + 2.0 ** -8 * 1.01) + TINY, "far swiglu")
    moe.moe_swiglu_grad(s, None, None, codes, scales, drows, rows, y.new_empty(R, H), h)
    g = (codes[-1].float() * scales[-1].repeat_interleave(128)).cpu()
    want = ref.swiglu_grad(g[:H], g[H:], drows[-1].cpu())[2]
    within(h[-1], want, want.abs() * (2.0 ** -20 + 2.0 ** -8 * 1.01) + TINY, "far h")


@pytest.mark.parametrize("T,k", [(64, 2), (129, 1), (43, 3), (341, 3), (4096, 1), (4097, 1), (1365, 3), (21845, 3), (65537, 1)])
@pytest.mark.parametrize("E", [1, 3, 64, 1024])
def test_dispatch_at_the_borders_of_its_ways(T, k, E):
    """Up to 128 pairs, 4 and 64 blocks of whole tokens, and more."""
    g = gen(T + E)
    idx = torch.randint(-1, E, (T, k), generator=g).to(torch.int32)  # repeated experts, empty slots
    x = randn(g, T, 9, dtype=torch.bfloat16).cuda()
    check_dispatch(idx, x, E)


# ---- together -------------------------------------------------------------------

class Layer:
    """The routed layer's step as a training program makes it from the operators."""

    def __init__(self, T, H, E, k, I, keep, score="softmax", seed=0):
        g = gen(seed)
        bf = torch.bfloat16
        self.T, self.H, self.E, self.k, self.I, self.keep = T, H, E, k, I, keep
        self.x, self.wr = randn(g, T, H, dtype=bf).cuda(), (randn(g, E, H) * H ** -0.5).to(bf).cuda()
        self.wg, self.wu = ((randn(g, E, I, H) * H ** -0.5).to(bf).cuda() for _ in range(2))
        self.wd = (randn(g, E, H, I) * I ** -0.5).to(bf).cuda()
        self.dy = randn(g, T, H, dtype=bf).cuda()
        n = T * k
        e = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        f, i32 = torch.float32, torch.int32
        self.logits, self.idx, self.w = e(T, E, dt=f), e(T, k, dt=i32), e(T, k, dt=f)
        self.offsets, self.src, self.of = e(E + 1, dt=i32), e(n, dt=i32), e(T, k, dt=i32)
        self.rows, self.gate, self.up, self.h, self.o, self.y = e(n, H), e(n, I), e(n, I), e(n, I), e(n, H), e(T, H)
        kb = -(-I // 128)
        self.codes, self.scales = (e(n, 256 * kb, dt=F8), e(n, 2 * kb, dt=f)) if keep else (None, None)
        self.do, self.dw, self.dh, self.dgate, self.dup, self.dlogits = (e(n, H), e(T, k, dt=f), e(n, I), e(n, I),
                                                                         e(n, I), e(T, E))
        self.drows, self.dx = e(n, H), e(T, H)
        self.gwg, self.gwu, self.gwd, self.gwr = (e(E, I, H, dt=f), e(E, I, H, dt=f), e(E, H, I, dt=f), e(1, E, H, dt=f))
        self.shape = moe.make_shape(T, H, E, k, I)
        self.router = moe.make_weights(self.wr, None, None, None)
        self.sel = moe.make_select(T, E, k, score=score)
        self.dis = moe.make_dispatch(T, H, E, k)
        self.ws = e(moe.moe_dispatch_workspace_bytes(self.dis), dt=torch.uint8)
        self.up_mm = moe.make_matmul_bf16(n, I, H, G=E)
        self.down_mm = moe.make_matmul_bf16(n, H, I, G=E)
        self.up_f, self.down_f = moe.make_matmul_bf16(n, I, H, G=E, out="f32"), moe.make_matmul_bf16(n, H, I, G=E, out="f32")
        self.rout, self.rout_f = moe.make_matmul_bf16(T, E, H), moe.make_matmul_bf16(T, E, H, out="f32")
        self.act, self.com = moe.make_swiglu(n, I), moe.make_combine(T, H, k, n)

    def step(self):
        s, off = self, self.offsets
        moe.moe_logits(s.shape, s.router, s.x, s.logits)
        moe.moe_select(s.sel, s.logits, None, s.idx, s.w)
        moe.moe_dispatch(s.dis, s.idx, s.x, None, s.rows, off, s.src, s.of, s.ws)
        moe.moe_matmul_bf16(s.up_mm, s.rows, s.wg, s.gate, off)
        moe.moe_matmul_bf16(s.up_mm, s.rows, s.wu, s.up, off)
        used = off[s.E:]
        moe.moe_swiglu(s.act, s.gate, s.up, s.h, s.codes, s.scales, used)
        moe.moe_matmul_bf16(s.down_mm, s.h, s.wd, s.o, off)
        moe.moe_combine(s.com, s.o, s.of, s.w, s.y)
        # backward
        moe.moe_combine_grad(s.com, s.dy, s.o, s.of, s.w, s.do, s.dw)
        moe.moe_matmul_bf16_dx(s.down_mm, s.do, s.wd, s.dh, off)
        g, u = (None, None) if s.keep else (s.gate, s.up)
        moe.moe_swiglu_grad(s.act, g, u, s.codes, s.scales, s.dh, s.dgate, s.dup, s.h, used)
        moe.moe_matmul_bf16_dw(s.down_f, s.do, s.h, s.gwd, off)
        moe.moe_matmul_bf16_dw(s.up_f, s.dgate, s.rows, s.gwg, off)
        moe.moe_matmul_bf16_dw(s.up_f, s.dup, s.rows, s.gwu, off)
        moe.moe_matmul_bf16_dx(s.up_mm, s.dgate, s.wg, s.drows, off)
        moe.moe_matmul_bf16_dx(s.up_mm, s.dup, s.wu, s.drows, off, s.drows)
        moe.moe_combine(s.com, s.drows, s.of, None, s.dx)
        moe.moe_select_grad(s.sel, s.logits, s.idx, s.dw, None, s.dlogits)
        moe.moe_matmul_bf16_dx(s.rout, s.dlogits, s.wr[None], s.dx, None, s.dx)
        moe.moe_matmul_bf16_dw(s.rout_f, s.dlogits, s.x, s.gwr)
        return {n: getattr(s, n) for n in ("y", "dx", "gwg", "gwu", "gwd", "gwr")}

    def definition(self):
        """The same by differentiation in 64 bits, with the routing's choice as it is."""
        d = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
        x, wr, wg, wu, wd = map(d, (self.x, self.wr, self.wg, self.wu, self.wd))
        idx = self.idx.cpu().long()
        l = x @ wr.t()
        s = torch.softmax(l, 1) if self.sel.score == moe.MOE_SCORE_SOFTMAX else torch.sigmoid(l)
        w = s.gather(1, idx)
        w = w / w.sum(1, keepdim=True)
        y = torch.zeros(self.T, self.H, dtype=torch.float64)
        for j in range(self.k):
            a = torch.einsum("th,tih->ti", x, wg[idx[:, j]])
            b = torch.einsum("th,tih->ti", x, wu[idx[:, j]])
            y = y + w[:, j:j + 1] * torch.einsum("ti,thi->th", a * torch.sigmoid(a) * b, wd[idx[:, j]])
        grads = torch.autograd.grad(y, (x, wg, wu, wd, wr), self.dy.double().cpu())
        return dict(zip(("y", "dx", "gwg", "gwu", "gwd", "gwr"), (y.detach(),) + grads))


@pytest.mark.parametrize("T,H,E,k,I,score", [(1, 256, 8, 2, 128, "softmax"), (37, 192, 8, 3, 192, "sigmoid"),
                                             (160, 256, 16, 4, 256, "softmax")])
@pytest.mark.parametrize("keep", [False, True])
def test_training_step_together(T, H, E, k, I, score, keep):
    """Each of the 12 tensors between the operators is rounded once to bf16 (2^-8 of each value at most, and of the
    norm), and a checkpoint moves gate and up by 2^-4 at most, which dgate, dup and h pass on with a slope of at
    most 1.1 each: norms of the differences below 12 * 2^-8, and 3 * 1.1 * 2^-4 more with the checkpoint.  The
    router's gradient is a difference of the dw, which the norm of dw's own error bounds relative to dw, not to
    the difference: three times that."""
    layer = Layer(T, H, E, k, I, keep, score)
    got = {n: v.clone() for n, v in layer.step().items()}
    want = layer.definition()
    for n in want:
        err = float((got[n].double().cpu().view(want[n].shape) - want[n]).norm() / want[n].norm())
        bar = 12 * 2.0 ** -8 + (3.3 * 2.0 ** -4 if keep and n != "y" else 0.0)
        bar *= 3 if n == "gwr" else 1
        print("%s: %.3g (bar %.3g)" % (n, err, bar), file=sys.stderr, flush=True)
        assert err <= bar, (n, err, bar)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_training_step_repeats_captures_and_other_streams(T):
    """The same bits from a second call, a replayed graph and another stream."""
    layer = Layer(T, 256, 16, 4, 128, True, seed=T)
    first = {n: v.clone() for n, v in layer.step().items()}

    def same(what):
        torch.cuda.synchronize()
        for n, v in first.items():
            assert torch.equal(getattr(layer, n), v), (what, n)
            getattr(layer, n).fill_(3.0)

    layer.step()
    same("again")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer.step()
    torch.cuda.current_stream().wait_stream(s)
    same("another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for i in range(3):
        graph.replay()
        same("replay %d" % i)
        torch.randn(1000, device="cuda").sum().item()
    layer.step()
    same("eager after replays")


def test_stream_argument_and_two_calls_at_once():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    g = gen(8)
    M, N, K = 700, 264, 328
    x, w = ints(g, M, K, dtype=torch.bfloat16).cuda(), ints(g, 1, N, K, dtype=torch.bfloat16).cuda()
    want = (x.double() @ w[0].double().t()).float()
    ys = [torch.zeros(M, N, device="cuda") for _ in range(2)]
    T, E, k = 5000, 64, 4
    idx = [routing(g, T, E, k, 0.1) for _ in range(2)]
    dev = [i.cuda() for i in idx]
    d = moe.make_dispatch(T, 64, E, k)
    xs = randn(g, T, 64, dtype=torch.bfloat16).cuda()
    outs = [(torch.zeros(T * k, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
             torch.zeros(T * k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, dtype=torch.int32, device="cuda"),
             torch.empty(moe.moe_dispatch_workspace_bytes(d), dtype=torch.uint8, device="cuda")) for _ in range(2)]
    torch.cuda.synchronize()
    m = moe.make_matmul_bf16(M, N, K, out="f32")
    for _ in range(3):
        for i, st in enumerate((a, b)):
            moe.moe_matmul_bf16(m, x, w, ys[i], stream=st)
            rows, off, src, of, ws = outs[i]
            moe.moe_dispatch(d, dev[i], xs, None, rows, off, src, of, ws, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(ys[i], want)
        woff, _, wof = ref.sort(idx[i], E)
        assert torch.equal(outs[i][1].cpu(), woff) and torch.equal(outs[i][3].cpu(), wof)


def test_binding_refuses_what_does_not_fit():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    m = moe.make_matmul_bf16(8, 16, 24)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_matmul_bf16(m, torch.zeros(8, 24, device="cuda"), bf(1, 16, 24), bf(8, 16))
    with pytest.raises(ValueError, match="holds"):
        moe.moe_matmul_bf16(m, bf(8, 24), bf(1, 15, 24), bf(8, 16))
    with pytest.raises(ValueError, match="not on a GPU"):
        moe.moe_matmul_bf16_dx(m, bf(8, 16).cpu(), bf(1, 16, 24), bf(8, 24))
    with pytest.raises(ValueError, match="strides"):
        moe.moe_matmul_bf16_dw(m, bf(8, 1).expand(8, 16), bf(8, 24), bf(1, 16, 24))
    with pytest.raises(ValueError, match="holds"):
        moe.moe_combine(moe.make_combine(4, 16, 2, 8), bf(7, 16), torch.zeros(4, 2, dtype=torch.int32, device="cuda"),
                        None, bf(4, 16))
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_swiglu(moe.make_swiglu(4, 16), bf(4, 16), bf(4, 16), bf(4, 16), bf(4, 256), torch.zeros(4, 2, device="cuda"))
    with pytest.raises(moe.MoeError):
        moe.moe_swiglu_grad(moe.make_swiglu(4, 16), None, None, None, None, bf(4, 16), bf(4, 16), bf(4, 16))
    with pytest.raises(moe.MoeError):
        moe.moe_dispatch(moe.make_dispatch(3, 16, 4, 2, x="fp8"), torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                         torch.zeros(3, 128, dtype=F8, device="cuda"), None, bf(6, 16),
                         torch.zeros(5, dtype=torch.int32, device="cuda"), None,
                         torch.zeros(3, 2, dtype=torch.int32, device="cuda"), None)
