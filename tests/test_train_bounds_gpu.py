"""What test_train_gpu.py leaves open: that what is not finite reaches every sum over it, and the
router's gradient within a bound made of the step's own numbers."""
import math
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import routed_expert_ffn_moe_amd as moe  # noqa: E402
from test_train_gpu import DT, Layer, gen, ints, run_matmul  # noqa: E402


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("grouped", [False, True])
@pytest.mark.parametrize("way", ["y", "dx", "dw"])
@pytest.mark.parametrize("M,N,K", [(20, 48, 64), (200, 264, 328), (700, 520, 136)])
def test_matmul_keeps_what_is_not_finite(M, N, K, way, grouped, odd, out):
    """A NaN of p and an infinity of q: the sums over either are not finite, all others are."""
    g = gen(1)
    N, K = N - odd, K - odd
    p, q = {"y": ((M, K), (N, K)), "dx": ((M, N), (N, K)), "dw": ((M, N), (M, K))}[way]
    a, b = ints(g, *p, dtype=torch.bfloat16), (ints(g, *q).abs() + 1).to(torch.bfloat16)
    a[p[0] // 2, p[1] // 3] = math.nan
    b[q[0] // 3, q[1] // 2] = math.inf
    off, G = None, 1
    if grouped:  # all rows in the second of three groups, whose matrix is the one with the infinity
        off, G = torch.tensor([0, 0, M, M], dtype=torch.int32, device="cuda"), 3
    if way != "dw":
        b = torch.cat([torch.ones(1, *q), b[None], torch.ones(1, *q)])[0 if grouped else 1:][:G].to(torch.bfloat16)
    shape = {"y": (M, N), "dx": (M, K), "dw": (G, N, K)}[way]
    res = torch.zeros(shape, dtype=DT[out], device="cuda")
    run_matmul(way, moe.make_matmul_bf16(M, N, K, G=G, out=out), a.cuda(), b.cuda(), res, off)
    bad = torch.zeros(shape[-2:], dtype=torch.bool)
    if way == "dw":
        bad[p[1] // 3] = True
        bad[:, q[1] // 2] = True
    else:
        bad[p[0] // 2] = True
        bad[:, q[0] // 3 if way == "y" else q[1] // 2] = True
    ok = torch.isfinite(res.cpu())
    if way == "dw":
        if grouped:
            assert (res[0] == 0).all() and (res[2] == 0).all()
        ok = ok[G // 2]
    assert ok[~bad].all() and not ok[bad].any()


@pytest.mark.parametrize("T,H,E,k,I,score", [(37, 192, 8, 3, 192, "sigmoid"), (160, 256, 16, 4, 256, "softmax"),
                                             (500, 320, 32, 6, 128, "softmax")])
def test_router_gradient_of_a_training_step(T, H, E, k, I, score):
    """dw = <dy, o>: the experts' rows o passed gate, up, h and their own rounding, 2^-8 of their norm each at
    most (with a slope of 1.1 of gate and up: 4.2), which have nothing to do with dy, so that the norm of dw's
    error is that share of dw's; twice that is allowed for what chance adds over T * k products.  A token's
    logits take dw through the matrix J (p and the selection's slope), so the norm of dlogits' error is at most
    the largest |J| times that of dw's, and 2^-8 of dlogits for their rounding; the gradient of the router's
    weights takes it times the largest singular value of x.  The checkpoint does not lie on this way: the same bits
    with it."""
    layer = Layer(T, H, E, k, I, False, score)
    got = {n: v.clone() for n, v in layer.step().items()}
    dw, dl = layer.dw.double().cpu(), layer.dlogits.double().cpu()
    kept = Layer(T, H, E, k, I, True, score)
    kept.step()
    assert torch.equal(kept.gwr, got["gwr"]) and torch.equal(kept.y, got["y"])

    x, wr, wg, wu, wd, dy = (t.double().cpu() for t in (layer.x, layer.wr, layer.wg, layer.wu, layer.wd, layer.dy))
    idx = layer.idx.cpu().long()
    want_dw = torch.empty(T, k, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            a = wg[e] @ x[t]
            want_dw[t, j] = dy[t] @ (wd[e] @ (a * torch.sigmoid(a) * (wu[e] @ x[t])))
    s = torch.softmax(x @ wr.t(), 1) if score == "softmax" else torch.sigmoid(x @ wr.t())
    s = s.gather(1, idx)
    p = s / s.sum(1, keepdim=True)
    slope = torch.ones_like(s) if score == "softmax" else 1 - s
    J = slope[:, :, None] * (torch.diag_embed(p) - p[:, :, None] * p[:, None, :])
    want_dl = torch.zeros(T, E, dtype=torch.float64).scatter_(1, idx, torch.matmul(J, want_dw[:, :, None])[:, :, 0])
    want = want_dl.t() @ x

    bar_dw = 2 * 4.2 * 2.0 ** -8 * float(want_dw.norm())
    bar_dl = float(torch.linalg.matrix_norm(J, 2).max()) * bar_dw + 2.0 ** -8 * float(want_dl.norm())
    bar = float(torch.linalg.matrix_norm(x, 2)) * bar_dl
    assert bar < 0.5 * float(want.norm())  # a gradient of half its size, or without half of its terms, does not pass
    for what, a, b, most in (("dw", dw, want_dw, bar_dw), ("dlogits", dl, want_dl, bar_dl),
                             ("router", got["gwr"].double().cpu()[0], want, bar)):
        err = float((a - b).norm())
        print("%s: %.3g of its norm (bar %.3g)" % (what, err / float(b.norm()), most / float(b.norm())), file=sys.stderr,
              flush=True)
        assert err <= most, (what, err, most)
