"""The training operators as a program keeps them: a captured step that is replayed on other
tokens, and a step with dropped slots in buffers that nobody cleared."""
import math
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import routed_expert_ffn_moe_amd as moe  # noqa: E402
from test_train_gpu import Layer, gen, randn  # noqa: E402

OUT = ("y", "dx", "gwg", "gwu", "gwd", "gwr")


def tokens(kind, T, H, seed):
    """Tokens that spread over the experts, that all go to the same few, or that are all alike."""
    x = randn(gen(seed), T, H)
    if kind == "few":
        x = x * 0.05 + x[:1] * 2
    elif kind == "one":
        x = x[:1].expand(T, H)
    return x.to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T,E,k", [(3, 16, 4), (64, 16, 4), (700, 40, 6)])
def test_captured_step_on_other_tokens(T, E, k):
    """A graph holds no routing: replayed on other tokens it gives what an eager step gives."""
    H, I = 256, 128
    layer, eager = (Layer(T, H, E, k, I, True, seed=T) for _ in range(2))
    layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    for i, kind in enumerate(("spread", "few", "one", "spread")):
        x, dy = tokens(kind, T, H, i), tokens("spread", T, H, 100 + i)
        for l in (layer, eager):
            l.x.copy_(x)
            l.dy.copy_(dy)
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        for n in OUT:
            assert torch.equal(getattr(layer, n), getattr(eager, n)), (kind, n)
        assert torch.equal(layer.offsets, eager.offsets)


@pytest.mark.parametrize("T,H,E,k,I,drop", [(5, 192, 8, 3, 128, 0.5), (90, 256, 16, 4, 192, 0.2), (300, 128, 40, 6, 136, 0.9),
                                            (40, 128, 8, 2, 64, 1.0)])
@pytest.mark.parametrize("keep", [False, True])
def test_step_with_dropped_slots_in_poisoned_buffers(T, H, E, k, I, drop, keep):
    """Slots dropped after the selection: their rows take no place, and what lies behind the last row (NaN in
    every buffer) reaches nothing.  The bounds are those of the step without drops: 12 roundings of 2^-8 of the
    norm, 3.3 * 2^-4 more behind a checkpoint; the router's gradient is checked by its finiteness and its
    untouched part alone."""
    layer = Layer(T, H, E, k, I, keep, seed=T)
    moe.moe_logits(moe.make_shape(T, H, E, k, 64), layer.router, layer.x, layer.logits)  # any I that a layer may have
    moe.moe_select(layer.sel, layer.logits, None, layer.idx, layer.w)
    gone = (torch.rand(T, k, generator=gen(T)) < drop).cuda()
    kept_idx = layer.idx.clone()
    idx = torch.where(gone, -1, kept_idx).contiguous()
    for n in ("rows", "gate", "up", "h", "o", "y", "do", "dw", "dh", "dgate", "dup", "dlogits", "drows", "dx", "gwg", "gwu",
              "gwd", "gwr"):
        getattr(layer, n).fill_(math.nan)
    if keep:
        layer.codes.view(torch.uint8).fill_(0x7F)  # NaN
        layer.scales.fill_(math.nan)
    s, off = layer, layer.offsets
    used = off[E:]
    moe.moe_dispatch(s.dis, idx, s.x, None, s.rows, off, s.src, s.of, s.ws)
    moe.moe_matmul_bf16(s.up_mm, s.rows, s.wg, s.gate, off)
    moe.moe_matmul_bf16(s.up_mm, s.rows, s.wu, s.up, off)
    moe.moe_swiglu(s.act, s.gate, s.up, s.h, s.codes, s.scales, used)
    moe.moe_matmul_bf16(s.down_mm, s.h, s.wd, s.o, off)
    moe.moe_combine(s.com, s.o, s.of, s.w, s.y)
    moe.moe_combine_grad(s.com, s.dy, s.o, s.of, s.w, s.do, s.dw)
    moe.moe_matmul_bf16_dx(s.down_mm, s.do, s.wd, s.dh, off)
    g, u = (None, None) if keep else (s.gate, s.up)
    moe.moe_swiglu_grad(s.act, g, u, s.codes, s.scales, s.dh, s.dgate, s.dup, s.h, used)
    moe.moe_matmul_bf16_dw(s.down_f, s.do, s.h, s.gwd, off)
    moe.moe_matmul_bf16_dw(s.up_f, s.dgate, s.rows, s.gwg, off)
    moe.moe_matmul_bf16_dw(s.up_f, s.dup, s.rows, s.gwu, off)
    moe.moe_matmul_bf16_dx(s.up_mm, s.dgate, s.wg, s.drows, off)
    moe.moe_matmul_bf16_dx(s.up_mm, s.dup, s.wu, s.drows, off, s.drows)
    moe.moe_combine(s.com, s.drows, s.of, None, s.dx)
    moe.moe_select_grad(s.sel, s.logits, kept_idx, s.dw, None, s.dlogits)
    torch.cuda.synchronize()
    n = int((~gone).sum())
    assert int(off[E]) == n
    for name in ("rows", "gate", "up", "h", "o", "do", "dh", "dgate", "dup", "drows"):
        v = getattr(s, name)
        assert torch.isfinite(v[:n]).all() and torch.isnan(v[n:]).all(), name
    assert (s.dw[gone] == 0).all() and torch.isfinite(s.dlogits).all()
    there = torch.zeros(T, E, dtype=torch.bool, device="cuda").scatter_(1, kept_idx.long(), True)
    assert (s.dlogits[~there] == 0).all()

    # the definition, with the weights as moe_select made them
    d = lambda t: t.double().cpu().requires_grad_()  # noqa: E731
    x, wg, wu, wd, w = map(d, (s.x, s.wg, s.wu, s.wd, s.w))
    live = (~gone).double().cpu()
    y = torch.zeros(T, H, dtype=torch.float64)
    for j in range(k):
        e = kept_idx.cpu().long()[:, j]
        a, b = ((m[e] * x[:, None, :]).sum(2) for m in (wg, wu))
        y = y + (w * live)[:, j:j + 1] * (wd[e] * (a * torch.sigmoid(a) * b)[:, None, :]).sum(2)
    grads = torch.autograd.grad(y, (x, wg, wu, wd), s.dy.double().cpu())
    for name, want in zip(("y", "dx", "gwg", "gwu", "gwd"), (y.detach(),) + grads):
        got = getattr(s, name).double().cpu().view(want.shape)
        bar = (12 * 2.0 ** -8 + (3.3 * 2.0 ** -4 if keep and name != "y" else 0.0)) * float(want.norm())
        err = float((got - want).norm())
        print("%s: %.3g (bar %.3g)" % (name, err, bar), file=sys.stderr, flush=True)
        assert err <= bar, (name, err, bar)
