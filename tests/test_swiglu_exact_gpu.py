"""SwiGLU of fp32 rows against 64 bits over every gate that fp32 tells apart from 0 and 1: the
bounds count the roundings of the sigmoid s, of its rest 1 - s and of the products."""
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import routed_expert_ffn_moe_amd as moe  # noqa: E402

STEP = 2.0 ** -24    # one rounding
ULP = 2.0 ** -23     # the exponential and the hardware's reciprocal
LEAST = 2.0 ** -149  # what fp32 leaves of a value below its normal ones


def rows():
    """(gate, up, dh): gates of every size, the up and dh of small gates so large that results are ordinary numbers."""
    g = torch.Generator().manual_seed(5)
    gate = torch.cat([
        torch.randn(2000, generator=g) * 3,
        torch.linspace(7.0, 30.0, 3001),        # 1 - s small, s next to 1
        torch.linspace(-30.0, -7.0, 1001),
        torch.linspace(-1.35, -1.2, 301),       # the slope passes 0
        torch.linspace(-87.2, -60.0, 1001),
        torch.linspace(-102.0, -87.3, 1001),    # s below the normal numbers
        torch.tensor([0.0, -0.0, 1e-40, -1e-40, 90.0, 200.0, 3e38, -110.0, -3e38])])
    up, dh = torch.randn(gate.numel(), generator=g), torch.randn(gate.numel(), generator=g)
    far = gate < -60
    up[far], dh[far] = up[far] * 2.0 ** 60, dh[far] * 2.0 ** 40
    up[gate > 1e30] = 0.5  # h stays finite
    n = gate.numel() // 16 * 16
    return tuple(t[-n:].view(16, -1) for t in (gate, up, dh))


def sigmoid(g):
    """(s, 1 - s) without cancellation."""
    e = torch.exp(-g.abs())
    return torch.where(g < 0, e, torch.ones_like(e)) / (1 + e), torch.where(g < 0, torch.ones_like(e), e) / (1 + e)


def errors(g):
    """(error of s, of 1 - s, of gate * s), as they come from e = exp(-|gate|) and r = 1 / (1 + e).  r: the sum's
    rounding and the reciprocal's ulp (e's own error, e / (1 + e) of itself, counts as one more ulp), e * r: that
    and the rounding of the product."""
    s, c = sigmoid(g)
    r = STEP + 2 * ULP
    er = r + ULP + STEP
    ds = s * torch.where(g < 0, er, r) + torch.where(g < 0, 3 * LEAST, 0.0)
    dc = c * torch.where(g < 0, r, er) + torch.where(g < 0, 0.0, 3 * LEAST)
    return ds, dc, g.abs() * ds + (g * s).abs() * STEP + LEAST


def within(got, want, bound, what):
    got = got.cpu()
    over = want.float().isinf()  # 3e38 times more than 1.13 is beyond fp32, whose rounding of it is infinite
    assert torch.equal(got[over], want.float()[over]), what
    d = torch.where(over, 0.0, (got.double() - want).abs())
    print("[%s] largest error %.3g of its bound" % (what, float((d / bound).max())), file=sys.stderr, flush=True)
    assert bool((d <= bound * 1.001 + LEAST).all()), (what, float((d / bound).max()))


def test_swiglu_of_every_gate():
    gate, up, dh = rows()
    g, u, d = gate.double(), up.double(), dh.double()
    s, c = sigmoid(g)
    ds, dc, dz = errors(g)
    z = g * s
    n = moe.make_swiglu(*gate.shape, dtype="f32")
    h, again, da, db = (torch.empty_like(gate, device="cuda") for _ in range(4))
    moe.moe_swiglu(n, gate.cuda(), up.cuda(), h)
    moe.moe_swiglu_grad(n, gate.cuda(), up.cuda(), None, None, dh.cuda(), da, db, again)
    within(h, z * u, u.abs() * dz + (z * u).abs() * STEP, "h")
    within(again, z * u, u.abs() * dz + (z * u).abs() * STEP, "h again")
    within(db, d * z, d.abs() * dz + (d * z).abs() * STEP, "dup")
    # s + z (1 - s), one rounding of the sum; then two products
    slope = s + z * c
    dslope = ds + dz * c + z.abs() * dc + slope.abs() * STEP
    within(da, d * u * slope, (d * u).abs() * (dslope + 2 * STEP * slope.abs()), "dgate")
