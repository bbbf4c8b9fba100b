"""The oracle's derivatives against central differences of its forward
definitions, in 64 bits on the CPU.  A difference over 2h is off by h^2 / 6 of the
third derivative and by 2^-53 / h of the value: with h = 1e-5 both are below 1e-9
for the values of order 1 here."""
import pytest
import torch

import train_ref as ref

H, TOL = 1e-5, 1e-8


def differences(f, x):
    """Gradient of the number f(x) by differences, element by element."""
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        v = float(flat[i])
        flat[i] = v + H
        up = f(x)
        flat[i] = v - H
        o[i] = (up - f(x)) / (2 * H)
        flat[i] = v
    return out


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_sort_is_stable_and_leaves_empty_slots_out():
    idx = torch.tensor([[2, 0], [-1, 2], [5, 1], [2, 2]], dtype=torch.int32)
    offsets, src, row_of = ref.sort(idx, 3)
    assert offsets.tolist() == [0, 1, 2, 6]
    assert src.tolist() == [1, 5, 0, 3, 6, 7]
    assert row_of.tolist() == [[2, 0], [-1, 3], [-1, 1], [4, 5]]


@pytest.mark.parametrize("weighted", [False, True])
def test_combine_grad(weighted):
    row_of = torch.tensor([[3, -1, 0], [1, 4, 9], [-1, -1, -1]], dtype=torch.int32)
    rows, dy = randn(1, 6, 4), randn(2, 3, 4)
    w = randn(3, 3, 3) if weighted else None
    drows, dw, _, named = ref.combine_grad(dy, rows, row_of, w)
    assert named.tolist() == [True, True, False, True, True, False]
    loss = lambda r, f: float((ref.combine(r, row_of, f)[0] * dy).sum())  # noqa: E731
    assert torch.allclose(drows, differences(lambda r: loss(r, w), rows), atol=TOL, rtol=0)
    if weighted:
        assert torch.allclose(dw, differences(lambda f: loss(rows, f), w), atol=TOL, rtol=0)


def test_swiglu_grad():
    gate, up, dh = (randn(i, 3, 7) * 2 for i in range(3))
    dgate, dup, h = ref.swiglu_grad(gate, up, dh)
    assert torch.equal(h, ref.swiglu(gate, up))
    assert torch.allclose(dgate, differences(lambda g: float((ref.swiglu(g, up) * dh).sum()), gate), atol=TOL, rtol=0)
    assert torch.allclose(dup, differences(lambda u: float((ref.swiglu(gate, u) * dh).sum()), up), atol=TOL, rtol=0)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("balance", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_select_grad(score, renorm, balance, masked):
    T, E, k = 3, 7, 3
    l, dw = randn(1, T, E), randn(2, T, k)
    dscore = randn(3, E) if balance else None
    bias = torch.zeros(E, dtype=torch.float64)
    idx = torch.tensor([[0, 4, 2], [6, 1, 0], [3, -1, 5]])
    if masked:
        l[0, 4] = -float("inf")
        bias[1] = -float("inf")

    def loss(x):
        v = 0.0
        for t in range(T):
            row, b = x[t].tolist(), bias.tolist()
            slots = [e for e in idx[t].tolist()]
            w = ref.weights(row, b, slots, score, renorm, 2.5)
            v += sum(a * float(d) for a, d in zip(w, dw[t]))
            if dscore is not None:
                s, on = ref._scores(row, b, score)
                v += sum(float(dscore[e]) * s[e] for e in range(E) if on[e])
        return v

    got, _ = ref.select_grad(l, bias, idx, dw, dscore, score, renorm, 2.5)
    want = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        for e in range(E):
            if l[t, e] > -float("inf"):
                up, down = l.clone(), l.clone()
                up[t, e] += H
                down[t, e] -= H
                want[t, e] = (loss(up) - loss(down)) / (2 * H)
    assert torch.allclose(got, want, atol=TOL, rtol=0)


@pytest.mark.parametrize("groups", [[0, 5], [0, 2, 2, 4], [1, 3, 4, 5]])
def test_matmul_grads(groups):
    M, N, K, G = 5, 3, 4, len(groups) - 1
    x, w, dy = randn(1, M, K), randn(2, G, N, K), randn(3, M, N)
    used = torch.zeros(M, 1, dtype=torch.bool)
    used[groups[0]:groups[-1]] = True

    def loss(x, w):
        y, _ = ref.matmul("y", x, w, groups, None, (M, N))
        return float((torch.where(used, y, 0.0) * dy).sum())

    dx, _ = ref.matmul("dx", dy, w, groups, None, (M, K))
    dw, _ = ref.matmul("dw", dy, x, groups, None, (G, N, K))
    assert torch.allclose(torch.where(used, dx, 0.0), differences(lambda v: loss(v, w), x), atol=TOL, rtol=0)
    assert torch.allclose(dw, differences(lambda v: loss(x, v), w), atol=TOL, rtol=0)
