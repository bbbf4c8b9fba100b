"""The training operators in 64 bits, on the CPU, from their definitions in
include/moe.h.  Derivatives are written as formulas; tests/test_train_ref.py
checks them against differences of the forward definitions."""
from __future__ import annotations

import math

import torch

import ops_ref

U32, UBF = ops_ref.U32, ops_ref.UBF
BIG = 3.4028234663852886e38


def half_step(dtype):
    """Relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


# ---- dispatch and combine ------------------------------------------------------

def sort(idx, E):
    """(offsets [E + 1], row_src, row_of [T, k]) one pair after the other."""
    T, k = idx.shape
    lists = [[] for _ in range(E)]
    for p, e in enumerate(idx.flatten().tolist()):
        if 0 <= e < E:
            lists[e].append(p)
    offsets = [0]
    for l in lists:
        offsets.append(offsets[-1] + len(l))
    src = [p for l in lists for p in l]
    row_of = [-1] * (T * k)
    for r, p in enumerate(src):
        row_of[p] = r
    return (torch.tensor(offsets, dtype=torch.int32), torch.tensor(src, dtype=torch.int32),
            torch.tensor(row_of, dtype=torch.int32).view(T, k))


def combine(rows, row_of, w):
    """(y, sum of the magnitudes)."""
    T, k = row_of.shape
    y = torch.zeros(T, rows.shape[1], dtype=torch.float64)
    mag = torch.zeros_like(y)
    for t in range(T):
        for j in range(k):
            r = int(row_of[t, j])
            if 0 <= r < rows.shape[0]:
                v = rows[r].double() * (1.0 if w is None else float(w[t, j]))
                y[t] += v
                mag[t] += v.abs()
    return y, mag


def combine_grad(dy, rows, row_of, w):
    """(drows, dw, magnitude of dw's sums, rows that are named)."""
    T, k = row_of.shape
    drows = torch.zeros(rows.shape, dtype=torch.float64)
    dw = torch.zeros(T, k, dtype=torch.float64)
    mag = torch.zeros(T, k, dtype=torch.float64)
    named = torch.zeros(rows.shape[0], dtype=torch.bool)
    for t in range(T):
        for j in range(k):
            r = int(row_of[t, j])
            if 0 <= r < rows.shape[0]:
                named[r] = True
                drows[r] = dy[t].double() * (1.0 if w is None else float(w[t, j]))
                p = dy[t].double() * rows[r].double()
                dw[t, j], mag[t, j] = p.sum(), p.abs().sum()
    return drows, dw, mag, named


# ---- SwiGLU -------------------------------------------------------------------

def swiglu(gate, up):
    gate, up = gate.double(), up.double()
    return gate * torch.sigmoid(gate) * up


def swiglu_grad(gate, up, dh):
    """(dgate, dup, h)."""
    gate, up, dh = gate.double(), up.double(), dh.double()
    s = torch.sigmoid(gate)
    return dh * up * s * (1 + gate * (1 - s)), dh * gate * s, gate * s * up


# ---- selection ------------------------------------------------------------------

def _scores(l, b, score):
    """(scores with the share of every unmasked logit, which of them count)."""
    E = len(l)
    v = [min(x, BIG) if x > -math.inf else None for x in l]
    if score == "sigmoid":
        s = [0.0 if x is None else 1.0 / (1.0 + math.exp(-x)) if x > -709.78 else 0.0 for x in v]
    else:
        m = max([x for x in v if x is not None], default=0.0)
        ex = [0.0 if x is None else math.exp(x - m) for x in v]
        z = math.fsum(ex)
        s = [x / z if z else 0.0 for x in ex]
    return s, [v[e] is not None and b[e] > -math.inf for e in range(E)]


def _rest(x):
    """1 - sigmoid(x), which the difference in 64 bits loses from x = 37 on (1 - s < 2^-53)."""
    x = min(x, BIG)
    return 1.0 / (1.0 + math.exp(x)) if x < 700 else 0.0


def weights(l, b, idx, score, renorm, scale):
    """The weights of one token's slots."""
    s, on = _scores(l, b, score)
    w = [s[e] if 0 <= e < len(l) and on[e] else 0.0 for e in idx]
    total = math.fsum(w)
    if renorm:
        w = [x / total if total else 0.0 for x in w]
    return [x * scale for x in w]


def select_grad(logits, bias, idx, dw, dscore, score="softmax", renorm=True, scale=1.0):
    """(dlogits, a bound's size: the same sums of magnitudes)."""
    T, E = logits.shape
    out = torch.zeros(T, E, dtype=torch.float64)
    mag = torch.zeros(T, E, dtype=torch.float64)
    b = [0.0] * E if bias is None else bias.double().tolist()
    for t in range(T):
        s, on = _scores(logits[t].double().tolist(), b, score)
        rest = [_rest(x) if x > -math.inf else 1.0 for x in logits[t].double().tolist()]
        slots = [(e, scale * float(dw[t, j])) for j, e in enumerate(idx[t].tolist())
                 if 0 <= e < E and on[e] and s[e] > 0.0]
        g = [0.0] * E
        gm = [0.0] * E
        if renorm:
            total = math.fsum(s[e] for e, _ in slots)
            for e, d in slots:
                p = s[e] / total
                inner = [s[i] / total * (d - di) for i, di in slots]
                slope = 1.0 if score == "softmax" else rest[e]
                out[t, e] += p * slope * math.fsum(inner)
                mag[t, e] += p * slope * math.fsum(map(abs, inner))
        else:
            for e, d in slots:
                g[e] += d
                gm[e] += abs(d)
        if dscore is not None:
            for e in range(E):
                if on[e]:
                    g[e] += float(dscore[e])
                    gm[e] += abs(float(dscore[e]))
        # the product scale * dw and the sum with dscore round to 2^-24 of the addends' magnitudes (gm), not of
        # their sum, which may be smaller than either
        if dscore is not None or not renorm:
            if score == "softmax":
                top = max(range(E), key=lambda e: s[e])
                d = [x - g[top] for x in g]
                mean = math.fsum(s[e] * d[e] for e in range(E))
                mabs = math.fsum(s[e] * abs(d[e]) for e in range(E))
                for e in range(E):
                    out[t, e] += s[e] * (d[e] - mean)
                    mag[t, e] += s[e] * (abs(d[e]) + mabs + 2.0 ** -6 * (gm[e] + gm[top]))
            else:
                for e in range(E):
                    out[t, e] += g[e] * s[e] * rest[e]
                    mag[t, e] += gm[e] * s[e] * rest[e]
    return out, mag


# ---- products -------------------------------------------------------------------

def matmul(way, p, q, ends, add, shape):
    """The groups' products with the sums of magnitudes; rows outside the groups are NaN."""
    out = torch.full(shape, math.nan, dtype=torch.float64)
    mag = torch.zeros(shape, dtype=torch.float64)
    M = p.shape[0]
    for g, (lo, hi) in enumerate(zip(ends, ends[1:])):
        lo, hi = min(max(lo, 0), M), min(max(hi, 0), M)
        rows = slice(lo, max(lo, hi))
        a = p[rows].double()
        for dst, f in ((out, lambda x: x), (mag, torch.abs)):
            if way == "y":
                dst[rows] = f(a) @ f(q[g].double()).t()
            elif way == "dx":
                dst[rows] = f(a) @ f(q[g].double())
            else:
                dst[g] = f(a).t() @ f(q[rows].double())
    if add is not None:
        out, mag = out + add.double(), mag + add.double().abs()
    return out, mag
