"""The routing and FP8 operators in 64 bits, on the CPU, from their
definitions in include/moe.h, with bounds on what fp32 arithmetic may differ.

Tolerances count roundings: an fp32 operation is off by at most 2^-24 of its
result (2^-23 where it may truncate), a bf16 result by 2^-8.  The FP8 matrix
instruction cuts the products of 8 consecutive K to multiples of 2^-13 of the
largest one's power of two: at most 7 cuts of 2^-13 of the largest product,
which is at most the product of the two operands' largest magnitudes."""
from __future__ import annotations

import math

import torch

BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -100
U32, UBF = 2.0 ** -24, 2.0 ** -8


def padded(n: int) -> int:
    return -(-n // BLOCK) * BLOCK


# ---- select -----------------------------------------------------------------

def select(logits, bias, k, score="softmax", n_group=1, topk_group=1, group_score="max", renorm=True,
           scale=1.0):
    """(idx [T, k], w [T, k] float64) one token and one expert at a time."""
    L = logits.double().cpu()
    T, E = L.shape
    b = torch.zeros(E, dtype=torch.float64) if bias is None else bias.double().cpu()
    big = 3.4028234663852886e38
    idx = torch.zeros(T, k, dtype=torch.int32)
    w = torch.zeros(T, k, dtype=torch.float64)
    gs = E // n_group
    for t in range(T):
        l = [min(float(v), big) if float(v) > -math.inf else None for v in L[t]]
        live = [v for v in l if v is not None]
        if score == "sigmoid":
            s = [0.0 if v is None else 1.0 / (1.0 + math.exp(-v)) if v > -700 else 0.0 for v in l]
        else:
            m = max(live) if live else 0.0
            ex = [0.0 if v is None else math.exp(v - m) for v in l]
            z = math.fsum(ex)
            s = [v / z if z else 0.0 for v in ex]
        key = []
        for e in range(E):
            be = float(b[e])
            if l[e] is None or not be > -math.inf:
                key.append(-math.inf)
                s[e] = 0.0
            else:
                key.append(s[e] + min(be, big))
        keep = range(n_group)
        if n_group > 1:
            val = []
            for g in range(n_group):
                top = sorted(key[g * gs:(g + 1) * gs], reverse=True)
                two = [v for v in top[:2] if v > -math.inf]
                val.append(top[0] if group_score == "max" or len(two) < 2 else two[0] + two[1])
            keep = sorted(range(n_group), key=lambda g: (-val[g], g))[:topk_group]
        cand = [e for g in keep for e in range(g * gs, (g + 1) * gs)]
        pick = sorted(cand, key=lambda e: (-key[e], e))[:k]
        tot = math.fsum(s[e] for e in pick)
        for j, e in enumerate(pick):
            idx[t, j] = e
            w[t, j] = scale * (s[e] if not renorm else s[e] / tot if tot > 0 else 0.0)
    return idx, w


# ---- quantisation -----------------------------------------------------------

def e4m3_grid(v):
    """(nearest E4M3 value, ties to even, the step there, distance to the nearest midpoint) of float64 values."""
    a = v.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(a)) - 3)
    q = torch.round(v / step) * step
    mid = (torch.floor(v / step) + 0.5) * step
    return q.clamp(-E4M3_MAX, E4M3_MAX), step, (v - mid).abs()


def quant(x, rows=1):
    """(code values, scales, quotients), float64, of x [R, K]."""
    x = x.double().cpu()
    R, K = x.shape
    Rp, Kp = -(-R // rows) * rows, padded(K)
    p = torch.zeros(Rp, Kp, dtype=torch.float64)
    p[:R, :K] = x
    p = p.view(Rp // rows, rows, Kp // BLOCK, BLOCK)
    top = p.abs().amax((1, 3)).clamp(min=TINY)
    v = p * E4M3_MAX / top[:, None, :, None]
    q = e4m3_grid(v)[0]
    return q.view(Rp, Kp)[:R], top / E4M3_MAX, v.view(Rp, Kp)[:R]


def rows_value(codes, scales):
    return codes.cpu().double() * scales.cpu().double().repeat_interleave(BLOCK, 1)


def matrix_value(codes, scales):
    N = codes.shape[0]
    s = scales.cpu().double().repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)
    return codes.cpu().double() * s


# ---- product ----------------------------------------------------------------

def product(av, bv, narrow=False):
    """(a b^T, bound of an fp32 blockwise sum's error) of the values av [M, Kp], bv [N, Kp]; narrow: by
    the FP8 matrix instruction."""
    kb = av.shape[1] // BLOCK
    # inside a block 128 additions (2^-23 each), then the two scales' product,
    # its product with the block's sum and one addition per block
    tol = (2 * 128 + kb + 4) * U32 * (av.abs() @ bv.abs().t())
    if narrow:
        top = [v.abs().view(v.shape[0], -1, 8).amax(2) for v in (av, bv)]
        tol = tol + 7 * 2.0 ** -13 * (top[0] @ top[1].t())
    return av @ bv.t(), tol


# ---- experts ----------------------------------------------------------------

def experts(x, wg, sg, wu, su, wd, sd, idx, w):
    """(y, bound) of the FP8 experts on x [T, H] with given routing; matrices as codes [E, N, K] and
    scales.  The bound covers the fp32 sums, h codes whose quotient lies so near a midpoint that
    those sums' errors may move them by a step, the bf16 staging row of each slot and the bf16 y."""
    T, H = x.shape
    E = wg.shape[0]
    k = idx.shape[1]
    qx, sx, _ = quant(x)
    xv = rows_value(qx, sx)
    o = torch.zeros(T, k, H, dtype=torch.float64)
    tol = torch.zeros(T, k, H, dtype=torch.float64)
    for e in range(E):
        t, j = (idx.cpu() == e).nonzero(as_tuple=True)
        if not t.numel():
            continue
        g, dg = product(xv[t], matrix_value(wg[e], sg[e]), True)
        u, du = product(xv[t], matrix_value(wu[e], su[e]), True)
        sig = torch.sigmoid(g)
        h = g * sig * u
        # silu' <= 1.1; exponential, sum, reciprocal (2 units each) and two products: 8 roundings, and the
        # exponential's argument -g log2(e), off by 2^-24 of itself, moves it by |g| 2^-24
        dh = 1.1 * dg * u.abs() + (g * sig).abs() * du + 1.1 * dg * du + (8 + g.abs()) * U32 * h.abs()
        qh, sh, v = quant(h)
        _, step, off = e4m3_grid(v)
        # error of the quotient: that of h and of the block's maximum, and 4 roundings
        top = sh.repeat_interleave(BLOCK, 1) * E4M3_MAX
        dtop = dh.view(len(t), -1, BLOCK).amax(2).repeat_interleave(BLOCK, 1)
        dv = (dh * E4M3_MAX + v.abs() * dtop) / top + 4 * U32 * v.abs()
        flip = torch.where(off <= dv, step, torch.zeros_like(step)) * sh.repeat_interleave(BLOCK, 1)
        wv = matrix_value(wd[e], sd[e])
        hv = rows_value(qh, sh)
        oe, do = product(hv, wv, True)
        do = do + flip @ wv.abs().t() + (hv.abs() * dtop / top) @ wv.abs().t()
        o[t, j] = oe
        tol[t, j] = do + UBF * (oe.abs() + do)
    wt = w.double().cpu()
    y = (o * wt[:, :, None]).sum(1)
    bound = ((tol + (k + 2) * U32 * o.abs()) * wt.abs()[:, :, None]).sum(1)
    return y, bound + UBF * (y.abs() + bound)
