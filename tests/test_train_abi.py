"""Refusals of the training operators, without a GPU: every call below has one
bad argument (pointers are made up and never followed), so nothing is launched."""
import ctypes

import pytest

import routed_expert_ffn_moe_amd as moe

BASE = 0x7F0000000000


def ptr(i):
    return BASE + (i << 32)


def fails(rc, word, code=moe.MOE_EINVAL):
    assert rc == code, (rc, moe.moe_last_error())
    assert word in moe.moe_last_error(), moe.moe_last_error()


# ---- dispatch -------------------------------------------------------------------

def call_dispatch(idx=ptr(1), x=ptr(2), sx=None, rows=ptr(3), offsets=ptr(4), src=ptr(5), of=ptr(6), ws=ptr(7),
                  ws_bytes=1 << 30, **kw):
    d = dict(T=40000, H=200, E=64, top_k=2, x_dtype=1, row_dtype=1, ldx=0, ldr=0)
    d.update(kw)
    return moe.load().moe_dispatch(ctypes.byref(moe.moe_dispatch_t(**d)), idx, x, sx, rows, offsets, src, of, ws,
                                   ws_bytes, None)


SIZES = [dict(T=-1), dict(H=0), dict(H=(1 << 30) + 1, T=1), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=17),
         dict(T=(1 << 30) // 2 + 1), dict(x_dtype=2), dict(x_dtype=4), dict(x_dtype=0), dict(row_dtype=0),
         dict(x_dtype=3, row_dtype=3, sx=ptr(8)), dict(x_dtype=3, row_dtype=2, sx=ptr(8)), dict(ldx=199),
         dict(ldx=-1), dict(ldr=199), dict(ldx=(1 << 31) + 1), dict(ldr=(1 << 31) + 1),
         dict(x_dtype=3, sx=ptr(8), ldx=200), dict(x_dtype=3, sx=ptr(8), ldx=264)]


@pytest.mark.parametrize("bad", SIZES + [
    dict(idx=0), dict(offsets=0), dict(of=0), dict(x=0), dict(rows=0), dict(x_dtype=3, sx=None),
    dict(idx=ptr(1) + 2), dict(offsets=ptr(4) + 1), dict(src=ptr(5) + 2), dict(of=ptr(6) + 2), dict(x=ptr(2) + 1),
    dict(rows=ptr(3) + 1), dict(x_dtype=3, sx=ptr(8), x=ptr(2) + 8), dict(x_dtype=3, sx=ptr(8) + 2),
    dict(ws=0), dict(ws=ptr(7) + 16), dict(rows=ptr(2) + 400), dict(of=ptr(1)), dict(of=ptr(4) + 64), dict(src=ptr(6)),
    dict(ws=ptr(3)), dict(offsets=ptr(2)), dict(x_dtype=3, sx=ptr(3) + 64),
])
def test_dispatch_refusals(bad):
    fails(call_dispatch(**bad), "moe_dispatch")


def test_dispatch_workspace():
    d = moe.make_dispatch(40000, 200, 64, 2)
    need = moe.moe_dispatch_workspace_bytes(d)
    assert need >= 256
    fails(call_dispatch(ws_bytes=need - 1), "moe_dispatch", moe.MOE_EWORKSPACE)
    assert moe.moe_dispatch_workspace_bytes(moe.make_dispatch(4, 0, 64, 2)) == 0
    assert moe.moe_dispatch_workspace_bytes(moe.make_dispatch(1, 64, 64, 2)) >= 256


def call_gather(of=ptr(1), x=ptr(2), sx=None, rows=ptr(3), **kw):
    d = dict(T=40000, H=200, E=64, top_k=2, x_dtype=1, row_dtype=1, ldx=0, ldr=0)
    d.update(kw)
    return moe.load().moe_gather(ctypes.byref(moe.moe_dispatch_t(**d)), of, x, sx, rows, None)


@pytest.mark.parametrize("bad", SIZES + [dict(of=0), dict(of=ptr(1) + 2), dict(x=0), dict(rows=0), dict(rows=ptr(2)),
                                         dict(rows=ptr(1) + 4), dict(x_dtype=3, sx=None)])
def test_gather_refusals(bad):
    fails(call_gather(**bad), "moe_gather")


def test_no_tokens_and_null_structs():
    lib = moe.load()
    assert call_gather(T=0, of=0, x=0, rows=0) == moe.MOE_OK
    fails(lib.moe_dispatch(None, *[ptr(i) for i in range(8)], 1 << 20, None), "moe_dispatch")
    fails(lib.moe_gather(None, ptr(1), ptr(2), None, ptr(3), None), "moe_gather")
    fails(lib.moe_combine(None, ptr(1), ptr(2), None, ptr(3), None), "moe_combine")
    fails(lib.moe_combine_grad(None, *[ptr(i) for i in range(6)], None), "moe_combine_grad")
    fails(lib.moe_swiglu(None, ptr(1), ptr(2), None, ptr(3), None, None, None), "moe_swiglu")
    fails(lib.moe_swiglu_grad(None, *[ptr(i) for i in range(9)], None), "moe_swiglu_grad")
    fails(lib.moe_select_grad(None, *[ptr(i) for i in range(6)], 0, None), "moe_select_grad")
    for name in ("moe_matmul_bf16", "moe_matmul_bf16_dx", "moe_matmul_bf16_dw"):
        fails(getattr(lib, name)(None, ptr(1), ptr(2), None, None, ptr(3), None), name)


# ---- combine --------------------------------------------------------------------

def call_combine(rows=ptr(1), of=ptr(2), w=ptr(3), y=ptr(4), **kw):
    d = dict(T=5, H=100, top_k=2, R=10, dtype=1, ldr=0, ldy=0)
    d.update(kw)
    return moe.load().moe_combine(ctypes.byref(moe.moe_combine_t(**d)), rows, of, w, y, None)


C_SIZES = [dict(T=-1), dict(H=0), dict(H=(1 << 30) + 1), dict(top_k=0), dict(top_k=17), dict(R=-1), dict(dtype=2), dict(dtype=3),
           dict(ldr=99), dict(ldy=99), dict(ldy=-1), dict(ldr=(1 << 31) + 1), dict(T=1 << 30)]


@pytest.mark.parametrize("bad", C_SIZES + [
    dict(rows=0), dict(of=0), dict(y=0), dict(rows=ptr(1) + 1), dict(y=ptr(4) + 1), dict(of=ptr(2) + 2),
    dict(w=ptr(3) + 2), dict(dtype=0, y=ptr(4) + 2), dict(y=ptr(1) + 200), dict(y=ptr(2) - 500), dict(y=ptr(3))])
def test_combine_refusals(bad):
    fails(call_combine(**bad), "moe_combine")


def call_combine_grad(dy=ptr(1), rows=ptr(2), of=ptr(3), w=ptr(4), drows=ptr(5), dw=ptr(6), **kw):
    d = dict(T=5, H=100, top_k=2, R=10, dtype=1, ldr=0, ldy=0)
    d.update(kw)
    return moe.load().moe_combine_grad(ctypes.byref(moe.moe_combine_t(**d)), dy, rows, of, w, drows, dw, None)


@pytest.mark.parametrize("bad", C_SIZES + [
    dict(dy=0), dict(rows=0), dict(of=0), dict(dy=ptr(1) + 1), dict(rows=ptr(2) + 1), dict(drows=ptr(5) + 1),
    dict(of=ptr(3) + 2), dict(w=ptr(4) + 1), dict(dw=ptr(6) + 2), dict(drows=ptr(2)), dict(drows=ptr(1) + 100),
    dict(dw=ptr(4)), dict(dw=ptr(5) + 40), dict(dw=ptr(3))])
def test_combine_grad_refusals(bad):
    fails(call_combine_grad(**bad), "moe_combine_grad")


def test_combine_of_nothing():
    assert call_combine(T=0, rows=0, of=0, y=0) == moe.MOE_OK
    assert call_combine_grad(drows=None, dw=None, dy=0) == moe.MOE_OK


# ---- SwiGLU ---------------------------------------------------------------------

def call_swiglu(gate=ptr(1), up=ptr(2), used=None, h=ptr(3), codes=ptr(4), scales=ptr(5), **kw):
    d = dict(R=5, I=200, dtype=1, ld=0, ldh=0)
    d.update(kw)
    return moe.load().moe_swiglu(ctypes.byref(moe.moe_swiglu_t(**d)), gate, up, used, h, codes, scales, None)


S_SIZES = [dict(R=-1), dict(I=0), dict(R=1, I=(1 << 30) + 1), dict(dtype=2), dict(dtype=3), dict(ld=199), dict(ldh=199), dict(ld=-8),
           dict(ld=(1 << 31) + 1), dict(R=1 << 30)]


@pytest.mark.parametrize("bad", S_SIZES + [
    dict(gate=0), dict(up=0), dict(h=0), dict(codes=0), dict(scales=0), dict(gate=ptr(1) + 1), dict(up=ptr(2) + 1),
    dict(h=ptr(3) + 1), dict(codes=ptr(4) + 8), dict(scales=ptr(5) + 2), dict(used=ptr(6) + 2), dict(h=ptr(1)),
    dict(h=ptr(2) + 64), dict(codes=ptr(1)), dict(scales=ptr(4) + 64), dict(h=ptr(4)), dict(used=ptr(3) + 8)])
def test_swiglu_refusals(bad):
    fails(call_swiglu(**bad), "moe_swiglu")


def call_swiglu_grad(gate=ptr(1), up=ptr(2), codes=None, scales=None, dh=ptr(3), used=None, dgate=ptr(4), dup=ptr(5),
                     h=ptr(6), **kw):
    d = dict(R=5, I=200, dtype=1, ld=0, ldh=0)
    d.update(kw)
    return moe.load().moe_swiglu_grad(ctypes.byref(moe.moe_swiglu_t(**d)), gate, up, codes, scales, dh, used, dgate,
                                      dup, h, None)


@pytest.mark.parametrize("bad", S_SIZES + [
    dict(gate=0), dict(up=0), dict(dh=0), dict(dgate=0), dict(dup=0), dict(codes=ptr(7)), dict(scales=ptr(8)),
    dict(codes=ptr(7) + 8, scales=ptr(8)), dict(codes=ptr(7), scales=ptr(8) + 1), dict(dgate=ptr(1)),
    dict(dup=ptr(1) + 32), dict(dgate=ptr(3)), dict(h=ptr(3)), dict(h=ptr(4)), dict(dup=ptr(4) + 400),
    dict(dup=ptr(4) + 400, ld=399), dict(dup=ptr(4) + 398, ld=400), dict(dup=ptr(4) + 402, ld=400),
    dict(dup=ptr(4)), dict(dup=ptr(4), ld=400),
    dict(dgate=ptr(7), codes=ptr(7), scales=ptr(8)), dict(used=ptr(4)), dict(h=ptr(6) + 1), dict(dh=ptr(3) + 1)])
def test_swiglu_grad_refusals(bad):
    fails(call_swiglu_grad(**bad), "moe_swiglu_grad")


def test_swiglu_of_nothing():
    assert call_swiglu(R=0, gate=0, up=0, h=0) == moe.MOE_OK
    assert call_swiglu_grad(R=0, dh=0) == moe.MOE_OK


# ---- selection ------------------------------------------------------------------

def call_select_grad(logits=ptr(1), bias=None, idx=ptr(2), dw=ptr(3), dscore=None, dl=ptr(4), out=0, **kw):
    d = dict(T=4, E=256, top_k=8, n_group=1, topk_group=1, score=1, group_score=0, renorm=1, logit_dtype=0,
             scale=1.0, ld=0)
    d.update(kw)
    return moe.load().moe_select_grad(ctypes.byref(moe.moe_select_t(**d)), logits, bias, idx, dw, dscore, dl, out,
                                      None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025), dict(top_k=0), dict(top_k=17), dict(E=4, top_k=5), dict(score=2),
    dict(logit_dtype=2), dict(out=2), dict(out=-1), dict(ld=255), dict(ld=(1 << 31) + 1), dict(logits=0), dict(idx=0),
    dict(dw=0), dict(dl=0), dict(logits=ptr(1) + 2), dict(dl=ptr(4) + 2), dict(idx=ptr(2) + 1), dict(dw=ptr(3) + 2),
    dict(bias=ptr(5) + 2), dict(dscore=ptr(6) + 2), dict(dl=ptr(1)), dict(dl=ptr(2)), dict(dl=ptr(3) - 64),
    dict(bias=ptr(4) + 64), dict(dscore=ptr(4))])
def test_select_grad_refusals(bad):
    fails(call_select_grad(**bad), "moe_select_grad")


# ---- products -------------------------------------------------------------------

def call_matmul(name, a=ptr(1), b=ptr(2), offsets=ptr(3), add=None, out=ptr(4), **kw):
    d = dict(M=64, N=48, K=40, G=4, out_dtype=1, ldx=0, ldw=0, ldy=0)
    d.update(kw)
    return getattr(moe.load(), name)(ctypes.byref(moe.moe_matmul_bf16_t(**d)), a, b, offsets, add, out, None)


@pytest.mark.parametrize("name", ["moe_matmul_bf16", "moe_matmul_bf16_dx", "moe_matmul_bf16_dw"])
@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(M=(1 << 30) + 1), dict(N=(1 << 30) + 1, G=1), dict(K=(1 << 30) + 1, G=1), dict(G=0), dict(G=65536), dict(out_dtype=2), dict(out_dtype=3), dict(ldx=39),
    dict(ldw=39), dict(ldy=47), dict(ldx=-8), dict(ldw=(1 << 31) + 1), dict(offsets=0),
    dict(N=1 << 30, ldw=1 << 31, G=9), dict(M=1 << 30, N=1 << 20, K=1 << 20), dict(a=0), dict(b=0), dict(out=0),
    dict(a=ptr(1) + 1), dict(b=ptr(2) + 1), dict(out=ptr(4) + 1), dict(out_dtype=0, out=ptr(4) + 2),
    dict(offsets=ptr(3) + 2), dict(out_dtype=0, add=ptr(5) + 2), dict(out=ptr(1)), dict(out=ptr(2) + 64),
    dict(out=ptr(3)), dict(add=ptr(4) + 2)])
def test_matmul_bf16_refusals(name, bad):
    fails(call_matmul(name, **bad), name)


def test_matmul_bf16_of_no_rows():
    assert call_matmul("moe_matmul_bf16", M=0, a=0, b=0, out=0) == moe.MOE_OK
    assert call_matmul("moe_matmul_bf16_dx", M=0, a=0, b=0, out=0) == moe.MOE_OK
    fails(call_matmul("moe_matmul_bf16_dw", M=0, a=0, b=0, out=0), "moe_matmul_bf16_dw")


# ---- largest sizes ----------------------------------------------------------------

def test_more_rows_than_offsets_in_bytes_hold():
    rows, ld = (1 << 31) - 1, 1 << 31  # of 4 bytes: 2^64 - 2^33 bytes, a negative number of 64 bits
    fails(call_combine(R=rows, ldr=ld, dtype=0), "2^30")
    fails(call_combine_grad(R=rows, ldr=ld, dtype=0), "2^30")
    fails(call_swiglu(R=rows, I=8, ld=ld, ldh=ld, dtype=0), "2^30")
    fails(call_swiglu_grad(R=rows, I=8, ld=ld, ldh=ld, dtype=0), "2^30")
    fails(call_select_grad(T=rows, ld=ld), "2^30")
