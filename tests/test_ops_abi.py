"""Refusals of the routing and FP8 operators, without a GPU: every call below
has one bad argument (pointers are made up and never followed), so nothing is
launched."""
import ctypes
import os

import pytest

import routed_expert_ffn_moe_amd as moe

P = ctypes.c_void_p
BASE = 0x7F0000000000


def ptr(i):
    return BASE + (i << 32)


def fails(rc, code, word):
    assert rc == code, (rc, moe.moe_last_error())
    assert word in moe.moe_last_error(), moe.moe_last_error()


# ---- moe_select ---------------------------------------------------------------

def call_select(logits=ptr(1), bias=None, idx=ptr(2), w=ptr(3), **kw):
    d = dict(T=4, E=256, top_k=8, n_group=8, topk_group=4, score=1, group_score=1, renorm=1,
             logit_dtype=0, scale=1.0, ld=0)
    d.update(kw)
    return moe.load().moe_select(ctypes.byref(moe.moe_select_t(**d)), logits, bias, idx, w, None)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025, n_group=1, topk_group=1), dict(top_k=0), dict(top_k=17),
    dict(E=8, top_k=9, n_group=1, topk_group=1), dict(score=2), dict(score=-1), dict(group_score=2),
    dict(logit_dtype=2), dict(logit_dtype=3), dict(n_group=0), dict(n_group=7), dict(n_group=128),
    dict(topk_group=0), dict(topk_group=9), dict(E=16, n_group=8, topk_group=1, top_k=3),
    dict(ld=255), dict(ld=-1), dict(logits=0), dict(idx=0), dict(logits=ptr(1) + 2),
    dict(idx=ptr(2) + 2), dict(w=ptr(3) + 1), dict(bias=ptr(4) + 2),
    dict(logits=ptr(1) + 1, logit_dtype=1),
])
def test_select_refusals(bad):
    fails(call_select(**bad), moe.MOE_EINVAL, "moe_select")


def test_select_null_struct_and_no_tokens():
    fails(moe.load().moe_select(None, ptr(1), None, ptr(2), None, None), moe.MOE_EINVAL, "moe_select")
    assert call_select(T=0, logits=0, idx=0) == moe.MOE_OK


# ---- moe_quant_fp8 --------------------------------------------------------------

def call_quant(x=ptr(1), codes=ptr(2), scales=ptr(3), **kw):
    d = dict(R=4, K=200, block_rows=1, src_dtype=1, ld=0)
    d.update(kw)
    return moe.load().moe_quant_fp8(ctypes.byref(moe.moe_quant_t(**d)), x, codes, scales, None)


@pytest.mark.parametrize("bad", [
    dict(R=-1), dict(K=0), dict(block_rows=0), dict(block_rows=64), dict(src_dtype=2), dict(ld=199),
    dict(R=1 << 30, K=1 << 20), dict(x=0), dict(codes=0), dict(scales=0), dict(x=ptr(1) + 1),
    dict(x=ptr(1) + 2, src_dtype=0), dict(codes=ptr(2) + 8), dict(scales=ptr(3) + 2),
    dict(codes=ptr(1) + 256), dict(scales=ptr(1)), dict(scales=ptr(2) + 64),
])
def test_quant_refusals(bad):
    fails(call_quant(**bad), moe.MOE_EINVAL, "moe_quant_fp8")


def test_quant_null_struct_and_no_rows():
    fails(moe.load().moe_quant_fp8(None, ptr(1), ptr(2), ptr(3), None), moe.MOE_EINVAL, "moe_quant_fp8")
    assert call_quant(R=0, x=0, codes=0, scales=0) == moe.MOE_OK


# ---- moe_matmul_fp8 -------------------------------------------------------------

def call_matmul(a=ptr(1), sa=ptr(2), b=ptr(3), sb=ptr(4), off=None, y=ptr(5), **kw):
    d = dict(M=8, N=96, K=200, G=1, out_dtype=1, lda=0, ldb=0, ldy=0)
    d.update(kw)
    return moe.load().moe_matmul_fp8(ctypes.byref(moe.moe_matmul_t(**d)), a, sa, b, sb, off, y, None)


@pytest.mark.parametrize("bad", [
    dict(M=-1), dict(N=0), dict(K=0), dict(G=0), dict(G=2), dict(G=65536, off=ptr(6)), dict(out_dtype=2),
    dict(out_dtype=3), dict(lda=200), dict(lda=264), dict(ldb=128), dict(ldb=260), dict(ldy=95),
    dict(N=1 << 30), dict(lda=1 << 25), dict(a=0), dict(sa=0), dict(b=0), dict(sb=0), dict(y=0),
    dict(a=ptr(1) + 8), dict(b=ptr(3) + 4), dict(sa=ptr(2) + 2), dict(sb=ptr(4) + 1),
    dict(off=ptr(6) + 2), dict(y=ptr(5) + 1), dict(y=ptr(5) + 2, out_dtype=0), dict(y=ptr(1)),
    dict(y=ptr(2)), dict(y=ptr(3)), dict(y=ptr(4)),
])
def test_matmul_refusals(bad):
    fails(call_matmul(**bad), moe.MOE_EINVAL, "moe_matmul_fp8")


def test_matmul_too_deep_null_struct_and_no_rows():
    fails(call_matmul(K=32769), moe.MOE_EUNSUPPORTED, "moe_matmul_fp8")
    fails(moe.load().moe_matmul_fp8(None, *[ptr(i) for i in range(1, 7)], None), moe.MOE_EINVAL,
          "moe_matmul_fp8")
    assert call_matmul(M=0, a=0, y=0) == moe.MOE_OK


# ---- moe_logits, moe_experts, FP8 layers ---------------------------------------------

def shape(**kw):
    d = dict(T=16, H=512, E=8, top_k=2, I=256, I_shared=0, chunk_T=0, act="bf16", w="fp8")
    d.update(kw)
    return moe.make_shape(**d)


def weights(**kw):
    d = dict(router_w=None, w_gate=ptr(1), w_up=ptr(2), w_down=ptr(3), s_gate=ptr(4), s_up=ptr(5),
             s_down=ptr(6), layout=moe.MOE_LAYOUT_ROWMAJOR)
    d.update(kw)
    return moe.moe_weights_t(**d)


def call_experts(sh=None, w=None, x=ptr(7), idx=ptr(8), tw=ptr(9), y=ptr(10), ws=ptr(11), nb=0):
    sh = shape() if sh is None else sh
    w = weights() if w is None else w
    return moe.load().moe_experts(ctypes.byref(sh), ctypes.byref(w), x, idx, tw, y, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(sh=shape(H=448)), moe.MOE_EINVAL), (dict(sh=shape(I=192)), moe.MOE_EINVAL),
    (dict(sh=shape(H=32896)), moe.MOE_EUNSUPPORTED), (dict(sh=shape(I=32896)), moe.MOE_EUNSUPPORTED),
    (dict(sh=shape(act="f32")), moe.MOE_EUNSUPPORTED), (dict(sh=shape(I_shared=256)), moe.MOE_EUNSUPPORTED),
    (dict(sh=shape(w="bf16", I_shared=256), w=weights(layout=1)), moe.MOE_EUNSUPPORTED),
    (dict(w=weights(layout=moe.MOE_LAYOUT_PACKED)), moe.MOE_EINVAL),
    (dict(w=weights(w_up=None)), moe.MOE_EINVAL), (dict(w=weights(s_down=None)), moe.MOE_EINVAL),
    (dict(w=weights(s_up=ptr(5) + 4)), moe.MOE_EINVAL), (dict(w=weights(w_gate=ptr(1) + 8)), moe.MOE_EINVAL),
    (dict(x=0), moe.MOE_EINVAL), (dict(y=0), moe.MOE_EINVAL), (dict(idx=0), moe.MOE_EINVAL),
    (dict(tw=0), moe.MOE_EINVAL), (dict(x=ptr(7) + 4), moe.MOE_EINVAL), (dict(idx=ptr(8) + 2), moe.MOE_EINVAL),
    (dict(ws=0), moe.MOE_EINVAL), (dict(ws=ptr(11) + 16), moe.MOE_EINVAL), (dict(nb=0), moe.MOE_EWORKSPACE),
    (dict(sh=shape(T=1 << 21, E=64, H=2048)), moe.MOE_EINVAL),
])
def test_experts_refusals(kw, code):
    assert call_experts(**kw) == code, moe.moe_last_error()
    assert moe.moe_last_error()


def test_experts_no_tokens_and_workspace():
    assert call_experts(sh=shape(T=0), x=0, idx=0, tw=0, y=0, ws=0) == moe.MOE_OK
    n = moe.moe_workspace_bytes(shape())
    # x codes, h codes and staging rows at least
    assert n >= 16 * 512 + 32 * 256 + 32 * 512 * 2
    assert moe.moe_workspace_bytes(shape(T=4096, chunk_T=16)) == n
    assert call_experts(nb=n - 1) == moe.MOE_EWORKSPACE
    assert moe.moe_workspace_bytes(shape(H=448)) == 0


def test_forward_takes_fp8_weights_row_major_only():
    sh = shape()
    w = weights(router_w=ptr(12), layout=moe.MOE_LAYOUT_PACKED)
    rc = moe.load().moe_forward(ctypes.byref(sh), ctypes.byref(w), ptr(7), ptr(10), ptr(8), None,
                                ptr(11), 1 << 40, None)
    fails(rc, moe.MOE_EINVAL, "row-major")


def test_logits_refusals():
    lib, sh = moe.load(), shape()
    w = weights(router_w=ptr(12))

    def call(w=w, x=ptr(7), out=ptr(8), sh=sh):
        return lib.moe_logits(ctypes.byref(sh), ctypes.byref(w), x, out, None)

    assert call(w=weights()) == moe.MOE_EINVAL
    assert call(w=weights(router_w=ptr(12) + 4)) == moe.MOE_EINVAL
    assert call(x=0) == moe.MOE_EINVAL
    assert call(out=0) == moe.MOE_EINVAL
    assert call(out=ptr(8) + 4) == moe.MOE_EINVAL
    assert call(sh=shape(E=0)) == moe.MOE_EINVAL
    assert call(sh=shape(T=0), x=0, out=0) == moe.MOE_OK


@pytest.mark.skipif(os.path.exists("/dev/kfd"),
                    reason="a GPU driver is present: a valid call would launch on made-up addresses")
def test_valid_calls_without_a_device_fail_loudly():
    for rc in (call_select(), call_quant(), call_matmul(),
               call_experts(nb=moe.moe_workspace_bytes(shape()))):
        assert rc == moe.MOE_EHIP
        assert "hipGetDevice" in moe.moe_last_error()


def test_binding_refuses_tensors_it_cannot_pass():
    import torch
    s = moe.make_select(4, 8, 2)
    cpu = torch.zeros(4, 8)
    i, w = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_select(s, cpu, None, i, w)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_select(s, cpu.half(), None, i, w)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_quant_fp8(moe.make_quant(4, 8, "f32"), cpu, i, w)
    with pytest.raises(ValueError, match="dtype"):
        moe.moe_matmul_fp8(moe.make_matmul(4, 4, 8), cpu, w, cpu, w, w)
    with pytest.raises(ValueError, match=r"\[R, K\]"):
        moe.quant_fp8(torch.zeros(4))
    with pytest.raises(ValueError, match="block_rows"):
        moe.quant_fp8(torch.zeros(2, 100, 128), block_rows=128)


@pytest.mark.parametrize("y", [ptr(6), ptr(6) + 4, ptr(6) - 8 * 96 * 2 + 2])
def test_matmul_refuses_a_y_that_overlaps_the_offsets(y):
    """Workgroups read the offsets while others store y."""
    fails(call_matmul(G=3, off=ptr(6), y=y), moe.MOE_EINVAL, "overlaps")
    assert call_matmul(G=3, off=ptr(6), y=ptr(6) + 16, M=0) == moe.MOE_OK


class OnGpu:
    """A CPU tensor that says it is on device 0, for the checks before a call."""

    def __init__(self, t):
        self.t, self.is_cuda = t, True

    def get_device(self):
        return 0

    def __getattr__(self, name):
        return getattr(self.t, name)


def fp8_parts(E=4, H=256, I=128, **kw):
    import torch
    f8 = torch.float8_e4m3fn
    d = dict(w_gate=torch.zeros(E, I, H, dtype=f8), w_up=torch.zeros(E, I, H, dtype=torch.uint8),
             w_down=torch.zeros(E, H, I, dtype=f8))
    for n, r, c in (("s_gate", I, H), ("s_up", I, H), ("s_down", H, I)):
        d[n] = torch.zeros(E, r // 128, c // 128)
    d.update(kw)
    return {n: t if t is None or isinstance(t, int) else OnGpu(t) for n, t in d.items()}


def test_binding_refuses_fp8_weights_that_the_shape_does_not_fit():
    """A matrix of fewer codes (packed 4-bit ones, say) or scales of one byte would be read out of range."""
    import torch
    u8, bf = torch.uint8, torch.bfloat16
    sh = moe.make_shape(2, 256, 4, 2, 128, w="fp8")
    fit = lambda **kw: moe._fp8_fit(sh, moe.make_weights(None, **fp8_parts(**kw)), 0)  # noqa: E731
    fit()
    fit(w_gate=torch.zeros(5, 128, 256, dtype=u8))   # a bank of more experts
    fit(s_up=None), fit(w_up=ptr(3))                 # NULL is the library's to refuse, a pointer the caller's to know
    for bad, word in [(dict(w_gate=torch.zeros(4, 128, 128, dtype=u8)), "w_gate"),
                      (dict(w_down=torch.zeros(3, 256, 128, dtype=u8)), "w_down"),
                      (dict(w_up=torch.zeros(4, 128, 256, dtype=bf)), "w_up"),
                      (dict(s_gate=torch.zeros(4, 1, 2, dtype=u8)), "s_gate"),
                      (dict(s_up=torch.zeros(4, 128, 8, dtype=u8)), "s_up"),
                      (dict(s_down=torch.zeros(4, 1, 1)), "s_down")]:
        with pytest.raises(ValueError, match=word):
            fit(**bad)
    with pytest.raises(ValueError, match="GPU"):
        moe._fp8_fit(sh, moe.make_weights(None, **{n: getattr(t, "t", t) for n, t in fp8_parts().items()}), 0)
    with pytest.raises(ValueError, match="cuda:0"):
        moe._fp8_fit(sh, moe.make_weights(None, **fp8_parts()), 1)


@pytest.mark.parametrize("call", ["moe_experts", "moe_forward", "moe_forward_noalloc"])
def test_calls_check_their_fp8_weights(call):
    import torch
    parts = {n: getattr(t, "t", t) for n, t in fp8_parts().items()}
    w = moe.make_weights(ptr(1), **parts)
    sh = moe.make_shape(2, 256, 4, 2, 128, w="fp8")
    args = {"moe_experts": (None, None, None, None, None), "moe_forward": (None, None, None, None, None),
            "moe_forward_noalloc": (None, None, None, None)}[call]
    with pytest.raises(ValueError, match="GPU"):
        getattr(moe, call)(sh, w, *args, stream=0)


def test_binding_refuses_single_rows_that_are_not_whole():
    """A row of `cols` elements lies in one row of a 2-D tensor that is not dense:
    the elements of its other rows (which may be the same ones) do not count."""
    import torch
    f32 = (torch.float32,)

    def mat(t, cols, rows=1):
        return moe._mat(OnGpu(t), "t", rows, cols, cols, f32, 0)

    buf = torch.zeros(4, 128)
    for good in (buf[:, :64], buf[1:2], buf, torch.zeros(64), torch.zeros(1, 64).expand(3, 64)):
        assert mat(good, 64) == good.data_ptr()
    for bad in (torch.zeros(1, 64).expand(2, 64), torch.zeros(80).as_strided((4, 40), (8, 1)), buf[:2, :64]):
        with pytest.raises(ValueError, match="holds"):
            mat(bad, 128)
    assert mat(buf, 128, rows=4) == buf.data_ptr()
    with pytest.raises(ValueError, match="holds|strides"):
        mat(buf[:, :64], 128, rows=2)


def test_experts_check_their_workspace_tensor():
    import torch
    sh = moe.make_shape(2, 256, 4, 2, 128, w="fp8")
    n = moe.moe_workspace_bytes(sh)
    ws = torch.zeros(n, dtype=torch.uint8)
    assert moe._workspace(OnGpu(ws), None, 0) == (ws.data_ptr(), n)
    assert moe._workspace(OnGpu(ws.view(torch.int16)), n - 256, 0) == (ws.data_ptr(), n - 256)
    assert moe._workspace(None, None, 0) == (None, 0)
    assert moe._workspace(ptr(1), n, 0) == (ptr(1), n)  # the caller's own pointer
    with pytest.raises(ValueError, match="GPU"):
        moe._workspace(ws, None, 0)
    with pytest.raises(ValueError, match="cuda:0"):
        moe._workspace(OnGpu(ws), None, 1)
    with pytest.raises(ValueError, match="holds"):
        moe._workspace(OnGpu(ws), n + 1, 0)
    with pytest.raises(ValueError, match="ws_bytes"):
        moe._workspace(ptr(1), None, 0)
    with pytest.raises(ValueError, match="GPU"):  # the call itself
        moe.moe_experts(sh, moe.make_weights(None, *(ptr(i) for i in (1, 2, 3)), s_gate=ptr(4), s_up=ptr(5),
                                             s_down=ptr(6)), None, None, None, None, ws, stream=0)


@pytest.mark.skipif(os.path.exists("/dev/kfd"),
                    reason="a GPU driver is present: a valid call would launch on made-up addresses")
@pytest.mark.parametrize("kw", [
    dict(T=1 << 20, H=4096, E=256, chunk_T=8192),           # as long as moe_forward's, in its passes
    dict(T=1 << 20, H=4096, E=256),
    dict(T=200000, H=4096, E=128, top_k=8, I=2048),         # rows of the experts do not count
    dict(T=1000, H=512, E=8, top_k=8, I=512 * 1024, w="bf16"),
])
def test_logits_take_any_number_of_tokens(kw):
    sh = shape(**kw)
    rc = moe.load().moe_logits(ctypes.byref(sh), ctypes.byref(weights(router_w=ptr(12))), ptr(7), ptr(8), None)
    fails(rc, moe.MOE_EHIP, "hipGetDevice")  # past every check


@pytest.mark.parametrize("bad", [dict(R=(1 << 31) - 1, K=1), dict(R=1 << 24, K=1 << 14), dict(R=(1 << 31) - 100, K=128)])
def test_quant_refuses_more_blocks_than_a_launch_has_threads_for(bad):
    """256 threads a block of 128 x 128; a grid of 2^32 threads would be launched short."""
    fails(call_quant(x=ptr(1), codes=ptr(200), scales=ptr(400), block_rows=128, **bad), moe.MOE_EINVAL, "blocks")
