"""Python binding of libmoe.so, the gfx950 routed-expert MoE FFN layer.

Argument marshalling only: torch tensors are passed by device pointer and
every step of the layer runs in the library's HIP kernels.  The functions
carry the names of the C entry points declared in ``include/moe.h``.

The library must have been built (``python -m routed_expert_ffn_moe_amd.build``);
importing the binding does not build it, and every call fails loudly when the
library is missing.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

__all__ = [
    "MOE_F32", "MOE_BF16", "MOE_MXFP4", "MOE_FP8", "MOE_LAYOUT_ROWMAJOR", "MOE_LAYOUT_PACKED", "MOE_OK",
    "MOE_EINVAL", "MOE_EWORKSPACE", "MOE_EUNSUPPORTED", "MOE_EHIP", "MoeError", "moe_shape_t", "moe_weights_t", "make_shape",
    "make_weights", "moe_workspace_bytes", "moe_forward", "moe_forward_noalloc",
    "MOE_NOALLOC_SCRATCH_BYTES", "moe_route", "moe_strerror",
    "moe_last_error", "moe_stage_timing_enable", "moe_stage_timing_read", "moe_pack_bf16",
    "pack_bf16", "moe_pack_mxfp4", "pack_mxfp4", "STAGES", "moe_probe_read", "moe_probe_mfma",
    "moe_probe_gather", "moe_probe_mxfp4",
    "MOE_SCORE_SOFTMAX", "MOE_SCORE_SIGMOID", "MOE_GROUP_MAX", "MOE_GROUP_TOP2", "moe_select_t",
    "moe_quant_t", "moe_matmul_t", "make_select", "make_quant", "make_matmul", "moe_logits",
    "moe_select", "moe_experts", "moe_quant_fp8", "quant_fp8", "moe_matmul_fp8",
    "moe_dispatch_t", "moe_combine_t", "moe_swiglu_t", "moe_matmul_bf16_t", "make_dispatch", "make_combine",
    "make_swiglu", "make_matmul_bf16", "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_gather",
    "moe_combine", "moe_combine_grad", "moe_swiglu", "moe_swiglu_grad", "moe_select_grad", "moe_matmul_bf16",
    "moe_matmul_bf16_dx", "moe_matmul_bf16_dw", "moe_matmul_bf16_tile",
    "lib_path", "load",
]

MOE_F32, MOE_BF16, MOE_MXFP4, MOE_FP8 = 0, 1, 2, 3
MOE_LAYOUT_ROWMAJOR, MOE_LAYOUT_PACKED = 0, 1
MOE_OK, MOE_EINVAL, MOE_EWORKSPACE, MOE_EUNSUPPORTED, MOE_EHIP = 0, -1, -2, -3, -4
_DT = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp4": MOE_MXFP4, "fp8": MOE_FP8}
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_GROUP_MAX, MOE_GROUP_TOP2 = 0, 1

_HERE = os.path.dirname(os.path.abspath(__file__))


def lib_path() -> str:
    return os.path.join(_HERE, "libmoe.so")


class MoeError(RuntimeError):
    def __init__(self, code: int, detail: str):
        super().__init__("%s (%d): %s" % (moe_strerror(code), code, detail))
        self.code = code


class moe_shape_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "H", "E", "top_k", "I", "I_shared", "chunk_T", "act_dtype", "w_dtype")]


class moe_weights_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("router_w", "router_bias", "w_gate", "w_up", "w_down", "s_gate", "s_up",
                 "s_down", "sh_gate", "sh_up", "sh_down")] + [("layout", ctypes.c_int32)]


class moe_select_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("T", "E", "top_k", "n_group", "topk_group", "score", "group_score", "renorm",
                 "logit_dtype")] + [("scale", ctypes.c_float), ("ld", ctypes.c_int64)]


class moe_quant_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "K", "block_rows", "src_dtype")] + \
        [("ld", ctypes.c_int64)]


class moe_matmul_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "G", "out_dtype")] + \
        [(n, ctypes.c_int64) for n in ("lda", "ldb", "ldy")]


class moe_dispatch_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "E", "top_k", "x_dtype", "row_dtype")] + \
        [(n, ctypes.c_int64) for n in ("ldx", "ldr")]


class moe_combine_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "H", "top_k", "R", "dtype")] + \
        [(n, ctypes.c_int64) for n in ("ldr", "ldy")]


class moe_swiglu_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "I", "dtype")] + \
        [(n, ctypes.c_int64) for n in ("ld", "ldh")]


class moe_matmul_bf16_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("M", "N", "K", "G", "out_dtype")] + \
        [(n, ctypes.c_int64) for n in ("ldx", "ldw", "ldy")]


_lib = None


def load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        path = lib_path()
        if not os.path.exists(path):
            raise RuntimeError("libmoe.so is not built: run `python -m routed_expert_ffn_moe_amd.build`")
        # torch ships its own HIP runtime (file libamdhip64.so, soname
        # libamdhip64.so.7).  Loaded first, it is the one libmoe.so binds to.
        # Loaded after libmoe.so, torch would bring a second runtime into the
        # process beside ROCm's, and the two cannot both own the device: the
        # library's calls would then fail with "no ROCm-capable device".
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        lib = ctypes.CDLL(path)
        P = ctypes.c_void_p
        lib.moe_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_workspace_bytes.argtypes = [P]
        lib.moe_forward.restype = ctypes.c_int
        lib.moe_forward.argtypes = [P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_forward_noalloc.restype = ctypes.c_int
        lib.moe_forward_noalloc.argtypes = [P, P, P, P, P, P, P]
        lib.moe_route.restype = ctypes.c_int
        lib.moe_route.argtypes = [P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_strerror.restype = ctypes.c_char_p
        lib.moe_strerror.argtypes = [ctypes.c_int]
        lib.moe_last_error.restype = ctypes.c_char_p
        lib.moe_last_error.argtypes = []
        lib.moe_stage_timing_enable.restype = ctypes.c_int
        lib.moe_stage_timing_enable.argtypes = [ctypes.c_int]
        lib.moe_stage_timing_read.restype = ctypes.c_int
        lib.moe_stage_timing_read.argtypes = [P, ctypes.c_int, P]
        lib.moe_pack_bf16.restype = ctypes.c_int
        lib.moe_pack_bf16.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, P, P, P]
        lib.moe_pack_mxfp4.restype = ctypes.c_int
        lib.moe_pack_mxfp4.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int, P, P, P, P, P]
        lib.moe_probe_read.restype = ctypes.c_int
        lib.moe_probe_read.argtypes = [P, ctypes.c_size_t, P]
        lib.moe_probe_mfma.restype = ctypes.c_int
        lib.moe_probe_mfma.argtypes = [ctypes.c_int, ctypes.c_int, P, P]
        lib.moe_probe_gather.restype = ctypes.c_int
        lib.moe_probe_gather.argtypes = [P, ctypes.c_size_t, ctypes.c_size_t, P, ctypes.c_int,
                                         ctypes.c_int, P]
        lib.moe_probe_mxfp4.restype = ctypes.c_int
        lib.moe_probe_mxfp4.argtypes = [P, P, ctypes.c_size_t, ctypes.c_int, P, P]
        lib.moe_logits.restype = ctypes.c_int
        lib.moe_logits.argtypes = [P, P, P, P, P]
        lib.moe_select.restype = ctypes.c_int
        lib.moe_select.argtypes = [P, P, P, P, P, P]
        lib.moe_experts.restype = ctypes.c_int
        lib.moe_experts.argtypes = [P, P, P, P, P, P, P, ctypes.c_size_t, P]
        lib.moe_quant_fp8.restype = ctypes.c_int
        lib.moe_quant_fp8.argtypes = [P, P, P, P, P]
        lib.moe_matmul_fp8.restype = ctypes.c_int
        lib.moe_matmul_fp8.argtypes = [P, P, P, P, P, P, P, P]
        lib.moe_dispatch_workspace_bytes.restype = ctypes.c_size_t
        lib.moe_dispatch_workspace_bytes.argtypes = [P]
        lib.moe_dispatch.argtypes = [P] * 9 + [ctypes.c_size_t, P]
        lib.moe_gather.argtypes = [P] * 6
        lib.moe_combine.argtypes = [P] * 6
        lib.moe_combine_grad.argtypes = [P] * 8
        lib.moe_swiglu.argtypes = [P] * 8
        lib.moe_swiglu_grad.argtypes = [P] * 11
        lib.moe_select_grad.argtypes = [P] * 7 + [ctypes.c_int, P]
        for name in ("moe_matmul_bf16", "moe_matmul_bf16_dx", "moe_matmul_bf16_dw"):
            getattr(lib, name).argtypes = [P] * 7
        lib.moe_matmul_bf16_tile.argtypes = [P, ctypes.c_int, ctypes.c_int, P]
        _lib = lib
    return _lib


def _ptr(t) -> Optional[int]:
    """Device pointer of a tensor (None -> NULL; ints pass through)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe must be contiguous")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(T, H, E, top_k, I, I_shared=0, chunk_T=0, act="bf16", w="bf16") -> moe_shape_t:
    return moe_shape_t(T, H, E, top_k, I, I_shared, chunk_T, _DT[act], _DT[w])


class _Weights:
    """moe_weights_t plus references keeping the tensors alive."""

    def __init__(self, layout, **tensors):
        self._keep = tensors
        self.c = moe_weights_t(**{k: _ptr(v) for k, v in tensors.items()}, layout=layout)
        # what lies behind those pointers, and the FP8 sizes (E, H, I, device) found to fit it
        self._held = {k: (v.dtype, v.numel(), v.get_device()) for k, v in tensors.items()
                      if v is not None and not isinstance(v, int)}
        self._fits = set()


def _is_packed(t) -> bool:
    return t is not None and getattr(t, "_moe_layout", None) == "packed"


def make_weights(router_w, w_gate, w_up, w_down, router_bias=None, s_gate=None, s_up=None,
                 s_down=None, sh_gate=None, sh_up=None, sh_down=None, layout=None) -> _Weights:
    """The weight struct.  `layout` (MOE_LAYOUT_*) defaults to PACKED when
    every expert matrix given came out of pack_bf16 / pack_mxfp4, else
    ROWMAJOR; the library refuses bf16 / MXFP4 matrices declared ROWMAJOR."""
    if layout is None:
        mats = [m for m in (w_gate, w_up, w_down, sh_gate, sh_up, sh_down) if m is not None]
        layout = MOE_LAYOUT_PACKED if all(_is_packed(m) for m in mats) else MOE_LAYOUT_ROWMAJOR
    return _Weights(layout, router_w=router_w, router_bias=router_bias, w_gate=w_gate, w_up=w_up,
                    w_down=w_down, s_gate=s_gate, s_up=s_up, s_down=s_down, sh_gate=sh_gate,
                    sh_up=sh_up, sh_down=sh_down)


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, moe_last_error())


def _fp8_fit(s, weights, dev) -> None:
    """Refuse expert matrices and scales that an FP8 shape would read out of
    range: of another type, on another device, or of fewer elements."""
    key = (s.E, s.H, s.I, dev)
    if s.w_dtype != MOE_FP8 or key in weights._fits:
        return
    if _SRC is None:
        _types()
    for name in ("w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down"):
        if name not in weights._held:  # NULL, which the library refuses, or the caller's own pointer
            continue
        dtype, held, on = weights._held[name]
        types, block = (_CODES, 1) if name[0] == "w" else (_F32, 128)
        if dtype not in types:
            raise ValueError("%s: dtype %s, expected %s" % (name, dtype, " or ".join(map(str, types))))
        if on < 0:
            raise ValueError("%s is not on a GPU" % name)
        if on != dev:
            raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (name, on, dev))
        need = s.E * (s.H // block) * (s.I // block)
        if held < need:
            raise ValueError("%s holds %d elements, E=%d, H=%d, I=%d take %d" % (name, held, s.E, s.H, s.I, need))
    weights._fits.add(key)


def moe_workspace_bytes(shape: moe_shape_t) -> int:
    return int(load().moe_workspace_bytes(ctypes.byref(shape)))


def moe_forward(shape, weights, x, y, topk_idx, topk_w, ws, ws_bytes=None, stream=None) -> None:
    """y[T,H] and the routing of x[T,H]; asynchronous on `stream`."""
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    if shape.w_dtype == MOE_FP8:
        _fp8_fit(shape, weights, _begin(stream)[1])
    _check(load().moe_forward(ctypes.byref(shape), ctypes.byref(weights.c), _ptr(x), _ptr(y),
                              _ptr(topk_idx), _ptr(topk_w), _ptr(ws), ws_bytes,
                              _stream(stream)))


MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


def moe_forward_noalloc(shape, weights, x, y, topk_idx, topk_w, stream=None) -> None:
    """moe_forward on the library's static device scratch (allocates nothing)."""
    if shape.w_dtype == MOE_FP8:
        _fp8_fit(shape, weights, _begin(stream)[1])
    _check(load().moe_forward_noalloc(ctypes.byref(shape), ctypes.byref(weights.c), _ptr(x),
                                      _ptr(y), _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


def moe_route(shape, weights, x, topk_idx, topk_w, counts, offsets, row_src, ws, ws_bytes=None,
              stream=None) -> None:
    """Router and permutation of one pass (see include/moe.h)."""
    if ws_bytes is None:
        ws_bytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().moe_route(ctypes.byref(shape), ctypes.byref(weights.c), _ptr(x),
                            _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                            _ptr(row_src), _ptr(ws), ws_bytes, _stream(stream)))


def moe_pack_bf16(E, N, K, w, w_out, stream=None) -> None:
    """Repack row-major bf16 matrices [E, N, K] into the layout moe_forward reads."""
    _check(load().moe_pack_bf16(E, N, K, _ptr(w), _ptr(w_out), _stream(stream)))


def pack_bf16(w, stream=None):
    """Packed copy of a bf16 device tensor [E, N, K] or [N, K]."""
    import torch
    E, N, K = (1, *w.shape) if w.dim() == 2 else w.shape
    out = torch.empty_like(w)
    moe_pack_bf16(E, N, K, w, out, stream)
    out._moe_layout = "packed"
    return out


def moe_pack_mxfp4(E, N, K, codes, scales, codes_out, scales_out, stream=None) -> None:
    """Repack OCP row-major MXFP4 matrices into the layout moe_forward reads."""
    _check(load().moe_pack_mxfp4(E, N, K, _ptr(codes), _ptr(scales), _ptr(codes_out),
                                 _ptr(scales_out), _stream(stream)))


def pack_mxfp4(codes, scales, stream=None):
    """Packed copies of codes [E, N, K/2] and scales [E, N, K/32] (uint8 device tensors)."""
    import torch
    E, N, K2 = codes.shape
    out_c = torch.empty_like(codes)
    out_s = torch.empty_like(scales)
    moe_pack_mxfp4(E, N, 2 * K2, codes, scales, out_c, out_s, stream)
    out_c._moe_layout = out_s._moe_layout = "packed"
    return out_c, out_s


def make_select(T, E, top_k, score="softmax", n_group=1, topk_group=1, group_score="max", renorm=True,
                scale=1.0, logits="f32", ld=0) -> moe_select_t:
    return moe_select_t(T, E, top_k, n_group, topk_group,
                        {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}[score],
                        {"max": MOE_GROUP_MAX, "top2": MOE_GROUP_TOP2}[group_score], int(renorm),
                        _DT[logits], scale, ld)


def make_quant(R, K, src="bf16", block_rows=1, ld=0) -> moe_quant_t:
    return moe_quant_t(R, K, block_rows, _DT[src], ld)


def make_matmul(M, N, K, G=1, out="bf16", lda=0, ldb=0, ldy=0) -> moe_matmul_t:
    return moe_matmul_t(M, N, K, G, _DT[out], lda, ldb, ldy)


# The operators below check what they are given (these calls are short: the
# ordinary tensor is passed after four comparisons).

def _types():
    """Element types by moe_dtype_t, once torch is there (load() imports it)."""
    global _SRC, _F32, _I32, _CODES
    import torch
    _SRC = {MOE_F32: (torch.float32,), MOE_BF16: (torch.bfloat16,)}
    _F32, _I32 = (torch.float32,), (torch.int32,)
    _CODES = (torch.float8_e4m3fn, torch.uint8)


_SRC = _F32 = _I32 = _CODES = None
_device = _raw_stream = None


def _begin(stream):
    """(library, current device, stream handle) of a call."""
    global _device, _raw_stream
    lib = _lib
    if lib is None:
        lib = load()
    if _device is None:
        import torch
        _types()
        if torch.cuda.is_available():
            torch.cuda.current_device()  # initialised from here on
            _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        else:
            _device = lambda: -1  # noqa: E731
        # the current stream's handle without building a Stream object
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    dev = _device()
    if stream is None:
        if dev < 0:
            return lib, dev, None
        return lib, dev, _raw_stream(dev) if _raw_stream else _stream(None)
    return lib, dev, _stream(stream)


def _mat(t, what, rows, cols, ld, types, dev) -> Optional[int]:
    """Device pointer of a tensor that a call reads or writes as `rows` rows
    of `cols` elements, `ld` apart (None -> NULL): of one of `types`, on the
    current device, and laid out so - dense, or 2-D with that row stride."""
    if t is None:
        return None
    if t.dtype in types and t.get_device() == dev and ld == cols and t.is_contiguous() and \
            t.numel() == rows * cols and dev >= 0:
        return t.data_ptr()
    return _mat_checked(t, what, rows, cols, ld, types, dev)


def _mat_checked(t, what, rows, cols, ld, types, dev):
    if t.dtype not in types:
        raise ValueError("%s: dtype %s, expected %s" % (what, t.dtype, " or ".join(map(str, types))))
    if not t.is_cuda:
        raise ValueError("%s is not on a GPU" % what)
    if t.get_device() != dev:
        raise ValueError("%s is on cuda:%d, the current device is cuda:%d" % (what, t.get_device(), dev))
    if rows <= 0 or cols <= 0:
        return t.data_ptr()
    need = (rows - 1) * ld + cols
    if t.dim() == 2 and rows > 1:
        # also a wider or longer tensor whose rows begin where the call's do
        ok = t.stride(0) == ld and (t.stride(1) == 1 or t.shape[1] == 1) and t.shape[1] >= cols
        held = t.stride(0) * (t.shape[0] - 1) + t.shape[1]
    else:
        ok = t.is_contiguous() or (t.dim() == 2 and t.stride(1) == 1)
        held = t.numel() if t.is_contiguous() else t.shape[1] if t.dim() == 2 else 0
    if not ok:
        raise ValueError("%s: strides %s, the call takes rows of %d elements, %d apart"
                         % (what, tuple(t.stride()), cols, ld))
    if held < need:
        raise ValueError("%s holds %d elements, the call needs %d" % (what, held, need))
    return t.data_ptr()


def moe_logits(shape, weights, x, logits, stream=None) -> None:
    """The router's logits [T, E] (float32) of x[T, H]."""
    lib, dev, st = _begin(stream)
    s = shape
    _check(lib.moe_logits(ctypes.byref(s), ctypes.byref(weights.c),
                          _mat(x, "x", s.T, s.H, s.H, _SRC.get(s.act_dtype, _CODES), dev),
                          _mat(logits, "logits", s.T, s.E, s.E, _F32, dev), st))


def moe_select(select, logits, bias, topk_idx, topk_w, stream=None) -> None:
    """topk_idx, topk_w [T, top_k] of the tokens with these logits (see include/moe.h)."""
    lib, dev, st = _begin(stream)
    s = select
    T, E, k = s.T, s.E, s.top_k
    rc = lib.moe_select(ctypes.byref(s),
                        _mat(logits, "logits", T, E, s.ld or E, _SRC.get(s.logit_dtype, _F32), dev),
                        _mat(bias, "bias", 1, E, E, _F32, dev),
                        _mat(topk_idx, "topk_idx", T, k, k, _I32, dev),
                        _mat(topk_w, "topk_w", T, k, k, _F32, dev), st)
    if rc:
        _check(rc)


def _workspace(ws, ws_bytes, dev):
    """(device pointer, bytes) of a workspace tensor; a caller's own pointer comes with its ws_bytes."""
    if ws is None or isinstance(ws, int):
        if ws and ws_bytes is None:
            raise ValueError("ws is a pointer: ws_bytes says how much lies behind it")
        return ws, ws_bytes or 0
    if not ws.is_cuda:
        raise ValueError("ws is not on a GPU")
    if ws.get_device() != dev:
        raise ValueError("ws is on cuda:%d, the current device is cuda:%d" % (ws.get_device(), dev))
    held = ws.numel() * ws.element_size()
    if ws_bytes is None:
        ws_bytes = held
    elif ws_bytes > held:
        raise ValueError("ws holds %d bytes, ws_bytes is %d" % (held, ws_bytes))
    return _ptr(ws), ws_bytes


def moe_experts(shape, weights, x, topk_idx, topk_w, y, ws, ws_bytes=None, stream=None) -> None:
    """y[T, H] of the routed experts with given routing (see include/moe.h)."""
    lib, dev, st = _begin(stream)
    s = shape
    T, H, k = s.T, s.H, s.top_k
    ws, ws_bytes = _workspace(ws, ws_bytes, dev)
    src = _SRC.get(s.act_dtype, _CODES)
    if s.w_dtype == MOE_FP8:
        _fp8_fit(s, weights, dev)
    rc = lib.moe_experts(ctypes.byref(s), ctypes.byref(weights.c), _mat(x, "x", T, H, H, src, dev),
                         _mat(topk_idx, "topk_idx", T, k, k, _I32, dev),
                         _mat(topk_w, "topk_w", T, k, k, _F32, dev), _mat(y, "y", T, H, H, src, dev),
                         ws, ws_bytes, st)
    if rc:
        _check(rc)


def moe_quant_fp8(quant, x, codes, scales, stream=None) -> None:
    """E4M3 codes [R, Kp] and their float32 block scales of x[R, K] (see include/moe.h)."""
    lib, dev, st = _begin(stream)
    q = quant
    R, K = q.R, q.K
    kb = -(-K // 128)
    rc = lib.moe_quant_fp8(ctypes.byref(q),
                           _mat(x, "x", R, K, q.ld or K, _SRC.get(q.src_dtype, _CODES), dev),
                           _mat(codes, "codes", R, kb * 128, kb * 128, _CODES, dev),
                           _mat(scales, "scales", -(-R // max(1, q.block_rows)), kb, kb, _F32, dev), st)
    if rc:
        _check(rc)


def quant_fp8(x, block_rows=1, stream=None):
    """(codes, scales) of a device tensor [R, K] or [E, N, K] (N a multiple of
    block_rows), bf16 or float32.  With `stream`, the outputs (and a copy of
    x, if its rows are not of unit stride) are allocated and written on it."""
    import torch
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            return quant_fp8(x, block_rows)
    if x.dim() not in (2, 3) or (x.dim() == 3 and x.shape[1] % block_rows):
        raise ValueError("quant_fp8 takes [R, K], or [E, N, K] with N a multiple of block_rows")
    if x.dim() == 3 or x.stride(1) != 1 or x.stride(0) < x.shape[1]:
        x = x.contiguous()
    lead, K = x.shape[:-1], x.shape[-1]
    R = x.numel() // max(1, K)
    kb = -(-K // 128)
    codes = torch.empty(*lead, kb * 128, dtype=torch.float8_e4m3fn, device=x.device)
    scales = torch.empty(*lead[:-1], -(-lead[-1] // block_rows), kb, dtype=torch.float32, device=x.device)
    src = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}.get(x.dtype, -1)
    moe_quant_fp8(moe_quant_t(R, K, block_rows, src, x.stride(0) if x.dim() == 2 and R > 1 else 0), x,
                  codes, scales)
    return codes, scales


def moe_matmul_fp8(matmul, a, sa, b, sb, y, offsets=None, stream=None) -> None:
    """y[M, N] of the codes a[M, Kp] and b[G, N, Kp] with their block scales
    (see include/moe.h); the rows of a are split among the b by `offsets`."""
    lib, dev, st = _begin(stream)
    m = matmul
    M, N, G = m.M, m.N, m.G
    kb = -(-m.K // 128)
    kp = kb * 128
    rc = lib.moe_matmul_fp8(ctypes.byref(m), _mat(a, "a", M, kp, m.lda or kp, _CODES, dev),
                            _mat(sa, "sa", M, kb, kb, _F32, dev),
                            _mat(b, "b", G * N, kp, m.ldb or kp, _CODES, dev),
                            _mat(sb, "sb", G * -(-N // 128), kb, kb, _F32, dev),
                            _mat(offsets, "offsets", 1, G + 1, G + 1, _I32, dev),
                            _mat(y, "y", M, N, m.ldy or N, _SRC.get(m.out_dtype, _CODES), dev), st)
    if rc:
        _check(rc)


def make_dispatch(T, H, E, top_k, x="bf16", rows=None, ldx=0, ldr=0) -> moe_dispatch_t:
    """rows: their type; by default x's, and bf16 where x is "fp8"."""
    return moe_dispatch_t(T, H, E, top_k, _DT[x], _DT[rows or ("bf16" if x == "fp8" else x)], ldx, ldr)


def make_combine(T, H, top_k, R, dtype="bf16", ldr=0, ldy=0) -> moe_combine_t:
    return moe_combine_t(T, H, top_k, R, _DT[dtype], ldr, ldy)


def make_swiglu(R, I, dtype="bf16", ld=0, ldh=0) -> moe_swiglu_t:
    return moe_swiglu_t(R, I, _DT[dtype], ld, ldh)


def make_matmul_bf16(M, N, K, G=1, out="bf16", ldx=0, ldw=0, ldy=0) -> moe_matmul_bf16_t:
    return moe_matmul_bf16_t(M, N, K, G, _DT[out], ldx, ldw, ldy)


def moe_dispatch_workspace_bytes(dispatch) -> int:
    return int(load().moe_dispatch_workspace_bytes(ctypes.byref(dispatch)))


def _tokens(d, x, sx, rows, dev):
    """Pointers of x, its scales and the rows in expert order."""
    T, H, kb = d.T, d.H, -(-d.H // 128)
    fp8 = d.x_dtype == MOE_FP8
    width = kb * 128 if fp8 else H
    return (_mat(x, "x", T, width, d.ldx or width, _CODES if fp8 else _SRC.get(d.x_dtype, _CODES), dev),
            _mat(sx, "sx", T, kb, kb, _F32, dev) if fp8 else None,
            _mat(rows, "rows", T * d.top_k, H, d.ldr or H, _SRC.get(d.row_dtype, _CODES), dev))


def moe_dispatch(dispatch, topk_idx, x, sx, rows, offsets, row_src, row_of, ws, ws_bytes=None, stream=None) -> None:
    """The pairs sorted by expert, offsets [E + 1], row_src [T * top_k] and row_of
    [T, top_k], and the rows [T * top_k, H] of x in that order (see include/moe.h);
    x and rows None: the order alone."""
    lib, dev, st = _begin(stream)
    d = dispatch
    T, E, k = d.T, d.E, d.top_k
    ws, ws_bytes = _workspace(ws, ws_bytes, dev)
    x, sx, rows = _tokens(d, x, sx, rows, dev)
    rc = lib.moe_dispatch(ctypes.byref(d), _mat(topk_idx, "topk_idx", T, k, k, _I32, dev), x, sx, rows,
                          _mat(offsets, "offsets", 1, E + 1, E + 1, _I32, dev),
                          _mat(row_src, "row_src", 1, T * k, T * k, _I32, dev),
                          _mat(row_of, "row_of", T, k, k, _I32, dev), ws, ws_bytes, st)
    if rc:
        _check(rc)


def moe_gather(dispatch, row_of, x, sx, rows, stream=None) -> None:
    """The rows of x by a row_of that moe_dispatch has made."""
    lib, dev, st = _begin(stream)
    d = dispatch
    x, sx, rows = _tokens(d, x, sx, rows, dev)
    rc = lib.moe_gather(ctypes.byref(d), _mat(row_of, "row_of", d.T, d.top_k, d.top_k, _I32, dev), x, sx, rows, st)
    if rc:
        _check(rc)


def moe_combine(combine, rows, row_of, topk_w, y, stream=None) -> None:
    """y[T, H], the weighted sum of each token's rows (topk_w None: weights of 1)."""
    lib, dev, st = _begin(stream)
    c = combine
    T, H, k = c.T, c.H, c.top_k
    src = _SRC.get(c.dtype, _CODES)
    rc = lib.moe_combine(ctypes.byref(c), _mat(rows, "rows", c.R, H, c.ldr or H, src, dev),
                         _mat(row_of, "row_of", T, k, k, _I32, dev), _mat(topk_w, "topk_w", T, k, k, _F32, dev),
                         _mat(y, "y", T, H, c.ldy or H, src, dev), st)
    if rc:
        _check(rc)


def moe_combine_grad(combine, dy, rows, row_of, topk_w, drows, dtopk_w, stream=None) -> None:
    """drows [R, H] and dtopk_w [T, top_k] of dy[T, H]; either may be None."""
    lib, dev, st = _begin(stream)
    c = combine
    T, H, k = c.T, c.H, c.top_k
    src = _SRC.get(c.dtype, _CODES)
    rc = lib.moe_combine_grad(ctypes.byref(c), _mat(dy, "dy", T, H, c.ldy or H, src, dev),
                              _mat(rows, "rows", c.R, H, c.ldr or H, src, dev),
                              _mat(row_of, "row_of", T, k, k, _I32, dev),
                              _mat(topk_w, "topk_w", T, k, k, _F32, dev),
                              _mat(drows, "drows", c.R, H, c.ldr or H, src, dev),
                              _mat(dtopk_w, "dtopk_w", T, k, k, _F32, dev), st)
    if rc:
        _check(rc)


def moe_swiglu(swiglu, gate, up, h, codes=None, scales=None, used=None, stream=None) -> None:
    """h[R, I] = silu(gate) * up, and with codes [R, 2 * Ip] and scales [R, 2 * Ip / 128]
    an 8-bit checkpoint of gate and up; used: an int32 tensor with the rows in use."""
    lib, dev, st = _begin(stream)
    s = swiglu
    R, I, kb = s.R, s.I, -(-s.I // 128)
    src = _SRC.get(s.dtype, _CODES)
    rc = lib.moe_swiglu(ctypes.byref(s), _mat(gate, "gate", R, I, s.ld or I, src, dev),
                        _mat(up, "up", R, I, s.ld or I, src, dev), _mat(used, "used", 1, 1, 1, _I32, dev),
                        _mat(h, "h", R, I, s.ldh or I, src, dev),
                        _mat(codes, "codes", R, 256 * kb, 256 * kb, _CODES, dev),
                        _mat(scales, "scales", R, 2 * kb, 2 * kb, _F32, dev), st)
    if rc:
        _check(rc)


def moe_swiglu_grad(swiglu, gate, up, codes, scales, dh, dgate, dup, h=None, used=None, stream=None) -> None:
    """dgate, dup and (unless None) h again, from gate and up or from their checkpoint."""
    lib, dev, st = _begin(stream)
    s = swiglu
    R, I, kb = s.R, s.I, -(-s.I // 128)
    src = _SRC.get(s.dtype, _CODES)
    ld, ldh = s.ld or I, s.ldh or I
    rc = lib.moe_swiglu_grad(ctypes.byref(s), _mat(gate, "gate", R, I, ld, src, dev), _mat(up, "up", R, I, ld, src, dev),
                             _mat(codes, "codes", R, 256 * kb, 256 * kb, _CODES, dev),
                             _mat(scales, "scales", R, 2 * kb, 2 * kb, _F32, dev),
                             _mat(dh, "dh", R, I, ldh, src, dev), _mat(used, "used", 1, 1, 1, _I32, dev),
                             _mat(dgate, "dgate", R, I, ld, src, dev), _mat(dup, "dup", R, I, ld, src, dev),
                             _mat(h, "h", R, I, ldh, src, dev), st)
    if rc:
        _check(rc)


def moe_select_grad(select, logits, topk_idx, dtopk_w, dscore, dlogits, bias=None, stream=None) -> None:
    """dlogits [T, E] (float32 or bfloat16) of the gradients dtopk_w [T, top_k] to
    moe_select's weights and dscore [E] (or None) to every token's scores; bias as
    moe_select had it."""
    lib, dev, st = _begin(stream)
    s = select
    T, E, k = s.T, s.E, s.top_k
    out = MOE_BF16 if dlogits is not None and dlogits.dtype in _SRC[MOE_BF16] else MOE_F32
    rc = lib.moe_select_grad(ctypes.byref(s),
                             _mat(logits, "logits", T, E, s.ld or E, _SRC.get(s.logit_dtype, _F32), dev),
                             _mat(bias, "bias", 1, E, E, _F32, dev),
                             _mat(topk_idx, "topk_idx", T, k, k, _I32, dev),
                             _mat(dtopk_w, "dtopk_w", T, k, k, _F32, dev),
                             _mat(dscore, "dscore", 1, E, E, _F32, dev),
                             _mat(dlogits, "dlogits", T, E, E, _SRC[out], dev), out, st)
    if rc:
        _check(rc)


def _bf16_mats(m, dev):
    """How the operands of the bf16 products lie: rows of x, matrices w, rows of y."""
    ldx, ldw, ldy = m.ldx or m.K, m.ldw or m.K, m.ldy or m.N

    def x(t, what, types):
        return _mat(t, what, m.M, m.K, ldx, types, dev)

    def w(t, what, types):
        if t is not None and t.dim() == 3 and not t.is_contiguous() and t.stride(0) == t.shape[1] * t.stride(1):
            t = t.flatten(0, 1)
        return _mat(t, what, m.G * m.N, m.K, ldw, types, dev)

    def y(t, what, types):
        return _mat(t, what, m.M, m.N, ldy, types, dev)

    return x, w, y, _SRC[MOE_BF16], _SRC.get(m.out_dtype, _CODES)


def moe_matmul_bf16(matmul, x, w, y, offsets=None, add=None, stream=None) -> None:
    """y[M, N] = x w[g]^T (+ add) for the rows of each group g (see include/moe.h)."""
    lib, dev, st = _begin(stream)
    m = matmul
    px, pw, py, src, out = _bf16_mats(m, dev)
    rc = lib.moe_matmul_bf16(ctypes.byref(m), px(x, "x", src), pw(w, "w", src),
                             _mat(offsets, "offsets", 1, m.G + 1, m.G + 1, _I32, dev), py(add, "add", out),
                             py(y, "y", out), st)
    if rc:
        _check(rc)


def moe_matmul_bf16_dx(matmul, dy, w, dx, offsets=None, add=None, stream=None) -> None:
    """dx[M, K] = dy w[g] (+ add)."""
    lib, dev, st = _begin(stream)
    m = matmul
    px, pw, py, src, out = _bf16_mats(m, dev)
    rc = lib.moe_matmul_bf16_dx(ctypes.byref(m), py(dy, "dy", src), pw(w, "w", src),
                                _mat(offsets, "offsets", 1, m.G + 1, m.G + 1, _I32, dev), px(add, "add", out),
                                px(dx, "dx", out), st)
    if rc:
        _check(rc)


def moe_matmul_bf16_dw(matmul, dy, x, dw, offsets=None, add=None, stream=None) -> None:
    """dw[G, N, K] = dy^T x over the rows of each group (+ add)."""
    lib, dev, st = _begin(stream)
    m = matmul
    px, pw, py, src, out = _bf16_mats(m, dev)
    rc = lib.moe_matmul_bf16_dw(ctypes.byref(m), py(dy, "dy", src), px(x, "x", src),
                                _mat(offsets, "offsets", 1, m.G + 1, m.G + 1, _I32, dev), pw(add, "add", out),
                                pw(dw, "dw", out), st)
    if rc:
        _check(rc)


def moe_matmul_bf16_tile(matmul, way, off16=False):
    """(rows, columns, groups of waves, 1 if copied in pieces of 16 bytes) of the tile that a product
    takes, way "y", "dx" or "dw"; off16: a pointer is not at a multiple of 16 bytes."""
    tile = (ctypes.c_int32 * 4)()
    _check(load().moe_matmul_bf16_tile(ctypes.byref(matmul), ("y", "dx", "dw").index(way), int(off16), tile))
    return tuple(tile)


STAGES = ("router", "permute", "gate_up", "down", "combine")


def moe_stage_timing_enable(on: bool) -> None:
    _check(load().moe_stage_timing_enable(1 if on else 0))


def moe_stage_timing_read():
    """(milliseconds summed per stage as a dict, number of timed calls)."""
    ms = (ctypes.c_float * len(STAGES))()
    n = ctypes.c_int(0)
    _check(load().moe_stage_timing_read(ms, len(STAGES), ctypes.byref(n)))
    return dict(zip(STAGES, [float(v) for v in ms])), n.value


def moe_probe_read(buf, stream=None) -> None:
    """Stream-read the device tensor `buf` (measurement aid, see moe.h)."""
    n = buf.numel() * buf.element_size()
    _check(load().moe_probe_read(_ptr(buf), n - n % 16, _stream(stream)))


def moe_probe_mfma(waves: int, iters: int, stream=None) -> None:
    """bf16 MFMA chains on every wave (measurement aid, see moe.h)."""
    _check(load().moe_probe_mfma(waves, iters, None, _stream(stream)))


def moe_probe_gather(pool, chunk_bytes: int, order, wgs: int, stream=None) -> None:
    """Read the chunks of `pool` listed in the int32 device tensor `order`
    (measurement aid, see moe.h)."""
    n = pool.numel() * pool.element_size()
    _check(load().moe_probe_gather(_ptr(pool), n, chunk_bytes, _ptr(order), order.numel(), wgs,
                                   _stream(stream)))


def moe_probe_mxfp4(codes, scales, out, stream=None) -> None:
    """Decode and sum the MXFP4 blocks of `codes` / `scales` (row-major OCP
    form); out (float32 device tensor) receives one sum per workgroup
    (measurement aid, see moe.h)."""
    nblk = scales.numel()
    assert codes.numel() * codes.element_size() >= 16 * nblk
    _check(load().moe_probe_mxfp4(_ptr(codes), _ptr(scales), nblk, out.numel(), _ptr(out),
                                  _stream(stream)))


def moe_strerror(code: int) -> str:
    return load().moe_strerror(code).decode()


def moe_last_error() -> str:
    return load().moe_last_error().decode()
