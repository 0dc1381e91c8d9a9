"""Group norm with an activation over NHWC feature maps (libcbr.so): :func:`group_norm_forward` and
:func:`group_norm_backward`, the norm for stems whose batch is too small for batch statistics.

``include/cbr.h`` has the formulas; calls behave as those of :mod:`conv_batchnorm_relu_gb300.tokens`.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import cbr
from .cbr import CBR_OK, CBRError
from .tokens import _DTYPE, _INVALID, _UNSUPPORTED, _bad, _get_device, _new, _raw_stream, _stream_of

_DESC = struct.Struct("@10q4if4x")   # cbr_group_norm_desc_t
_ACT = {"none": 0, "relu": 1, "silu": 2}

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = cbr.load()
        vp, d, size = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_size_t
        lib.cbr_group_norm_workspace_size.argtypes = [d, ctypes.POINTER(size), ctypes.POINTER(size)]
        lib.cbr_group_norm_forward.argtypes = [d] + [vp] * 7 + [size, vp]
        lib.cbr_group_norm_backward.argtypes = [d] + [vp] * 10 + [size, vp]
        for f in ("cbr_group_norm_workspace_size", "cbr_group_norm_forward", "cbr_group_norm_backward"):
            getattr(lib, f).restype = ctypes.c_int32
        _lib = lib
    return _lib


def _map(t: torch.Tensor, shape, pixels: int, dtype, index: int, what: str):
    """Checks a feature map [images][...][channels] whose pixels lie a fixed step apart; (image, pixel) strides, address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _bad(f"{what} has to be {list(shape)} {dtype} on cuda:{index}: {list(t.shape)} {t.dtype} on {t.device}")
    if t.is_contiguous():
        return (pixels or 1) * shape[-1], shape[-1], t.data_ptr()
    s = t.stride()
    if s[-1] != 1 and shape[-1] > 1:
        _bad(f"{what}: a pixel's channels have to be adjacent")
    step, reach = shape[-1], None     # of the pixels, from the last axis of several
    for n, st in zip(shape[-2:0:-1], s[-2:0:-1]):
        if n == 1:
            continue
        if reach is None:
            step, reach = st, st * n
        elif st != reach:
            _bad(f"{what}: its pixels have to lie a fixed step apart")
        else:
            reach = st * n
    return s[0], step, t.data_ptr()


def _floats(t: torch.Tensor | None, n: int, index: int, what: str):
    """Checks an optional contiguous fp32 tensor of n elements; its address."""
    if t is None:
        return None
    if t.numel() != n or t.dtype is not torch.float32 or t.get_device() != index or not t.is_contiguous():
        _bad(f"{what} has to be {n} contiguous fp32 values on cuda:{index}")
    return t.data_ptr()


def _shape(x: torch.Tensor, groups: int, act: str):
    """(shape, pixels, channels, type, its code, device, activation's code) of a map."""
    shape, dt, index = x.shape, x.dtype, x.get_device()
    if len(shape) < 2 or index < 0:
        _bad("x has to be an [images][...][channels] CUDA tensor")
    if groups < 1:
        _bad(f"{groups} groups")
    if index != _get_device():
        _bad(f"tensors on {x.device}, which is not the current device", 5)
    code, what = _DTYPE.get(dt), _ACT.get(act)
    if code is None:
        _bad(f"x: {dt}", _UNSUPPORTED)
    if what is None:
        _bad(f"act {act!r}: one of {sorted(_ACT)}")
    pixels = 1
    for n in shape[1:-1]:
        pixels *= n
    return shape, pixels, shape[-1], dt, code, index, what


def _pack(images, pixels, x, y, dy, dx, channels, groups, act, code, eps) -> bytes:
    """The descriptor; a number that its 32 bits cannot hold is refused like one that the library refuses."""
    try:
        return _DESC.pack(images, pixels, x[0], x[1], y[0], y[1], dy[0], dy[1], dx[0], dx[1], channels, groups, act, code, eps)
    except (struct.error, OverflowError) as e:
        raise CBRError(_INVALID, f"arguments: {e}") from None


_NONE = (0, 0)
_sizes: dict = {}   # cbr_group_norm_workspace_size's answers: they go by shapes alone


def _bytes(images, pixels, channels, groups, code) -> tuple[int, int]:
    key = (images, pixels, channels, groups, code)
    known = _sizes.get(key)
    if known is None:
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        desc = _pack(images, pixels, _NONE, _NONE, _NONE, _NONE, channels, groups, 0, code, 1.0)
        status = _load().cbr_group_norm_workspace_size(desc, ctypes.byref(f), ctypes.byref(b))
        if status != CBR_OK:
            raise CBRError(status, "cbr_group_norm_workspace_size")
        if len(_sizes) > 4096:
            _sizes.clear()
        known = _sizes[key] = (f.value, b.value)
    return known


def _workspace(n: int, dev, index: int, ws):
    """The workspace (None: none is needed), its address and its bytes."""
    if ws is None:
        if not n:
            return None, None, 0
        ws = _new((n,), torch.uint8, dev)
    elif ws.get_device() != index or not ws.is_contiguous():
        _bad(f"ws has to be contiguous on cuda:{index}")
    return ws, ws.data_ptr(), ws.numel() * ws.element_size()


def _given(out, name: str, shape, dtype, dev):
    t = out.get(name) if out else None
    return _new(shape, dtype, dev) if t is None else t


def group_norm_forward(x, gamma, beta, groups, *, eps=1e-5, act="none", ws=None, out=None) -> dict:
    """cbr_group_norm_forward -> dict(y, mean [images][groups], rstd [images][groups]), the statistics fp32.

    x [images][...][channels] (an NHWC feature map; f32, f16 or bf16), whose pixels lie a fixed step apart; gamma
    and beta fp32 [channels], or both None; act "none", "relu" or "silu".  out may hold "y" (x itself, to save
    its memory), "mean" and "rstd" (NaN for a map without pixels).  ws: a workspace
    (:func:`group_norm_workspace_size`) to use instead of a new one."""
    shape, pixels, channels, dt, code, index, act = _shape(x, groups, act)
    images, dev = shape[0], x.device
    sx = _map(x, shape, pixels, dt, index, "x")
    y = _given(out, "y", shape, dt, dev)
    sy = _map(y, shape, pixels, dt, index, "y")
    n = images * groups
    mean = _given(out, "mean", (images, groups), torch.float32, dev)
    rstd = _given(out, "rstd", (images, groups), torch.float32, dev)
    desc = _pack(images, pixels, sx, sy, _NONE, _NONE, channels, groups, act, code, eps)
    ws, ws_at, ws_n = _workspace(_bytes(images, pixels, channels, groups, code)[0], dev, index, ws)
    status = (_lib or _load()).cbr_group_norm_forward(
        desc, sx[2], _floats(gamma, channels, index, "gamma"), _floats(beta, channels, index, "beta"), sy[2],
        _floats(mean, n, index, "mean"), _floats(rstd, n, index, "rstd"), ws_at, ws_n,
        _raw_stream(index) if _raw_stream else _stream_of(dev))
    if status != CBR_OK:
        raise CBRError(status, "cbr_group_norm_forward")
    if not pixels:      # the mean of no values
        mean.fill_(math.nan)
        rstd.fill_(math.nan)
    return {"y": y, "mean": mean, "rstd": rstd}


def group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, *, act="none", ws=None, out=None) -> dict:
    """cbr_group_norm_backward -> dict(dx, dgamma, dbeta); the last two None without a gamma.

    dy: the gradient at y; mean and rstd from :func:`group_norm_forward`; the rest as there.  out may hold "dx" (dy
    itself, to save its memory), "dgamma" and "dbeta".  ws: as there."""
    shape, pixels, channels, dt, code, index, act = _shape(x, groups, act)
    images, dev = shape[0], x.device
    sx = _map(x, shape, pixels, dt, index, "x")
    sdy = _map(dy, shape, pixels, dt, index, "dy")
    dx = _given(out, "dx", shape, dt, dev)
    sdx = _map(dx, shape, pixels, dt, index, "dx")
    n = images * groups
    dgamma = dbeta = None
    if gamma is not None:
        dgamma = _given(out, "dgamma", (channels,), torch.float32, dev)
        dbeta = _given(out, "dbeta", (channels,), torch.float32, dev)
    desc = _pack(images, pixels, sx, _NONE, sdy, sdx, channels, groups, act, code, 1.0)
    ws, ws_at, ws_n = _workspace(_bytes(images, pixels, channels, groups, code)[1], dev, index, ws)
    status = (_lib or _load()).cbr_group_norm_backward(
        desc, sdy[2], sx[2], _floats(gamma, channels, index, "gamma"), _floats(beta, channels, index, "beta"),
        _floats(mean, n, index, "mean"), _floats(rstd, n, index, "rstd"), sdx[2], _floats(dgamma, channels, index, "dgamma"),
        _floats(dbeta, channels, index, "dbeta"), ws_at, ws_n, _raw_stream(index) if _raw_stream else _stream_of(dev))
    if status != CBR_OK:
        raise CBRError(status, "cbr_group_norm_backward")
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def group_norm_workspace_size(x, groups) -> tuple[int, int]:
    """Workspace bytes of (:func:`group_norm_forward`, :func:`group_norm_backward`) for a map of x's shape."""
    shape, pixels, channels, _, code, _, _ = _shape(x, groups, "none")
    return _bytes(shape[0], pixels, channels, groups, code)
