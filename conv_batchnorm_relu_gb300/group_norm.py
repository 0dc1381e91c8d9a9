"""Group norm with an activation over NHWC feature maps (libcbr.so): :func:`group_norm_forward` and
:func:`group_norm_backward`, the norm for stems whose batch is too small for batch statistics.

``include/cbr.h`` has the formulas; calls behave as those of :mod:`conv_batchnorm_relu_gb300.tokens`.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import cbr
from .cbr import _check
from .tokens import _bad, _device_of, _dtype, _given, _new, _pack, _stream_of, _vector

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


def _map(t: torch.Tensor, shape, dtype, dev, what: str):
    """Checks a feature map [images][...][channels] whose pixels lie a fixed step apart; (image, pixel) strides."""
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        _bad(f"{what} has to be {list(shape)} {dtype} on {dev}: {list(t.shape)} {t.dtype} on {t.device}")
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
    return (s[0], step), t.data_ptr()


def _act(act: str) -> int:
    if act not in _ACT:
        _bad(f"act {act!r}: one of {sorted(_ACT)}")
    return _ACT[act]


def _shape(x: torch.Tensor, what: str):
    """(images, pixels, channels)"""
    if x.dim() < 2 or not x.is_cuda:
        _bad(f"{what} has to be an [images][...][channels] CUDA tensor")
    pixels = 1
    for n in x.shape[1:-1]:
        pixels *= n
    return x.shape[0], pixels, x.shape[-1]


def _workspace(desc, ws, dev, backward: bool):
    """The workspace (None: none is needed), its address and its bytes."""
    if ws is not None:
        if ws.device != dev or not ws.is_contiguous():
            _bad(f"ws has to be contiguous on {dev}")
        return ws, ws.data_ptr(), ws.numel() * ws.element_size()
    size = ctypes.c_size_t()
    at = ctypes.byref(size)
    _check(_load().cbr_group_norm_workspace_size(desc, None if backward else at, at if backward else None),
           "cbr_group_norm_workspace_size")
    if not size.value:
        return None, None, 0
    ws = _new((size.value,), torch.uint8, dev)
    return ws, ws.data_ptr(), size.value


def group_norm_forward(x, gamma, beta, groups, *, eps=1e-5, act="none", ws=None, out=None) -> dict:
    """cbr_group_norm_forward -> dict(y, mean [images][groups], rstd [images][groups]), the statistics fp32.

    x [images][...][channels] (an NHWC feature map; f32, f16 or bf16), whose pixels lie a fixed step apart; gamma
    and beta fp32 [channels], or both None; act "none", "relu" or "silu".  out may hold "y" (x itself, to save
    its memory), "mean" and "rstd".  ws: a workspace (:func:`group_norm_workspace_size`) to use instead of a new
    one."""
    images, pixels, channels = _shape(x, "x")
    dev, dt = _device_of(x), x.dtype
    code = _dtype(x, "x")
    sx, x_at = _map(x, x.shape, dt, dev, "x")
    y = _given(out, "y", x.shape, dt, dev)
    sy, y_at = _map(y, x.shape, dt, dev, "y")
    n = images * groups
    mean = _given(out, "mean", (images, groups), torch.float32, dev)
    rstd = _given(out, "rstd", (images, groups), torch.float32, dev)
    desc = _pack(_DESC, images, pixels, *sx, *sy, 0, 0, 0, 0, channels, groups, _act(act), code, eps)
    ws, ws_at, ws_n = _workspace(desc, ws, dev, False)
    _check(_load().cbr_group_norm_forward(
        desc, x_at, _vector(gamma, channels, dev, "gamma"), _vector(beta, channels, dev, "beta"), y_at,
        _vector(mean, n, dev, "mean"), _vector(rstd, n, dev, "rstd"), ws_at, ws_n, _stream_of(dev)),
        "cbr_group_norm_forward")
    return {"y": y, "mean": mean, "rstd": rstd}


def group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, *, act="none", ws=None, out=None) -> dict:
    """cbr_group_norm_backward -> dict(dx, dgamma, dbeta); the last two None without a gamma.

    dy: the gradient at y; mean and rstd from :func:`group_norm_forward`; the rest as there.  out may hold "dx" (dy
    itself, to save its memory), "dgamma" and "dbeta".  ws: as there."""
    images, pixels, channels = _shape(x, "x")
    dev, dt = _device_of(x), x.dtype
    code = _dtype(x, "x")
    sx, x_at = _map(x, x.shape, dt, dev, "x")
    sdy, dy_at = _map(dy, x.shape, dt, dev, "dy")
    dx = _given(out, "dx", x.shape, dt, dev)
    sdx, dx_at = _map(dx, x.shape, dt, dev, "dx")
    n = images * groups
    dgamma = dbeta = None
    if gamma is not None:
        dgamma = _given(out, "dgamma", (channels,), torch.float32, dev)
        dbeta = _given(out, "dbeta", (channels,), torch.float32, dev)
    desc = _pack(_DESC, images, pixels, *sx, 0, 0, *sdy, *sdx, channels, groups, _act(act), code, 1.0)
    ws, ws_at, ws_n = _workspace(desc, ws, dev, True)
    _check(_load().cbr_group_norm_backward(
        desc, dy_at, x_at, _vector(gamma, channels, dev, "gamma"), _vector(beta, channels, dev, "beta"),
        _vector(mean, n, dev, "mean"), _vector(rstd, n, dev, "rstd"), dx_at, _vector(dgamma, channels, dev, "dgamma"),
        _vector(dbeta, channels, dev, "dbeta"), ws_at, ws_n, _stream_of(dev)),
        "cbr_group_norm_backward")
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def group_norm_workspace_size(x, groups) -> tuple[int, int]:
    """Workspace bytes of (:func:`group_norm_forward`, :func:`group_norm_backward`) for a map of x's shape."""
    images, pixels, channels = _shape(x, "x")
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    desc = _pack(_DESC, images, pixels, *([0] * 8), channels, groups, 0, _dtype(x, "x"), 1.0)
    _check(_load().cbr_group_norm_workspace_size(desc, ctypes.byref(f), ctypes.byref(b)), "cbr_group_norm_workspace_size")
    return f.value, b.value
