"""The end of a training step (libcbr.so): :func:`gradient_norm` over many tensors and :func:`clip_gradients`.

``include/cbr.h`` has the formulas; calls behave as those of :mod:`conv_batchnorm_relu_gb300.tokens`.  Nothing is
kept between calls, and nothing waits for the device: the norm stays there, so a step can be captured.
"""
from __future__ import annotations

import ctypes
import math
from array import array

import torch

from . import cbr
from .cbr import _check
from .tokens import _DTYPE, _UNSUPPORTED, _bad, _device_of, _given, _new, _stream_of, _vector

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = cbr.load()
        vp, f, size = ctypes.c_void_p, ctypes.c_float, ctypes.c_size_t
        lib.cbr_clip_workspace_size.argtypes = [ctypes.c_int64, ctypes.POINTER(size)]
        lib.cbr_clip_gradients.argtypes = [ctypes.c_int64] + [vp] * 4 + [f, f] + [vp] * 3 + [size, vp]
        for name in ("cbr_clip_workspace_size", "cbr_clip_gradients"):
            getattr(lib, name).restype = ctypes.c_int32
        _lib = lib
    return _lib


# A call is over many tensors: their attributes through map, without a line of Python for each.
_T = torch.Tensor
_dtype_of = _T.dtype.__get__


def _addresses(tensors, dev, what: str) -> array:
    if set(map(_T.get_device, tensors)) != {dev.index} or not all(map(_T.is_contiguous, tensors)):
        _bad(f"{what} have to be contiguous on {dev}")
    return array("Q", map(_T.data_ptr, tensors))


def _run(grads, outs, max_norm, unscale, ws, out):
    if not grads:
        _bad("no gradients")
    if not grads[0].is_cuda:
        _bad("gradients have to be CUDA tensors")
    dev, n = _device_of(grads[0]), len(grads)
    at = _addresses(grads, dev, "gradients")
    dtypes, sizes = list(map(_dtype_of, grads)), array("q", map(_T.numel, grads))
    try:
        types = array("i", [_DTYPE[dtypes[0]]]) * n if dtypes.count(dtypes[0]) == n else array("i", map(_DTYPE.__getitem__, dtypes))
    except KeyError as e:
        _bad(f"gradients: {e}", _UNSUPPORTED)
    out_at = at
    if outs is not grads and outs is not None:
        if len(outs) != n:
            _bad(f"{len(outs)} outs for {n} gradients")
        out_at = _addresses(outs, dev, "outs")
        if list(map(_dtype_of, outs)) != dtypes or array("q", map(_T.numel, outs)) != sizes:
            _bad("an out has to have its gradient's type and number of elements")
    norm = _given(out, "norm", (), torch.float32, dev)
    scale = _given(out, "scale", (), torch.float32, dev)
    if ws is None:
        ws = _new((clip_workspace_size(n),), torch.uint8, dev)
    elif ws.device != dev or not ws.is_contiguous():
        _bad(f"ws has to be contiguous on {dev}")
    _check(_load().cbr_clip_gradients(
        n, at.buffer_info()[0], sizes.buffer_info()[0], types.buffer_info()[0],
        out_at.buffer_info()[0] if outs is not None else None, max_norm, unscale, _vector(norm, 1, dev, "norm"),
        _vector(scale, 1, dev, "scale"), ws.data_ptr(), ws.numel() * ws.element_size(), _stream_of(dev)),
        "cbr_clip_gradients")
    return norm, scale


_sizes: dict = {}   # clip_workspace_size's answers


def clip_workspace_size(count: int) -> int:
    """Workspace bytes of the calls below for `count` tensors."""
    known = _sizes.get(count)
    if known is None:
        size = ctypes.c_size_t()
        _check(_load().cbr_clip_workspace_size(count, ctypes.byref(size)), "cbr_clip_workspace_size")
        known = _sizes[count] = size.value
    return known


def gradient_norm(grads, *, unscale=1.0, ws=None) -> torch.Tensor:
    """unscale times the norm of all the gradients together, a fp32 scalar on their device."""
    return _run(list(grads), None, math.inf, float(unscale), ws, None)[0]


def clip_gradients(grads, max_norm, *, unscale=1.0, ws=None, out=None, scalars=None) -> dict:
    """cbr_clip_gradients -> dict(norm, scale), fp32 scalars on the device; the gradients are scaled in place.

        norm = unscale * sqrt(sum of all squares),  scale = unscale * min(1, max_norm / norm)

    grads: contiguous tensors (f32, f16, bf16 in any mixture).  unscale takes a loss scale off.  out: tensors
    of the same sizes and types to write instead of the gradients.  A tensor that is written may not share memory with
    another (the same gradient twice, for one).  scalars: {"norm": ..., "scale": ...} to
    write.  ws: a workspace of :func:`clip_workspace_size` bytes to use instead of a new one.  An infinite
    gradient makes the scale 0, a NaN makes it NaN; a step that is to be skipped then can look at "norm"."""
    grads = list(grads)
    norm, scale = _run(grads, grads if out is None else list(out), float(max_norm), float(unscale), ws, scalars)
    return {"norm": norm, "scale": scale}
