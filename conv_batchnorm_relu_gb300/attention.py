"""Attention over a trunk's tokens (libcbr.so): :func:`attention_forward`, and :func:`attention_backward`, which
computes the probabilities again instead of keeping them.

``include/cbr.h`` has the formulas.  As in :mod:`conv_batchnorm_relu_gb300.tokens`, each call checks its
arguments, allocates what it returns (or takes it in ``out``), launches on the current stream and raises
:class:`~conv_batchnorm_relu_gb300.cbr.CBRError` on a refusal; there is no fallback.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import cbr
from .cbr import _check
from .tokens import _bad, _device_of, _dtype, _given, _heads, _new, _pack, _stream_of, _vector

_DESC = struct.Struct("@27q5if")   # cbr_attention_desc_t
_NONE = (0, 0, 0)

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = cbr.load()
        vp, d, size = ctypes.c_void_p, ctypes.c_char_p, ctypes.c_size_t
        lib.cbr_attention_workspace_size.argtypes = [d, ctypes.POINTER(size), ctypes.POINTER(size)]
        lib.cbr_attention_forward.argtypes = [d] + [vp] * 8 + [size, vp]
        lib.cbr_attention_backward.argtypes = [d] + [vp] * 12 + [size, vp]
        for f in ("cbr_attention_workspace_size", "cbr_attention_forward", "cbr_attention_backward"):
            getattr(lib, f).restype = ctypes.c_int32
        _lib = lib
    return _lib


def _places(t: torch.Tensor | None, batch: int, dev, what: str):
    """Checks an optional contiguous int32 [batch]; its address."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.device != dev or t.dim() != 1 or t.shape[0] != batch or not t.is_contiguous():
        _bad(f"{what} has to be contiguous int32 [{batch}] on {dev}")
    return t.data_ptr()


class _Call:
    """The checked operands that both directions share, and the descriptor's fields."""

    def __init__(self, q, k, v, scale, causal, key_lengths, query_start):
        if q.dim() != 4 or not q.is_cuda:
            _bad("q has to be a [batch][tokens][heads][head_dim] CUDA tensor")
        if k.dim() != 4:
            _bad("k has to be a [batch][tokens][heads][head_dim] tensor")
        self.dev, self.dt = _device_of(q), q.dtype
        self.code = _dtype(q, "q")
        self.batch, self.tq, self.hq, self.dim = q.shape
        self.tk, self.hk = k.shape[1], k.shape[2]
        self.sq, _, self.q = self.heads(q, self.tq, self.hq, "q")
        self.sk, _, self.k = self.heads(k, self.tk, self.hk, "k")
        self.sv, _, self.v = self.heads(v, self.tk, self.hk, "v")
        self.lengths = _places(key_lengths, self.batch, self.dev, "key_lengths")
        self.start = _places(query_start, self.batch, self.dev, "query_start")
        self.scale = float(self.dim ** -0.5 if scale is None else scale)
        self.causal = 1 if causal else 0

    def heads(self, t, tokens, heads, what):
        got = _heads(t, self.batch, tokens, self.dim, self.dt, self.dev, what)
        if got[1] != heads:
            _bad(f"{what} has {got[1]} heads, not {heads}")
        return got

    def desc(self, so, sdo=_NONE, sdq=_NONE, sdk=_NONE, sdv=_NONE) -> bytes:
        return _pack(_DESC, self.batch, self.tq, self.tk, *self.sq, *self.sk, *self.sv, *so, *sdo, *sdq, *sdk, *sdv,
                     self.hq, self.hk, self.dim, self.causal, self.code, self.scale)

    def workspace(self, desc, ws, backward: bool):
        """(address, bytes) of the workspace, and the tensor that holds it."""
        if ws is not None:
            if ws.device != self.dev or not ws.is_contiguous():
                _bad(f"ws has to be contiguous on {self.dev}")
            return ws, ws.data_ptr(), ws.numel() * ws.element_size()
        n = ctypes.c_size_t()
        at = ctypes.byref(n)
        _check(_load().cbr_attention_workspace_size(desc, None if backward else at, at if backward else None),
               "cbr_attention_workspace_size")
        if not n.value:
            return None, None, 0
        ws = _new((n.value,), torch.uint8, self.dev)
        return ws, ws.data_ptr(), n.value


def attention_workspace_size(q, k) -> tuple[int, int]:
    """Workspace bytes of (:func:`attention_forward`, :func:`attention_backward`) on operands of these shapes."""
    c = _Call(q, k, k, None, False, None, None)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_load().cbr_attention_workspace_size(c.desc(_NONE), ctypes.byref(f), ctypes.byref(b)),
           "cbr_attention_workspace_size")
    return f.value, b.value


def attention_forward(q, k, v, *, scale=None, causal=False, key_lengths=None, query_start=None, want_lse=True, ws=None,
                      out=None) -> dict:
    """cbr_attention_forward -> dict(o [batch][tq][heads_q][head_dim], lse [batch][heads_q][tq] fp32).

    q [batch][tq][heads_q][head_dim], k and v [batch][tk][heads_k][head_dim], f16 or bf16, with any strides of
    the first three axes that are multiples of 8 elements, as views of a fused product; heads_q a multiple of
    heads_k (shared key heads); head_dim a multiple of 8 up to 128.  scale: of the scores, head_dim**-0.5 where
    None.  key_lengths int32 [batch]: the keys a sequence has, where the rest is padding.  causal: query i
    of sequence b sees the keys up to query_start[b] + i (int32 [batch]; None: 0), so a single new token after
    n keys (its own among them) has query_start n - 1.  A query that sees no key has o = 0 and lse = -inf.
    ws: a workspace (:func:`attention_workspace_size`) to use instead of a new one."""
    c = _Call(q, k, v, scale, causal, key_lengths, query_start)
    o = _given(out, "o", (c.batch, c.tq, c.hq, c.dim), c.dt, c.dev)
    so, _, o_at = c.heads(o, c.tq, c.hq, "o")
    n = c.batch * c.hq * c.tq
    lse = _given(out, "lse", (c.batch, c.hq, c.tq), torch.float32, c.dev) if want_lse else None
    desc = c.desc(so)
    keep, ws_at, ws_n = c.workspace(desc, ws, False)
    _check(_load().cbr_attention_forward(desc, c.q, c.k, c.v, c.lengths, c.start, o_at, _vector(lse, n, c.dev, "lse"),
                                         ws_at, ws_n, _stream_of(c.dev)), "cbr_attention_forward")
    return {"o": o, "lse": lse}


def attention_backward(do, q, k, v, o, lse, *, scale=None, causal=False, key_lengths=None, query_start=None, ws=None,
                       out=None) -> dict:
    """cbr_attention_backward -> dict(dq, dk, dv), contiguous where ``out`` does not give them.

    do: the gradient at o; o and lse from :func:`attention_forward`; the rest as there.  The gradients of a key
    head are summed over the query heads that read it, those of keys from key_lengths on are 0."""
    c = _Call(q, k, v, scale, causal, key_lengths, query_start)
    so, _, o_at = c.heads(o, c.tq, c.hq, "o")
    sdo, _, do_at = c.heads(do, c.tq, c.hq, "do")
    dq = _given(out, "dq", (c.batch, c.tq, c.hq, c.dim), c.dt, c.dev)
    dk = _given(out, "dk", (c.batch, c.tk, c.hk, c.dim), c.dt, c.dev)
    dv = _given(out, "dv", (c.batch, c.tk, c.hk, c.dim), c.dt, c.dev)
    sdq, _, dq_at = c.heads(dq, c.tq, c.hq, "dq")
    sdk, _, dk_at = c.heads(dk, c.tk, c.hk, "dk")
    sdv, _, dv_at = c.heads(dv, c.tk, c.hk, "dv")
    desc = c.desc(so, sdo, sdq, sdk, sdv)
    keep, ws_at, ws_n = c.workspace(desc, ws, True)
    _check(_load().cbr_attention_backward(desc, do_at, c.q, c.k, c.v, o_at,
                                          _vector(lse, c.batch * c.hq * c.tq, c.dev, "lse"), c.lengths, c.start, dq_at,
                                          dk_at, dv_at, ws_at, ws_n, _stream_of(c.dev)), "cbr_attention_backward")
    return {"dq": dq, "dk": dk, "dv": dv}
