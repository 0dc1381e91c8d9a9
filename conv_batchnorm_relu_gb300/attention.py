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
from .cbr import CBR_OK, CBRError
from .tokens import _DTYPE, _INVALID, _UNSUPPORTED, _bad, _empty_cuda, _get_device, _new, _raw_stream, _stream_of

_DESC = struct.Struct("@27q5if")   # cbr_attention_desc_t

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


# A small call's time is host time, so the checks ask a tensor for each thing once.

def _heads(t: torch.Tensor, shape, dtype, index: int, what: str):
    """Checks a [batch][tokens][heads][head_dim] tensor; its strides and its address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        _bad(f"{what} has to be {list(shape)} {dtype} on cuda:{index}: {list(t.shape)} {t.dtype} on {t.device}")
    s = t.stride()
    if s[3] != 1:
        _bad(f"{what}: a head's elements have to be adjacent")
    return s, t.data_ptr()


def _flat(t: torch.Tensor | None, shape, dtype, index: int, what: str):
    """Checks an optional contiguous tensor; its address."""
    if t is None:
        return None
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        _bad(f"{what} has to be contiguous {list(shape)} {dtype} on cuda:{index}")
    return t.data_ptr()


def _operands(q, k):
    """(shape of q, shape of k, type, its code, device) of checked operands."""
    qs, ks, dt, index = q.shape, k.shape, q.dtype, q.get_device()
    if len(qs) != 4 or index < 0:
        _bad("q has to be a [batch][tokens][heads][head_dim] CUDA tensor")
    if len(ks) != 4 or ks[0] != qs[0] or ks[3] != qs[3]:
        _bad(f"k {list(ks)} does not go with q {list(qs)}")
    if index != _get_device():
        _bad(f"tensors on {q.device}, which is not the current device", 5)
    code = _DTYPE.get(dt)
    if code is None:
        _bad(f"q: {dt}", _UNSUPPORTED)
    return qs, ks, dt, code, index


def _empty(shape, dtype, index: int) -> torch.Tensor:
    """A new contiguous tensor of four axes on the current device."""
    if _empty_cuda is None:
        return torch.empty(shape, dtype=dtype, device=index)
    a, b = shape[3], shape[2] * shape[3]
    return _empty_cuda(tuple(shape), ((shape[1] or 1) * b, b, a, 1), dtype)


_sizes: dict = {}   # cbr_attention_workspace_size's answers: they go by shapes alone


def _workspace(qs, ks, code, index, ws, backward: bool):
    """The workspace (None: none is needed), its address and its bytes."""
    if ws is not None:
        if ws.get_device() != index or not ws.is_contiguous():
            _bad(f"ws has to be contiguous on cuda:{index}")
        return ws, ws.data_ptr(), ws.numel() * ws.element_size()
    key = (qs, ks[1], ks[2], code)
    known = _sizes.get(key)
    if known is None:
        f, b = ctypes.c_size_t(), ctypes.c_size_t()
        desc = _pack(qs, ks, code, 1.0, False, *([(0, 0, 0)] * 8))
        status = _load().cbr_attention_workspace_size(desc, ctypes.byref(f), ctypes.byref(b))
        if status != CBR_OK:
            raise CBRError(status, "cbr_attention_workspace_size")
        if len(_sizes) > 4096:
            _sizes.clear()
        known = _sizes[key] = (f.value, b.value)
    n = known[backward]
    if not n:
        return None, None, 0
    ws = _new((n,), torch.uint8, torch.device("cuda", index)) if _empty_cuda is None else _empty_cuda((n,), (1,), torch.uint8)
    return ws, ws.data_ptr(), n


def _pack(qs, ks, code, scale, causal, q, k, v, o, do=(0, 0, 0), dq=(0, 0, 0), dk=(0, 0, 0), dv=(0, 0, 0)) -> bytes:
    """The descriptor; a number that its 32 bits cannot hold is refused like one that the library refuses."""
    try:
        return _DESC.pack(qs[0], qs[1], ks[1], q[0], q[1], q[2], k[0], k[1], k[2], v[0], v[1], v[2], o[0], o[1], o[2], do[0],
                          do[1], do[2], dq[0], dq[1], dq[2], dk[0], dk[1], dk[2], dv[0], dv[1], dv[2], qs[2], ks[2], qs[3],
                          1 if causal else 0, code, scale)
    except (struct.error, OverflowError) as e:
        raise CBRError(_INVALID, f"arguments: {e}") from None


def attention_workspace_size(q, k) -> tuple[int, int]:
    """Workspace bytes of (:func:`attention_forward`, :func:`attention_backward`) on operands of these shapes."""
    qs, ks, _, code, _ = _operands(q, k)
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    desc = _pack(qs, ks, code, 1.0, False, *([(0, 0, 0)] * 8))
    status = _load().cbr_attention_workspace_size(desc, ctypes.byref(f), ctypes.byref(b))
    if status != CBR_OK:
        raise CBRError(status, "cbr_attention_workspace_size")
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
    qs, ks, dt, code, index = _operands(q, k)
    sq, q_at = _heads(q, qs, dt, index, "q")
    sk, k_at = _heads(k, ks, dt, index, "k")
    sv, v_at = _heads(v, ks, dt, index, "v")
    n = qs[:1]
    lengths = _flat(key_lengths, n, torch.int32, index, "key_lengths")
    start = _flat(query_start, n, torch.int32, index, "query_start")
    rows = (qs[0], qs[2], qs[1])
    o = out.get("o") if out else None
    if o is None:
        o = _empty(qs, dt, index)
    so, o_at = _heads(o, qs, dt, index, "o")
    lse = lse_at = None
    if want_lse:
        lse = out.get("lse") if out else None
        if lse is None:
            lse = _new(rows, torch.float32, q.device)
        lse_at = _flat(lse, rows, torch.float32, index, "lse")
    desc = _pack(qs, ks, code, qs[3] ** -0.5 if scale is None else scale, causal, sq, sk, sv, so)
    ws, ws_at, ws_n = _workspace(qs, ks, code, index, ws, False)
    status = (_lib or _load()).cbr_attention_forward(desc, q_at, k_at, v_at, lengths, start, o_at, lse_at, ws_at, ws_n,
                                                     _raw_stream(index) if _raw_stream else _stream_of(q.device))
    if status != CBR_OK:
        raise CBRError(status, "cbr_attention_forward")
    return {"o": o, "lse": lse}


def attention_backward(do, q, k, v, o, lse, *, scale=None, causal=False, key_lengths=None, query_start=None, ws=None,
                       out=None) -> dict:
    """cbr_attention_backward -> dict(dq, dk, dv), contiguous where ``out`` does not give them.

    do: the gradient at o; o and lse from :func:`attention_forward`; the rest as there.  The gradients of a key
    head are summed over the query heads that read it, those of keys from key_lengths on are 0."""
    qs, ks, dt, code, index = _operands(q, k)
    sq, q_at = _heads(q, qs, dt, index, "q")
    sk, k_at = _heads(k, ks, dt, index, "k")
    sv, v_at = _heads(v, ks, dt, index, "v")
    so, o_at = _heads(o, qs, dt, index, "o")
    sdo, do_at = _heads(do, qs, dt, index, "do")
    n = qs[:1]
    lengths = _flat(key_lengths, n, torch.int32, index, "key_lengths")
    start = _flat(query_start, n, torch.int32, index, "query_start")
    lse_at = _flat(lse, (qs[0], qs[2], qs[1]), torch.float32, index, "lse")
    given = out.get if out else (lambda name: None)
    dq, dk, dv = given("dq"), given("dk"), given("dv")
    dq = _empty(qs, dt, index) if dq is None else dq
    dk = _empty(ks, dt, index) if dk is None else dk
    dv = _empty(ks, dt, index) if dv is None else dv
    sdq, dq_at = _heads(dq, qs, dt, index, "dq")
    sdk, dk_at = _heads(dk, ks, dt, index, "dk")
    sdv, dv_at = _heads(dv, ks, dt, index, "dv")
    desc = _pack(qs, ks, code, qs[3] ** -0.5 if scale is None else scale, causal, sq, sk, sv, so, sdo, sdq, sdk, sdv)
    ws, ws_at, ws_n = _workspace(qs, ks, code, index, ws, True)
    status = (_lib or _load()).cbr_attention_backward(desc, do_at, q_at, k_at, v_at, o_at, lse_at, lengths, start, dq_at, dk_at,
                                                      dv_at, ws_at, ws_n,
                                                      _raw_stream(index) if _raw_stream else _stream_of(q.device))
    if status != CBR_OK:
        raise CBRError(status, "cbr_attention_backward")
    return {"dq": dq, "dk": dk, "dv": dv}
