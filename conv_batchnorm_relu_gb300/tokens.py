"""Token operators of libcbr.so: what a trunk of blocks and a training objective need on top of a
CBR stem, whose NHWC feature map is a grid of tokens.

* :func:`distill_forward`, :func:`distill_backward`, :func:`distill_forward_backward` -- the
  distillation loss from a teacher's top logits and its gradient;
* :func:`block_norm_forward`, :func:`block_norm_backward` -- the norms after one block and before
  the next, with the block's gate and the residual scale, in one pass;
* :func:`rotary_forward`, :func:`rotary_backward` -- rotary positions over several axes, with
  :func:`rotary_table` and :func:`grid_positions` for their inputs.

``include/cbr.h`` has the formulas.  As in :mod:`conv_batchnorm_relu_gb300.cbr`, each call checks
its arguments, allocates what it returns (or takes it in ``out``), launches on the current stream
and raises :class:`~conv_batchnorm_relu_gb300.cbr.CBRError` on a refusal; there is no fallback.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import cbr
from .cbr import CBRError, _check, _ptr, _stream

_INVALID, _UNSUPPORTED = 1, 3
_DTYPE = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_KIND = {"rms": 0, "layer": 1}
_LAYOUT = {"halves": 0, "neighbours": 1}

# The descriptors of include/cbr.h, packed: rebuilt on every call, cheaper than a ctypes.Structure.
_DISTILL = struct.Struct("@7q3if")
_NORM = struct.Struct("@11q2i3f4x")
_ROTARY = struct.Struct("@17q7i4x")

_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = cbr.load()
        vp, d = ctypes.c_void_p, ctypes.c_char_p
        lib.cbr_distill_forward.argtypes = [d] + [vp] * 8
        lib.cbr_distill_backward.argtypes = [d] + [vp] * 9
        lib.cbr_distill_forward_backward.argtypes = [d] + [vp] * 9
        lib.cbr_block_norm_forward.argtypes = [d] + [vp] * 9
        lib.cbr_block_norm_workspace_size.argtypes = [d, ctypes.POINTER(ctypes.c_size_t)]
        lib.cbr_block_norm_backward.argtypes = [d] + [vp] * 14 + [ctypes.c_size_t, vp]
        lib.cbr_rotary_forward.argtypes = [d] + [vp] * 8
        lib.cbr_rotary_backward.argtypes = [d] + [vp] * 8
        for f in ("cbr_distill_forward", "cbr_distill_backward", "cbr_distill_forward_backward",
                  "cbr_block_norm_forward", "cbr_block_norm_workspace_size", "cbr_block_norm_backward",
                  "cbr_rotary_forward", "cbr_rotary_backward"):
            getattr(lib, f).restype = ctypes.c_int32
        _lib = lib
    return _lib


def _bad(what: str, status: int = _INVALID):
    raise CBRError(status, what)


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        _bad(f"{what}: {t.dtype}", _UNSUPPORTED)
    return code


def _matrix(t: torch.Tensor, rows: int, width: int, dtype, like: torch.Tensor, what: str) -> int:
    """Checks a [rows][width] tensor whose rows lie anywhere but are contiguous; its row stride."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != width or t.dtype != dtype or t.device != like.device:
        _bad(f"{what} has to be [{rows}][{width}] {dtype} on {like.device}: {list(t.shape)} {t.dtype} on {t.device}")
    s, e = t.stride()
    if e != 1 and width > 1:
        _bad(f"{what}: a row has to be contiguous")
    return s if rows > 1 else width


def _vector(t: torch.Tensor | None, n: int, like: torch.Tensor, what: str):
    """Checks an optional contiguous fp32 tensor of n elements."""
    if t is not None and (t.numel() != n or t.dtype != torch.float32 or t.device != like.device or
                          not t.is_contiguous()):
        _bad(f"{what} has to be {n} contiguous fp32 values on {like.device}")


def _given(out: dict | None, name: str, shape, dtype, like: torch.Tensor) -> torch.Tensor:
    """The caller's output of that name, or a new one."""
    if out and name in out:
        return out[name]
    return torch.empty(shape, dtype=dtype, device=like.device)


# ------------------------------------------------------------------------------- distillation

def _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits):
    if logits.dim() != 2 or not logits.is_cuda:
        _bad("logits have to be a [rows][vocab] CUDA tensor")
    rows, vocab = logits.shape
    dtype = _dtype(logits, "logits")
    top_dtype = _dtype(top_logits, "top_logits")
    if top_ids.dtype not in (torch.int32, torch.int64):
        _bad(f"top_ids: {top_ids.dtype}", _UNSUPPORTED)
    k = top_ids.shape[-1] if top_ids.dim() else 0
    s = _matrix(logits, rows, vocab, logits.dtype, logits, "logits")
    s_id = _matrix(top_ids, rows, k, top_ids.dtype, logits, "top_ids")
    s_top = _matrix(top_logits, rows, k, top_logits.dtype, logits, "top_logits")
    _vector(teacher_lse, rows, logits, "teacher_lse")
    _vector(row_weight, rows, logits, "row_weight")
    s_out = vocab if dlogits is None else _matrix(dlogits, rows, vocab, logits.dtype, logits, "dlogits")
    return _DISTILL.pack(rows, vocab, k, s, s_out, s_id, s_top, dtype, top_dtype, top_ids.element_size(),
                         float(temperature))


def distill_forward(logits, top_ids, top_logits, *, temperature=1.0, teacher_lse=None, row_weight=None,
                    out=None) -> dict:
    """cbr_distill_forward -> dict(loss [rows], stats [rows][3]), fp32.

    logits [rows][vocab]; top_ids (int32 or int64; an id outside the vocabulary marks an absent entry)
    and top_logits [rows][k]: the teacher's entries.  Without ``teacher_lse`` the teacher is renormalised
    over its entries; with it (the log-sum-exp of the teacher's logits / temperature over its whole
    vocabulary, [rows]) the mass it leaves out is one more class.  ``row_weight`` [rows] scales a row;
    0 masks it."""
    desc = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, None)
    rows = logits.shape[0]
    loss = _given(out, "loss", rows, torch.float32, logits)
    stats = _given(out, "stats", (rows, 3), torch.float32, logits)
    _vector(loss, rows, logits, "loss")
    _vector(stats, 3 * rows, logits, "stats")
    _check(_load().cbr_distill_forward(desc, _ptr(logits), _ptr(top_ids), _ptr(top_logits), _ptr(teacher_lse),
                                       _ptr(row_weight), _ptr(loss), _ptr(stats), _stream()), "cbr_distill_forward")
    return {"loss": loss, "stats": stats}


def distill_backward(dloss, logits, top_ids, top_logits, stats, *, temperature=1.0, teacher_lse=None,
                     row_weight=None, out=None) -> torch.Tensor:
    """cbr_distill_backward -> dlogits [rows][vocab] (``out`` may be the logits themselves).

    dloss [rows] fp32 or None (ones); stats from :func:`distill_forward`; the rest as there."""
    dlogits = torch.empty_like(logits, memory_format=torch.contiguous_format) if out is None else out
    desc = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits)
    rows = logits.shape[0]
    _vector(dloss, rows, logits, "dloss")
    _vector(stats, 3 * rows, logits, "stats")
    _check(_load().cbr_distill_backward(desc, _ptr(dloss), _ptr(logits), _ptr(top_ids), _ptr(top_logits),
                                        _ptr(teacher_lse), _ptr(row_weight), _ptr(stats), _ptr(dlogits), _stream()),
           "cbr_distill_backward")
    return dlogits


def distill_forward_backward(logits, top_ids, top_logits, *, temperature=1.0, teacher_lse=None, row_weight=None,
                             out=None) -> dict:
    """cbr_distill_forward_backward -> dict(loss [rows], dlogits [rows][vocab]): the loss and its gradient
    (a mean is a row_weight of 1 / rows) with one read of the logits.  ``out`` may hold "dlogits" (the
    logits themselves, to save their memory), "loss" and "stats"."""
    dlogits = out["dlogits"] if out and "dlogits" in out else torch.empty_like(
        logits, memory_format=torch.contiguous_format)
    desc = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits)
    rows = logits.shape[0]
    loss = _given(out, "loss", rows, torch.float32, logits)
    stats = out.get("stats") if out else None
    _vector(loss, rows, logits, "loss")
    _vector(stats, 3 * rows, logits, "stats")
    _check(_load().cbr_distill_forward_backward(
        desc, _ptr(logits), _ptr(top_ids), _ptr(top_logits), _ptr(teacher_lse), _ptr(row_weight), _ptr(loss),
        _ptr(stats), _ptr(dlogits), _stream()), "cbr_distill_forward_backward")
    return {"loss": loss, "dlogits": dlogits} if stats is None else {"loss": loss, "dlogits": dlogits, "stats": stats}


# ------------------------------------------------------------------------------- block norms

def _kind(kind: str) -> int:
    if kind not in _KIND:
        _bad(f"kind {kind!r}: one of {sorted(_KIND)}")
    return _KIND[kind]


def _gate_rows(gate, rows: int, dim: int, like) -> int:
    """Rows of one gate, from the gate's [dim] or [groups][dim]."""
    if gate is None:
        return 0
    if gate.dtype != torch.float32 or gate.device != like.device or gate.dim() not in (1, 2) or \
            gate.shape[-1] != dim or not gate.is_contiguous():
        _bad(f"gate has to be contiguous fp32 [{dim}] or [groups][{dim}] on {like.device}")
    groups = gate.shape[0] if gate.dim() == 2 else 1
    if groups < 1 or rows % groups:
        _bad(f"{rows} rows do not split over {groups} gates")
    return max(1, rows // groups)


def _norm_weights(x, branch, post_weight, gate, pre_weight, dim):
    if (branch is None) != (post_weight is None):
        _bad("branch and post_weight go together")
    if branch is None and gate is not None:
        _bad("a gate needs a branch")
    if branch is None and pre_weight is None:
        _bad("neither a branch nor a pre_weight")
    _vector(post_weight, dim, x, "post_weight")
    _vector(pre_weight, dim, x, "pre_weight")


def block_norm_forward(x, branch=None, post_weight=None, gate=None, pre_weight=None, *, kind="rms", eps=1e-6,
                       residual_scale=1.0, branch_scale=1.0, want_stats=True, out=None) -> dict:
    """cbr_block_norm_forward -> dict(x_out, h, stats).

        x_out = residual_scale * x + branch_scale * gate * norm(branch) * post_weight
        h     = norm(x_out) * pre_weight

    x and branch [rows][dim]; gate [dim], or [groups][dim] with rows / groups consecutive rows each, or
    None.  Without a branch there is no join: h is the norm of x and "x_out" is None.  Without a
    pre_weight "h" is None.  kind: "rms", or "layer" (the mean is taken off).  stats [rows][4] fp32
    serve the backward (None without want_stats)."""
    if x.dim() != 2 or not x.is_cuda:
        _bad("x has to be a [rows][dim] CUDA tensor")
    rows, dim = x.shape
    dtype = _dtype(x, "x")
    s_x = _matrix(x, rows, dim, x.dtype, x, "x")
    _norm_weights(x, branch, post_weight, gate, pre_weight, dim)
    s_f = s_xo = s_h = dim
    x_out = h = stats = None
    if branch is not None:
        s_f = _matrix(branch, rows, dim, x.dtype, x, "branch")
        x_out = _given(out, "x_out", (rows, dim), x.dtype, x)
        s_xo = _matrix(x_out, rows, dim, x.dtype, x, "x_out")
    if pre_weight is not None:
        h = _given(out, "h", (rows, dim), x.dtype, x)
        s_h = _matrix(h, rows, dim, x.dtype, x, "h")
    if want_stats:
        stats = _given(out, "stats", (rows, 4), torch.float32, x)
        _vector(stats, 4 * rows, x, "stats")
    desc = _NORM.pack(rows, dim, _gate_rows(gate, rows, dim, x), s_x, s_f, s_xo, s_h, 0, 0, 0, 0, dtype,
                      _kind(kind), eps, residual_scale, branch_scale)
    _check(_load().cbr_block_norm_forward(desc, _ptr(x), _ptr(branch), _ptr(post_weight), _ptr(gate),
                                          _ptr(pre_weight), _ptr(x_out), _ptr(h), _ptr(stats), _stream()),
           "cbr_block_norm_forward")
    return {"x_out": x_out, "h": h, "stats": stats}


def block_norm_workspace_size(rows: int, dim: int, dtype=torch.float16) -> int:
    """Workspace bytes of :func:`block_norm_backward`."""
    n = ctypes.c_size_t()
    desc = _NORM.pack(rows, dim, 0, dim, dim, dim, dim, dim, dim, dim, dim, _DTYPE[dtype], 0, 1.0, 1.0, 1.0)
    _check(_load().cbr_block_norm_workspace_size(desc, ctypes.byref(n)), "cbr_block_norm_workspace_size")
    return n.value


def block_norm_backward(dx_out, dh, x_out, branch=None, post_weight=None, gate=None, pre_weight=None, stats=None, *,
                        kind="rms", residual_scale=1.0, branch_scale=1.0, ws=None, out=None) -> dict:
    """cbr_block_norm_backward -> dict(dx, dbranch, dpost_weight, dgate, dpre_weight), None for what has no
    part in the call.

    dx_out: the gradient at x_out from later in the residual stream, or None; dh: that at h (None without
    a pre_weight); x_out: the forward's (without a branch: its x); stats: the forward's.  ws: a workspace of
    block_norm_workspace_size bytes to use instead of a new one."""
    given = dx_out if dx_out is not None else dh
    if given is None or given.dim() != 2 or not given.is_cuda:
        _bad("dx_out or dh has to be a [rows][dim] CUDA tensor")
    rows, dim = given.shape
    dt, dtype = given.dtype, _dtype(given, "the gradient")
    _norm_weights(given, branch, post_weight, gate, pre_weight, dim)
    if (pre_weight is None) != (dh is None):
        _bad("dh and pre_weight go together")
    if stats is None:
        _bad("the backward needs the forward's stats")
    _vector(stats, 4 * rows, given, "stats")
    s_f = s_xo = s_dxo = s_dh = s_df = dim
    if dx_out is not None:
        s_dxo = _matrix(dx_out, rows, dim, dt, given, "dx_out")
    dpre = dpost = dgate = dbranch = None
    if pre_weight is not None:
        s_xo = _matrix(x_out, rows, dim, dt, given, "x_out")
        s_dh = _matrix(dh, rows, dim, dt, given, "dh")
        dpre = _given(out, "dpre_weight", dim, torch.float32, given)
        _vector(dpre, dim, given, "dpre_weight")
    gate_rows = _gate_rows(gate, rows, dim, given)
    if branch is not None:
        s_f = _matrix(branch, rows, dim, dt, given, "branch")
        dbranch = _given(out, "dbranch", (rows, dim), dt, given)
        s_df = _matrix(dbranch, rows, dim, dt, given, "dbranch")
        dpost = _given(out, "dpost_weight", dim, torch.float32, given)
        _vector(dpost, dim, given, "dpost_weight")
        if gate is not None:
            dgate = _given(out, "dgate", gate.shape, torch.float32, given)
            _vector(dgate, gate.numel(), given, "dgate")
            if rows == 0:
                dgate.zero_()
    dx = _given(out, "dx", (rows, dim), dt, given)
    s_dx = _matrix(dx, rows, dim, dt, given, "dx")
    desc = _NORM.pack(rows, dim, gate_rows, dim, s_f, s_xo, dim, s_dxo, s_dh, s_dx, s_df, dtype, _kind(kind), 1.0,
                      residual_scale, branch_scale)
    lib = _load()
    if ws is None:
        n = ctypes.c_size_t()
        _check(lib.cbr_block_norm_workspace_size(desc, ctypes.byref(n)), "cbr_block_norm_workspace_size")
        ws = torch.empty(n.value, dtype=torch.uint8, device=given.device)
    _check(lib.cbr_block_norm_backward(
        desc, _ptr(dx_out), _ptr(dh), _ptr(x_out) if pre_weight is not None else None, _ptr(branch),
        _ptr(post_weight), _ptr(gate), _ptr(pre_weight), _ptr(stats), _ptr(dx), _ptr(dbranch), _ptr(dpost),
        _ptr(dgate), _ptr(dpre), _ptr(ws), ws.numel() * ws.element_size(), _stream()), "cbr_block_norm_backward")
    return {"dx": dx, "dbranch": dbranch, "dpost_weight": dpost, "dgate": dgate, "dpre_weight": dpre}


# ------------------------------------------------------------------------------- rotary positions

def rotary_table(pairs_per_axis, theta: float = 10000.0, *, order: str = "blocks", spectrum: str = "shared",
                 device="cuda") -> tuple[torch.Tensor, torch.Tensor]:
    """(freq int64 [pairs], axis uint8 [pairs]) of cbr_rotary_forward: made once, kept by the caller.

    pairs_per_axis: how many of a head's pairs follow each axis, as (8, 12, 12).  order "blocks": the
    first axis has the first pairs, and so on; "cycled": the axes take turns until theirs are used up.
    spectrum "shared": pair i of n turns by theta**(-i / n), whatever its axis; "own": the pairs of an
    axis, j of m, by theta**(-j / m)."""
    counts = [int(n) for n in pairs_per_axis]
    if not counts or min(counts) < 0 or sum(counts) < 1 or len(counts) > 8 or not theta > 0:
        _bad("pairs_per_axis: counts of 1 to 8 axes, and a theta above 0")
    if order == "blocks":
        axis = [a for a, n in enumerate(counts) for _ in range(n)]
    elif order == "cycled":
        axis = [a for j in range(max(counts)) for a, n in enumerate(counts) if j < n]
    else:
        _bad(f"order {order!r}: blocks or cycled")
    n, used, freq = len(axis), [0] * len(counts), []
    for i, a in enumerate(axis):
        if spectrum == "shared":
            f = theta ** (-i / n)
        elif spectrum == "own":
            f = theta ** (-used[a] / counts[a])
        else:
            _bad(f"spectrum {spectrum!r}: shared or own")
        used[a] += 1
        # a fraction of a turn in 64 bits; whole turns fall away
        turn = int(round(f / (2 * math.pi) * 2.0 ** 64)) & (2 ** 64 - 1)
        freq.append(turn - 2 ** 64 if turn >= 2 ** 63 else turn)
    return (torch.tensor(freq, dtype=torch.int64).to(device), torch.tensor(axis, dtype=torch.uint8).to(device))


def grid_positions(*extents: int, device="cuda") -> torch.Tensor:
    """Positions [tokens][axes] int32 of a grid's cells in row-major order: grid_positions(p, q) for
    the pixels of one image of an NHWC feature map."""
    axes = [torch.arange(n, dtype=torch.int32, device=device) for n in extents]
    return torch.stack(torch.meshgrid(*axes, indexing="ij"), -1).reshape(-1, len(extents))


def _heads(t, batch, tokens, head_dim, like, what):
    if t.dim() != 4 or t.shape[0] != batch or t.shape[1] != tokens or t.shape[3] != head_dim or \
            t.dtype != like.dtype or t.device != like.device:
        _bad(f"{what} has to be [{batch}][{tokens}][heads][{head_dim}] {like.dtype} on {like.device}")
    sb, st, sh, se = t.stride()
    if se != 1:
        _bad(f"{what}: a head's elements have to be adjacent")
    return sb, st, sh, t.shape[2]


def _rotary(f, q, k, positions, freq, axis, layout, out):
    first = q if q is not None else k
    if first is None or first.dim() != 4 or not first.is_cuda:
        _bad("q or k has to be a [batch][tokens][heads][head_dim] CUDA tensor")
    batch, tokens, _, head_dim = first.shape
    dtype = _dtype(first, "q and k")
    if layout not in _LAYOUT:
        _bad(f"layout {layout!r}: one of {sorted(_LAYOUT)}")
    if positions.dtype != torch.int32 or positions.dim() not in (2, 3) or positions.device != first.device:
        _bad(f"positions have to be int32 [tokens][axes] or [batch][tokens][axes] on {first.device}")
    if positions.shape[-2] != tokens or (positions.dim() == 3 and positions.shape[0] not in (1, batch)):
        _bad(f"positions {list(positions.shape)} do not go with {batch} x {tokens} tokens")
    sp = positions.stride()
    if positions.dim() == 2 or positions.shape[0] == 1:
        sp = (0,) + sp[-2:]
    pairs = freq.numel()
    if freq.dtype != torch.int64 or axis.dtype != torch.uint8 or axis.numel() != pairs or \
            not freq.is_contiguous() or not axis.is_contiguous() or freq.device != first.device or \
            axis.device != first.device:
        _bad("freq (int64) and axis (uint8) have to be contiguous, one each for every pair")
    strides, heads, res = [], [], []
    for i, t in enumerate((q, k)):
        if t is None:
            strides.append((0, 0, 0, 0, 0, 0))
            heads.append(0)
            res.append(None)
            continue
        sb, st, sh, n = _heads(t, batch, tokens, head_dim, first, "qk"[i])
        o = out[i] if out is not None else torch.empty_like(t, memory_format=torch.contiguous_format)
        ob, ot, oh, m = _heads(o, batch, tokens, head_dim, first, "out")
        if m != n:
            _bad("out has another number of heads")
        strides.append((sb, st, sh, ob, ot, oh))
        heads.append(n)
        res.append(o)
    (a, b) = strides
    desc = _ROTARY.pack(batch, tokens, *a[:3], *b[:3], *a[3:], *b[3:], *sp, heads[0], heads[1], head_dim, 2 * pairs,
                        positions.shape[-1], _LAYOUT[layout], dtype)
    lib = _load()
    _check(getattr(lib, f)(desc, _ptr(q), _ptr(k), _ptr(positions), _ptr(freq), _ptr(axis), _ptr(res[0]),
                           _ptr(res[1]), _stream()), f)
    return tuple(res)


def rotary_forward(q, k, positions, freq, axis, *, layout="halves", out=None) -> tuple:
    """cbr_rotary_forward -> (q rotated, k rotated); either may be None.

    q [batch][tokens][heads][head_dim] and k (its own number of heads) with any strides of the first
    three axes, as views of a fused product; positions int32 [tokens][axes] or [batch][tokens][axes];
    (freq, axis) from :func:`rotary_table`: the first 2 * pairs elements of each head are rotated, in
    pairs (i, i + pairs) ("halves") or (2 i, 2 i + 1) ("neighbours").  out: (q_out, k_out), which may be
    q and k themselves."""
    return _rotary("cbr_rotary_forward", q, k, positions, freq, axis, layout, out)


def rotary_backward(dq_out, dk_out, positions, freq, axis, *, layout="halves", out=None) -> tuple:
    """cbr_rotary_backward -> (dq, dk): the rotation by the opposite angle; arguments as the forward's."""
    return _rotary("cbr_rotary_backward", dq_out, dk_out, positions, freq, axis, layout, out)
