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
from .cbr import CBRError, _check, _stream

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


def _pack(form: struct.Struct, *values) -> bytes:
    """The descriptor; a number that its 32 bits cannot hold is refused like one that the library refuses."""
    try:
        return form.pack(*values)
    except (struct.error, OverflowError) as e:
        raise CBRError(_INVALID, f"arguments: {e}") from None


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        _bad(f"{what}: {t.dtype}", _UNSUPPORTED)
    return code


def _matrix(t: torch.Tensor, shape, dtype, dev, what: str) -> int:
    """Checks a [rows][width] tensor whose rows lie anywhere but are contiguous; its row stride."""
    if t.shape != shape or t.dtype != dtype or t.device != dev:
        _bad(f"{what} has to be {list(shape)} {dtype} on {dev}: {list(t.shape)} {t.dtype} on {t.device}")
    s, e = t.stride()
    if e != 1 and shape[1] > 1:
        _bad(f"{what}: a row has to be contiguous")
    return s if shape[0] > 1 else shape[1]


def _vector(t: torch.Tensor | None, n: int, dev, what: str):
    """Checks an optional contiguous fp32 tensor of n elements; its address."""
    if t is None:
        return None
    if t.numel() != n or t.dtype != torch.float32 or t.device != dev or not t.is_contiguous():
        _bad(f"{what} has to be {n} contiguous fp32 values on {dev}")
    return t.data_ptr()


# A small call's time is host time: torch's short ways to a new tensor, the current stream and the current
# device, where it has them.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_empty_cuda = getattr(getattr(getattr(torch._C, "_dynamo", None), "guards", None), "_empty_strided_cuda", None)


def _new(shape, dtype, dev) -> torch.Tensor:
    """A new contiguous tensor on the current device."""
    if _empty_cuda is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not shape:
        return _empty_cuda((), (), dtype)
    strides = [1]
    for n in shape[:0:-1]:
        strides.append(strides[-1] * (n or 1))
    return _empty_cuda(tuple(shape), tuple(strides[::-1]), dtype)


def _given(out: dict | None, name: str, shape, dtype, dev) -> torch.Tensor:
    """The caller's output of that name, or a new one."""
    if out and name in out:
        return out[name]
    return _new(shape, dtype, dev)


def _device_of(t: torch.Tensor):
    """The tensor's device, which has to be the current one: the library launches there."""
    dev = t.device
    if dev.index != _get_device():
        _bad(f"tensors on {dev}, which is not the current device", 5)
    return dev


def _stream_of(dev) -> int:
    return _raw_stream(dev.index) if _raw_stream is not None else _stream()


# ------------------------------------------------------------------------------- distillation

def _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits):
    """The packed descriptor and the addresses of the calls' common arguments."""
    if logits.dim() != 2 or not logits.is_cuda:
        _bad("logits have to be a [rows][vocab] CUDA tensor")
    shape, dev = logits.shape, _device_of(logits)
    rows, vocab = shape
    dtype = _dtype(logits, "logits")
    top_dtype = _dtype(top_logits, "top_logits")
    if top_ids.dtype not in (torch.int32, torch.int64):
        _bad(f"top_ids: {top_ids.dtype}", _UNSUPPORTED)
    k = top_ids.shape[-1] if top_ids.dim() else 0
    s = _matrix(logits, shape, logits.dtype, dev, "logits")
    s_id = _matrix(top_ids, (rows, k), top_ids.dtype, dev, "top_ids")
    s_top = _matrix(top_logits, (rows, k), top_logits.dtype, dev, "top_logits")
    s_out = vocab if dlogits is None else _matrix(dlogits, shape, logits.dtype, dev, "dlogits")
    desc = _pack(_DISTILL, rows, vocab, k, s, s_out, s_id, s_top, dtype, top_dtype, top_ids.element_size(),
                 float(temperature))
    return desc, (logits.data_ptr(), top_ids.data_ptr(), top_logits.data_ptr(),
                  _vector(teacher_lse, rows, dev, "teacher_lse"), _vector(row_weight, rows, dev, "row_weight"))


def distill_forward(logits, top_ids, top_logits, *, temperature=1.0, teacher_lse=None, row_weight=None,
                    out=None) -> dict:
    """cbr_distill_forward -> dict(loss [rows], stats [rows][3]), fp32.

    logits [rows][vocab]; top_ids (int32 or int64; an id outside the vocabulary marks an absent entry)
    and top_logits [rows][k]: the teacher's entries.  Without ``teacher_lse`` the teacher is renormalised
    over its entries; with it (the log-sum-exp of the teacher's logits / temperature over its whole
    vocabulary, [rows]) the mass it leaves out is one more class.  ``row_weight`` [rows] scales a row;
    0 masks it."""
    desc, args = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, None)
    rows, dev = logits.shape[0], logits.device
    loss = _given(out, "loss", (rows,), torch.float32, dev)
    stats = _given(out, "stats", (rows, 3), torch.float32, dev)
    _check(_load().cbr_distill_forward(desc, *args, _vector(loss, rows, dev, "loss"),
                                       _vector(stats, 3 * rows, dev, "stats"), _stream_of(dev)), "cbr_distill_forward")
    return {"loss": loss, "stats": stats}


def distill_backward(dloss, logits, top_ids, top_logits, stats, *, temperature=1.0, teacher_lse=None,
                     row_weight=None, out=None) -> torch.Tensor:
    """cbr_distill_backward -> dlogits [rows][vocab] (``out`` may be the logits themselves).

    dloss [rows] fp32 or None (ones); stats from :func:`distill_forward`; the rest as there."""
    dlogits = _new(logits.shape, logits.dtype, logits.device) if out is None and logits.is_cuda else out
    desc, args = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits)
    rows, dev = logits.shape[0], logits.device
    _check(_load().cbr_distill_backward(desc, _vector(dloss, rows, dev, "dloss"), *args,
                                        _vector(stats, 3 * rows, dev, "stats"), dlogits.data_ptr(), _stream_of(dev)),
           "cbr_distill_backward")
    return dlogits


def distill_forward_backward(logits, top_ids, top_logits, *, temperature=1.0, teacher_lse=None, row_weight=None,
                             out=None) -> dict:
    """cbr_distill_forward_backward -> dict(loss [rows], dlogits [rows][vocab]): the loss and its gradient
    (a mean is a row_weight of 1 / rows) with one read of the logits.  ``out`` may hold "dlogits" (the
    logits themselves, to save their memory), "loss" and "stats"."""
    dlogits = out["dlogits"] if out and "dlogits" in out else None
    if dlogits is None and logits.is_cuda:
        dlogits = _new(logits.shape, logits.dtype, logits.device)
    desc, args = _distill_args(logits, top_ids, top_logits, temperature, teacher_lse, row_weight, dlogits)
    rows, dev = logits.shape[0], logits.device
    loss = _given(out, "loss", (rows,), torch.float32, dev)
    stats = out.get("stats") if out else None
    _check(_load().cbr_distill_forward_backward(
        desc, *args, _vector(loss, rows, dev, "loss"), _vector(stats, 3 * rows, dev, "stats"), dlogits.data_ptr(),
        _stream_of(dev)), "cbr_distill_forward_backward")
    return {"loss": loss, "dlogits": dlogits} if stats is None else {"loss": loss, "dlogits": dlogits, "stats": stats}


# ------------------------------------------------------------------------------- block norms

def _kind(kind: str) -> int:
    if kind not in _KIND:
        _bad(f"kind {kind!r}: one of {sorted(_KIND)}")
    return _KIND[kind]


def _gate(gate, rows: int, dim: int, dev):
    """(rows of one gate, address, number of elements) of a gate [dim] or [groups][dim]."""
    if gate is None:
        return 0, None
    if gate.dtype != torch.float32 or gate.device != dev or gate.dim() not in (1, 2) or gate.shape[-1] != dim or \
            not gate.is_contiguous():
        _bad(f"gate has to be contiguous fp32 [{dim}] or [groups][{dim}] on {dev}")
    groups = gate.shape[0] if gate.dim() == 2 else 1
    if groups < 1 or rows % groups:
        _bad(f"{rows} rows do not split over {groups} gates")
    return max(1, rows // groups), gate.data_ptr()


def _forms(branch, post_weight, gate, pre_weight):
    if (branch is None) != (post_weight is None):
        _bad("branch and post_weight go together")
    if branch is None and gate is not None:
        _bad("a gate needs a branch")
    if branch is None and pre_weight is None:
        _bad("neither a branch nor a pre_weight")


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
    shape, dt, dev = x.shape, x.dtype, _device_of(x)
    rows, dim = shape
    dtype = _dtype(x, "x")
    s_x = _matrix(x, shape, dt, dev, "x")
    _forms(branch, post_weight, gate, pre_weight)
    s_f = s_xo = s_h = dim
    x_out = h = stats = f_at = xo_at = h_at = None
    if branch is not None:
        s_f = _matrix(branch, shape, dt, dev, "branch")
        x_out = _given(out, "x_out", shape, dt, dev)
        s_xo = _matrix(x_out, shape, dt, dev, "x_out")
        f_at, xo_at = branch.data_ptr(), x_out.data_ptr()
    if pre_weight is not None:
        h = _given(out, "h", shape, dt, dev)
        s_h = _matrix(h, shape, dt, dev, "h")
        h_at = h.data_ptr()
    if want_stats:
        stats = _given(out, "stats", (rows, 4), torch.float32, dev)
    gate_rows, gate_at = _gate(gate, rows, dim, dev)
    desc = _pack(_NORM, rows, dim, gate_rows, s_x, s_f, s_xo, s_h, 0, 0, 0, 0, dtype, _kind(kind), eps, residual_scale,
                 branch_scale)
    _check(_load().cbr_block_norm_forward(
        desc, x.data_ptr(), f_at, _vector(post_weight, dim, dev, "post_weight"), gate_at,
        _vector(pre_weight, dim, dev, "pre_weight"), xo_at, h_at, _vector(stats, 4 * rows, dev, "stats"),
        _stream_of(dev)), "cbr_block_norm_forward")
    return {"x_out": x_out, "h": h, "stats": stats}


_sizes: dict = {}   # block_norm_workspace_size's answers


def block_norm_workspace_size(rows: int, dim: int, dtype=torch.float16) -> int:
    """Workspace bytes of :func:`block_norm_backward` (they go by dim alone)."""
    size = _sizes.get(dim)
    if size is None:
        n = ctypes.c_size_t()
        desc = _pack(_NORM, rows, dim, 0, dim, dim, dim, dim, dim, dim, dim, dim, _DTYPE[dtype], 0, 1.0, 1.0, 1.0)
        _check(_load().cbr_block_norm_workspace_size(desc, ctypes.byref(n)), "cbr_block_norm_workspace_size")
        size = _sizes[dim] = n.value
    return size


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
    shape, dt, dev = given.shape, given.dtype, _device_of(given)
    rows, dim = shape
    dtype = _dtype(given, "the gradient")
    _forms(branch, post_weight, gate, pre_weight)
    if (pre_weight is None) != (dh is None):
        _bad("dh and pre_weight go together")
    if stats is None:
        _bad("the backward needs the forward's stats")
    s_f = s_xo = s_dxo = s_dh = s_df = dim
    dpre = dpost = dgate = dbranch = dxo_at = xo_at = dh_at = f_at = df_at = None
    if dx_out is not None:
        s_dxo = _matrix(dx_out, shape, dt, dev, "dx_out")
        dxo_at = dx_out.data_ptr()
    if pre_weight is not None:
        s_xo = _matrix(x_out, shape, dt, dev, "x_out")
        s_dh = _matrix(dh, shape, dt, dev, "dh")
        xo_at, dh_at = x_out.data_ptr(), dh.data_ptr()
        dpre = _given(out, "dpre_weight", (dim,), torch.float32, dev)
    gate_rows, gate_at = _gate(gate, rows, dim, dev)
    if branch is not None:
        s_f = _matrix(branch, shape, dt, dev, "branch")
        dbranch = _given(out, "dbranch", shape, dt, dev)
        s_df = _matrix(dbranch, shape, dt, dev, "dbranch")
        f_at, df_at = branch.data_ptr(), dbranch.data_ptr()
        dpost = _given(out, "dpost_weight", (dim,), torch.float32, dev)
        if gate is not None:
            dgate = _given(out, "dgate", gate.shape, torch.float32, dev)
            if rows == 0:
                dgate.zero_()
    dx = _given(out, "dx", shape, dt, dev)
    s_dx = _matrix(dx, shape, dt, dev, "dx")
    desc = _pack(_NORM, rows, dim, gate_rows, dim, s_f, s_xo, dim, s_dxo, s_dh, s_dx, s_df, dtype, _kind(kind), 1.0,
                 residual_scale, branch_scale)
    if ws is None:
        ws = _new((block_norm_workspace_size(rows, dim, dt),), torch.uint8, dev)
    elif ws.device != dev or not ws.is_contiguous():
        _bad(f"ws has to be contiguous on {dev}")
    _check(_load().cbr_block_norm_backward(
        desc, dxo_at, dh_at, xo_at, f_at, _vector(post_weight, dim, dev, "post_weight"), gate_at,
        _vector(pre_weight, dim, dev, "pre_weight"), _vector(stats, 4 * rows, dev, "stats"), dx.data_ptr(), df_at,
        _vector(dpost, dim, dev, "dpost_weight"), _vector(dgate, dgate.numel() if dgate is not None else 0, dev, "dgate"),
        _vector(dpre, dim, dev, "dpre_weight"), ws.data_ptr(), ws.numel() * ws.element_size(), _stream_of(dev)),
        "cbr_block_norm_backward")
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


def _heads(t, batch, tokens, head_dim, dtype, dev, what):
    """Checks a [batch][tokens][heads][head_dim] tensor; its strides, its heads and its address."""
    n = t.shape
    if len(n) != 4 or n[0] != batch or n[1] != tokens or n[3] != head_dim or t.dtype != dtype or t.device != dev:
        _bad(f"{what} has to be [{batch}][{tokens}][heads][{head_dim}] {dtype} on {dev}")
    sb, st, sh, se = t.stride()
    if se != 1:
        _bad(f"{what}: a head's elements have to be adjacent")
    return (sb, st, sh), n[2], t.data_ptr()


def _rotary(f, q, k, positions, freq, axis, layout, out):
    first = q if q is not None else k
    if first is None or first.dim() != 4 or not first.is_cuda:
        _bad("q or k has to be a [batch][tokens][heads][head_dim] CUDA tensor")
    batch, tokens, _, head_dim = first.shape
    dt, dev = first.dtype, _device_of(first)
    dtype = _dtype(first, "q and k")
    code = _LAYOUT.get(layout)
    if code is None:
        _bad(f"layout {layout!r}: one of {sorted(_LAYOUT)}")
    p = positions.shape
    if positions.dtype != torch.int32 or len(p) not in (2, 3) or positions.device != dev:
        _bad(f"positions have to be int32 [tokens][axes] or [batch][tokens][axes] on {dev}")
    if p[-2] != tokens or (len(p) == 3 and p[0] not in (1, batch)):
        _bad(f"positions {list(p)} do not go with {batch} x {tokens} tokens")
    sp = positions.stride()
    if len(p) == 2 or p[0] == 1:
        sp = (0,) + sp[-2:]
    pairs = freq.numel()
    if freq.dtype != torch.int64 or axis.dtype != torch.uint8 or axis.numel() != pairs or freq.device != dev or \
            axis.device != dev or not freq.is_contiguous() or not axis.is_contiguous():
        _bad("freq (int64) and axis (uint8) have to be contiguous, one each for every pair")
    none = (0, 0, 0)
    sq = sqo = sk = sko = none
    hq = hk = 0
    q_at = k_at = qo_at = ko_at = q_out = k_out = None
    if q is not None:
        sq, hq, q_at = _heads(q, batch, tokens, head_dim, dt, dev, "q")
        q_out = out[0] if out is not None else _new(q.shape, dt, dev)
        sqo, n, qo_at = _heads(q_out, batch, tokens, head_dim, dt, dev, "out[0]")
        if n != hq:
            _bad("out[0] has another number of heads")
    if k is not None:
        sk, hk, k_at = _heads(k, batch, tokens, head_dim, dt, dev, "k")
        k_out = out[1] if out is not None else _new(k.shape, dt, dev)
        sko, n, ko_at = _heads(k_out, batch, tokens, head_dim, dt, dev, "out[1]")
        if n != hk:
            _bad("out[1] has another number of heads")
    desc = _pack(_ROTARY, batch, tokens, *sq, *sk, *sqo, *sko, *sp, hq, hk, head_dim, 2 * pairs, p[-1], code, dtype)
    _check(getattr(_load(), f)(desc, q_at, k_at, positions.data_ptr(), freq.data_ptr(), axis.data_ptr(), qo_at, ko_at,
                               _stream_of(dev)), f)
    return q_out, k_out


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
