"""Plain 64-bit forms of the trunk operators, on the CPU, and the error bounds their kernels are held to.

The bounds are derived here, before any run.  u: the unit roundoff of the storage type; w = 2^-24, that of
the 32-bit arithmetic in between.  A product on the tensor cores adds exact products of 16-bit values in 32
bits, each step off by at most 2 w of the magnitudes added so far (rounded towards zero), so a sum of
n terms is off by 2 (n / 16 + 16) w of the sum of magnitudes at the most.
"""
import math

import torch

from token_reference import TINY, U, W, close, rounds  # noqa: F401


def mma(n: int) -> float:
    return 2 * (n / 16 + 16) * W


# ------------------------------------------------------------------------------- attention

def visible(batch, tq, tk, causal=False, lengths=None, start=None):
    j = torch.arange(tk)[None, None]
    n = torch.full((batch,), tk) if lengths is None else lengths.cpu().long().clamp(0, tk)
    see = (j < n[:, None, None]).expand(batch, tq, tk)
    if causal:
        first = torch.zeros(batch, dtype=torch.long) if start is None else start.cpu().long()
        see = see & (j <= first[:, None, None] + torch.arange(tq)[None, :, None])
    return see


def _operands(q, k, v, lengths):
    """[batch][heads_q][tokens][dim] in 64 bits, key heads repeated, padding zero."""
    group = q.shape[2] // k.shape[2]
    q, k, v = (t.detach().cpu().double().permute(0, 2, 1, 3) for t in (q, k, v))
    if lengths is not None:
        behind = torch.arange(k.shape[2])[None] >= lengths.cpu()[:, None]
        k, v = (t.masked_fill(behind[:, None, :, None], 0.0) for t in (k, v))
    return q, k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)


def attention(q, k, v, scale, causal=False, lengths=None, start=None):
    """dict(o, lse, p, o_bound, lse_bound) in the operands' layout (p: [batch][heads_q][tq][tk])."""
    dt, dim = q.dtype, q.shape[3]
    see = visible(q.shape[0], q.shape[1], k.shape[1], causal, lengths, start)[:, None]
    q, k, v = _operands(q, k, v, lengths)
    s = (scale * q @ k.transpose(-1, -2)).masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True) if s.shape[-1] else torch.full(s.shape[:-1] + (1,), -math.inf, dtype=s.dtype)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    e = torch.exp(s - top)
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    o, lse = p @ v, (top + torch.log(total))[..., 0]
    # a score's error: the product's, the largest score's (both enter the exponent), two roundings of it
    mag = scale * (q.abs() @ k.abs().transpose(-1, -2))
    es = (mma(dim) + 4 * W) * torch.where(see, mag, torch.zeros_like(mag))
    es = es + es.amax(-1, keepdim=True) if s.shape[-1] else es
    n = s.shape[-1]
    # p enters the second product rounded to the storage type (f16: 2^6 times as large, so its subnormals are
    # 2^-31 of the largest p); the exponential is good to 4 w and a rescaling of the sums to 2 w each
    ep = U[dt] + 2.0 ** -30 + es + 32 * W
    o_bound = (ep * p) @ v.abs() + (mma(n) + rounds(n)) * (p @ v.abs()) + (2.0 ** -31 * (p > 0).double()) @ v.abs()
    lse_bound = (es * p).sum(-1) + (es.amax(-1) if n else 0.0) + rounds(n) + 32 * W + 4 * W * torch.where(
        torch.isinf(lse), torch.zeros_like(lse), lse.abs())
    back = lambda t: t.permute(0, 2, 1, 3)  # noqa: E731
    return {"o": back(o), "lse": lse, "p": p, "es": es, "o_bound": back(o_bound), "lse_bound": lse_bound}


def attention_backward(do, q, k, v, o, lse, scale, causal=False, lengths=None, start=None):
    """dict(dq, dk, dv, dq_bound, ...) of the formulas of include/cbr.h for these o and lse."""
    dt, dim, group = q.dtype, q.shape[3], q.shape[2] // k.shape[2]
    tq, tk = q.shape[1], k.shape[1]
    see = visible(q.shape[0], tq, tk, causal, lengths, start)[:, None]
    q, k, v = _operands(q, k, v, lengths)
    do, o, lse = do.cpu().double().permute(0, 2, 1, 3), o.cpu().double().permute(0, 2, 1, 3), lse.cpu().double()
    s = scale * q @ k.transpose(-1, -2)
    p = torch.exp(torch.where(see, s - lse[..., None], torch.full_like(s, -math.inf)))
    delta = (do * o).sum(-1, keepdim=True)
    dp = do @ v.transpose(-1, -2)
    ds = p * (dp - delta)
    dv, dq, dk = p.transpose(-1, -2) @ do, scale * ds @ k, scale * ds.transpose(-1, -2) @ q
    mag = torch.where(see, scale * (q.abs() @ k.abs().transpose(-1, -2)) + lse.abs().masked_fill(torch.isinf(lse), 0.0)[..., None],
                      torch.zeros_like(s))
    ep = (mma(dim) + 4 * W) * mag + 16 * W
    edp = (mma(dim) + 4 * W) * (do.abs() @ v.abs().transpose(-1, -2) + (do.abs() * o.abs()).sum(-1, keepdim=True))
    # f16: p and ds are scaled before they are rounded; what is left of the subnormals is 2^-36 of the largest p and
    # 2^-30 of the largest |do| |v|, as lengths of vectors
    low = 2.0 ** -36 * see.double()
    ds_low = torch.zeros_like(p)
    if dt == torch.float16 and tk and tq:
        big = do.norm(dim=-1).amax(-1)[..., None, None] * torch.maximum(v.norm(dim=-1), o.norm(dim=-1).amax(-1, keepdim=True)).amax(-1)[..., None, None]
        big = big.amax(1, keepdim=True)
        ds_low = 2.0 ** -30 * big * see
    e_p = p * (U[dt] + ep) + low
    # p itself is a 32-bit number: below 2^-126 its exponential is 0, so ds is off by that much of |dp - D|
    e_ds = ds.abs() * (U[dt] + ep + 4 * W) + p * (1 + ep) * edp + ds_low + 2.0 ** -126 * (dp - delta).abs() * see
    nq, nk = tq * group, tk
    dv_b = e_p.transpose(-1, -2) @ do.abs() + mma(nq) * (p.transpose(-1, -2) @ do.abs())
    dq_b = scale * (e_ds @ k.abs() + mma(nk) * (ds.abs() @ k.abs()))
    dk_b = scale * (e_ds.transpose(-1, -2) @ q.abs() + mma(nq) * (ds.abs().transpose(-1, -2) @ q.abs()))

    def shared(t):
        b, h = t.shape[:2]
        return t.reshape(b, h // group, group, tk, dim).sum(2).permute(0, 2, 1, 3)

    return {"dq": dq.permute(0, 2, 1, 3), "dk": shared(dk), "dv": shared(dv), "dq_bound": dq_b.permute(0, 2, 1, 3) * (1 + 8 * W),
            "dk_bound": shared(dk_b) * (1 + 8 * W), "dv_bound": shared(dv_b) * (1 + 8 * W)}


# ------------------------------------------------------------------------------- group norm

def sums(n: int) -> float:
    """A sum of n terms over at least 32 lanes that take turns, then trees of them."""
    return (n / 32 + 48) * W


def _groups(x, groups):
    n, c = x.shape[0], x.shape[-1]
    return x.reshape(n, -1, groups, c // groups)


def activation(z, act):
    if act == "relu":
        return z.clamp(min=0)
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def slope(z, act):
    if act == "relu":
        return (z > 0).double()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def group_norm(x, gamma, beta, groups, eps, act):
    dt, shape = x.dtype, x.shape
    x = _groups(x.cpu().double(), groups)
    c = shape[-1]
    gamma = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.cpu().double()
    beta = torch.zeros(c, dtype=torch.float64) if beta is None else beta.cpu().double()
    n = x.shape[1] * x.shape[3]
    mean = x.mean((1, 3), keepdim=True)
    var = ((x - mean) ** 2).mean((1, 3), keepdim=True)
    rstd = (var + eps).rsqrt()
    xh = ((x - mean) * rstd)
    z = xh.reshape(shape) * gamma + beta
    # means are merged from shifted partial sums: off by a sum's rounding of the deviations and of the mean itself
    dev = (x - mean).abs().mean((1, 3), keepdim=True)
    em = 2 * sums(n) * dev + 4 * W * mean.abs()
    er = rstd * (4 * sums(n) * var + em ** 2 + 4 * em * dev) * rstd ** 2 + 4 * W * rstd
    ex = (xh.abs() * (er / rstd + 4 * W) + rstd * em).reshape(shape)
    bound = 1.1 * (ex * gamma.abs() + 2 * W * (xh.reshape(shape) * gamma).abs() + 2 * W * z.abs()) + 16 * W * z.abs()
    return {"y": activation(z, act), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0], "y_bound": bound,
            "mean_bound": em[:, 0, :, 0], "rstd_bound": er[:, 0, :, 0], "dtype": dt}


def group_norm_backward(dy, x, gamma, beta, mean, rstd, groups, act):
    """dict(dx, dgamma, dbeta and their bounds) of the formulas for these statistics.  Where z is nearer to the
    ReLU's edge than its own rounding, either side is right: the bounds allow for both."""
    shape = x.shape
    c = shape[-1]
    x, dy = _groups(x.cpu().double(), groups), dy.cpu().double()
    gamma = torch.ones(c, dtype=torch.float64) if gamma is None else gamma.cpu().double()
    beta = torch.zeros(c, dtype=torch.float64) if beta is None else beta.cpu().double()
    mean, rstd = mean.cpu().double()[:, None, :, None], rstd.cpu().double()[:, None, :, None]
    xh = (x - mean) * rstd
    flat = xh.reshape(shape)
    z = flat * gamma + beta
    g = dy * slope(z, act)
    unsure = torch.zeros_like(g)
    if act == "relu":
        unsure = dy.abs() * (z.abs() <= 8 * W * ((flat * gamma).abs() + beta.abs()))
    eg = g.abs() * 8 * W + unsure + (dy.abs() * 64 * W * (1 + z.abs()) if act == "silu" else 0.0)
    n = x.shape[1] * x.shape[3]
    u, eu = _groups(g * gamma, groups), _groups(eg * gamma.abs(), groups)
    m1, m2 = u.mean((1, 3), keepdim=True), (u * xh).mean((1, 3), keepdim=True)
    e1 = sums(n) * u.abs().mean((1, 3), keepdim=True) + eu.mean((1, 3), keepdim=True)
    e2 = (sums(n) + 8 * W) * (u * xh).abs().mean((1, 3), keepdim=True) + (eu * xh.abs()).mean((1, 3), keepdim=True)
    dx = rstd * (u - m1 - xh * m2)
    ex = 4 * W * xh.abs() + 2 * W * rstd * mean.abs()   # the difference is rounded once, at the mean's size at most
    bound = rstd * (eu + e1 + xh.abs() * e2 + ex * m2.abs() + 8 * W * (u.abs() + m1.abs() + (xh * m2).abs()))
    axes = tuple(range(len(shape) - 1))
    rows = n * x.shape[0] // (c // groups)
    exf = ex.reshape(shape)
    dgamma, dbeta = (g * flat).sum(axes), g.sum(axes)
    return {"dx": dx.reshape(shape), "dgamma": dgamma, "dbeta": dbeta, "dx_bound": bound.reshape(shape),
            "dgamma_bound": (sums(rows) * (g * flat).abs() + eg * flat.abs() + g.abs() * exf).sum(axes),
            "dbeta_bound": (sums(rows) * g.abs() + eg).sum(axes)}


# ------------------------------------------------------------------------------- clipping

def clip(grads, max_norm, unscale=1.0):
    """(norm, scale, scaled gradients) in 64 bits."""
    total = math.fsum(float((g.cpu().double() ** 2).sum()) for g in grads)
    norm = unscale * math.sqrt(total)
    scale = unscale * min(1.0, max_norm / norm) if norm > 0 else unscale
    return norm, scale, [g.cpu().double() * scale for g in grads]
