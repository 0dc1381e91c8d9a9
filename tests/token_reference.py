"""Plain 64-bit forms of the token operators, on the CPU, and the error bounds their kernels are held to.

The bounds are derived here, before any run, from the unit roundoffs: u of the storage type (one
rounding of the result; 2^-24, 2^-11, 2^-8 for f32, f16, bf16, and the smallest subnormal of the
f16 where a result underflows) and w = 2^-24 of the 32-bit arithmetic in between, times a count of
roundings and the magnitudes that enter: a sum of n terms is taken in partial sums of at most n / 32
terms each (a warp) and a tree, so it is good to (n / 32 + 16) w of the sum of its terms' magnitudes.
"""
import math

import torch

W = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}
HUGE = 1e300
INF = math.inf


def rounds(n: int) -> float:
    return (n / 32 + 16) * W


def close(got, want, bound, name, dtype=torch.float32):
    """|got - want| <= bound + the result's own rounding, and the same infinities and NaN."""
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{name}: NaN in other places"
    big = torch.isinf(want)
    assert torch.equal(got[big], want[big]) and not torch.isinf(got[~big]).any(), f"{name}: infinities differ"
    ok = ~big & ~torch.isnan(want)
    if not bool(ok.any()):
        return
    allowed = (bound + U[dtype] * want.abs() + TINY[dtype])[ok]
    err = (got - want).abs()[ok]
    worst = int(torch.argmax(err - allowed))
    assert bool((err <= allowed).all()), f"{name}: error {float(err[worst]):.3g} > {float(allowed[worst]):.3g}"


# ------------------------------------------------------------------------------- distillation

def distill(logits, ids, top, temperature=1.0, teacher_lse=None, row_weight=None):
    """dict(loss, dlogits, stats, loss_bound, grad_bound) of the formulas of include/cbr.h."""
    r, v = logits.shape
    z = logits.cpu().double()
    ids, top = ids.cpu().long(), top.cpu().double()
    k = ids.shape[1]
    w = torch.ones(r, dtype=torch.float64) if row_weight is None else row_weight.cpu().double()
    out = {"loss": torch.zeros(r, dtype=torch.float64), "dlogits": torch.zeros(r, v, dtype=torch.float64),
           "stats": torch.zeros(r, 3, dtype=torch.float64), "loss_bound": torch.zeros(r, dtype=torch.float64),
           "grad_bound": torch.zeros(r, v, dtype=torch.float64)}
    for i in range(r):
        here = [j for j in range(k) if 0 <= int(ids[i, j]) < v]
        if float(w[i]) == 0 or not here:
            continue
        at = ids[i, here]
        t = top[i, here] / temperature
        if teacher_lse is None:
            if bool((t == -INF).all()):
                continue
            p = torch.exp(t - torch.logsumexp(t, 0))
        else:
            p = torch.exp(t - float(teacher_lse[i]))
        if bool((z[i] == -INF).all()):
            continue
        x = z[i] / temperature
        top_x = x.max()
        e = torch.exp(x - top_x)
        total = e.sum()
        q = e / total
        log_q = x - top_x - torch.log(total)
        listed = torch.zeros(v, dtype=torch.bool)
        listed[at] = True
        unlisted = e[~listed].sum()
        q_rest = unlisted / total
        rest = 0.0
        if teacher_lse is not None and not float(q_rest) == 0:
            rest = max(0.0, float(1 - p.sum()))
        terms = torch.where(p == 0, torch.zeros_like(p), p * (torch.log(p) - log_q[at]))
        loss = terms.sum()
        # each term: the two logarithms and their arguments to some roundings, the sums inside them
        per = rounds(v) + rounds(k) + 16 * W
        mag = (p * (1 + torch.log(p.clamp(min=1e-300)).abs() + log_q[at].abs().clamp(max=HUGE)
                    + t.abs().clamp(max=HUGE))).sum()
        bound = mag * per
        if rest > 0:
            loss = loss + rest * (math.log(rest) - torch.log(q_rest))
            # rest = 1 - sum p: an absolute error of the sum's
            bound = bound + (p.sum() + 1) * per * (1 + abs(math.log(rest)) + abs(float(torch.log(q_rest)))) \
                + rest * per
        full = torch.zeros(v, dtype=torch.float64)
        full.index_add_(0, at, p)
        grad = q * (p.sum() + rest) - full
        gb = (q * (1 + log_q.abs().clamp(max=200.0)) * (p.sum() + 1) + full * (1 + t.abs().max().clamp(max=HUGE))) * per
        if rest > 0:
            grad = torch.where(listed, grad, grad - q * rest / q_rest)
            gb = gb + torch.where(listed, torch.zeros_like(q), q / q_rest * (p.sum() + 1) * (2 + log_q.abs().clamp(max=200.0)) * per)
        # an exponential (at most 1 before it is scaled) below the normal range
        gb = gb + 2.0 ** -149 * (p.sum() + 1 + (rest / q_rest if rest > 0 else 0.0))
        s = float(w[i]) * temperature
        out["loss"][i], out["loss_bound"][i] = loss * s * temperature, bound * abs(s) * temperature
        out["dlogits"][i], out["grad_bound"][i] = grad * s, gb * abs(s)
        out["stats"][i] = torch.stack([z[i].max(), total, unlisted])
    return out


# ------------------------------------------------------------------------------- block norms

def _norm(a, kind, eps):
    m = a.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(a[:, :1])
    return m, ((a - m).pow(2).mean(1, keepdim=True) + eps).rsqrt()


def _cpu(t):
    return None if t is None else t.detach().cpu().double()


def norm_forward(x, branch, w1, gate, w2, kind, eps, rho, beta):
    x, branch, w1, gate, w2 = map(_cpu, (x, branch, w1, gate, w2))
    rows, dim = x.shape
    zero = torch.zeros(rows, 1, dtype=torch.float64)
    m1 = r1 = m2 = r2 = zero
    out = {"x_out": None, "h": None}
    c = rounds(dim) + 16 * W
    mag, joined = x.abs(), x
    if branch is not None:
        m1, r1 = _norm(branch, kind, eps)
        g = torch.ones(1, dim, dtype=torch.float64) if gate is None else gate.reshape(-1, dim)
        g = g.repeat_interleave(max(1, rows // g.shape[0]), 0)[:rows] if rows else g[:0]
        n = (branch - m1) * r1 * w1
        joined = rho * x + beta * g * n
        # the branch's mean cancels in (f - m1): its magnitude counts
        mag = (rho * x).abs() + (beta * g * w1).abs() * r1 * (branch.abs() + branch.abs().mean(1, keepdim=True))
        out["x_out"], out["x_bound"] = joined, mag * c
    if w2 is not None:
        m2, r2 = _norm(joined, kind, eps)
        out["h"] = (joined - m2) * r2 * w2
        lift = mag + mag.pow(2).mean(1, keepdim=True).sqrt() * (1 + ((joined - m2) * r2).abs())
        out["h_bound"] = r2 * w2.abs() * lift * c
    out["stats"] = torch.cat([m1, r1, m2, r2], 1)
    return out


def norm_backward(dx_out, dh, x_out, branch, w1, gate, w2, stats, kind, rho, beta):
    dx_out, dh, x_out, branch, w1, gate, w2, stats = map(_cpu, (dx_out, dh, x_out, branch, w1, gate, w2, stats))
    rows, dim = (dx_out if dx_out is not None else dh).shape
    m1, r1, m2, r2 = stats.split(1, 1)
    c = rounds(dim) + 32 * W
    rows_c = rounds(rows) + c
    center = kind == "layer"
    d = torch.zeros(rows, dim, dtype=torch.float64) if dx_out is None else dx_out
    mag = d.abs()
    out = dict.fromkeys(("dx", "dbranch", "dpost_weight", "dgate", "dpre_weight"))

    def pull(up, unit, rstd):
        return rstd * (up - (up.mean(1, keepdim=True) if center else 0.0) - unit * (up * unit).mean(1, keepdim=True))

    def pull_mag(up, unit, unit_mag, rstd):
        return rstd * (up + up.mean(1, keepdim=True) + unit_mag * (up * unit_mag).mean(1, keepdim=True))

    if w2 is not None:
        unit = (x_out - m2) * r2
        unit_mag = (x_out.abs() + m2.abs()) * r2
        d = d + pull(dh * w2, unit, r2)
        mag = mag + pull_mag((dh * w2).abs(), unit, unit_mag, r2)
        out["dpre_weight"] = (dh * unit).sum(0)
        out["dpre_bound"] = (dh.abs() * unit_mag).sum(0) * rows_c
    if branch is not None:
        unit = (branch - m1) * r1
        unit_mag = (branch.abs() + m1.abs()) * r1
        groups = 1 if gate is None else gate.reshape(-1, dim).shape[0]
        g = torch.ones(1, dim, dtype=torch.float64) if gate is None else gate.reshape(-1, dim)
        g = g.repeat_interleave(max(1, rows // groups), 0)[:rows]
        b, bm = beta * d, abs(beta) * mag
        if gate is not None:
            per = (b * unit * w1).reshape(groups, -1, dim)
            out["dgate"] = per.sum(1).reshape(gate.shape)
            out["dgate_bound"] = ((bm * unit_mag * w1.abs()).reshape(groups, -1, dim).sum(1) * rows_c).reshape(gate.shape)
        out["dpost_weight"] = (b * g * unit).sum(0)
        out["dpost_bound"] = (bm * g.abs() * unit_mag).sum(0) * rows_c
        out["dbranch"] = pull(b * g * w1, unit, r1)
        out["dbranch_bound"] = pull_mag(bm * (g * w1).abs(), unit, unit_mag, r1) * c
        d, mag = rho * d, abs(rho) * mag
    out["dx"], out["dx_bound"] = d, mag * c
    return out


# ------------------------------------------------------------------------------- rotary positions

def rotary(a, positions, freq, axis, layout, backward=False):
    """(rotated, bound): angles from whole numbers, modulo 2^64 as Python has them."""
    a = a.detach().cpu().double()
    b, t, h, d = a.shape
    pos = positions.cpu()
    pos = pos[None] if pos.dim() == 2 else pos
    pos = pos.expand(b, -1, -1).tolist()
    f, ax = [v % 2 ** 64 for v in freq.tolist()], axis.tolist()
    n = len(f)
    turns = [[[(pos[i][j][ax[p]] * f[p] % 2 ** 64) / 2.0 ** 64 for p in range(n)] for j in range(t)] for i in range(b)]
    angle = torch.tensor(turns, dtype=torch.float64).reshape(b, t, n) * (2 * math.pi)
    if backward:
        angle = -angle
    cos, sin = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    one = slice(0, n) if layout == "halves" else slice(0, 2 * n, 2)
    two = slice(n, 2 * n) if layout == "halves" else slice(1, 2 * n, 2)
    out, bound = a.clone(), torch.zeros_like(a)
    x1, x2 = a[..., one], a[..., two]
    out[..., one], out[..., two] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    # the angle to 2^-24 of half a turn and 2^-32 of one, its functions and the products to a rounding or two
    bound[..., one] = bound[..., two] = (x1.abs() + x2.abs()) * 8 * W
    return out, bound
