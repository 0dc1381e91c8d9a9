"""The token operators (conv_batchnorm_relu_gb300.tokens) as measured cases: a distillation loss
from a teacher's top logits, the norms around a gated residual block, and rotary positions over
several axes.  They are the parts of one training step of a hybrid student: a Conv-BN-ReLU stem
whose NHWC feature map becomes a grid of tokens, a trunk of blocks on those tokens, and a loss
against a teacher's stored logits.

``run`` computes an operator either in elementary torch operations (``own = False``: products,
sums, exponentials and indexing in 32 bits, rounded once at the end) or through the package's
kernels (``own = True``).  ``exact`` is the same definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
FORMS = {"pre": (0, 1), "post": (1, 0), "both": (1, 1)}   # (branch joins the residual, next norm)


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # a small batch of image-class logits (1000 classes) against a teacher's ten best: latency
        dict(name="distill_step_8x1000", op="distill", mode="step", rows=8, vocab=1000, topk=10, dtype="f32",
             temperature=2.0, tail=False, masked=0.0, ragged=False, dead=0),
        # a training step's loss and gradient, 2048 tokens of a 32000-word vocabulary
        dict(name="distill_step_2048x32000", op="distill", mode="step", rows=2048, vocab=32000, topk=64, dtype="bf16",
             temperature=1.0, tail=False, masked=0.0, ragged=False, dead=0),
        # loss and gradient as two calls (an autograd pair) on an odd vocabulary, whose rows start at
        # every 2-byte phase; padding tokens masked, the teacher cut at a share of its mass, tail class
        dict(name="distill_pair_1021x50257", op="distill", mode="pair", rows=1021, vocab=50257, topk=33, dtype="f16",
             temperature=2.0, tail=True, masked=0.3, ragged=True, dead=0),
        # the largest step: 4096 tokens of a 131072-word vocabulary, the last columns padding
        dict(name="distill_step_4096x131072", op="distill", mode="step", rows=4096, vocab=131072, topk=128,
             dtype="bf16", temperature=2.0, tail=True, masked=0.0, ragged=False, dead=100),
        # one token through the join of a block: the smallest call
        dict(name="norm_forward_1x2048", op="norm", mode="forward", form="both", kind="rms", rows=1, dim=2048,
             groups=1, dtype="bf16"),
        # the backward over a 56x56x64 feature map's tokens, 16 images, a gate for each image
        dict(name="norm_backward_50176x64", op="norm", mode="backward", form="both", kind="layer", rows=50176, dim=64,
             groups=16, dtype="f16"),
        # an odd width: no row but the first starts on a 16-byte boundary
        dict(name="norm_forward_4099x1001", op="norm", mode="forward", form="both", kind="layer", rows=4099, dim=1001,
             groups=1, dtype="f32"),
        # the join of a wide block, forward and backward: 8 sequences of 4096 tokens
        dict(name="norm_forward_32768x4096", op="norm", mode="forward", form="both", kind="rms", rows=32768, dim=4096,
             groups=8, dtype="bf16"),
        dict(name="norm_backward_32768x4096", op="norm", mode="backward", form="both", kind="rms", rows=32768, dim=4096,
             groups=8, dtype="bf16"),
        # one new token's queries and keys
        dict(name="rotary_forward_1x1", op="rotary", mode="forward", batch=1, t=1, y=1, x=1, heads_q=16, heads_k=4,
             head_dim=128, rot_dim=128, layout="halves", fused=False, dtype="bf16"),
        # the backward on views of a fused query/key/value product, 2 clips of 8 frames of 28x28
        # positions, part of each head rotated, neighbouring pairs
        dict(name="rotary_backward_2x8x28x28", op="rotary", mode="backward", batch=2, t=8, y=28, x=28, heads_q=12,
             heads_k=12, head_dim=80, rot_dim=72, layout="neighbours", fused=True, dtype="f16"),
        # long sequences with shared key heads
        dict(name="rotary_forward_2x32x32x32", op="rotary", mode="forward", batch=2, t=32, y=32, x=32, heads_q=32,
             heads_k=8, head_dim=128, rot_dim=128, layout="halves", fused=False, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["distill", "norm", "rotary"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "distill":
        while True:
            rows, vocab = _spread(rng, 1, 4096), _spread(rng, 100, 131072)
            if vocab != 3072 and rows != 3072 and rows * vocab * SIZE[dtype] <= 4096 * 131072:
                break
        return dict(op=op, mode=rng.choice(["step", "pair", "forward"]), rows=rows, vocab=vocab,
                    topk=min(_spread(rng, 1, 128), vocab), dtype=dtype, temperature=rng.choice([1.0, 2.0, 4.0]),
                    tail=rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.25]), ragged=rng.random() < 0.5,
                    dead=rng.choice([0, 0, 17]))
    if op == "norm":
        while True:
            groups, per = rng.choice([0, 1, 1, 3, 8]), _spread(rng, 1, 16384)
            rows, dim = per * max(1, groups), _spread(rng, 32, 4096)
            if rng.random() < 0.6:
                dim = dim // 8 * 8
            if rows <= 32768 and dim != 3072 and rows != 3072 and rows * dim * SIZE[dtype] <= 32768 * 4096:
                break
        return dict(op=op, mode=rng.choice(["forward", "backward"]), form=rng.choice(["both", "both", "pre", "post"]),
                    kind=rng.choice(["rms", "layer"]), rows=rows, dim=dim, groups=groups, dtype=dtype)
    while True:
        batch, t, y, x = rng.choice([1, 2, 3]), _spread(rng, 1, 32), _spread(rng, 1, 48), _spread(rng, 1, 48)
        heads_k = rng.choice([1, 2, 4, 8])
        heads_q, head_dim = heads_k * rng.choice([1, 2, 3, 4]), rng.choice([40, 64, 72, 80, 96, 128, 256])
        n = batch * t * y * x * (heads_q + heads_k) * head_dim * SIZE[dtype]
        if n <= 2 * 32768 * 40 * 128 and 3072 not in (t * y * x, batch * t * y * x, heads_q * head_dim):
            break
    return dict(op=op, mode=rng.choice(["forward", "backward"]), batch=batch, t=t, y=y, x=x, heads_q=heads_q,
                heads_k=heads_k, head_dim=head_dim, rot_dim=head_dim - rng.choice([0, 0, 8]),
                layout=rng.choice(["halves", "neighbours"]), fused=rng.random() < 0.5, dtype=dtype)


def _masked_rows(case):
    return int(case["masked"] * case["rows"])


def work(case):
    """Each input read once, each output written once; a masked row is not read, its zeros are written."""
    e = SIZE[case["dtype"]]
    if case["op"] == "distill":
        r, v, k = case["rows"], case["vocab"], case["topk"]
        live = r - _masked_rows(case)
        reads = {"forward": 1, "step": 1, "pair": 2}[case["mode"]]
        b = live * v * e * reads + live * k * (4 + e) + r * 8
        if case["mode"] != "forward":
            b += r * v * e
        return {"bytes": b, "flops": live * v * (5 if case["mode"] == "forward" else 9)}
    if case["op"] == "norm":
        join, nxt = FORMS[case["form"]]
        n = case["rows"] * case["dim"]
        small = 4 * case["dim"] * (join + nxt + (case["groups"] if join else 0)) + 16 * case["rows"]
        if case["mode"] == "forward":   # x (and the branch) in; x_out and / or h out
            return {"bytes": n * e * (1 + join + join + nxt) + small, "flops": n * (6 * join + 4 * nxt)}
        # x_out and dh for the second norm, dx_out, the branch; dx and dbranch out
        return {"bytes": n * e * (2 * nxt + 1 + join + 1 + join) + 2 * small, "flops": n * (14 * join + 10 * nxt)}
    tokens = case["batch"] * case["t"] * case["y"] * case["x"]
    n = tokens * (case["heads_q"] + case["heads_k"])
    return {"bytes": 2 * n * case["head_dim"] * e + 12 * tokens, "flops": 3 * n * case["rot_dim"]}


# ------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    s = {"case": case}
    s.update({"distill": _prepare_distill, "norm": _prepare_norm, "rotary": _prepare_rotary}[case["op"]](
        case, _gen(seed)))
    return s


def _prepare_distill(c, g):
    r, v, k, dt = c["rows"], c["vocab"], c["topk"], DTYPES[c["dtype"]]
    logits = torch.randn((r, v), generator=g, device="cuda", dtype=dt).mul_(2.0)
    # distinct ids: from a start, in steps short enough not to come round
    live = v - min(c["dead"], v - k)
    step = 1 + (torch.rand((r, 1), generator=g, device="cuda") * (live // k)).long().clamp_(max=live // k - 1)
    start = (torch.rand((r, 1), generator=g, device="cuda") * live).long().clamp_(max=live - 1)
    ids = (start + step * torch.arange(k, device="cuda")) % live
    # a student that has learned something: the listed words stand out by about as much as the teacher's
    top = torch.randn((r, k), generator=g, device="cuda").sort(dim=1, descending=True).values * 2 + 6
    logits.scatter_(1, ids, (top + torch.randn((r, k), generator=g, device="cuda")).to(dt))
    if c["dead"]:
        logits[:, live:] = float("-inf")       # columns that pad the vocabulary
    top = top.to(dt)
    ids = ids.to(torch.int32)
    if c["ragged"]:                            # fewer entries than k, now and then none; the rest is junk
        count = (torch.rand((r, 1), generator=g, device="cuda") * (k + 1)).long()
        absent = torch.arange(k, device="cuda") >= count
        ids = torch.where(absent, torch.full_like(ids, -1), ids)
        top = torch.where(absent, torch.full_like(top, float("nan")), top)
    present = ids >= 0
    lse = None
    if c["tail"]:                              # the listed words hold 61% to all of the teacher's mass
        x = torch.where(present, top.float() / c["temperature"], torch.full_like(top, float("-inf"), dtype=torch.float32))
        lse = torch.logsumexp(x, 1) + 0.5 * torch.rand((r,), generator=g, device="cuda")
        lse = torch.where(present.any(1), lse, torch.zeros_like(lse))
    # the mean over live tokens; with 16-bit floating gradients times a loss scale
    weight = torch.full((r,), (1024.0 if c["dtype"] == "f16" else 1.0) / max(1, r - _masked_rows(c)), device="cuda")
    if c["masked"]:
        rows = torch.rand((r,), generator=g, device="cuda").argsort()[:_masked_rows(c)]
        weight[rows] = 0.0
        logits[rows[: len(rows) // 2]] = float("nan")   # what stands in a padding token's row is nobody's business
    return {"logits": logits, "ids": ids, "top": top, "lse": lse, "weight": weight,
            "dloss": torch.ones((r,), device="cuda")}


def _prepare_norm(c, g):
    r, d, dt = c["rows"], c["dim"], DTYPES[c["dtype"]]
    join, nxt = FORMS[c["form"]]
    s = {"x": _normal((r, d), g, dt, 2.0), "rho": 1.0 if c["kind"] == "rms" else 0.9, "beta": 0.7, "eps": 1e-6}
    s["branch"] = _normal((r, d), g, dt, 3.0) if join else None
    s["w1"] = 1 + _normal((d,), g, torch.float32, 0.2) if join else None
    s["gate"] = _normal((c["groups"], d), g, torch.float32, 0.5) if join and c["groups"] else None
    s["w2"] = 1 + _normal((d,), g, torch.float32, 0.2) if nxt else None
    if c["mode"] == "backward":
        x_out, _, stats = _plain_norm_forward(c, s)
        s["x_out"] = x_out if join else s["x"]
        s["stats"] = stats
        s["dx_out"] = _normal((r, d), g, dt)
        s["dh"] = _normal((r, d), g, dt) if nxt else None
        del s["x"]
    return s


def _pairs_per_axis(pairs):
    """The pairs of a head over time, height and width: about a quarter for time, the rest halved."""
    t = pairs // 4
    h = (pairs - t) // 2
    return [t, h, pairs - t - h]


def _prepare_rotary(c, g):
    b, n, dt = c["batch"], c["t"] * c["y"] * c["x"], DTYPES[c["dtype"]]
    hq, hk, d = c["heads_q"], c["heads_k"], c["head_dim"]
    if c["fused"]:
        qkv = _normal((b, n, hq + 2 * hk, d), g, dt)
        q, k = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
    else:
        q, k = _normal((b, n, hq, d), g, dt), _normal((b, n, hk, d), g, dt)
    # the grid's positions, each clip at its own time
    t0 = (torch.rand((b, 1), generator=g, device="cuda") * 100000).int()
    i = torch.arange(n, device="cuda", dtype=torch.int32)
    plane = c["y"] * c["x"]
    t = t0 + (i // plane)[None]
    y, x = ((i % plane) // c["x"]).expand(b, n), (i % c["x"]).expand(b, n)
    pos = torch.stack([t, y, x], -1).to(torch.int32).contiguous()
    pairs = c["rot_dim"] // 2
    axis = [a for a, m in enumerate(_pairs_per_axis(pairs)) for _ in range(m)]
    turns = [int(round(10000.0 ** (-i / pairs) / (2 * math.pi) * 2.0 ** 64)) for i in range(pairs)]
    return {"q": q, "k": k, "pos": pos, "axis": torch.tensor(axis, dtype=torch.uint8, device="cuda"),
            "freq": torch.tensor(turns, dtype=torch.int64, device="cuda")}


# ------------------------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"distill": _plain_distill, "norm": _plain_norm, "rotary": _plain_rotary}[c["op"]](c, state)


def _own(c, s):
    from conv_batchnorm_relu_gb300 import tokens
    if c["op"] == "distill":
        kw = dict(temperature=c["temperature"], teacher_lse=s["lse"], row_weight=s["weight"])
        if c["mode"] == "step":
            o = tokens.distill_forward_backward(s["logits"], s["ids"], s["top"], **kw)
            return {"loss": o["loss"], "dlogits": o["dlogits"]}
        o = tokens.distill_forward(s["logits"], s["ids"], s["top"], **kw)
        if c["mode"] == "forward":
            return {"loss": o["loss"], "stats": o["stats"]}
        return {"loss": o["loss"], "dlogits": tokens.distill_backward(s["dloss"], s["logits"], s["ids"], s["top"],
                                                                      o["stats"], **kw)}
    if c["op"] == "norm":
        kw = dict(kind=c["kind"], residual_scale=s["rho"], branch_scale=s["beta"])
        if c["mode"] == "forward":
            return tokens.block_norm_forward(s["x"], s["branch"], s["w1"], s["gate"], s["w2"], eps=s["eps"], **kw)
        return tokens.block_norm_backward(s["dx_out"], s["dh"], s["x_out"], s["branch"], s["w1"], s["gate"], s["w2"],
                                          s["stats"], **kw)
    f = tokens.rotary_forward if c["mode"] == "forward" else tokens.rotary_backward
    return f(s["q"], s["k"], s["pos"], s["freq"], s["axis"], layout=c["layout"])


def _plain_distill(c, s):
    temp, r = c["temperature"], c["rows"]
    present = s["ids"] >= 0
    ids = s["ids"].long().clamp(min=0)
    live = (s["weight"] != 0) & present.any(1)
    x = s["logits"].float() / temp
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    del x
    total = e.sum(1, keepdim=True)
    zero = torch.zeros((), device="cuda")
    t = torch.where(present, s["top"].float() / temp, zero - math.inf)
    if s["lse"] is None:
        p = torch.exp(t - t.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = torch.exp(t - s["lse"][:, None])
    logq = s["logits"].float().gather(1, ids) / temp - m - torch.log(total)
    terms = torch.where(p > 0, p * (torch.log(p) - logq), zero)
    loss = terms.sum(1)
    mass, tail = p.sum(1), torch.zeros(r, device="cuda")
    # the exponentials of the words that are not listed (an absent entry marks an extra last column)
    mark = torch.zeros((r, c["vocab"] + 1), dtype=torch.bool, device="cuda")
    mark.scatter_(1, torch.where(present, ids, torch.full_like(ids, c["vocab"])), True)
    mark = mark[:, :-1]
    rest = torch.where(mark, zero, e).sum(1)
    qrest = rest / total[:, 0]
    if s["lse"] is not None:
        tail = torch.where(qrest > 0, (1 - mass).clamp(min=0), zero)
        loss = loss + torch.where(tail > 0, tail * (torch.log(tail) - torch.log(qrest)), zero)
    loss = torch.where(live, loss * temp * temp * s["weight"], zero)
    if c["mode"] == "forward":
        stats = torch.stack([m[:, 0] * temp, total[:, 0], rest], 1)
        return {"loss": loss, "stats": torch.where(live[:, None], stats, zero)}
    grad = e.mul_(((mass + tail) / total[:, 0])[:, None])
    if s["lse"] is not None:
        keep = torch.where(tail > 0, 1 - tail / (qrest * (mass + tail)), zero + 1)
        grad = grad * torch.where(mark, zero + 1, keep[:, None])
    grad.scatter_add_(1, ids, torch.where(present, -p, zero))
    grad.mul_((s["weight"] * temp * (s["dloss"] if c["mode"] == "pair" else 1.0))[:, None])
    grad = torch.where(live[:, None], grad, zero)
    return {"loss": loss, "dlogits": grad.to(s["logits"].dtype)}


def _spans(c, s):
    """The gate of each row, or None."""
    return None if s["gate"] is None else s["gate"].repeat_interleave(c["rows"] // s["gate"].shape[0], 0)


def _moments(a, kind, eps):
    m = a.mean(1, keepdim=True) if kind == "layer" else torch.zeros((a.shape[0], 1), device=a.device)
    return m, 1.0 / torch.sqrt(((a - m) ** 2).mean(1, keepdim=True) + eps)


def _plain_norm_forward(c, s):
    x = s["x"].float()
    none = torch.zeros((c["rows"], 1), device="cuda")
    m1 = r1 = m2 = r2 = none
    if s["branch"] is not None:
        f = s["branch"].float()
        m1, r1 = _moments(f, c["kind"], s["eps"])
        n = (f - m1) * r1 * s["w1"]
        g = _spans(c, s)
        x = s["rho"] * x + s["beta"] * (n if g is None else g * n)
    h = None
    if s["w2"] is not None:
        m2, r2 = _moments(x, c["kind"], s["eps"])
        h = ((x - m2) * r2 * s["w2"]).to(s["x"].dtype)
    x_out = x.to(s["x"].dtype) if s["branch"] is not None else None
    return x_out, h, torch.cat([m1, r1, m2, r2], 1)


def _plain_norm(c, s):
    if c["mode"] == "forward":
        x_out, h, stats = _plain_norm_forward(c, s)
        return {"x_out": x_out, "h": h, "stats": stats}
    m1, r1, m2, r2 = s["stats"].split(1, 1)
    out = {"dx": None, "dbranch": None, "dpost_weight": None, "dgate": None, "dpre_weight": None}
    dx = s["dx_out"].float()
    center = c["kind"] == "layer"
    if s["dh"] is not None:
        dh = s["dh"].float()
        n = (s["x_out"].float() - m2) * r2
        u = dh * s["w2"]
        dx = dx + r2 * (u - (u.mean(1, keepdim=True) if center else 0.0) - n * (u * n).mean(1, keepdim=True))
        out["dpre_weight"] = (dh * n).sum(0)
    if s["branch"] is not None:
        n = (s["branch"].float() - m1) * r1
        b = s["beta"] * dx
        g = _spans(c, s)
        if g is not None:
            out["dgate"] = (b * n * s["w1"]).view(s["gate"].shape[0], -1, c["dim"]).sum(1)
            b = b * g
        out["dpost_weight"] = (b * n).sum(0)
        v = b * s["w1"]
        out["dbranch"] = (r1 * (v - (v.mean(1, keepdim=True) if center else 0.0)
                                - n * (v * n).mean(1, keepdim=True))).to(s["branch"].dtype)
        dx = s["rho"] * dx
    out["dx"] = dx.to(s["dx_out"].dtype)
    return out


def _plain_rotary(c, s):
    # pos * frequency in turns, as a fixed-point fraction of 64 bits that wraps; the top 32 bits, signed
    fraction = (s["pos"].long()[:, :, s["axis"].long()] * s["freq"]) >> 32
    angle = fraction.float() * (2 * math.pi / 2.0 ** 32)
    cos, sin = torch.cos(angle)[:, :, None], torch.sin(angle)[:, :, None]
    if c["mode"] == "backward":
        sin = -sin
    return tuple(_turn(a.float(), cos, sin, c["layout"], c["rot_dim"]).to(a.dtype) for a in (s["q"], s["k"]))


def _turn(a, cos, sin, layout, rot):
    out = a.clone(memory_format=torch.contiguous_format)
    if layout == "halves":
        one, two = a[..., :rot // 2], a[..., rot // 2:rot]
        out[..., :rot // 2], out[..., rot // 2:rot] = one * cos - two * sin, two * cos + one * sin
    else:
        one, two = a[..., 0:rot:2], a[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = one * cos - two * sin, two * cos + one * sin
    return out


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"distill": _exact_distill, "norm": _exact_norm, "rotary": _exact_rotary}[case["op"]](case, s)


def _exact_distill(c, s):
    temp, r, v = c["temperature"], c["rows"], c["vocab"]
    f64 = dict(dtype=torch.float64, device="cuda")
    loss, grad, stats = torch.zeros(r, **f64), torch.zeros((r, v), **f64), torch.zeros((r, 3), **f64)
    block = max(1, (1 << 26) // v)
    for a in range(0, r, block):
        b = min(r, a + block)
        w = s["weight"][a:b].double()
        here = s["ids"][a:b] >= 0
        on = (w != 0) & here.any(1)
        z = s["logits"][a:b].double()
        q = torch.softmax(z / temp, 1)
        t = (s["top"][a:b].double() / temp).masked_fill(~here, -math.inf)
        p = torch.softmax(t, 1) if s["lse"] is None else (t - s["lse"][a:b, None].double()).exp()
        at = s["ids"][a:b].long().masked_fill(~here, v)
        # the teacher's distribution over the vocabulary and one junk column
        full = torch.zeros((b - a, v + 1), **f64).scatter_add_(1, at, p)[:, :v]
        listed_ = torch.zeros((b - a, v + 1), **f64).scatter_(1, at, 1.0)[:, :v]
        qk = torch.log_softmax(z / temp, 1).gather(1, at.clamp(max=v - 1))
        part = (torch.special.xlogy(p, p) - p * qk).masked_fill(p == 0, 0.0).sum(1)
        out = (q * (1 - listed_)).sum(1)
        rest = (1 - p.sum(1)).clamp(min=0) if s["lse"] is not None else torch.zeros(b - a, **f64)
        rest = rest.masked_fill(out == 0, 0.0)
        part = part + (torch.special.xlogy(rest, rest) - torch.special.xlogy(rest, out))
        total = p.sum(1) + rest
        loss[a:b] = (part * temp ** 2 * w).masked_fill(~on, 0.0)
        slope = (rest / out).masked_fill(rest == 0, 0.0)
        d = (q * total[:, None] - full - q * (1 - listed_) * slope[:, None]) * (w * temp)[:, None]
        grad[a:b] = d.masked_fill(~on[:, None], 0.0)
        top = z.amax(1)
        sums = ((z - top[:, None]) / temp).exp().sum(1)
        stats[a:b] = torch.stack([top, sums, sums * out], 1).masked_fill(~on[:, None], 0.0)
    return {"loss": loss, "stats": stats} if c["mode"] == "forward" else {"loss": loss, "dlogits": grad}


def _wide(v):
    return v.double() if isinstance(v, torch.Tensor) else v


def _exact_norm(c, s):
    """Rows in blocks; the gradients from the Jacobian's definition of each norm."""
    d, r, center = c["dim"], c["rows"], c["kind"] == "layer"
    s = {k: v if k in ("x", "branch", "x_out", "dx_out", "dh") else _wide(v) for k, v in s.items()}
    block = max(1, (1 << 25) // d)
    per = r // s["gate"].shape[0] if s["gate"] is not None else 1
    back = c["mode"] == "backward"
    names = ("dx", "dbranch") if back else ("x_out", "h", "stats")
    pieces = {n: [] for n in names}
    sums = {n: torch.zeros(d, dtype=torch.float64, device="cuda") for n in ("dpost_weight", "dpre_weight")}
    dgate = torch.zeros_like(s["gate"]) if s["gate"] is not None else None

    def scale_of(a):
        mu = a.sum(1) / d if center else a.new_zeros(len(a))
        return mu, ((a - mu[:, None]).pow(2).sum(1) / d + s["eps"]).rsqrt()

    def pull(up, unit, rstd):
        """The gradient at a norm's input from that at its unscaled output."""
        along = (up * unit).sum(1, keepdim=True) / d
        level = up.sum(1, keepdim=True) / d if center else 0.0
        return (up - level - unit * along) * rstd[:, None]

    for a in range(0, r, block):
        i = torch.arange(a, min(r, a + block), device="cuda")
        gate = s["gate"][i // per] if s["gate"] is not None else 1.0
        take = {k: s[k][a:a + block].double() if s.get(k) is not None else None
                for k in ("x", "branch", "x_out", "dx_out", "dh")}
        if not back:
            x, st = take["x"], torch.zeros((len(i), 4), dtype=torch.float64, device="cuda")
            if take["branch"] is not None:
                st[:, 0], st[:, 1] = scale_of(take["branch"])
                x = x * s["rho"] + gate * s["w1"] * s["beta"] * (take["branch"] - st[:, :1]) * st[:, 1:2]
                pieces["x_out"].append(x)
            if s["w2"] is not None:
                st[:, 2], st[:, 3] = scale_of(x)
                pieces["h"].append((x - st[:, 2:3]) * st[:, 3:4] * s["w2"])
            pieces["stats"].append(st)
            continue
        st = s["stats"][a:a + block]
        up = take["dx_out"]
        if take["dh"] is not None:
            unit = (take["x_out"] - st[:, 2:3]) * st[:, 3:4]
            sums["dpre_weight"] += (take["dh"] * unit).sum(0)
            up = up + pull(take["dh"] * s["w2"], unit, st[:, 3])
        if take["branch"] is not None:
            unit = (take["branch"] - st[:, :1]) * st[:, 1:2]
            sums["dpost_weight"] += (up * gate * unit).sum(0) * s["beta"]
            if dgate is not None:
                dgate.index_add_(0, i // per, up * unit * s["w1"] * s["beta"])
            pieces["dbranch"].append(pull(up * gate * s["w1"] * s["beta"], unit, st[:, 1]))
            up = up * s["rho"]
        pieces["dx"].append(up)
    out = {n: torch.cat(v) if v else None for n, v in pieces.items()}
    if back:
        out.update(dgate=dgate, dpost_weight=sums["dpost_weight"] if s["branch"] is not None else None,
                   dpre_weight=sums["dpre_weight"] if s["w2"] is not None else None)
    return out


def _exact_rotary(c, s):
    """Each pair as a complex number, turned by exp(i angle)."""
    pairs = c["rot_dim"] // 2
    f = torch.tensor([10000.0 ** (-i / pairs) for i in range(pairs)], dtype=torch.float64, device="cuda")
    angle = s["pos"].double()[:, :, s["axis"].long()] * f
    turn = torch.polar(torch.ones_like(angle), -angle if c["mode"] == "backward" else angle)[:, :, None]
    out = []
    for a in (s["q"], s["k"]):
        a = a.double()
        rot, rest = a[..., :c["rot_dim"]], a[..., c["rot_dim"]:]
        if c["layout"] == "halves":
            z = torch.complex(rot[..., :pairs], rot[..., pairs:]) * turn
            rot = torch.cat([z.real, z.imag], -1)
        else:
            z = torch.complex(rot[..., 0::2].contiguous(), rot[..., 1::2].contiguous()) * turn
            rot = torch.view_as_real(z).flatten(-2)
        out.append(torch.cat([rot, rest], -1))
    return tuple(out)
