"""The trunk operators of a student's training step as measured cases: attention (forward, and the
backward that recomputes the probabilities), group norm with an activation over NHWC feature maps, and
the global gradient norm with clipping.  They stand beside the Conv-BN-ReLU stem and the token
operators: a norm for stems whose batch is too small for batch statistics, the mixing of a trunk's
tokens, and the end of the step.

``run`` computes an operator either in elementary torch operations (``own = False``: products, sums,
exponentials and indexing in 32 bits, rounded once at the end) or through the package's kernels
(``own = True``).  ``exact`` is the same definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
MOST_SCORES = 2 * 16 * 8192 * 8192        # of a drawn attention case: what the largest listed one has
MOST_GROUP_NORM = 128 * 112 * 112 * 128 * 2   # bytes of one feature map
MOST_GRADIENT = 400_000_000 * 4           # bytes of one set of gradients


# ------------------------------------------------------------------------------------ the cases

def _attention(name, mode, batch, tq, tk, heads_q, heads_k, head_dim, dtype, causal=False, ragged=False, at_end=False,
               fused=False):
    return dict(name=name, op="attention", mode=mode, batch=batch, tq=tq, tk=tk, heads_q=heads_q, heads_k=heads_k,
                head_dim=head_dim, dtype=dtype, causal=causal, ragged=ragged, at_end=at_end, fused=fused)


def _group_norm(name, mode, n, h, w, c, groups, act, dtype):
    return dict(name=name, op="group_norm", mode=mode, n=n, h=h, w=w, c=c, groups=groups, act=act, dtype=dtype)


def _clip(name, tensors, elements, dtype, flat, share, loss_scale, shapes):
    return dict(name=name, op="clip", tensors=tensors, elements=elements, dtype=dtype, flat=flat, share=share,
                loss_scale=loss_scale, shapes=shapes)


def listed():
    return [
        # the attention of one 7x7 feature map's tokens: latency
        _attention("attention_forward_1x49", "forward", 1, 49, 49, 4, 4, 64, "bf16"),
        # one new token a sequence against the keys of those before it, eight query heads to a key head;
        # what stands behind each sequence's last key is junk
        _attention("attention_forward_4x1_of_16384", "forward", 4, 1, 16384, 32, 4, 128, "f16", causal=True, ragged=True,
                   at_end=True),
        # training forward on long causal sequences with shared key heads
        _attention("attention_forward_2x8192", "forward", 2, 8192, 8192, 16, 4, 128, "bf16", causal=True),
        # the backward over the 28x28 tokens of 16 images, on views of a fused query/key/value product
        _attention("attention_backward_16x784", "backward", 16, 784, 784, 12, 12, 64, "f16", fused=True),
        # a padded batch of odd lengths (one of them empty), shared key heads, a head of 80
        _attention("attention_backward_4x1025", "backward", 4, 1025, 1025, 12, 4, 80, "bf16", ragged=True),
        # the backward of the long training step
        _attention("attention_backward_2x8192", "backward", 2, 8192, 8192, 16, 4, 128, "bf16", causal=True),
        # a small deep feature map: latency
        _group_norm("group_norm_forward_1x7x7x512", "forward", 1, 7, 7, 512, 32, "silu", "f32"),
        # the largest map of a stem, whose samples (6 MB) are larger than what one block can hold
        _group_norm("group_norm_forward_128x112x112x128", "forward", 128, 112, 112, 128, 32, "relu", "bf16"),
        # odd sides and groups of an odd number of channels
        _group_norm("group_norm_backward_8x61x45x60", "backward", 8, 61, 45, 60, 4, "silu", "f16"),
        # a training step's 56x56x64 maps
        _group_norm("group_norm_backward_256x56x56x64", "backward", 256, 56, 56, 64, 16, "relu", "f16"),
        # a small student's gradients, types mixed, in allocations of their own
        _clip("clip_24_tensors", 24, 300_000, "mixed", False, 0.5, 1.0, 1),
        # a large model's gradients, one flat buffer whose tensors start at any element
        _clip("clip_400_tensors", 400, 400_000_000, "f32", True, 0.25, 1.0, 2),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "group_norm", "clip"])
    if op == "attention":
        while True:
            batch, heads_k = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 4, 8, 12])
            heads_q = heads_k * rng.choice([1, 1, 2, 3, 4, 8])
            tk = _spread(rng, 1, 16384)
            kind = rng.choice(["self", "self", "few", "cross"])
            tq = {"self": tk, "few": rng.choice([1, 1, 2, 5]), "cross": _spread(rng, 1, 8192)}[kind]
            mode = "forward" if kind == "few" and rng.random() < 0.7 else rng.choice(["forward", "backward"])
            causal = rng.random() < 0.5
            # a query that sees one key has no gradient but roundings': a backward's queries mostly see more
            many = mode == "forward" or tk >= 16 and (tq >= 16 or kind == "few" or not causal)
            if many and batch * heads_q * tq * tk <= MOST_SCORES and batch * heads_q * (tq + tk) <= 4 * 16 * 16384:
                break
        c = _attention("", mode, batch, tq, tk, heads_q, heads_k, rng.choice([16, 40, 64, 64, 72, 80, 96, 128, 128]),
                       rng.choice(["f16", "bf16"]), causal=causal, ragged=rng.random() < 0.4,
                       at_end=kind == "few", fused=kind == "self" and rng.random() < 0.5)
    elif op == "group_norm":
        while True:
            dtype, groups = rng.choice(["f32", "f16", "bf16"]), rng.choice([1, 2, 4, 8, 16, 32])
            n, h, w = _spread(rng, 1, 256), _spread(rng, 1, 224), _spread(rng, 1, 224)
            channels = groups * _spread(rng, 1, 64)
            # (the gradient of a norm over one or two elements is nothing but roundings)
            if n * h * w * channels * SIZE[dtype] <= MOST_GROUP_NORM and channels <= 1024 and h * w * channels // groups >= 8:
                break
        c = _group_norm("", rng.choice(["forward", "backward"]), n, h, w, channels, groups,
                        rng.choice(["none", "relu", "silu"]), dtype)
    else:
        dtype = rng.choice(["f32", "f16", "bf16", "mixed"])
        c = _clip("", _spread(rng, 1, 500), _spread(rng, 1000, MOST_GRADIENT // SIZE.get(dtype, 4)), dtype,
                  rng.random() < 0.5, rng.choice([0.25, 0.5, 2.0]), rng.choice([1.0, 1024.0]), rng.randrange(1 << 20))
    del c["name"]
    return c


def _lengths(c):
    """The keys of each sequence: all of them, or (ragged) fewer, and none in the second of several."""
    if not c["ragged"]:
        return [c["tk"]] * c["batch"]
    return [0 if b == 1 and c["batch"] > 2 else c["tk"] - (b * 131) % (c["tk"] // 2 + 1) for b in range(c["batch"])]


def _starts(c):
    """The place of each sequence's first query among its keys."""
    return [max(0, n - c["tq"]) if c["at_end"] else 0 for n in _lengths(c)]


def _seen(c):
    """Pairs of a query and a key that it sees, over the batch, for one head."""
    total = 0
    for n, start in zip(_lengths(c), _starts(c)):
        if not c["causal"]:
            total += c["tq"] * n
            continue
        rising = min(c["tq"], max(0, n - start))          # queries i with start + i < n see start + i + 1 keys
        total += rising * start + rising * (rising + 1) // 2 + (c["tq"] - rising) * n
    return total


def _dtype_names(c):
    return ["f32", "f16", "bf16"] if c["dtype"] == "mixed" else [c["dtype"]]


def _sizes(c):
    """(type, elements) of each gradient: from single elements to a large share of all."""
    rng = random.Random(c["shapes"])
    names = _dtype_names(c)
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(c["tensors"])]
    whole = sum(share)
    return [(names[i % len(names)], max(1, int(c["elements"] * v / whole))) for i, v in enumerate(share)]


def work(case):
    """Each input read once, each output written once."""
    c = case
    if c["op"] == "attention":
        e, d = SIZE[c["dtype"]], c["head_dim"]
        q = c["batch"] * c["tq"] * c["heads_q"] * d
        k = sum(_lengths(c)) * c["heads_k"] * d
        rows = 4 * c["batch"] * c["tq"] * c["heads_q"]
        if c["mode"] == "forward":
            return {"bytes": e * (2 * q + 2 * k) + rows, "flops": 4 * _seen(c) * c["heads_q"] * d}
        k_all = c["batch"] * c["tk"] * c["heads_k"] * d
        return {"bytes": e * (4 * q + 2 * k + 2 * k_all) + rows, "flops": 10 * _seen(c) * c["heads_q"] * d}
    if c["op"] == "group_norm":
        n = c["n"] * c["h"] * c["w"] * c["c"]
        small = 8 * c["n"] * c["groups"] + 8 * c["c"]
        if c["mode"] == "forward":
            return {"bytes": 2 * n * SIZE[c["dtype"]] + small, "flops": 8 * n}
        return {"bytes": 3 * n * SIZE[c["dtype"]] + small + 8 * c["c"], "flops": 16 * n}
    sizes = _sizes(c)
    return {"bytes": 2 * sum(SIZE[t] * n for t, n in sizes), "flops": 3 * sum(n for _, n in sizes)}


# ------------------------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def prepare(case, seed):
    s = {"case": case}
    s.update({"attention": _prepare_attention, "group_norm": _prepare_group_norm, "clip": _prepare_clip}[case["op"]](
        case, _gen(seed)))
    return s


def _prepare_attention(c, g):
    b, tq, tk, hq, hk, d, dt = c["batch"], c["tq"], c["tk"], c["heads_q"], c["heads_k"], c["head_dim"], DTYPES[c["dtype"]]
    if c["fused"]:
        qkv = _normal((b, tk, hq + 2 * hk, d), g, dt, 1.25)
        q, k, v = qkv.split([hq, hk, hk], dim=2)
    else:
        q, k, v = (_normal((b, t, h, d), g, dt, 1.25) for t, h in ((tq, hq), (tk, hk), (tk, hk)))
    s = {"q": q, "k": k, "v": v, "scale": d ** -0.5, "lengths": None, "start": None}
    if c["ragged"]:
        s["lengths"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
        behind = torch.arange(tk, device="cuda")[None] >= s["lengths"][:, None]
        k[behind] = float("nan")               # what stands behind a sequence's last key is nobody's business
        v[behind] = float("nan")
    if c["at_end"]:
        s["start"] = torch.tensor(_starts(c), dtype=torch.int32, device="cuda")
    if c["mode"] == "backward":
        s["o"], s["lse"] = _plain_attention_forward(c, s)
        s["do"] = _normal((b, tq, hq, d), g, dt)
    return s


def _prepare_group_norm(c, g):
    shape, dt = (c["n"], c["h"], c["w"], c["c"]), DTYPES[c["dtype"]]
    # a convolution's output: channels with means and spreads of their own
    level, spread = _normal((c["c"],), g, torch.float32, 0.5), 1.0 + 0.5 * torch.rand(c["c"], generator=g, device="cuda")
    x = (torch.randn(shape, generator=g, device="cuda") * spread + level).to(dt)
    s = {"x": x, "gamma": 1 + _normal((c["c"],), g, torch.float32, 0.2), "beta": _normal((c["c"],), g, torch.float32, 0.2),
         "eps": 1e-5}
    if c["mode"] == "backward":
        o = _plain_group_norm_forward(c, s)
        s["mean"], s["rstd"] = o["mean"], o["rstd"]
        s["dy"] = _normal(shape, g, dt)
    return s


def _prepare_clip(c, g):
    sizes, spread = _sizes(c), 1e-2 * c["loss_scale"]
    grads, out, flat = [], [], {}
    offset = {}
    for name in _dtype_names(c):
        n = sum(m for t, m in sizes if t == name)
        flat[name] = torch.empty(n, dtype=DTYPES[name], device="cuda")
        if c["flat"]:
            offset[name] = [0, _normal((n,), g, DTYPES[name], spread)]
        else:
            offset[name] = [0, None]
    for t, m in sizes:
        at, source = offset[t]
        out.append(flat[t][at:at + m])
        grads.append(source[at:at + m] if source is not None else _normal((m,), g, DTYPES[t], spread))
        offset[t][0] = at + m
    # the norm of what is drawn, nearly
    expected = 1e-2 * math.sqrt(sum(m for _, m in sizes))
    return {"grads": grads, "out": out, "flat": flat, "max_norm": c["share"] * expected, "unscale": 1.0 / c["loss_scale"]}


# ------------------------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"attention": _plain_attention, "group_norm": _plain_group_norm, "clip": _plain_clip}[c["op"]](c, state)


def _own(c, s):
    from conv_batchnorm_relu_gb300 import attention, gradients, group_norm
    if c["op"] == "attention":
        kw = dict(scale=s["scale"], causal=c["causal"], key_lengths=s["lengths"], query_start=s["start"])
        if c["mode"] == "forward":
            return attention.attention_forward(s["q"], s["k"], s["v"], **kw)
        return attention.attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], **kw)
    if c["op"] == "group_norm":
        if c["mode"] == "forward":
            return group_norm.group_norm_forward(s["x"], s["gamma"], s["beta"], c["groups"], eps=s["eps"], act=c["act"])
        return group_norm.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], s["mean"], s["rstd"], c["groups"],
                                              act=c["act"])
    o = gradients.clip_gradients(s["grads"], s["max_norm"], unscale=s["unscale"], out=s["out"])
    return {"norm": o["norm"], "scale": o["scale"], "grads": s["flat"]}


def _visible(c, s):
    """[batch][1][tq][tk]: which keys a query sees."""
    j = torch.arange(c["tk"], device="cuda")[None, None, None]
    see = torch.ones((1, 1, c["tq"], c["tk"]), dtype=torch.bool, device="cuda")
    if s["lengths"] is not None:
        see = see & (j < s["lengths"][:, None, None, None])
    if c["causal"]:
        first = torch.zeros(1, device="cuda") if s["start"] is None else s["start"]
        see = see & (j <= first[:, None, None, None] + torch.arange(c["tq"], device="cuda")[None, None, :, None])
    return see


def _by_heads(a, c, s):
    """Keys or values as [batch][heads_q][tk][head_dim] in 32 bits; what stands behind the keys is zero."""
    a = a.float().permute(0, 2, 1, 3)
    if s["lengths"] is not None:
        behind = torch.arange(c["tk"], device="cuda")[None] >= s["lengths"][:, None]
        a = a.masked_fill(behind[:, None, :, None], 0.0)
    return a.repeat_interleave(c["heads_q"] // c["heads_k"], 1)


def _plain_attention_forward(c, s):
    q = s["q"].float().permute(0, 2, 1, 3)
    k, v = _by_heads(s["k"], c, s), _by_heads(s["v"], c, s)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).masked_fill_(~_visible(c, s), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = x.sub_(m).exp_()
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 2, 1, 3).contiguous().to(s["q"].dtype), (m + torch.log(total))[..., 0]


def _plain_attention(c, s):
    if c["mode"] == "forward":
        o, lse = _plain_attention_forward(c, s)
        return {"o": o, "lse": lse}
    q, do, o = (s[n].float().permute(0, 2, 1, 3) for n in ("q", "do", "o"))
    k, v = _by_heads(s["k"], c, s), _by_heads(s["v"], c, s)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).sub_(s["lse"][..., None])
    p = x.exp_().masked_fill_(~_visible(c, s), 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    dq = torch.matmul(ds, k) * s["scale"]
    dk = torch.matmul(ds.transpose(-1, -2), q) * s["scale"]
    shared = (c["batch"], c["heads_k"], -1, c["tk"], c["head_dim"])
    dk, dv = dk.reshape(shared).sum(2), dv.reshape(shared).sum(2)
    dt = s["q"].dtype
    return {n: a.permute(0, 2, 1, 3).contiguous().to(dt) for n, a in (("dq", dq), ("dk", dk), ("dv", dv))}


def _grouped(a, c):
    return a.float().reshape(c["n"], c["h"] * c["w"], c["groups"], c["c"] // c["groups"])


def _plain_group_norm_forward(c, s):
    x = _grouped(s["x"], c)
    mean = x.mean((1, 3), keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean((1, 3), keepdim=True) + s["eps"])
    y = ((x - mean) * rstd).reshape(s["x"].shape) * s["gamma"] + s["beta"]
    if c["act"] == "relu":
        y = torch.where(y > 0, y, torch.zeros_like(y))
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0, :, 0], "rstd": rstd[:, 0, :, 0]}


def _plain_group_norm(c, s):
    if c["mode"] == "forward":
        return _plain_group_norm_forward(c, s)
    shape = s["x"].shape
    mean, rstd = s["mean"][:, None, :, None], s["rstd"][:, None, :, None]
    xh = ((_grouped(s["x"], c) - mean) * rstd)
    flat = xh.reshape(shape)
    g = s["dy"].float()
    pre = flat * s["gamma"] + s["beta"]
    if c["act"] == "relu":
        g = torch.where(pre > 0, g, torch.zeros_like(g))
    elif c["act"] == "silu":
        sig = 1 / (1 + torch.exp(-pre))
        g = g * sig * (1 + pre * (1 - sig))
    dbeta, dgamma = g.sum((0, 1, 2)), (g * flat).sum((0, 1, 2))
    u = _grouped(g * s["gamma"], c)
    dx = rstd * (u - u.mean((1, 3), keepdim=True) - xh * (u * xh).mean((1, 3), keepdim=True))
    return {"dx": dx.reshape(shape).to(s["x"].dtype), "dgamma": dgamma, "dbeta": dbeta}


def _plain_clip(c, s):
    squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
    norm = squares.sum().sqrt().mul(s["unscale"]).float()
    scale = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)) * s["unscale"]
    for g, o in zip(s["grads"], s["out"]):
        o.copy_(g.float() * scale)
    return {"norm": norm, "scale": scale, "grads": s["flat"]}


# ------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "group_norm": _exact_group_norm, "clip": _exact_clip}[case["op"]](case, s)


def _exact_attention(c, s):
    """One key head of one sequence at a time, over the keys that the sequence has; its query heads stacked."""
    group, d, tq = c["heads_q"] // c["heads_k"], c["head_dim"], c["tq"]
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(s["q"].shape, **f64), torch.full((c["batch"], c["heads_q"], tq), -math.inf, **f64)
    dq, dk, dv = (torch.zeros(s[n].shape, **f64) for n in ("q", "k", "v"))
    for b, (n, start) in enumerate(zip(_lengths(c), _starts(c))):
        if n == 0:
            continue
        hidden = None
        if c["causal"]:
            hidden = torch.ones((tq, n), dtype=torch.bool, device="cuda").triu(start + 1)
        for h in range(c["heads_k"]):
            here = slice(h * group, (h + 1) * group)
            k, v = s["k"][b, :n, h].double(), s["v"][b, :n, h].double()
            logits = torch.einsum("igd,jd->gij", s["q"][b, :, here].double(), k) * s["scale"]
            if hidden is not None:
                logits.masked_fill_(hidden, -math.inf)
            if c["mode"] == "forward":
                lse[b, here] = torch.logsumexp(logits, -1)
                o[b, :, here] = torch.einsum("gij,jd->igd", torch.softmax(logits, -1), v)
                continue
            p = (logits - s["lse"][b, here].double()[..., None]).exp()
            up = s["do"][b, :, here].double()
            dv[b, :n, h] = torch.einsum("gij,igd->jd", p, up)
            along = (up * s["o"][b, :, here].double()).sum(-1).t()
            slope = p * (torch.einsum("igd,jd->gij", up, v) - along[..., None]) * s["scale"]
            dq[b, :, here] = torch.einsum("gij,jd->igd", slope, k)
            dk[b, :n, h] = torch.einsum("gij,igd->jd", slope, s["q"][b, :, here].double())
    return {"o": o, "lse": lse} if c["mode"] == "forward" else {"dq": dq, "dk": dk, "dv": dv}


def _exact_group_norm(c, s):
    """A sample at a time, its groups' elements in rows; the gradient through the norm's Jacobian."""
    shape, per = s["x"].shape, c["c"] // c["groups"]
    f64 = dict(dtype=torch.float64, device="cuda")
    gamma, beta = s["gamma"].double(), s["beta"].double()
    y, mean, rstd = torch.empty(shape, **f64), torch.empty((c["n"], c["groups"]), **f64), torch.empty((c["n"], c["groups"]), **f64)
    dgamma, dbeta = torch.zeros(c["c"], **f64), torch.zeros(c["c"], **f64)

    def rows(a):
        return a.reshape(-1, c["groups"], per).transpose(0, 1).reshape(c["groups"], -1)

    def pixels(a):
        return a.reshape(c["groups"], -1, per).transpose(0, 1).reshape(-1, c["c"])

    for i in range(c["n"]):
        x = rows(s["x"][i].double())
        if c["mode"] == "forward":
            var, mean[i] = torch.var_mean(x, 1, correction=0)
            rstd[i] = (var + s["eps"]).rsqrt()
            z = torch.addcmul(beta, pixels((x - mean[i][:, None]) * rstd[i][:, None]), gamma)
            z = z.clamp(min=0) if c["act"] == "relu" else z * torch.sigmoid(z) if c["act"] == "silu" else z
            y[i] = z.view(shape[1:])
            continue
        r = s["rstd"][i].double()[:, None]
        unit = (x - s["mean"][i].double()[:, None]) * r
        flat, up = pixels(unit), s["dy"][i].double().reshape(-1, c["c"])
        z = torch.addcmul(beta, flat, gamma)
        if c["act"] == "relu":
            up = up * (z > 0)
        elif c["act"] == "silu":
            t = torch.tanh(z / 2)
            up = up * (0.5 * (1 + t) + z * 0.25 * (1 - t * t))
        dbeta += up.sum(0)
        dgamma += (up * flat).sum(0)
        u = rows(up * gamma)
        n = u.shape[1]
        y[i] = pixels((u - u.sum(1, keepdim=True) / n - unit * ((u * unit).sum(1, keepdim=True) / n)) * r).view(shape[1:])
    return {"y": y, "mean": mean, "rstd": rstd} if c["mode"] == "forward" else {"dx": y, "dgamma": dgamma, "dbeta": dbeta}


def _exact_clip(c, s):
    norm = s["unscale"] * math.sqrt(math.fsum(float(torch.dot(g.double(), g.double())) for g in s["grads"]))
    scale = s["unscale"] * min(1.0, s["max_norm"] / norm)
    grads = {name: torch.cat([g.double() * scale for g in s["grads"] if g.dtype == DTYPES[name]]) for name in s["flat"]
             if any(g.dtype == DTYPES[name] for g in s["grads"])}
    f64 = dict(dtype=torch.float64, device="cuda")
    return {"norm": torch.tensor(norm, **f64), "scale": torch.tensor(scale, **f64),
            "grads": {name: grads.get(name, torch.empty(0, **f64)) for name in s["flat"]}}
