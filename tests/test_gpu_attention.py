"""Attention, forward and backward, against its plain 64-bit form: types, heads, lengths from one token on, odd
sizes, masks that leave rows empty, junk in the padding, strides and orders of axes, streams, graphs."""
import math

import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import attention as att
from conv_batchnorm_relu_gb300 import cbr

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


def tensor(shape, dtype, g, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype]).cuda()


def make(batch, tq, tk, hq, hk, dim, dtype, seed=0, lengths=None, start=None, size=1.25):
    g = torch.Generator().manual_seed(seed)
    s = {"q": tensor((batch, tq, hq, dim), dtype, g, size), "k": tensor((batch, tk, hk, dim), dtype, g, size),
         "v": tensor((batch, tk, hk, dim), dtype, g), "do": tensor((batch, tq, hq, dim), dtype, g),
         "lengths": None, "start": None}
    if lengths is not None:
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        behind = torch.arange(tk, device="cuda")[None] >= s["lengths"][:, None]
        s["k"][behind] = NAN
        s["v"][behind] = NAN
    if start is not None:
        s["start"] = torch.tensor(start, dtype=torch.int32, device="cuda")
    return s


def check(s, causal=False, scale=None, backward=True, **kw):
    """One forward and one backward against the formulas; what they returned."""
    dim = s["q"].shape[3]
    scale = dim ** -0.5 if scale is None else scale
    args = dict(scale=scale, causal=causal, key_lengths=s["lengths"], query_start=s["start"])
    got = att.attention_forward(s["q"], s["k"], s["v"], **args, **kw)
    torch.cuda.synchronize()
    assert cbr.stream_status_code() == 0
    dt = s["q"].dtype
    want = ref.attention(s["q"], s["k"], s["v"], scale, causal, s["lengths"], s["start"])
    ref.close(got["lse"], want["lse"], want["lse_bound"], "lse")
    ref.close(got["o"], want["o"], want["o_bound"], "o", dt)
    if not backward:
        return got, None
    back = att.attention_backward(s["do"], s["q"], s["k"], s["v"], got["o"], got["lse"], **args)
    torch.cuda.synchronize()
    assert cbr.stream_status_code() == 0
    wb = ref.attention_backward(s["do"], s["q"], s["k"], s["v"], got["o"], got["lse"], scale, causal, s["lengths"], s["start"])
    for n in ("dv", "dq", "dk"):
        ref.close(back[n], wb[n], wb[n + "_bound"], n, dt)
    return got, back


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("batch,tq,tk,hq,hk,dim", [
    (1, 1, 1, 1, 1, 64), (2, 1, 300, 4, 4, 64), (1, 49, 49, 4, 4, 64), (1, 128, 128, 1, 1, 128), (2, 129, 127, 2, 1, 128),
    (1, 200, 70, 3, 1, 40), (2, 65, 257, 4, 2, 80), (1, 300, 513, 2, 2, 8), (1, 385, 640, 1, 1, 96), (1, 700, 900, 2, 1, 128),
    (1, 900, 300, 4, 1, 16), (3, 2, 1, 2, 2, 24)])
def test_shapes(batch, tq, tk, hq, hk, dim, causal, dtype):
    check(make(batch, tq, tk, hq, hk, dim, dtype, seed=tq * 7 + tk), causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,start,causal", [
    ([0, 1, 260, 259], None, False), ([128, 127, 129, 2], None, True), ([300, 0, 260, 200], [-5, 0, 100, 259], True),
    ([64, 256, 3, 260], [-400, -128, 2147483647, -2147483648], True), ([-7, 2147483647, 260, 5], [0, 0, 0, 0], True)])
def test_masks_that_leave_rows_empty(lengths, start, causal, dtype):
    s = make(4, 133, 260, 4, 2, 64, dtype, 3, [min(max(n, 0), 260) for n in lengths], start)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    got, back = check(s, causal)
    empty = torch.isinf(got["lse"]).permute(0, 2, 1)
    assert not got["o"][empty].any() and not back["dq"][empty].any()
    for b, n in enumerate(lengths):
        assert not back["dk"][b, max(0, n):].any() and not back["dv"][b, max(0, n):].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tq,tk,hq,hk,dim", [(1, 5000, 8, 1, 128), (1, 4097, 4, 4, 64), (3, 2500, 6, 2, 80), (130, 4500, 1, 1, 64),
                                             (1, 3000, 32, 4, 128)])
def test_few_queries_on_long_keys(tq, tk, hq, hk, dim, dtype):
    """Single new tokens: the keys before them, and their own, split among blocks and joined."""
    lengths, ends = [tk, tk // 2 + 1, tq, 0], [tk - tq, tk // 2 + 1 - tq, 0, -tq]
    check(make(4, tq, tk, hq, hk, dim, dtype, 5, lengths, ends), True)
    check(make(1, tq, tk, hq, hk, dim, dtype, 6), False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("batch,tq,tk,hq,hk,dim,causal", [
    (20, 300, 300, 8, 8, 64, True), (11, 260, 390, 24, 3, 128, True), (16, 513, 200, 12, 4, 80, False), (40, 129, 70, 4, 4, 32, True)])
def test_many_heads(batch, tq, tk, hq, hk, dim, causal, dtype):
    """More blocks than SMs, each with several tiles of queries, odd numbers of them and of rows in the last."""
    g = torch.Generator().manual_seed(batch)
    lengths = [int(torch.randint(0, tk + 1, (1,), generator=g)) for _ in range(batch)]
    start = [int(torch.randint(-tq, tk, (1,), generator=g)) for _ in range(batch)] if causal else None
    check(make(batch, tq, tk, hq, hk, dim, dtype, 20, lengths, start), causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tq,tk,hq,hk,causal", [(3000, 40, 4, 1, False), (2100, 2100, 3, 1, True), (5000, 1, 1, 1, False)])
def test_many_queries_on_few_keys(tq, tk, hq, hk, causal, dtype):
    check(make(1, tq, tk, hq, hk, 64, dtype, 8), causal)


def test_strides_and_orders_of_axes():
    g = torch.Generator().manual_seed(4)
    batch, t, hq, hk, dim = 2, 150, 4, 2, 72
    qkv = tensor((batch, t, hq + 2 * hk, dim), "bf16", g)
    q, k, v = qkv.split([hq, hk, hk], dim=2)
    s = {"q": q, "k": k, "v": v, "do": tensor((batch, t, hq, dim), "bf16", g), "lengths": None, "start": None}
    got, back = check(s, True)
    # heads before tokens; tokens before sequences; rows far apart; padded heads
    flip = {n: s[n].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for n in ("q", "k", "v", "do")}
    turn = {n: s[n].permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3) for n in ("q", "k", "v", "do")}
    wide = {}
    for n in ("q", "k", "v", "do"):
        room = torch.full((batch, t, s[n].shape[2], 3 * 72 + 8), NAN, dtype=torch.bfloat16, device="cuda")
        room[..., 8:80] = s[n]
        wide[n] = room[..., 8:80]
    for other in (flip, turn, wide):
        o = att.attention_forward(other["q"], other["k"], other["v"], causal=True)
        assert torch.equal(o["o"], got["o"]) and torch.equal(o["lse"], got["lse"])
        b = att.attention_backward(other["do"], other["q"], other["k"], other["v"], got["o"], got["lse"], causal=True)
        assert all(torch.equal(b[n], back[n]) for n in back)
    # outputs of the caller's, in views of one buffer; what lies between them stays
    room = torch.full((batch, t, hq + 2 * hk + 1, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    dq, dk, dv, left = room.split([hq, hk, hk, 1], dim=2)
    att.attention_backward(s["do"], q, k, v, got["o"], got["lse"], causal=True, out={"dq": dq, "dk": dk, "dv": dv})
    assert torch.equal(dq, back["dq"]) and torch.equal(dk, back["dk"]) and torch.equal(dv, back["dv"]) and bool((left == 7).all())
    o = torch.full((batch, hq, t, dim + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    att.attention_forward(q, k, v, causal=True, out={"o": o[..., :dim].permute(0, 2, 1, 3)})
    assert torch.equal(o[..., :dim].permute(0, 2, 1, 3), got["o"]) and bool((o[..., dim:] == 7).all())


def test_inputs_that_repeat():
    """Keys that all sequences share, queries that all heads share; their gradients come per use."""
    g = torch.Generator().manual_seed(9)
    q, k, v = tensor((3, 70, 1, 64), "f16", g), tensor((1, 90, 2, 64), "f16", g), tensor((1, 90, 1, 64), "f16", g)
    check({"q": q.expand(3, 70, 4, 64), "k": k.expand(3, 90, 2, 64), "v": v.expand(3, 90, 2, 64),
           "do": tensor((1, 70, 1, 64), "f16", g).expand(3, 70, 4, 64), "lengths": None, "start": None})


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size,scale", [(8.0, None), (1.0, 0.0), (0.01, 1.0), (30.0, 0.01)])
def test_scores_of_other_magnitudes(size, scale, dtype):
    check(make(2, 140, 270, 2, 1, 64, dtype, 12, size=size), False, scale)


@pytest.mark.parametrize("up", [1e-5, 3e-4, 200.0])
def test_small_and_large_gradients_in_f16(up):
    s = make(1, 260, 520, 2, 1, 64, "f16", 13)
    s["do"] = (s["do"].float() * up).half()
    check(s)


def test_rising_scores_move_the_maximum_in_every_tile():
    s = make(1, 130, 700, 1, 1, 64, "bf16", 14)
    s["q"][:] = 0
    s["k"][:] = 0
    s["q"][..., 0] = 8.0
    s["k"][0, :, 0, 0] = torch.linspace(-60, 60, 700).to(torch.bfloat16).cuda()
    check(s, False, 1.0)
    s["k"][0, :, 0, 0] = torch.linspace(60, -60, 700).to(torch.bfloat16).cuda()
    check(s, False, 1.0)


def test_a_sequence_of_nan_stays_by_itself():
    s = make(3, 150, 150, 2, 1, 64, "bf16", 15)
    clean = att.attention_forward(s["q"], s["k"], s["v"])
    back = att.attention_backward(s["do"], s["q"], s["k"], s["v"], clean["o"], clean["lse"])
    bad = {n: s[n].clone() for n in ("q", "k", "v", "do")}
    for n in bad:
        bad[n][1] = NAN
    o = att.attention_forward(bad["q"], bad["k"], bad["v"])
    b = att.attention_backward(bad["do"], bad["q"], bad["k"], bad["v"], o["o"], o["lse"])
    assert torch.isnan(o["o"][1]).all() and torch.isnan(b["dq"][1]).all() and torch.isnan(b["dk"][1]).all()
    for i in (0, 2):
        assert torch.equal(o["o"][i], clean["o"][i]) and all(torch.equal(b[n][i], back[n][i]) for n in b)


def test_empty_calls():
    for batch, tq, tk in ((0, 4, 4), (2, 0, 5), (2, 5, 0), (1, 0, 0)):
        s = make(batch, tq, tk, 2, 1, 64, "bf16")
        o = att.attention_forward(s["q"], s["k"], s["v"])
        assert not o["o"].any() and torch.isinf(o["lse"]).all()
        b = att.attention_backward(s["do"], s["q"], s["k"], s["v"], o["o"], o["lse"])
        torch.cuda.synchronize()
        assert not b["dq"].any() and not b["dk"].any() and not b["dv"].any()
    assert att.attention_forward(s["q"], s["k"], s["v"], want_lse=False)["lse"] is None


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    s = make(2, 300, 1500, 4, 2, 128, "bf16", 16, [1500, 700])
    small = make(2, 1, 1500, 4, 2, 128, "bf16", 17, [1500, 700])

    def run():
        out = []
        for x in (s, small):
            o = att.attention_forward(x["q"], x["k"], x["v"], key_lengths=x["lengths"])
            b = att.attention_backward(x["do"], x["q"], x["k"], x["v"], o["o"], o["lse"], key_lengths=x["lengths"])
            out += [o["o"], o["lse"], b["dq"], b["dk"], b["dv"]]
        return out

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run()
    for t in third:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)
    # another step's inputs in the graph's buffers
    s["q"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, c in zip(run(), third):
        assert torch.equal(a, c)


def test_a_workspace_of_the_callers():
    s = make(1, 5, 4000, 2, 1, 64, "f16", 18)
    fwd, bwd = att.attention_workspace_size(s["q"], s["k"])
    ws = torch.full((max(fwd, bwd, 16) + 64,), 255, dtype=torch.uint8, device="cuda")
    want = att.attention_forward(s["q"], s["k"], s["v"])
    got = att.attention_forward(s["q"], s["k"], s["v"], ws=ws[:fwd] if fwd else None)
    assert torch.equal(got["o"], want["o"])
    b0 = att.attention_backward(s["do"], s["q"], s["k"], s["v"], want["o"], want["lse"])
    b1 = att.attention_backward(s["do"], s["q"], s["k"], s["v"], want["o"], want["lse"], ws=ws[:bwd])
    assert all(torch.equal(b0[n], b1[n]) for n in b0)
    assert bool((ws[max(fwd, bwd):] == 255).all())
    with pytest.raises(cbr.CBRError):
        att.attention_backward(s["do"], s["q"], s["k"], s["v"], want["o"], want["lse"], ws=ws[:bwd - 1])


def test_refusals():
    s = make(2, 8, 8, 2, 1, 64, "f16", 19)
    q, k, v = s["q"], s["k"], s["v"]
    bad = [
        dict(q=q.float(), k=k.float(), v=v.float()), dict(q=q.bfloat16()), dict(k=k[:1]), dict(v=v[:, :7]), dict(q=q[..., :60], k=k[..., :60], v=v[..., :60]),
        dict(q=q.cpu()), dict(q=q[0]), dict(q=q[:, :, :1].expand(2, 8, 3, 64), k=k.expand(2, 8, 2, 64), v=v.expand(2, 8, 2, 64)),
        dict(q=torch.zeros(2, 8, 2, 136, dtype=torch.float16, device="cuda"), k=torch.zeros(2, 8, 1, 136, dtype=torch.float16, device="cuda"),
             v=torch.zeros(2, 8, 1, 136, dtype=torch.float16, device="cuda")),
        dict(k=torch.zeros(2 * 8 * 65 + 1, dtype=torch.float16, device="cuda")[1:].view(2, 8, 1, 65)[..., :64]),
        dict(k=torch.zeros(2 * 8 * 64 + 4, dtype=torch.float16, device="cuda")[4:].view(2, 8, 1, 64)),
        dict(k=k[:, :1].expand(2, 8, 1, 64)), dict(key_lengths=torch.zeros(2, dtype=torch.int64, device="cuda")),
        dict(key_lengths=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(query_start=torch.zeros(2, dtype=torch.int32)),
        dict(scale=-1.0), dict(scale=math.inf), dict(scale=NAN), dict(scale=1e39), dict(out={"o": q}), dict(out={"o": q.float()}),
        dict(out={"o": torch.zeros(2, 8, 1, 64, dtype=torch.float16, device="cuda").expand(2, 8, 2, 64)})]
    for kw in bad:
        args = {"q": q, "k": k, "v": v, **kw}
        with pytest.raises(cbr.CBRError):
            att.attention_forward(**args)
    o = att.attention_forward(q, k, v)
    for kw in (dict(lse=o["lse"].double()), dict(lse=o["lse"][:1]), dict(do=s["do"][:, :7]), dict(out={"dq": q}),
               dict(out={"dk": torch.zeros_like(v)[:, :7]}), dict(ws=torch.zeros(1, dtype=torch.uint8, device="cuda"))):
        args = {"do": s["do"], "q": q, "k": k, "v": v, "o": o["o"], "lse": o["lse"], **kw}
        with pytest.raises(cbr.CBRError):
            att.attention_backward(**args)
