"""Group norm with an activation against its plain 64-bit form: types, channels that are and are not whole
vectors, images from one pixel on to ones that no block holds, strides, in place, streams and graphs."""
import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import cbr
from conv_batchnorm_relu_gb300 import group_norm as gn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def make(shape, dtype, seed=0, offset=0.5, affine=True):
    g = torch.Generator().manual_seed(seed)
    c = shape[-1]
    level = offset + 0.5 * torch.randn(c, generator=g)
    s = {"x": (torch.randn(shape, generator=g) + level).to(DT[dtype]).cuda(), "dy": torch.randn(shape, generator=g).to(DT[dtype]).cuda(),
         "gamma": None, "beta": None}
    if affine:
        s["gamma"] = (1 + 0.2 * torch.randn(c, generator=g)).cuda()
        s["beta"] = (0.2 * torch.randn(c, generator=g)).cuda()
    return s


def check(s, groups, act, **kw):
    got = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS, act=act)
    torch.cuda.synchronize()
    want = ref.group_norm(s["x"], s["gamma"], s["beta"], groups, EPS, act)
    dt = s["x"].dtype
    ref.close(got["mean"], want["mean"], want["mean_bound"], "mean")
    ref.close(got["rstd"], want["rstd"], want["rstd_bound"], "rstd")
    ref.close(got["y"], want["y"], want["y_bound"], "y", dt)
    back = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], got["mean"], got["rstd"], groups, act=act)
    torch.cuda.synchronize()
    assert cbr.stream_status_code() == 0
    wb = ref.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], got["mean"], got["rstd"], groups, act)
    ref.close(back["dx"], wb["dx"], wb["dx_bound"], "dx", dt)
    for n in ("dgamma", "dbeta"):
        if s["gamma"] is None:
            assert back[n] is None
        else:
            ref.close(back[n], wb[n], wb[n + "_bound"], n)
    return got, back


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups,act", [
    ((1, 1, 1, 1), 1, "none"), ((2, 1, 1, 8), 1, "silu"), ((3, 7, 7, 512), 32, "silu"), ((2, 13, 9, 60), 4, "relu"), ((5, 3, 17, 7), 7, "silu"),
    ((2, 31, 33, 64), 64, "relu"), ((2, 56, 56, 64), 16, "relu"), ((1, 5, 4, 1000), 8, "none"), ((9, 8, 8, 30), 5, "silu"),
    ((1, 2, 3, 4096), 1, "relu"), ((300, 2, 2, 16), 2, "silu"), ((1, 3, 1, 16384), 32, "none"), ((2, 40, 50, 3), 3, "relu"),
    ((3, 100, 64), 4, "relu"), ((4, 96), 8, "silu")])
def test_shapes(shape, groups, act, dtype):
    check(make(shape, dtype, seed=shape[-1]), groups, act)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,groups,act", [((2, 224, 224, 64), 32, "relu"), ((1, 301, 211, 40), 5, "silu"), ((3, 112, 112, 128), 32, "silu")])
def test_images_that_no_block_holds(shape, groups, act, dtype):
    check(make(shape, dtype, seed=3), groups, act)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups,act", [((2, 9, 11, 333), 1, "silu"), ((3, 5, 7, 2056), 4, "relu"), ((1, 60, 41, 1026), 3, "silu"), ((40, 2, 2, 515), 5, "none")])
def test_more_channels_than_a_block_has_columns_for(shape, groups, act, dtype):
    check(make(shape, dtype, seed=14), groups, act)


@pytest.mark.parametrize("offset", [30.0, -1000.0])
def test_means_far_from_zero(offset):
    check(make((2, 28, 28, 64), "f32", 5, offset), 8, "none")


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_without_parameters(act):
    check(make((3, 14, 15, 48), "f16", 6, affine=False), 6, act)


def test_an_image_without_spread():
    s = make((2, 9, 9, 16), "f32", 7)
    s["x"][0] = 3.25
    got, _ = check(s, 4, "relu")
    assert bool((got["mean"][0] == 3.25).all())


def test_strides_and_in_place():
    s = make((3, 20, 21, 64), "bf16", 8)
    got, back = check(s, 8, "silu")
    for first in (0, 8, 1, 135):
        room = torch.full((3, 20, 21, 200), float("nan"), dtype=torch.bfloat16, device="cuda")
        x = room[..., first:first + 64]
        x.copy_(s["x"])
        o = gn.group_norm_forward(x, s["gamma"], s["beta"], 8, eps=EPS, act="silu")
        for n in ("mean", "rstd"):
            ref.close(o[n], got[n].cpu(), 1e-6 * got[n].cpu().abs().double(), n)
        dy = torch.empty_like(room)[..., first:first + 64]
        dy.copy_(s["dy"])
        ref_b = ref.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], got["mean"], got["rstd"], 8, "silu")
        b = gn.group_norm_backward(dy, x, s["gamma"], s["beta"], got["mean"], got["rstd"], 8, act="silu", out={"dx": dy})
        assert b["dx"] is dy
        ref.close(dy, ref_b["dx"], ref_b["dx_bound"], "dx", torch.bfloat16)
        rest = [c for c in range(200) if not first <= c < first + 64]
        assert bool(torch.isnan(room[..., rest]).all()) and torch.equal(x, s["x"])
    # images in another order, and y in x's place
    x = s["x"].flip(0).flip(0).clone()
    y = gn.group_norm_forward(x, s["gamma"], s["beta"], 8, eps=EPS, act="silu", out={"y": x})["y"]
    assert y is x and torch.equal(y, got["y"])
    far = s["x"].permute(1, 2, 0, 3).contiguous().permute(2, 0, 1, 3)   # images next to one another
    assert torch.equal(gn.group_norm_forward(far, s["gamma"], s["beta"], 8, eps=EPS, act="silu")["y"], got["y"])


def test_large_images_in_place():
    s = make((2, 224, 200, 64), "f32", 9)
    got, back = check(s, 32, "relu")
    x, dy = s["x"].clone(), s["dy"].clone()
    gn.group_norm_forward(x, s["gamma"], s["beta"], 32, eps=EPS, act="relu", out={"y": x})
    gn.group_norm_backward(dy, s["x"], s["gamma"], s["beta"], got["mean"], got["rstd"], 32, act="relu", out={"dx": dy})
    assert torch.equal(x, got["y"]) and torch.equal(dy, back["dx"])


def test_nan_and_infinity_stay_in_their_group():
    s = make((2, 10, 10, 32), "f32", 10)
    clean = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], 4, act="relu")
    for value in (float("nan"), float("inf"), float("-inf")):
        x = s["x"].clone()
        x[1, 5, 5, 9] = value
        o = gn.group_norm_forward(x, s["gamma"], s["beta"], 4, act="relu")
        assert torch.isnan(o["y"][1, 5, 5, 9])
        keep = torch.ones(2, 10, 10, 32, dtype=torch.bool, device="cuda")
        keep[1, :, :, 8:16] = False
        assert torch.equal(o["y"][keep], clean["y"][keep])


def test_empty_calls():
    for shape in ((0, 4, 4, 8), (2, 0, 4, 8)):
        s = make(shape, "f16")
        o = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], 2)
        b = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], o["mean"], o["rstd"], 2)
        torch.cuda.synchronize()
        assert not b["dgamma"].any() and not b["dbeta"].any()


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    s, t = make((6, 30, 31, 64), "bf16", 11), make((2, 112, 112, 96), "f16", 12)

    def run():
        out = []
        for x, groups in ((s, 16), (t, 6)):
            o = gn.group_norm_forward(x["x"], x["gamma"], x["beta"], groups, act="silu")
            b = gn.group_norm_backward(x["dy"], x["x"], x["gamma"], x["beta"], o["mean"], o["rstd"], groups, act="silu")
            out += [*o.values(), *b.values()]
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
    s["x"].mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c, d in zip(first, second, third, run()):
        assert torch.equal(a, b) and torch.equal(c, d)


def test_refusals():
    s = make((2, 6, 6, 16), "f16", 13)
    x, gamma, beta = s["x"], s["gamma"], s["beta"]
    for kw in (dict(groups=3), dict(groups=0), dict(groups=17), dict(x=x.cpu()), dict(x=x.double()), dict(gamma=gamma[:8]), dict(gamma=None),
               dict(beta=beta.half()), dict(act="gelu"), dict(eps=0.0), dict(eps=float("nan")), dict(x=x[..., ::2], gamma=gamma[:8], beta=beta[:8], groups=2),
               dict(x=x[:, ::2, ::2]), dict(x=x.transpose(1, 2)), dict(out={"y": x.float()}), dict(out={"mean": torch.zeros(2, 3, device="cuda")}),
               dict(out={"y": x[:1].expand(2, 6, 6, 16)})):
        args = {"x": x, "gamma": gamma, "beta": beta, "groups": 4, **kw}
        with pytest.raises(cbr.CBRError):
            gn.group_norm_forward(**args)
    o = gn.group_norm_forward(x, gamma, beta, 4)
    n = gn.group_norm_workspace_size(x, 4)[1]
    for kw in (dict(dy=s["dy"].float()), dict(mean=o["mean"][:1]), dict(out={"dx": x}), dict(ws=torch.zeros(n - 1, dtype=torch.uint8, device="cuda")),
               dict(ws=torch.zeros(n, dtype=torch.uint8)), dict(gamma=None, beta=None, out={"dx": x})):
        args = {"dy": s["dy"], "x": x, "gamma": gamma, "beta": beta, "mean": o["mean"], "rstd": o["rstd"], "groups": 4, **kw}
        with pytest.raises(cbr.CBRError):
            gn.group_norm_backward(**args)
