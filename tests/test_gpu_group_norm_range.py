"""Group norm over fp32's whole range, in every layout that the kernels have (slices of the channels, clusters, the stream
of tasks, pixels wider than a block)."""
import math

import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import cbr
from conv_batchnorm_relu_gb300 import group_norm as gn
from test_gpu_group_norm import DT, EPS, make

pytestmark = pytest.mark.gpu

LAYOUTS = {"slices": ((2, 7, 7, 512), 32), "cluster": ((3, 28, 28, 64), 8), "stream": ((2, 160, 150, 96), 8), "wide": ((2, 9, 11, 333), 3)}


# coefficients of a gradient of subnormal size are each off by half a step of 2^-149, and |g| and |xh| are below 8
SUBNORMAL = 32 * 2.0 ** -150


def check(s, groups, act="silu"):
    """Forward and backward against 64 bits."""
    x, dt = s["x"], s["x"].dtype
    assert bool(x.isfinite().all())
    got = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS, act=act)
    want = ref.group_norm(x, s["gamma"], s["beta"], groups, EPS, act)
    ref.close(got["mean"], want["mean"], want["mean_bound"], "mean")
    ref.close(got["rstd"], want["rstd"], want["rstd_bound"], "rstd")
    ref.close(got["y"], want["y"], want["y_bound"], "y", dt)
    back = gn.group_norm_backward(s["dy"], x, s["gamma"], s["beta"], got["mean"], got["rstd"], groups, act=act)
    wb = ref.group_norm_backward(s["dy"], x, s["gamma"], s["beta"], got["mean"], got["rstd"], groups, act)
    ref.close(back["dx"], wb["dx"], wb["dx_bound"] + SUBNORMAL, "dx", dt)
    for n in ("dgamma", "dbeta"):
        ref.close(back[n], wb[n], wb[n + "_bound"], n)
    assert cbr.stream_status_code() == 0
    return got


def group(c, groups, g):
    """The channels of group g."""
    return slice(g * (c // groups), (g + 1) * (c // groups))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("mean,spread", [(1e20, 1e16), (-3e20, 1e16), (-3e30, 1e26), (1e37, 1e34)])
def test_means_whose_squares_leave_the_range(layout, mean, spread):
    """(The spreads' own squares: the last two's.)"""
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=21)
    s["x"] = mean + spread * s["x"]
    check(s, groups, "none")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spread", [1e15, 3e19, 1e25, 3e37])
def test_spreads_whose_squares_leave_the_range(layout, dtype, spread):
    shape, groups = LAYOUTS[layout]
    s = make(shape, dtype, seed=22)
    s["x"] = (s["x"].float() * spread).to(DT[dtype])
    check(s, groups, "silu" if dtype == "f32" else "relu")


@pytest.mark.parametrize("layout", LAYOUTS)
def test_values_at_both_ends_of_the_range(layout):
    """Half of a group is the largest number, half its negative: differences are past the range."""
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=23)
    s["x"] = torch.where(s["x"] > 0, 1.0, -1.0) * torch.finfo(torch.float32).max
    check(s, groups, "none")


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_constant_in_each_run_of_pixels(layout):
    """No spread in a thread's, row's or run's values, only among them."""
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=24)
    pixels = math.prod(shape[1:-1])
    level = 1e30 * torch.randn(8, generator=torch.Generator().manual_seed(1))
    s["x"] = level[torch.arange(pixels) * 8 // pixels].view(1, *shape[1:-1], 1).expand(shape).contiguous().cuda()
    check(s, groups, "none")


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("spread", [1e22, 1e36])
def test_the_other_groups_keep_their_bits(layout, spread):
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=25)
    clean = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS)
    far = group(shape[-1], groups, 1)
    s["x"][1][..., far] *= spread
    got = check(s, groups)
    again = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS)
    keep = torch.ones(shape[0], groups, dtype=torch.bool, device="cuda")
    keep[1, 1] = False
    for n in ("mean", "rstd"):
        assert torch.equal(got[n][keep], clean[n][keep])
    assert torch.equal(again["y"][0], clean["y"][0])
    ordinary = torch.ones(shape[-1], dtype=torch.bool, device="cuda")
    ordinary[far] = False
    # y of the image's other groups: the same values up to the order of two roundings
    a, b = again["y"][1][..., ordinary], clean["y"][1][..., ordinary]
    assert bool(((a - b).abs() <= 4 * ref.W * (1 + b.abs())).all())


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_nan_and_infinity_at_any_place(layout, act, value):
    """The group's rstd and all its results are NaN, and its mean is what the sum is, wherever the value stands."""
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=26)
    clean = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS, act=act)
    c, pixels = shape[-1], math.prod(shape[1:-1])
    here = group(c, groups, 1)
    keep = torch.ones(shape, dtype=torch.bool, device="cuda")
    keep[1][..., here] = False
    for i in range(pixels) if pixels < 100 else [0, 1, 2, 3, 15, 16, 31, 100, 255, 256, 700, pixels // 3, pixels // 2, pixels - 1]:
        x = s["x"].clone()
        x.view(shape[0], pixels, c)[1, i, here.start + i % (c // groups)] = value
        o = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS, act=act)
        assert torch.isnan(o["rstd"][1, 1]), i
        assert torch.equal(o["mean"][1, 1].cpu(), torch.tensor(value)) or math.isnan(value) and torch.isnan(o["mean"][1, 1]), i
        assert bool(torch.isnan(o["y"][~keep]).all()), i
        assert torch.equal(o["y"][keep], clean["y"][keep]), i
        b = gn.group_norm_backward(s["dy"], x, s["gamma"], s["beta"], o["mean"], o["rstd"], groups, act=act)
        assert bool(torch.isnan(b["dx"][~keep]).all()) and bool(b["dx"][keep].isfinite().all()), i
    x = s["x"].clone()      # both infinities: the mean is none
    x.view(shape[0], pixels, c)[1, [0, pixels - 1], here.start] = torch.tensor([math.inf, -math.inf], device="cuda")
    o = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS, act=act)
    assert torch.isnan(o["mean"][1, 1]) and torch.isnan(o["rstd"][1, 1]) and bool(torch.isnan(o["y"][~keep]).all())


@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_map_of_nan_in_place(layout):
    """Every sum is taken again, in a map that its own results replace."""
    shape, groups = LAYOUTS[layout]
    x = torch.full(shape, math.nan, device="cuda")
    o = gn.group_norm_forward(x, None, None, groups, act="relu", out={"y": x})
    assert bool(torch.isnan(x).all()) and bool(torch.isnan(o["rstd"]).all()) and bool(torch.isnan(o["mean"]).all())
    x = torch.randn(shape, generator=torch.Generator().manual_seed(2)).cuda() * 1e30
    want = gn.group_norm_forward(x, None, None, groups, act="relu")
    got = gn.group_norm_forward(x, None, None, groups, act="relu", out={"y": x})
    assert all(torch.equal(got[n], want[n]) for n in want)
    cbr.stream_status()


@pytest.mark.parametrize("shape", [(2, 0, 4, 8), (3, 5, 0, 8)])
def test_a_map_without_pixels_has_no_statistics(shape):
    x = torch.empty(shape, device="cuda")
    out = {n: torch.full((shape[0], 2), 7.0, device="cuda") for n in ("mean", "rstd")}
    o = gn.group_norm_forward(x, None, None, 2, out=out)
    assert bool(torch.isnan(o["mean"]).all()) and bool(torch.isnan(o["rstd"]).all())


def test_silu_over_its_range():
    """z is beta exactly where an image is constant.  exp is good to (2 + 1.173 |z|) steps of 2^-23 of it, the quotient to two,
    the sum in between to half of one; below -87 the quotient's divisor is past 2^126 and the result 0."""
    z = torch.linspace(-110, 90, 1600, dtype=torch.float64).float()
    x = torch.full((1, 3, 5, 1600), 2.5, device="cuda")
    y = gn.group_norm_forward(x, torch.ones(1600, device="cuda"), z.cuda(), 4, act="silu")["y"][0, 1, 2]
    z = z.double()
    want = z * torch.sigmoid(z)
    ref.close(y, want, (5 + 1.2 * z.abs()) * 2.0 ** -23 * want.abs() + 2.0 ** -118, "y")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape,groups", [((2, 24, 20, 1536), 24), ((3, 7, 9, 2048), 32), ((2, 60, 61, 1048), 8), ((1, 100, 90, 1024), 1)])
def test_wide_pixels_that_a_block_has_columns_for(shape, groups, dtype):
    check(make(shape, dtype, seed=27), groups, "relu")


@pytest.mark.parametrize("shape,groups", [((2, 20, 21, 512), 1), ((2, 70, 71, 1024), 2), ((2, 9, 5, 2056), 1)])
def test_groups_wider_than_a_block(shape, groups):
    """Values far apart, and one NaN, in groups of more channels than a block has threads; strided, and in place."""
    s = make(shape, "bf16", seed=28)
    s["x"] = (s["x"].float() * 1e27).to(torch.bfloat16)
    want = check(s, groups, "relu")
    c = shape[-1]
    room = torch.full((*shape[:-1], c + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    x = room[..., 8:8 + c]
    x.copy_(s["x"])
    got = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS, act="relu", out={"y": x})
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert bool((room[..., :8] == 7).all()) and bool((room[..., 8 + c:] == 7).all())
    s["x"][1, 3, 4, c - 1] = math.nan
    got = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS, act="relu")
    bad = torch.zeros(shape[0], groups, dtype=torch.bool, device="cuda")
    bad[1, groups - 1] = True
    assert torch.equal(torch.isnan(got["mean"]), bad) and torch.equal(torch.isnan(got["rstd"]), bad)
    assert torch.equal(torch.isnan(got["y"]).flatten(1, -2).any(1), bad.repeat_interleave(c // groups, 1))
