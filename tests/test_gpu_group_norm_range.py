"""Group norm over fp32's whole range, in every layout that the kernels have (slices of the channels, clusters, the stream
of tasks, pixels wider than a block)."""
import math

import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import group_norm as gn
from test_gpu_group_norm import EPS, make

pytestmark = pytest.mark.gpu

LAYOUTS = {"slices": ((2, 7, 7, 512), 32), "cluster": ((3, 28, 28, 64), 8), "stream": ((2, 160, 150, 96), 8), "wide": ((2, 9, 11, 333), 3)}


def group(c, groups, g):
    """The channels of group g."""
    return slice(g * (c // groups), (g + 1) * (c // groups))


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("mean,spread", [(1e20, 1e16), (-3e20, 1e16)])
def test_means_whose_squares_leave_the_range(layout, mean, spread):
    shape, groups = LAYOUTS[layout]
    s = make(shape, "f32", seed=21)
    s["x"] = mean + spread * s["x"]
    x, want = s["x"], ref.group_norm(s["x"], s["gamma"], s["beta"], groups, EPS, "none")
    got = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS)
    ref.close(got["mean"], want["mean"], want["mean_bound"], "mean")
    ref.close(got["rstd"], want["rstd"], want["rstd_bound"], "rstd")
    ref.close(got["y"], want["y"], want["y_bound"], "y")


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_nan_and_infinity_at_any_place(layout, act, value):
    """The group's rstd and all its results are NaN, wherever the value stands."""
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
        assert bool(torch.isnan(o["y"][~keep]).all()), i
        assert torch.equal(o["y"][keep], clean["y"][keep]), i
        b = gn.group_norm_backward(s["dy"], x, s["gamma"], s["beta"], o["mean"], o["rstd"], groups, act=act)
        assert bool(torch.isnan(b["dx"][~keep]).all()) and bool(b["dx"][keep].isfinite().all()), i
    x = s["x"].clone()      # both infinities
    x.view(shape[0], pixels, c)[1, [0, pixels - 1], here.start] = torch.tensor([math.inf, -math.inf], device="cuda")
    o = gn.group_norm_forward(x, s["gamma"], s["beta"], groups, eps=EPS, act=act)
    assert torch.isnan(o["rstd"][1, 1]) and bool(torch.isnan(o["y"][~keep]).all())
