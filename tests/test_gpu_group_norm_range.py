"""Group norm over fp32's whole range, in every layout that the kernels have (slices of the channels, clusters, the stream
of tasks, pixels wider than a block)."""
import pytest

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import group_norm as gn
from test_gpu_group_norm import EPS, make

pytestmark = pytest.mark.gpu

LAYOUTS = {"slices": ((2, 7, 7, 512), 32), "cluster": ((3, 28, 28, 64), 8), "stream": ((2, 160, 150, 96), 8), "wide": ((2, 9, 11, 333), 3)}


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
