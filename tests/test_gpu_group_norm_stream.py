"""Group norm's stream of tasks with many images, so that moments, merges and results of different images are under way
at once; and results written between values that have to stay as they were."""
import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import cbr
from conv_batchnorm_relu_gb300 import group_norm as gn
from test_gpu_group_norm import EPS, check, make

pytestmark = pytest.mark.gpu

MANY = (40, 112, 112, 64)


def test_many_images():
    check(make((40, 96, 100, 64), "f16", seed=31), 16, "relu")


@pytest.mark.parametrize("dtype,act", [("f16", "silu"), ("f32", "relu")])
def test_many_images_as_each_alone(dtype, act):
    """Statistics and results of the whole batch are held against 64 bits, a few images at a time."""
    s = make(MANY, dtype, seed=32)
    got = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], 16, eps=EPS, act=act)
    back = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], got["mean"], got["rstd"], 16, act=act)
    for i in range(0, 40, 8):
        part = slice(i, i + 8)
        want = ref.group_norm(s["x"][part], s["gamma"], s["beta"], 16, EPS, act)
        for n in ("mean", "rstd"):
            ref.close(got[n][part], want[n], want[n + "_bound"], n)
        ref.close(got["y"][part], want["y"], want["y_bound"], "y", s["x"].dtype)
        wb = ref.group_norm_backward(s["dy"][part], s["x"][part], s["gamma"], s["beta"], got["mean"][part], got["rstd"][part], 16, act)
        ref.close(back["dx"][part], wb["dx"], wb["dx_bound"], "dx", s["x"].dtype)
    cbr.stream_status()


@pytest.mark.parametrize("first", [0, 8, 1])
def test_many_images_in_place_and_strided(first):
    """The same bits in place, and with gaps between the pixels that stay as they were."""
    s = make(MANY, "bf16", seed=33)
    want = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], 8, eps=EPS, act="relu")
    back = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], want["mean"], want["rstd"], 8, act="relu")
    room = torch.full((*MANY[:3], 80), 7.0, dtype=torch.bfloat16, device="cuda")
    x, dy = room[..., first:first + 64], room.clone()[..., first:first + 64]
    x.copy_(s["x"])
    dy.copy_(s["dy"])
    other = dy._base
    b = gn.group_norm_backward(dy, x, s["gamma"], s["beta"], want["mean"], want["rstd"], 8, act="relu", out={"dx": dy})
    o = gn.group_norm_forward(x, s["gamma"], s["beta"], 8, eps=EPS, act="relu", out={"y": x})
    if first == 1:      # single elements: the sums are shared out another way
        for n in ("mean", "rstd"):
            ref.close(o[n], want[n].cpu(), 1e-5 * (want[n].abs() + 0.1).double().cpu(), n)
        assert bool(((x - want["y"]).abs().float() <= 2.0 ** -7 * (want["y"].abs().float() + 0.01)).all())
    else:
        assert all(torch.equal(o[n], want[n]) for n in want)
    assert torch.equal(o["y"], x) and torch.equal(b["dx"], dy)
    if first == 0:
        assert torch.equal(dy, back["dx"]) and torch.equal(b["dgamma"], back["dgamma"]) and torch.equal(b["dbeta"], back["dbeta"])
    rest = [c for c in range(80) if not first <= c < first + 64]
    assert bool((room[..., rest] == 7).all()) and bool((other[..., rest] == 7).all())


LAYOUTS = [((2, 7, 7, 512), 32), ((3, 20, 21, 64), 8), ((2, 160, 150, 96), 8), ((2, 9, 11, 333), 3), ((3, 5, 7, 2056), 4)]


@pytest.mark.parametrize("shape,groups", LAYOUTS)
@pytest.mark.parametrize("first", [0, 8, 1, 135])
def test_strided_results_and_what_lies_between_them(shape, groups, first):
    """x, dy and both results in rooms of their own at any alignment: values, gradients of the parameters, gaps."""
    s = make(shape, "bf16", seed=34)
    c = shape[-1]
    rooms = {n: torch.full((*shape[:-1], c + 140), 7.0, dtype=torch.bfloat16, device="cuda") for n in ("x", "dy", "y", "dx")}
    v = {n: r[..., first:first + c] for n, r in rooms.items()}
    v["x"].copy_(s["x"])
    v["dy"].copy_(s["dy"])
    for in_place in (False, True):
        names = ("dy", "x") if in_place else ("dx", "y")
        want = ref.group_norm(s["x"], s["gamma"], s["beta"], groups, EPS, "silu")
        o = gn.group_norm_forward(v["x"], s["gamma"], s["beta"], groups, eps=EPS, act="silu", out={"y": v["y"]})
        for n in ("mean", "rstd"):
            ref.close(o[n], want[n], want[n + "_bound"], n)
        b = gn.group_norm_backward(v["dy"], v["x"], s["gamma"], s["beta"], o["mean"], o["rstd"], groups, act="silu", out={"dx": v[names[0]]})
        if in_place:
            again = gn.group_norm_forward(v["x"], s["gamma"], s["beta"], groups, eps=EPS, act="silu", out={"y": v["x"]})
            assert torch.equal(again["y"], v["y"])
        wb = ref.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], o["mean"], o["rstd"], groups, "silu")
        ref.close(v[names[1]], want["y"], want["y_bound"], "y", torch.bfloat16)
        ref.close(v[names[0]], wb["dx"], wb["dx_bound"], "dx", torch.bfloat16)
        for n in ("dgamma", "dbeta"):
            ref.close(b[n], wb[n], wb[n + "_bound"], n)
    rest = [i for i in range(c + 140) if not first <= i < first + c]
    for n, r in rooms.items():
        assert bool((r[..., rest] == 7).all()), n
    cbr.stream_status()


@pytest.mark.parametrize("shape,groups", LAYOUTS + [((40, 60, 60, 64), 16)])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_a_workspace_of_the_reported_size(shape, groups, dtype):
    s = make(shape, dtype, seed=35)
    want = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS, act="relu")
    back = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], want["mean"], want["rstd"], groups, act="relu")
    for i, n in enumerate(gn.group_norm_workspace_size(s["x"], groups)):
        room = torch.full((n + 512,), 85, dtype=torch.uint8, device="cuda")
        ws = room[256:256 + n]
        if i == 0:
            got, right = gn.group_norm_forward(s["x"], s["gamma"], s["beta"], groups, eps=EPS, act="relu", ws=ws), want
        else:
            got, right = gn.group_norm_backward(s["dy"], s["x"], s["gamma"], s["beta"], want["mean"], want["rstd"], groups, act="relu", ws=ws), back
        assert all(torch.equal(got[k], right[k]) for k in right)
        assert bool((room[:256] == 85).all()) and bool((room[256 + n:] == 85).all())
