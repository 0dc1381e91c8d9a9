"""The global gradient norm and clipping against 64 bits: types mixed, sizes from none on, any alignment, more
tensors than one launch takes, magnitudes at the ends of the range, infinities and NaN, streams and graphs."""
import math

import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import cbr, gradients

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# a thread sums at most 64 squares in 32 bits, the rest is in 64: 64 roundings of a sum of positive terms and a
# few of the square root's, the quotient's and the scale's halve to well under this
NORM = 64 * ref.W


def make(sizes, dtypes, seed=0, scale=1e-2, shift=0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n + shift, generator=g) * scale).to(DT[dtypes[i % len(dtypes)]]).cuda()[shift:] for i, n in enumerate(sizes)]


def check(grads, share, unscale=1.0, in_place=False):
    norm, _, _ = ref.clip(grads, math.inf, unscale)
    top = float(torch.tensor(norm * share if math.isfinite(norm * share) else 1.0, dtype=torch.float32))
    norm, scale, want = ref.clip(grads, top, unscale)
    rooms = [torch.full((g.numel() + 2,), 7.0, dtype=g.dtype, device="cuda") for g in grads]
    out = [r[1:-1] for r in rooms]
    if in_place:
        for o, g in zip(out, grads):
            o.copy_(g)
        got = gradients.clip_gradients(out, top, unscale=unscale)
    else:
        before = [g.clone() for g in grads]
        got = gradients.clip_gradients(grads, top, unscale=unscale, out=out)
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
    ref.close(got["norm"], torch.tensor(norm), NORM * norm, "norm")
    ref.close(got["scale"], torch.tensor(scale), 2 * NORM * scale, "scale")
    for r, w in zip(rooms, want):
        ref.close(r[1:-1], w, 3 * NORM * w.abs(), "out", r.dtype)
        assert r[0] == 7 and r[-1] == 7
    assert float(gradients.gradient_norm(grads, unscale=unscale)) == float(got["norm"])


@pytest.mark.parametrize("dtypes", [["f32"], ["f16"], ["bf16"], ["f32", "f16", "bf16"]])
@pytest.mark.parametrize("sizes", [[1], [3, 0, 5], [8191, 8192, 8193], [100, 1, 70001, 33, 0, 4096, 12345, 7], [3_000_001]])
@pytest.mark.parametrize("share", [0.3, 4.0])
def test_sizes_and_types(sizes, dtypes, share):
    grads = make(sizes, dtypes, seed=len(sizes))
    check(grads, share)
    check(grads, share, in_place=True)


@pytest.mark.parametrize("count", [63, 64, 65, 511, 512, 513, 1200])
def test_more_tensors_than_a_launch_takes(count):
    check(make([(i * 37) % 300 for i in range(count)], ["f32", "bf16"], seed=count), 0.5)


@pytest.mark.parametrize("shift", [1, 2, 3, 5])
def test_any_alignment(shift):
    check(make([5000, 17, 20000], ["f16", "f32", "bf16"], seed=shift, shift=shift), 0.25, 0.5)


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-25, 1e18, 1e30, 1e37])
def test_magnitudes_at_the_ends_of_the_range(scale):
    check(make([5000, 100], ["f32"], 3, scale), 0.5)
    mixed = make([300, 300], ["f32"], 4, scale) + make([5000], ["bf16"], 5, 1.0)
    check(mixed, 2.0)


def test_a_loss_scale_comes_off():
    check(make([1000, 2000], ["f16"], 6, 10.0), 0.5, 1.0 / 1024)
    check(make([1000, 2000], ["f16"], 7, 10.0), 8.0, 1.0 / 1024, in_place=True)


def test_zeros_infinities_and_nan():
    g = [torch.zeros(100, device="cuda"), torch.zeros(5, device="cuda", dtype=torch.float16)]
    o = gradients.clip_gradients(g, 1.0, unscale=0.5)
    assert float(o["norm"]) == 0 and float(o["scale"]) == 0.5 and not g[0].any()
    g = [torch.full((4,), 3e38, device="cuda"), torch.ones(3, device="cuda")]
    o = gradients.clip_gradients(g, 1.0)
    # the norm, 6e38, is past fp32's range; the scale goes by it all the same (a subnormal, to 2^-149)
    assert math.isinf(float(o["norm"])) and abs(float(o["scale"]) - 1 / 6e38) < 2e-45
    assert bool(((g[0] - 0.5).abs() < 1e-6).all())
    for value, scale in ((math.inf, 0.0), (math.nan, math.nan)):
        g = [torch.ones(10, device="cuda", dtype=torch.bfloat16), torch.tensor([1.0, value], device="cuda")]
        o = gradients.clip_gradients(g, 1.0)
        s = float(o["scale"])
        assert s == scale or math.isnan(s) and math.isnan(scale)
        assert torch.isnan(g[1][1])
    g = [torch.ones(4, device="cuda")]
    assert float(gradients.clip_gradients(g, 0.0)["scale"]) == 0 and not g[0].any()
    g = [torch.ones(4, device="cuda")]
    assert float(gradients.clip_gradients(g, 2.0)["scale"]) == 1 and bool((g[0] == 1).all())      # the norm is 2
    assert float(gradients.clip_gradients(g, math.inf)["scale"]) == 1


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    grads = make([70000, 3, 1234, 40000], ["f32", "bf16"], 8)
    keep = [g.clone() for g in grads]

    def run():
        out = [torch.empty_like(g) for g in grads]
        o = gradients.clip_gradients(grads, 0.1, out=out)
        return out + [o["norm"], o["scale"]]

    first = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third = run()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, second, third))
    for g, k in zip(grads, keep):
        g.copy_(k * 3)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run(), third))


def test_refusals():
    g = [torch.ones(8, device="cuda"), torch.ones(4, device="cuda", dtype=torch.float16)]
    bad = [([], 1.0, {}), ([torch.ones(3)], 1.0, {}), ([g[0].double()], 1.0, {}), ([g[0][::2]], 1.0, {}), (g, -1.0, {}), (g, math.nan, {}),
           (g, 1.0, dict(unscale=0.0)), (g, 1.0, dict(unscale=math.inf)), (g, 1.0, dict(unscale=1e39)), (g, 1.0, dict(out=g[:1])),
           (g, 1.0, dict(out=[g[0].half(), g[1]])), (g, 1.0, dict(out=[g[0][:4], g[1]])), (g, 1.0, dict(ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))),
           (g, 1.0, dict(scalars={"norm": torch.zeros(2, device="cuda")}))]
    for grads, top, kw in bad:
        with pytest.raises(cbr.CBRError):
            gradients.clip_gradients(grads, top, **kw)
    assert bool((g[0] == 1).all())
