"""Clipping of far more tensors than one launch takes: what the scale of each costs does not grow with their number."""
import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import gradients
from test_gpu_clip import NORM

pytestmark = pytest.mark.gpu


def captured(count):
    """A graph of one call over `count` tensors of eight values; its inputs and outputs."""
    flat = torch.randn(8 * count, generator=torch.Generator().manual_seed(count)).cuda()
    out = torch.zeros_like(flat)
    grads, outs = list(flat.view(count, 8)), list(out.view(count, 8))
    gradients.clip_gradients(grads, 1.0, out=outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gradients.clip_gradients(grads, 1.0, out=outs)
    return graph, flat, out, got


def milliseconds(graph):
    times = []
    for _ in range(7):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end))
    return sorted(times)[3]


def test_time_grows_with_the_number_of_tensors():
    """16 times the tensors are 16 times the launches; a sum over all of them in each launch would be 256 times the work."""
    few, many = captured(2 ** 12), captured(2 ** 16)
    assert milliseconds(many[0]) < 24 * milliseconds(few[0])
    for _, flat, out, got in (few, many):
        norm, scale, _ = ref.clip([flat], 1.0)
        ref.close(got["norm"], torch.tensor(norm), NORM * norm, "norm")
        ref.close(got["scale"], torch.tensor(scale), 2 * NORM * scale, "scale")
        ref.close(out, flat.cpu().double() * scale, 3 * NORM * scale * flat.abs().cpu().double(), "out")


@pytest.mark.parametrize("count", [513, 1500])
@pytest.mark.parametrize("top,unscale", [(0.5, 1.0), (1e9, 1.0), (1e9, 0.25)])
def test_in_place_over_several_launches(count, top, unscale):
    """In place, where the scale is 1 too: the same bits as into other tensors."""
    grads = [torch.randn(1 + i % 37, generator=torch.Generator().manual_seed(i)).to((torch.float32, torch.bfloat16)[i % 2]).cuda() for i in range(count)]
    outs = [torch.empty_like(g) for g in grads]
    want = gradients.clip_gradients(grads, top, unscale=unscale, out=outs)
    got = gradients.clip_gradients(grads, top, unscale=unscale)
    assert torch.equal(got["norm"], want["norm"]) and torch.equal(got["scale"], want["scale"])
    assert all(torch.equal(g, o) for g, o in zip(grads, outs))
    norm, scale, _ = ref.clip([o.float() for o in outs], float("inf"))
    assert abs(norm - min(top, want["norm"].item())) < 2 ** -8 * norm
