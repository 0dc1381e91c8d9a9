"""The trunk operators as calls meet: elements past 32 bits of offset, two streams at once, two captured graphs on one
workspace, a gradient named twice."""
import math

import pytest
import torch

from conv_batchnorm_relu_gb300 import attention as att
from conv_batchnorm_relu_gb300 import cbr, gradients
from conv_batchnorm_relu_gb300 import group_norm as gn

pytestmark = pytest.mark.gpu


def normal(*shape, seed=0, dtype=torch.float16):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def far_view(t, axis):
    """t's values in a view whose last step along `axis` begins past 2^31 elements; gaps between its steps."""
    stride = -(-(2 ** 31 + 64) // (t.shape[axis] - 1) // 64) * 64 + 64
    inner = list(t.stride())
    inner[axis] = stride
    room = torch.empty(stride * (t.shape[axis] - 1) + t.numel(), dtype=t.dtype, device="cuda")
    view = room.as_strided(t.shape, inner)
    view.copy_(t)
    return view


@pytest.mark.parametrize("axis", [0, 1])
def test_attention_past_32_bits(axis):
    """The same bits as of contiguous operands, with every operand's and result's steps that far apart."""
    q, k, v, do = (normal(2, 130, 1, 64, seed=i) for i in range(4))
    want = att.attention_forward(q, k, v, causal=True)
    back = att.attention_backward(do, q, k, v, want["o"], want["lse"], causal=True)
    far = [far_view(t, axis) for t in (q, k, v, do)]
    out = {n: far_view(torch.zeros_like(q), axis) for n in ("o", "dq", "dk", "dv")}
    got = att.attention_forward(*far[:3], causal=True, out=out)
    grads = att.attention_backward(far[3], *far[:3], got["o"], got["lse"], causal=True, out=out)
    assert torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
    assert all(torch.equal(grads[n], back[n]) for n in back)
    cbr.stream_status()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_cache_that_is_not_written_yet(dtype):
    """Causal, no lengths: what lies behind the last query's own key may be NaN, in keys as in values."""
    start = torch.tensor([0, 37, 150, -3, 292], dtype=torch.int32, device="cuda")
    q, do = normal(5, 8, 4, 64, seed=1, dtype=dtype), normal(5, 8, 4, 64, seed=2, dtype=dtype)
    k, v = normal(5, 300, 2, 64, seed=3, dtype=dtype), normal(5, 300, 2, 64, seed=4, dtype=dtype)
    behind = torch.arange(300, device="cuda") >= start[:, None] + 8
    want = att.attention_forward(q, k, v, causal=True, query_start=start)
    back = att.attention_backward(do, q, k, v, want["o"], want["lse"], causal=True, query_start=start)
    k, v = (t.masked_fill(behind[:, :, None, None], math.nan) for t in (k, v))
    got = att.attention_forward(q, k, v, causal=True, query_start=start)
    grads = att.attention_backward(do, q, k, v, got["o"], got["lse"], causal=True, query_start=start)
    assert bool(got["o"].isfinite().all()) and torch.equal(got["o"], want["o"]) and torch.equal(got["lse"], want["lse"])
    assert all(torch.equal(grads[n], back[n]) for n in back)
    assert bool((grads["dk"][behind] == 0).all()) and bool((grads["dv"][behind] == 0).all())


@pytest.mark.parametrize("axis,shape", [(0, (3, 40, 64)), (1, (1, 70, 64)), (1, (1, 6000, 64)), (0, (2, 9, 2200))])
def test_group_norm_past_32_bits(axis, shape):
    x, dy = normal(*shape, seed=5), normal(*shape, seed=6)
    gamma, beta = normal(shape[-1], seed=7, dtype=torch.float32), normal(shape[-1], seed=8, dtype=torch.float32)
    want = gn.group_norm_forward(x, gamma, beta, 4, act="silu")
    back = gn.group_norm_backward(dy, x, gamma, beta, want["mean"], want["rstd"], 4, act="silu")
    x, dy = far_view(x, axis), far_view(dy, axis)
    got = gn.group_norm_forward(x, gamma, beta, 4, act="silu", out={"y": far_view(torch.zeros(shape, dtype=x.dtype, device="cuda"), axis)})
    grads = gn.group_norm_backward(dy, x, gamma, beta, got["mean"], got["rstd"], 4, act="silu",
                                   out={"dx": far_view(torch.zeros(shape, dtype=x.dtype, device="cuda"), axis)})
    assert all(torch.equal(got[n], want[n]) for n in want) and all(torch.equal(grads[n], back[n]) for n in back)
    cbr.stream_status()


def test_a_gradient_past_32_bits():
    """2^32 + 5 values of which six are not 0: the norm is theirs, and so is what is scaled (exactly: a scale of 1/4)."""
    g = torch.zeros(2 ** 32 + 5, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1, 2 ** 31, 2 ** 32 - 1, 2 ** 32, 2 ** 32 + 4], device="cuda")
    g[at] = torch.tensor([8.0, 8.0, 8.0, 4.0, 4.0, 4.0], dtype=torch.bfloat16, device="cuda")
    got = gradients.clip_gradients([g], 0.25 * math.sqrt(240.0))
    assert abs(got["norm"].item() - math.sqrt(240.0)) < 1e-5
    assert g[at].tolist() == [2.0, 2.0, 2.0, 1.0, 1.0, 1.0] and int(torch.count_nonzero(g[: 2 ** 31])) == 2


def maps(seed):
    """A map that no cluster holds, its gradient and parameters."""
    return [normal(2, 160, 150, 96, seed=seed, dtype=torch.bfloat16), normal(2, 160, 150, 96, seed=seed + 1, dtype=torch.bfloat16),
            normal(96, seed=seed + 2, dtype=torch.float32), normal(96, seed=seed + 3, dtype=torch.float32)]


def both_norms(x, dy, gamma, beta, ws=None):
    o = gn.group_norm_forward(x, gamma, beta, 8, act="relu", ws=ws)
    b = gn.group_norm_backward(dy, x, gamma, beta, o["mean"], o["rstd"], 8, act="relu", ws=ws)
    return [*o.values(), *b.values()]


def both_attentions(q, k, v, do, ws=None):
    o = att.attention_forward(q, k, v, ws=ws)
    return [o["o"], o["lse"], *att.attention_backward(do, q, k, v, o["o"], o["lse"], ws=ws).values()]


def test_two_streams_at_once():
    """Calls of one stream in the other's midst: resident grids, clusters and workspaces of their own."""
    m = [maps(1), maps(11)]
    a = [[normal(2, 300, 4, 64, seed=s + i) for i in range(4)] for s in (21, 31)]
    grads = [[normal(70001, seed=s), normal(333, seed=s + 1, dtype=torch.float32)] for s in (41, 51)]

    def run(i):
        clipped = gradients.clip_gradients(grads[i], 1.0, out=[torch.empty_like(g) for g in grads[i]])
        return both_norms(*m[i]) + both_attentions(*a[i]) + list(clipped.values())

    want = [run(0), run(1)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None]
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                got[i] = run(i)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for i in (0, 1) for x, y in zip(want[i], got[i]))
    cbr.stream_status()


def test_two_graphs_on_one_workspace():
    """Each replayed after the other, twice: nothing of a call is left for the next."""
    m = [maps(1), maps(11)]
    a = [[normal(2, 5, 4, 64, seed=s), *(normal(2, 3000, 1, 64, seed=s + i) for i in (1, 2)), normal(2, 5, 4, 64, seed=s + 3)] for s in (21, 31)]
    n = max(*gn.group_norm_workspace_size(m[0][0], 8), *att.attention_workspace_size(*a[0][:2]))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    want = [both_norms(*m[i]) + both_attentions(*a[i]) for i in (0, 1)]
    graphs, got = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    ws.fill_(255)
    torch.cuda.synchronize()
    for i in (0, 1):
        with torch.cuda.graph(graphs[i]):
            got.append(both_norms(*m[i], ws=ws) + both_attentions(*a[i], ws=ws))
    for _ in range(2):
        for i in (0, 1):
            for t in got[i]:
                t.zero_()
            graphs[i].replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(want[i], got[i])), i
    cbr.stream_status()


def test_a_gradient_named_twice():
    g, h = normal(1000, seed=1), normal(500, seed=2)
    before = g.clone()
    for grads, out in (([g, g], None), ([g, g[100:200]], None), ([g, h], [g, g[:500]]), ([g, h], [h.new_empty(1000), g[:500]])):
        with pytest.raises(cbr.CBRError):
            gradients.clip_gradients(grads, 0.5, out=out)
    assert torch.equal(g, before)
    out = gradients.clip_gradients([g, g], 0.5, out=[torch.empty_like(g), torch.empty_like(g)])      # read twice: counted twice
    assert abs(out["norm"].item() - math.sqrt(2) * before.double().norm().item()) < 1e-5 * out["norm"].item()
