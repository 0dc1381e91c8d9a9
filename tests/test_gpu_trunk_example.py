"""The trunk example's training step: its logits, loss, gradients and their norm against the same network in plain
64-bit torch operations; several steps run, and the whole step as a captured graph repeats them."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain(student, p, x, ids, top, lse, temperature):
    """The student's network and loss in 64 bits."""
    n, t, d, heads, hd = student.images, student.size ** 2, student.dim, student.heads, student.head_dim
    group = heads // student.key_heads

    def rms(a, w):
        return a / (a.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w

    z = torch.nn.functional.conv2d(x.double().permute(0, 3, 1, 2), p["filter"].permute(0, 3, 1, 2), padding=1)
    z = z.permute(0, 2, 3, 1).reshape(n * t, d)
    z = (z - z.mean(0)) / (z.var(0, unbiased=False) + 1e-5).sqrt() * p["gamma"] + p["beta"]
    z = z.relu().view(n, t, student.groups, d // student.groups)
    z = (z - z.mean((1, 3), keepdim=True)) / (z.var((1, 3), unbiased=False, keepdim=True) + 1e-5).sqrt()
    z = z.reshape(n * t, d) * p["group_gamma"] + p["group_beta"]
    x = z * torch.sigmoid(z)
    h = rms(x, p["norm0"])
    q, k, v = (h @ p["qkv"].t()).view(n, t, heads + 2 * student.key_heads, hd).split([heads, student.key_heads, student.key_heads], 2)
    angle = (student.positions.double()[:, student.axis.long()] * (student.freq.double() / 2.0 ** 64) * 2 * torch.pi)[None, :, None]

    def turn(a):
        one, two = a.chunk(2, -1)
        return torch.cat([one * angle.cos() - two * angle.sin(), two * angle.cos() + one * angle.sin()], -1)

    q, k, v = turn(q), turn(k).repeat_interleave(group, 2), v.repeat_interleave(group, 2)
    scores = torch.einsum("nthd,nshd->nhts", q, k) * hd ** -0.5
    mixed = torch.einsum("nhts,nshd->nthd", scores.softmax(-1), v).reshape(n * t, heads * hd)
    x = x + p["gate1"] * rms(mixed @ p["proj"].t(), p["post1"])
    h = rms(x, p["norm1"])
    x = x + p["gate2"] * rms((h @ p["up"].t()).relu() @ p["down"].t(), p["post2"])
    logits = rms(x, p["norm2"]).view(n, t, d).mean(1) @ p["head"].t()
    log_q = torch.log_softmax(logits / temperature, 1)
    prob = (top.double() / temperature - lse.double()[:, None]).exp()
    rest = 1 - prob.sum(1)
    kept = torch.ones_like(log_q, dtype=torch.bool).scatter_(1, ids, False)
    log_rest = torch.logsumexp(log_q.masked_fill(~kept, -torch.inf), 1)
    loss = (prob * (prob.log() - log_q.gather(1, ids))).sum(1) + rest * (rest.log() - log_rest)
    return logits, loss.mean() * temperature ** 2


def test_step_against_plain_network():
    """Activations are rounded to 8 significant bits some twenty-five times on the way to the loss and back: relative
    errors of 25 * 2^-8 / sqrt(3), under 6%, in the 2-norm of a gradient, if they add up at worst as they come; the
    loss, a mean over rows of near-independent errors, within 2%; the gradients' norm as they are."""
    import trunk_student as ex
    from conv_batchnorm_relu_gb300 import gradients
    student = ex.Student()
    x, ids, top, lse, temperature = ex.make_batch(student)
    p = {k: v.detach().double().requires_grad_() for k, v in student.p.items()}
    want_logits, want = plain(student, p, x, ids, top, lse, temperature)
    want_grads = torch.autograd.grad(want, list(p.values()))
    logits = student(x)
    loss = ex.Distill.apply(logits, ids, top, lse, temperature)
    grads = [g.contiguous() for g in torch.autograd.grad(loss, list(student.p.values()))]
    assert ((logits.double() - want_logits).norm() / want_logits.norm()).item() < 0.06
    assert abs(loss.item() - want.item()) < 0.02 * want.item()
    for name, got, ref in zip(p, grads, want_grads):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 0.06, name
    norm = math.sqrt(math.fsum(float(g.double().pow(2).sum()) for g in grads))
    top_norm = 0.25 * norm
    want_scaled = [g.double() * (top_norm / norm) for g in grads]
    got = gradients.clip_gradients(grads, top_norm)
    assert abs(got["norm"].item() - norm) < 1e-5 * norm
    for g, w in zip(grads, want_scaled):
        assert ((g.double() - w).norm() / w.norm()).item() < 2 * torch.finfo(g.dtype).eps


def test_steps_run():
    import trunk_student as ex
    losses, norms = ex.train(5)
    assert len(losses) == len(norms) == 5 and all(math.isfinite(v) and v > 0 for v in losses + norms)


def test_a_captured_step_repeats():
    """Forward, loss, backward and clipping in one graph, replayed: the gradients of the eager step, bit for bit."""
    import trunk_student as ex
    from conv_batchnorm_relu_gb300 import gradients
    student = ex.Student()
    x, ids, top, lse, temperature = ex.make_batch(student)

    def step():
        loss = ex.Distill.apply(student(x), ids, top, lse, temperature)
        grads = [g.contiguous() for g in torch.autograd.grad(loss, list(student.p.values()))]
        norm = gradients.clip_gradients(grads, 0.1)["norm"]
        return [loss.detach(), norm, *grads]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        eager = [t.clone() for t in step()]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, captured):
        assert torch.equal(a, b)
