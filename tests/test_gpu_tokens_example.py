"""The example's training step: its logits, loss and gradients against the same network in plain 64-bit
torch operations, and the loss over its steps."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def plain(student, p, x, ids, top, lse, temperature):
    """The student's network and loss in 64 bits."""
    n, t, d, heads = student.images, student.size ** 2, student.dim, student.heads

    def rms(a, w):
        return a / (a.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w

    z = torch.nn.functional.conv2d(x.double().permute(0, 3, 1, 2), p["filter"].permute(0, 3, 1, 2), padding=1)
    z = z.permute(0, 2, 3, 1).reshape(n * t, d)
    z = (z - z.mean(0)) / (z.var(0, unbiased=False) + 1e-5).sqrt() * p["gamma"] + p["beta"]
    x = z.relu()
    h = rms(x, p["norm0"])
    q, k, v = (h @ p["qkv"].t()).view(n, t, 3 * heads, d // heads).split(heads, dim=2)
    turns = student.positions.double()[:, student.axis.long()] * (student.freq.double() / 2.0 ** 64)
    angle = (turns * 2 * torch.pi)[None, :, None]

    def turn(a):
        one, two = a.chunk(2, -1)
        return torch.cat([one * angle.cos() - two * angle.sin(), two * angle.cos() + one * angle.sin()], -1)

    scores = torch.einsum("nthd,nshd->nhts", turn(q), turn(k)) * (d // heads) ** -0.5
    mixed = torch.einsum("nhts,nshd->nthd", scores.softmax(-1), v).reshape(n * t, d)
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
    """Activations are rounded to 8 significant bits some twenty times on the way to the loss and back:
    relative errors of 20 * 2^-8 / sqrt(3), under 5%, in the 2-norm of a gradient, if they add up at worst
    as they come; the loss, a mean over rows of near-independent errors, within 2%."""
    import distill_student as ex
    student = ex.Student()
    x, ids, top, lse, temperature = ex.make_batch(student)
    p = {k: v.detach().double().requires_grad_() for k, v in student.p.items()}
    want_logits, want = plain(student, p, x, ids, top, lse, temperature)
    want_grads = torch.autograd.grad(want, list(p.values()))
    logits = student(x)
    loss = ex.Distill.apply(logits, ids, top, lse, temperature)
    grads = torch.autograd.grad(loss, list(student.p.values()))
    assert ((logits.double() - want_logits).norm() / want_logits.norm()).item() < 0.05
    assert abs(loss.item() - want.item()) < 0.02 * want.item()
    for name, got, ref in zip(p, grads, want_grads):
        assert ((got.double() - ref).norm() / ref.norm()).item() < 0.05, name


def test_loss_falls():
    import distill_student as ex
    losses = ex.train(30)
    assert losses[-1] < 0.9 * losses[0] and all(l == l for l in losses)
