"""Trains a small hybrid student from a teacher's stored top logits, with this package's kernels.

A Conv-BN-ReLU stem turns images into a feature map, whose pixels are the tokens of a trunk: one block of
attention and one of a two-layer network, each between two norms and with a gate on its way into the
residual stream; queries and keys are rotated by their pixel's row and column; the pooled features'
logits learn from the ten best logits a teacher left for each image.

    python examples/distill_student.py [--steps 30]

The stem, the norms, the rotation and the loss are the package's; the matrix products between them and
the attention's softmax are torch's, and torch.autograd strings the backward calls together.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from conv_batchnorm_relu_gb300 import cbr, tokens  # noqa: E402

DTYPE = torch.bfloat16


class Stem(torch.autograd.Function):
    """images NHWC -> relu(batch norm(conv)), NHWC."""

    @staticmethod
    def forward(ctx, x, w, gamma, beta, layer, running, ws):
        o = cbr.forward_train(layer, x, w, gamma, beta, *running, ws=ws[0])
        ctx.save_for_backward(x, w, gamma, o["mask"], o["z"], o["saved_mean"], o["saved_inv_var"])
        ctx.layer, ctx.ws = layer, ws[1]
        return o["y"]

    @staticmethod
    def backward(ctx, dy):
        x, w, gamma, mask, z, mean, inv_var = ctx.saved_tensors
        o = cbr.backward(ctx.layer, dy.contiguous(), x, w, mask, cbr.CBR_MASK_BITS, z, gamma, mean, inv_var, ws=ctx.ws,
                         need_dx=False)
        return None, o["dw"].to(w.dtype), o["dgamma"], o["dbeta"], None, None, None


class Join(torch.autograd.Function):
    """(x, branch) -> (the residual stream after the branch has joined it, its norm)."""

    @staticmethod
    def forward(ctx, x, branch, post_weight, gate, pre_weight):
        o = tokens.block_norm_forward(x, branch, post_weight, gate, pre_weight)
        ctx.save_for_backward(o["x_out"], branch, post_weight, gate, pre_weight, o["stats"])
        return o["x_out"], o["h"]

    @staticmethod
    def backward(ctx, dx_out, dh):
        x_out, branch, post_weight, gate, pre_weight, stats = ctx.saved_tensors
        o = tokens.block_norm_backward(dx_out.contiguous(), dh.contiguous(), x_out, branch, post_weight, gate, pre_weight,
                                       stats)
        return o["dx"], o["dbranch"], o["dpost_weight"], o["dgate"], o["dpre_weight"]


class Norm(torch.autograd.Function):
    """The norm before the first block."""

    @staticmethod
    def forward(ctx, x, weight):
        o = tokens.block_norm_forward(x, pre_weight=weight)
        ctx.save_for_backward(x, weight, o["stats"])
        return o["h"]

    @staticmethod
    def backward(ctx, dh):
        x, weight, stats = ctx.saved_tensors
        o = tokens.block_norm_backward(None, dh.contiguous(), x, pre_weight=weight, stats=stats)
        return o["dx"], o["dpre_weight"]


class Rotate(torch.autograd.Function):
    """Queries and keys turned by their tokens' places."""

    @staticmethod
    def forward(ctx, q, k, positions, freq, axis):
        ctx.place = positions, freq, axis
        return tokens.rotary_forward(q, k, positions, freq, axis)

    @staticmethod
    def backward(ctx, dq, dk):
        return (*tokens.rotary_backward(dq.contiguous(), dk.contiguous(), *ctx.place), None, None, None)


class Distill(torch.autograd.Function):
    """The mean distillation loss; its gradient comes with it."""

    @staticmethod
    def forward(ctx, logits, top_ids, top_logits, teacher_lse, temperature):
        rows = logits.shape[0]
        weight = torch.full((rows,), 1.0 / rows, device=logits.device)
        o = tokens.distill_forward_backward(logits, top_ids, top_logits, temperature=temperature,
                                            teacher_lse=teacher_lse, row_weight=weight)
        ctx.save_for_backward(o["dlogits"])
        return o["loss"].sum()

    @staticmethod
    def backward(ctx, up):
        (dlogits,) = ctx.saved_tensors
        return dlogits * up.to(dlogits.dtype), None, None, None, None


class Student:
    """Weights (the stem's filter and the matrices in 16 bits, the rest in 32) and the forward pass."""

    def __init__(self, images=16, size=12, c_in=16, dim=64, heads=4, classes=1000, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype=DTYPE):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype).requires_grad_()

        def ones(n, value=1.0):
            return torch.full((n,), value, device="cuda").requires_grad_()

        self.layer = cbr.Layer(images, size, size, c_in, dim, dtype=DTYPE)
        self.ws = [cbr.new_workspace(n) for n in cbr.workspace_size(self.layer)]
        self.running = torch.zeros(dim, device="cuda"), torch.ones(dim, device="cuda")
        self.images, self.size, self.dim, self.heads = images, size, dim, heads
        self.p = {
            "filter": normal(dim, 3, 3, c_in, std=(2.0 / (9 * c_in)) ** 0.5), "gamma": ones(dim), "beta": ones(dim, 0.0),
            "norm0": ones(dim), "qkv": normal(3 * dim, dim, std=dim ** -0.5), "proj": normal(dim, dim, std=dim ** -0.5),
            "post1": ones(dim), "gate1": ones(dim, 0.5), "norm1": ones(dim),
            "up": normal(4 * dim, dim, std=dim ** -0.5), "down": normal(dim, 4 * dim, std=(4 * dim) ** -0.5),
            "post2": ones(dim), "gate2": ones(dim, 0.5), "norm2": ones(dim),
            "head": normal(classes, dim, std=dim ** -0.5),
        }
        # the tokens of an image are its pixels: half of a head's pairs turn with the row, half with the column
        self.positions = tokens.grid_positions(size, size)
        pairs = dim // heads // 2
        self.freq, self.axis = tokens.rotary_table((pairs // 2, pairs - pairs // 2), theta=100.0, spectrum="own")

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        p, n, t, d = self.p, self.images, self.size * self.size, self.dim
        x = Stem.apply(x, p["filter"], p["gamma"], p["beta"], self.layer, self.running, self.ws).view(n * t, d)
        h = Norm.apply(x, p["norm0"])
        qkv = (h @ p["qkv"].t()).view(n, t, 3 * self.heads, d // self.heads)
        q, k, v = qkv.split(self.heads, dim=2)
        q, k = Rotate.apply(q, k, self.positions, self.freq, self.axis)
        scores = torch.einsum("nthd,nshd->nhts", q, k).float() * (d // self.heads) ** -0.5
        mixed = torch.einsum("nhts,nshd->nthd", scores.softmax(-1).to(DTYPE), v).reshape(n * t, d)
        x, h = Join.apply(x, mixed @ p["proj"].t(), p["post1"], p["gate1"], p["norm1"])
        _, h = Join.apply(x, (h @ p["up"].t()).relu() @ p["down"].t(), p["post2"], p["gate2"], p["norm2"])
        return h.view(n, t, d).float().mean(1).to(DTYPE) @ p["head"].t()


def make_batch(student: Student, classes=1000, top=10, temperature=2.0, seed=1):
    """Images and what a teacher left for them: its ten best classes, their logits and the log-sum-exp of
    all its logits / temperature."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer = student.layer
    x = torch.randn(layer.n, layer.h, layer.w, layer.c_in, generator=g, device="cuda").to(DTYPE)
    logits = torch.randn(layer.n, classes, generator=g, device="cuda") * 2
    best = logits.topk(top, dim=1)
    return x, best.indices, best.values, torch.logsumexp(logits / temperature, 1), temperature


def train(steps=30, rate=1.0, quiet=True) -> list[float]:
    """Plain gradient steps on one batch; the losses."""
    student = Student()
    x, ids, top, lse, temperature = make_batch(student)
    losses = []
    for i in range(steps):
        loss = Distill.apply(student(x), ids, top, lse, temperature)
        grads = torch.autograd.grad(loss, list(student.p.values()))
        with torch.no_grad():
            for w, dw in zip(student.p.values(), grads):
                w.sub_(rate * dw.to(w.dtype))
        losses.append(loss.item())
        if not quiet:
            print(f"step {i:3d}  loss {losses[-1]:.4f}")
    cbr.stream_status()
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps, quiet=False)
