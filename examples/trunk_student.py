"""Trains a student whose trunk runs on this package's kernels from its norm to the end of its step.

A Conv-BN-ReLU stem turns images into a feature map, which a group norm with SiLU takes over a few channels at a
time; its pixels are the tokens of a block of attention (three query heads to a key head, queries and keys rotated by
their pixel's place) and one of a two-layer network, between norms, with gates; the pooled features' logits learn
from the ten best logits a teacher left for each image; the step's gradients are clipped to a norm, on the device.

    python examples/trunk_student.py [--steps 30]

Between the package's calls are torch's matrix products, and torch.autograd strings the backward calls together.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from conv_batchnorm_relu_gb300 import attention, cbr, gradients, group_norm, tokens  # noqa: E402
from distill_student import DTYPE, Distill, Join, Norm, Rotate, Stem, make_batch  # noqa: E402


class GroupNorm(torch.autograd.Function):
    """silu(group norm(x)) of an NHWC feature map."""

    @staticmethod
    def forward(ctx, x, gamma, beta, groups):
        o = group_norm.group_norm_forward(x, gamma, beta, groups, act="silu")
        ctx.save_for_backward(x, gamma, beta, o["mean"], o["rstd"])
        ctx.groups = groups
        return o["y"]

    @staticmethod
    def backward(ctx, dy):
        x, gamma, beta, mean, rstd = ctx.saved_tensors
        o = group_norm.group_norm_backward(dy.contiguous(), x, gamma, beta, mean, rstd, ctx.groups, act="silu")
        return o["dx"], o["dgamma"], o["dbeta"], None


class Attention(torch.autograd.Function):
    """What each query takes from the values of its image; the probabilities are not kept."""

    @staticmethod
    def forward(ctx, q, k, v):
        o = attention.attention_forward(q, k, v)
        ctx.save_for_backward(q, k, v, o["o"], o["lse"])
        return o["o"]

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse = ctx.saved_tensors
        g = attention.attention_backward(do.contiguous(), q, k, v, o, lse)
        return g["dq"], g["dk"], g["dv"]


class Student:
    """Weights (the stem's filter and the matrices in 16 bits, the rest in 32) and the forward pass."""

    def __init__(self, images=16, size=12, c_in=16, dim=64, heads=6, key_heads=2, head_dim=32, groups=8, classes=1000, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std, dtype=DTYPE):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype).requires_grad_()

        def full(n, value=1.0):
            return torch.full((n,), value, device="cuda").requires_grad_()

        self.layer = cbr.Layer(images, size, size, c_in, dim, dtype=DTYPE)
        self.ws = [cbr.new_workspace(n) for n in cbr.workspace_size(self.layer)]
        self.running = torch.zeros(dim, device="cuda"), torch.ones(dim, device="cuda")
        self.images, self.size, self.dim, self.groups = images, size, dim, groups
        self.heads, self.key_heads, self.head_dim = heads, key_heads, head_dim
        inner = heads * head_dim
        self.p = {
            "filter": normal(dim, 3, 3, c_in, std=(2.0 / (9 * c_in)) ** 0.5), "gamma": full(dim), "beta": full(dim, 0.0),
            "group_gamma": full(dim), "group_beta": full(dim, 0.1), "norm0": full(dim),
            "qkv": normal(inner + 2 * key_heads * head_dim, dim, std=dim ** -0.5), "proj": normal(dim, inner, std=inner ** -0.5),
            "post1": full(dim), "gate1": full(dim, 0.5), "norm1": full(dim),
            "up": normal(4 * dim, dim, std=dim ** -0.5), "down": normal(dim, 4 * dim, std=(4 * dim) ** -0.5),
            "post2": full(dim), "gate2": full(dim, 0.5), "norm2": full(dim),
            "head": normal(classes, dim, std=dim ** -0.5),
        }
        self.positions = tokens.grid_positions(size, size)
        pairs = head_dim // 2
        self.freq, self.axis = tokens.rotary_table((pairs // 2, pairs - pairs // 2), theta=100.0, spectrum="own")

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        p, n, t, d = self.p, self.images, self.size * self.size, self.dim
        x = Stem.apply(x, p["filter"], p["gamma"], p["beta"], self.layer, self.running, self.ws)
        x = GroupNorm.apply(x, p["group_gamma"], p["group_beta"], self.groups).view(n * t, d)
        h = Norm.apply(x, p["norm0"])
        qkv = (h @ p["qkv"].t()).view(n, t, self.heads + 2 * self.key_heads, self.head_dim)
        q, k, v = qkv.split([self.heads, self.key_heads, self.key_heads], dim=2)
        q, k = Rotate.apply(q, k, self.positions, self.freq, self.axis)
        mixed = Attention.apply(q, k, v).reshape(n * t, self.heads * self.head_dim)
        x, h = Join.apply(x, mixed @ p["proj"].t(), p["post1"], p["gate1"], p["norm1"])
        _, h = Join.apply(x, (h @ p["up"].t()).relu() @ p["down"].t(), p["post2"], p["gate2"], p["norm2"])
        return h.view(n, t, d).float().mean(1).to(DTYPE) @ p["head"].t()


def train(steps=30, rate=1.0, max_norm=0.1, quiet=True) -> tuple[list[float], list[float]]:
    """Plain gradient steps on one batch, each clipped; the losses and the gradients' norms."""
    student = Student()
    x, ids, top, lse, temperature = make_batch(student)
    weights, losses, norms = list(student.p.values()), [], []
    for i in range(steps):
        loss = Distill.apply(student(x), ids, top, lse, temperature)
        grads = [g.contiguous() for g in torch.autograd.grad(loss, weights)]
        clipped = gradients.clip_gradients(grads, max_norm)
        with torch.no_grad():
            for w, dw in zip(weights, grads):
                w.sub_(rate * dw.to(w.dtype))
        losses.append(loss.item())
        norms.append(clipped["norm"].item())
        if not quiet:
            print(f"step {i:3d}  loss {losses[-1]:.4f}  gradient norm {norms[-1]:.4f}")
    cbr.stream_status()
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=30)
    train(ap.parse_args().steps, quiet=False)
