"""A mixture-of-experts layer's training step from the framework's operators.

    y = x + W2_e swiglu(W13_e norm(x)),   rows of x grouped by expert e

Forward and backward pass in bf16 (layer norm, the experts' products, the
SwiGLU of the MXFP8 library) and the update of the experts' weights by
orthogonalised momentum.  Where a run casts to MXFP8, mxfp8_gated_fwd_grouped
and mxfp8_grouped_gemm take the places of swiglu and the products; the norm,
the high-precision products and the update stay as here.

    python examples/expert_layer_step.py [--tokens 4096 --experts 8 --dim 1024 --hidden 2048 --steps 20]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import swiglu_activation_cast_amd as mx  # noqa: E402


class ExpertLayer:
    """Parameters (bf16 weights, fp32 norm and momentum) of one layer."""

    def __init__(self, experts: int, dim: int, hidden: int, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def weight(n, k):
            return (torch.randn((experts, n, k), generator=g, device=device) / math.sqrt(k)).to(torch.bfloat16)

        self.w13 = weight(2 * hidden, dim)  # [gate | up]
        self.w2 = weight(dim, hidden)
        self.norm_w = torch.ones(dim, device=device)
        self.norm_b = torch.zeros(dim, device=device)
        self.momentum = {"w13": torch.zeros(self.w13.shape, device=device),
                         "w2": torch.zeros(self.w2.shape, device=device)}
        self.hidden = hidden

    def forward(self, x: torch.Tensor, ends: torch.Tensor):
        """y, and what the backward pass needs."""
        n, mean, rstd = mx.mxtrain_layer_norm_fwd(x, self.norm_w, self.norm_b)
        gu = mx.mxtrain_grouped_gemm(n, self.w13, ends)
        h = mx.mxfp8_swiglu_fwd_bf16(gu[:, : self.hidden], gu[:, self.hidden:])
        y = x + mx.mxtrain_grouped_gemm(h, self.w2, ends)
        return y, (x, ends, n, mean, rstd, gu, h)

    def backward(self, dy: torch.Tensor, saved):
        """dx and the gradients of the weights (fp32)."""
        x, ends, n, mean, rstd, gu, h = saved
        grads = {"w2": mx.mxtrain_grouped_gemm_k(dy, h, ends)}
        dh = mx.mxtrain_grouped_gemm(dy, self.w2, ends, transpose_b=False)
        dgu = mx.mxfp8_swiglu_bwd_bf16(dh, gu[:, : self.hidden], gu[:, self.hidden:])
        grads["w13"] = mx.mxtrain_grouped_gemm_k(dgu, n, ends)
        dn = mx.mxtrain_grouped_gemm(dgu, self.w13, ends, transpose_b=False)
        dx, grads["norm_w"], grads["norm_b"] = mx.mxtrain_layer_norm_bwd(dn, x, mean, rstd, self.norm_w)
        return dy + dx, grads

    def update(self, grads, lr: float, beta: float = 0.95) -> None:
        """Momentum, orthogonalised for the experts' matrices."""
        for name in ("w13", "w2"):
            m, w = self.momentum[name], getattr(self, name)
            m.mul_(beta).add_(grads[name])
            step = mx.mxtrain_newton_schulz(m)
            scale = lr * math.sqrt(max(1.0, w.shape[1] / w.shape[2]))
            w.copy_(w.float() - scale * step)
        self.norm_w -= lr * grads["norm_w"].sign()
        self.norm_b -= lr * grads["norm_b"].sign()


def train(tokens: int, experts: int, dim: int, hidden: int, steps: int, lr: float = 0.01, seed: int = 0, report=print):
    """Fits the layer to another one's outputs; returns the losses."""
    layer, teacher = ExpertLayer(experts, dim, hidden, seed), ExpertLayer(experts, dim, hidden, seed + 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    losses = []
    for i in range(steps):
        x = torch.randn((tokens, dim), generator=g, device="cuda").to(torch.bfloat16)
        route = torch.randint(0, experts, (tokens,), generator=g, device="cuda")
        ends = torch.bincount(route, minlength=experts).cumsum(0).to(torch.int32)  # rows of x sorted by expert
        target, _ = teacher.forward(x, ends)
        y, saved = layer.forward(x, ends)
        err = y.float() - target.float()
        _, grads = layer.backward((err * (2.0 / err.numel())).to(torch.bfloat16), saved)
        layer.update(grads, lr)
        losses.append(float(err.square().mean()))
        if report and (i % 5 == 0 or i == steps - 1):
            report(f"step {i}: loss {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("experts", 8), ("dim", 1024), ("hidden", 2048), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    train(a.tokens, a.experts, a.dim, a.hidden, a.steps)
