"""A mixture-of-experts layer's training step from the framework's operators.

    y = x + W2_e swiglu(W13_e norm(x)),   rows of x grouped by expert e

Forward and backward pass in bf16 (layer norm, the experts' products, the
SwiGLU of the MXFP8 library) and the update of the experts' weights by
orthogonalised momentum.  Where a run casts to MXFP8, mxfp8_gated_fwd_grouped
and mxfp8_grouped_gemm take the places of swiglu and the products; the norm,
the high-precision products and the update stay as here.

    python examples/expert_layer_step.py [--tokens 4096 --experts 8 --dim 1024 --hidden 2048 --steps 20]

With --top-k, the layer gets words instead of sorted rows: an embedding, a
router that sends each token to k experts, and dropout before the residual,

    y = x + drop(sum_j w_j W2_ej swiglu(W13_ej norm(x))),   x = scale table[word]

with the tokens sorted by expert, moved there and back, and the gradients of
all of it, the embedding's added to a running one.

    python examples/expert_layer_step.py --top-k 2 [--words 32768 --dropout 0.1 ...]
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


class RoutedLayer(ExpertLayer):
    """An ExpertLayer behind an embedding and a router, with dropout in front of the residual."""

    def __init__(self, words: int, top_k: int, dropout: float, experts: int, dim: int, hidden: int, seed: int = 0,
                 device="cuda"):
        super().__init__(experts, dim, hidden, seed, device)
        g = torch.Generator(device=device)
        g.manual_seed(seed + 1000)
        self.table = (torch.randn((words, dim), generator=g, device=device) / math.sqrt(dim)).to(torch.bfloat16)
        self.table_grad = torch.zeros((words, dim), device=device)
        self.router = torch.randn((experts, dim), generator=g, device=device) / math.sqrt(dim)
        self.scale, self.top_k, self.p, self.seed = math.sqrt(dim), top_k, dropout, seed

    def forward(self, words: torch.Tensor, step: int):
        """y [T, dim] for words [T], and what the backward pass needs; `step` numbers the dropout's mask."""
        x = mx.mxtrain_embedding_fwd(self.table, words, scale=self.scale)
        n, mean, rstd = mx.mxtrain_layer_norm_fwd(x, self.norm_w, self.norm_b)
        top = torch.topk(n.float() @ self.router.T, self.top_k, dim=1)
        weights = torch.softmax(top.values, 1)
        ns, rank, ends, _ = mx.mxtrain_sort_dispatch(n, top.indices, self.router.shape[0])
        gu = mx.mxtrain_grouped_gemm(ns, self.w13, ends)
        h = mx.mxfp8_swiglu_fwd_bf16(gu[:, : self.hidden], gu[:, self.hidden:])
        ys = mx.mxtrain_grouped_gemm(h, self.w2, ends)
        c = mx.mxtrain_combine_fwd(ys, rank, weights)
        y = mx.mxtrain_dropout_fwd(c, self.p, self.seed, step, residual=x)
        return y, (words, step, x, n, mean, rstd, top.indices, weights, ns, rank, ends, gu, h, ys)

    def backward(self, dy: torch.Tensor, saved):
        """dx and the gradients (fp32); the table's is added to table_grad."""
        words, step, x, n, mean, rstd, ids, weights, ns, rank, ends, gu, h, ys = saved
        dc = mx.mxtrain_dropout_bwd(dy, self.p, self.seed, step)
        dys, dweights = mx.mxtrain_combine_bwd(dc, ys, rank, weights)
        grads = {"w2": mx.mxtrain_grouped_gemm_k(dys, h, ends)}
        dh = mx.mxtrain_grouped_gemm(dys, self.w2, ends, transpose_b=False)
        dgu = mx.mxfp8_swiglu_bwd_bf16(dh, gu[:, : self.hidden], gu[:, self.hidden:])
        grads["w13"] = mx.mxtrain_grouped_gemm_k(dgu, ns, ends)
        dn = mx.mxtrain_dispatch_bwd(mx.mxtrain_grouped_gemm(dgu, self.w13, ends, transpose_b=False), rank)
        # the weights are a softmax over the chosen experts' scores
        dscores = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        dlogits = torch.zeros((dy.shape[0], self.router.shape[0]), device=dy.device).scatter_(1, ids, dscores)
        grads["router"] = dlogits.T @ n.float()
        dn = (dn.float() + dlogits @ self.router).to(dn.dtype)
        dx, grads["norm_w"], grads["norm_b"] = mx.mxtrain_layer_norm_bwd(dn, x, mean, rstd, self.norm_w)
        dx = dy + dx
        mx.mxtrain_embedding_bwd(dx, words, self.table.shape[0], scale=self.scale, out=self.table_grad, accumulate=True)
        return dx, grads

    def update(self, grads, lr: float, beta: float = 0.95) -> None:
        super().update(grads, lr, beta)
        self.router -= lr * grads["router"].sign()
        self.table.copy_(self.table.float() - lr * self.table_grad.sign() / math.sqrt(self.table.shape[1]))
        self.table_grad.zero_()


def train_routed(tokens: int, words: int, top_k: int, dropout: float, experts: int, dim: int, hidden: int, steps: int,
                 lr: float = 0.01, seed: int = 0, report=print):
    """Fits a routed layer to another one's outputs; returns the losses."""
    layer = RoutedLayer(words, top_k, dropout, experts, dim, hidden, seed)
    teacher = RoutedLayer(words, top_k, 0.0, experts, dim, hidden, seed + 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 2)
    losses = []
    for i in range(steps):
        batch = torch.randint(0, words, (tokens,), generator=g, device="cuda")
        target, _ = teacher.forward(batch, i)
        y, saved = layer.forward(batch, i)
        err = y.float() - target.float()
        _, grads = layer.backward((err * (2.0 / err.numel())).to(torch.bfloat16), saved)
        layer.update(grads, lr)
        losses.append(float(err.square().mean()))
        if report and (i % 5 == 0 or i == steps - 1):
            report(f"step {i}: loss {losses[-1]:.4f}")
    return losses


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
    ap.add_argument("--top-k", type=int, default=0, help="experts of a token; 0: sorted rows instead of words")
    ap.add_argument("--words", type=int, default=32768)
    ap.add_argument("--dropout", type=float, default=0.1)
    a = ap.parse_args()
    if a.top_k:
        train_routed(a.tokens, a.words, a.top_k, a.dropout, a.experts, a.dim, a.hidden, a.steps)
    else:
        train(a.tokens, a.experts, a.dim, a.hidden, a.steps)
