"""The training operators together: a mixture-of-experts layer's step
(examples/expert_layer_step.py) against the same layer in fp32, its fit, and
the step's calls in one HIP graph."""
import importlib.util
import os

import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("expert_layer_step", os.path.join(ROOT, "examples", "expert_layer_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_match_the_layer_in_fp32():
    """The layer's activations are bf16: seven roundings (norm, products,
    SwiGLU's two, and theirs on the way back), each at most 2^-8 of its values and
    independent, against one fp32 evaluation: 7 * 2^-8 = 2.7% of a gradient's
    norm if they all added up."""
    ex = example()
    layer = ex.ExpertLayer(3, 64, 96)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((150, 64), generator=g, device="cuda").to(torch.bfloat16)
    dy = torch.randn((150, 64), generator=g, device="cuda").to(torch.bfloat16)
    ends = torch.tensor([61, 61, 150], dtype=torch.int32, device="cuda")
    y, saved = layer.forward(x, ends)
    dx, grads = layer.backward(dy, saved)
    p = {k: getattr(layer, k).float().requires_grad_() for k in ("w13", "w2", "norm_w", "norm_b")}
    xr = x.float().requires_grad_()
    n = torch.nn.functional.layer_norm(xr, (64,), p["norm_w"], p["norm_b"], 1e-5)
    out, lo = [], 0
    for e, hi in enumerate(ends.tolist()):
        gu = n[lo:hi] @ p["w13"][e].T
        out.append((torch.nn.functional.silu(gu[:, :96]) * gu[:, 96:]) @ p["w2"][e].T)
        lo = hi
    ref = xr + torch.cat(out)
    ref.backward(dy.float())
    off = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    assert off(y, ref.detach()) < 0.027 and off(dx, xr.grad) < 0.027
    for k, v in grads.items():
        assert off(v, p[k].grad) < 0.027, k
    assert not grads["w13"][1].any() and not grads["w2"][1].any()  # the expert without tokens


def test_layer_learns():
    losses = example().train(1024, 4, 128, 256, 30, report=None)
    assert losses[-1] < 0.6 * losses[0]


def test_graph_replays_match_eager():
    """No call allocates, synchronizes, copies to the host or records a
    memset: a step's calls capture into one graph."""
    T, G, N, K = 300, 4, 264, 136
    g = torch.Generator(device="cuda")
    x, dy = (torch.empty((T, w), dtype=torch.bfloat16, device="cuda") for w in (K, N))
    w = torch.empty((G, N, K), dtype=torch.bfloat16, device="cuda")
    ends = torch.tensor([10, 10, 200, 300], dtype=torch.int32, device="cuda")
    gamma, beta = torch.randn(K, device="cuda"), torch.randn(K, device="cuda")

    def step():
        n, mean, rstd = mx.mxtrain_layer_norm_fwd(x, gamma, beta)
        y = mx.mxtrain_grouped_gemm(n, w, ends)
        dn = mx.mxtrain_grouped_gemm(dy, w, ends, transpose_b=False)
        dw = mx.mxtrain_grouped_gemm_k(dy, n, ends)
        return (y, dw, mx.mxtrain_newton_schulz(dw), *mx.mxtrain_layer_norm_bwd(dn, x, mean, rstd, gamma))

    def fill(seed):
        g2 = torch.Generator(device="cuda")
        g2.manual_seed(seed)
        for t in (x, dy, w):
            t.copy_(torch.randn(t.shape, generator=g2, device="cuda"))

    fill(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (2, 3, 4):
        fill(seed)
        ends.copy_(torch.tensor([seed * 20, 150, 150 + seed, 300], dtype=torch.int32))
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
