"""The token operators together: a routed layer's step from words to gradients
(examples/expert_layer_step.py) against the same layer in fp32, the step's
calls in one HIP graph, another stream, two graphs with one workspace."""
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
    """Against one fp32 evaluation with the same choice of experts and the same
    mask.  bf16 roundings on the way to a gradient: lookup, norm, both products,
    SwiGLU, combine, dropout, and nine on the way back (dropout, weighting, two
    products, SwiGLU, their sum over the choices, the router's share, the norm, the
    residual); each at most 2^-8 of its values and independent of the others, 16 *
    2^-8 = 6.3% of a gradient's norm if they all added up."""
    ex = example()
    T, words, k, E, dim, hidden, p = 200, 90, 2, 5, 64, 96, 0.25
    layer = ex.RoutedLayer(words, k, p, E, dim, hidden)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    batch = torch.randint(0, words - 3, (T,), generator=g, device="cuda")
    dy = torch.randn((T, dim), generator=g, device="cuda").to(torch.bfloat16)
    y, saved = layer.forward(batch, 5)
    ids = saved[6]
    dx, grads = layer.backward(dy, saved)
    keep = mx.mxtrain_dropout_fwd(torch.ones((T, dim), device="cuda"), p, layer.seed, 5) != 0
    assert 0.7 < float(keep.float().mean()) < 0.8  # 12800 elements of probability 3/4: 13 standard deviations
    q = {n: getattr(layer, n).float().requires_grad_() for n in ("table", "router", "w13", "w2", "norm_w", "norm_b")}
    x = q["table"][batch] * layer.scale
    n = torch.nn.functional.layer_norm(x, (dim,), q["norm_w"], q["norm_b"], 1e-5)
    w = torch.softmax((n @ q["router"].T).gather(1, ids), 1)
    c = 0
    for e in range(E):
        gu = n @ q["w13"][e].T
        out = (torch.nn.functional.silu(gu[:, :hidden]) * gu[:, hidden:]) @ q["w2"][e].T
        c = c + (w * (ids == e)).sum(1, keepdim=True) * out
    ref = x + torch.where(keep, c * (1 / (1 - p)), 0.0)
    ref.backward(dy.float())
    off = lambda a, b: float((a.float() - b).norm() / b.norm())  # noqa: E731
    assert off(y, ref.detach()) < 0.063
    for name, grad in grads.items():
        assert off(grad, q[name].grad) < 0.063, name
    assert off(layer.table_grad, q["table"].grad) < 0.063
    assert not layer.table_grad[words - 3:].any()  # words that no token has


def test_the_example_runs():
    losses = example().train_routed(512, 300, 2, 0.1, 4, 128, 256, 3, report=None)
    assert len(losses) == 3 and all(v == v for v in losses)


class Step:
    """Words to gradients by the new operators, around a plain product; every buffer's contents may change between
    calls."""

    def __init__(self, T=700, k=3, E=9, H=136, V=500):
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        self.E, self.V = E, V
        self.table = torch.empty((V, H), dtype=torch.bfloat16, device="cuda")
        self.words = torch.empty(T, dtype=torch.int64, device="cuda")
        self.ids = torch.empty((T, k), dtype=torch.int64, device="cuda")
        self.w = torch.empty((T, k), device="cuda")
        self.dy = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        self.state = torch.zeros(2, dtype=torch.int64, device="cuda")

    def fill(self, seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for t in (self.table, self.w, self.dy):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        self.words.copy_(torch.randint(0, self.V, self.words.shape, generator=g, device="cuda"))
        # a few dropped pairs, which leave rows behind the last
        self.ids.copy_(torch.randint(-1, self.E, self.ids.shape, generator=g, device="cuda"))
        self.state.copy_(torch.tensor([seed, 7 * seed]))

    def run(self, rows=None, drows=None, workspace=None):
        x = mx.mxtrain_embedding_fwd(self.table, self.words, scale=3.0)
        xs, rank, ends, order = mx.mxtrain_sort_dispatch(x, self.ids, self.E, out=rows)
        c = mx.mxtrain_combine_fwd(xs, rank, self.w, residual=x)
        y = mx.mxtrain_dropout_fwd(c, 0.2, 11, 12, residual=x, state=self.state)
        dc = mx.mxtrain_dropout_bwd(self.dy, 0.2, 11, 12, state=self.state)
        dxs, dw = mx.mxtrain_combine_bwd(dc, xs, rank, self.w, out=drows)
        dx = mx.mxtrain_dispatch_bwd(dxs, rank)
        dt = mx.mxtrain_embedding_bwd(dx, self.words, self.V, scale=3.0, workspace=workspace)
        return y, rank, ends, order, dw, dx, dt


def buffers(s):
    n = s.ids.numel()
    return [torch.zeros((n, s.dy.shape[1]), dtype=torch.bfloat16, device="cuda") for _ in range(2)]


@pytest.mark.parametrize("sizes", [dict(), dict(T=40, k=2), dict(T=9000, k=2, V=3000), dict(T=2500, k=4, V=9000),
                                   dict(T=6000, k=2, E=1500), dict(T=33000, k=1, E=2000, V=5000)])
def test_graph_replays_match_eager(sizes):
    """Each form of the sort: with the move in one launch, by comparing, in tiles, by digits with and without counts
    between the workgroups."""
    s = Step(**sizes)
    s.fill(1)
    rows = buffers(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(*rows)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = s.run(*rows)
    masks = []
    for seed in (2, 3, 4):
        s.fill(seed)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = s.run(*buffers(s))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        masks.append(mx.mxtrain_dropout_fwd(torch.ones((50, 50), device="cuda"), 0.2, 11, 12, state=s.state) == 0)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])


def test_two_graphs_share_a_workspace():
    """One after the other on one stream, each call writes its workspace before it reads it."""
    a, b = Step(T=9000, V=3000), Step(T=8500, V=200)
    ws = torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for s in (a, b):
        s.fill(1)
        rows = buffers(s)
        s.run(*rows, ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(s.run(*rows, ws))
    for seed in (5, 6):
        a.fill(seed)
        b.fill(seed + 10)
        ws.fill_(255)
        for g in (graphs[0], graphs[1], graphs[0], graphs[1]):
            g.replay()
        torch.cuda.synchronize()
        for s, out in zip((a, b), outs):
            assert all(torch.equal(p, q) for p, q in zip(out, s.run(*buffers(s))))


@pytest.mark.parametrize("as_handle", [False, True])
def test_handover_to_another_stream(as_handle):
    """Called for a side stream from the current one: what the call reads is ready and what it allocated is not reused
    before the side stream is done."""
    s = Step(T=9000, V=3000)
    s.fill(3)
    want = s.run(*buffers(s))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    on = side.cuda_stream if as_handle else side
    for _ in range(3):
        x = mx.mxtrain_embedding_fwd(s.table, s.words, scale=3.0, stream=on)
        r1, r2 = buffers(s)
        xs, rank, ends, order = mx.mxtrain_sort_dispatch(x, s.ids, s.E, out=r1, stream=on)
        c = mx.mxtrain_combine_fwd(xs, rank, s.w, residual=x, stream=on)
        y = mx.mxtrain_dropout_fwd(c, 0.2, 11, 12, residual=x, state=s.state, stream=on)
        dc = mx.mxtrain_dropout_bwd(s.dy, 0.2, 11, 12, state=s.state, stream=on)
        dxs, dw = mx.mxtrain_combine_bwd(dc, xs, rank, s.w, out=r2, stream=on)
        dx = mx.mxtrain_dispatch_bwd(dxs, rank, stream=on)
        dt = mx.mxtrain_embedding_bwd(dx, s.words, s.V, scale=3.0, stream=on)
        junk = torch.full((1 << 24,), float("nan"), device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip((y, rank, ends, order, dw, dx, dt), want))
        del junk


def test_calls_at_once_on_two_streams():
    """Two steps side by side give what each gives alone."""
    a, b = Step(T=9000, V=3000), Step(T=7000, k=2, E=300, V=20000)
    a.fill(1)
    b.fill(2)
    want = [s.run(*buffers(s)) for s in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i] = s.run(*buffers(s))
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(got[i], want[i]))
