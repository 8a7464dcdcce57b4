"""The token operators past 2^31 pieces of rows, where their numbers need 64 bits
and a launch's grid goes round: narrow rows, moved by element, reach that in a
few gigabytes."""
import numpy as np
import pytest
import torch

import swiglu_activation_cast_amd as mx
from test_gpu_dropout import philox

pytestmark = pytest.mark.gpu
T, H = 310_000_000, 7  # 2.17e9 elements


def ids(V, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)


def test_lookup():
    table = torch.arange(5 * H, device="cuda").view(5, H).to(torch.bfloat16)
    words = ids(5, 1)
    y = mx.mxtrain_embedding_fwd(table, words, scale=2.0)
    for lo in range(0, T, 1 << 26):
        assert torch.equal(y[lo:lo + (1 << 26)], 2 * table[words[lo:lo + (1 << 26)].long()])


def test_moves():
    """k = 1 and ranks that turn the rows round: dispatch, its gradient and combine's."""
    x = torch.arange(T, device="cuda", dtype=torch.int32).remainder(251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    rank = torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.int32)[:, None]
    xs = mx.mxtrain_dispatch_fwd(x, rank)
    for lo in range(0, T, 1 << 26):
        n = min(1 << 26, T - lo)
        assert torch.equal(xs[lo:lo + n], x[T - lo - n:T - lo].flip(0))
    assert torch.equal(mx.mxtrain_dispatch_bwd(xs, rank), x)
    w = torch.full((T, 1), 0.5, device="cuda")
    dys, dw = mx.mxtrain_combine_bwd(x, xs, rank, w, out=xs.clone())
    assert torch.equal(dys, xs * 0.5)
    assert torch.equal(dw[:, 0], H * x[:, 0].float().square())  # whole numbers below 2^24


@pytest.mark.parametrize("tokens", [5, 3000])
def test_zeros_of_a_long_table(tokens):
    words = torch.arange(tokens, device="cuda") * (T // tokens) + 3
    dw = mx.mxtrain_embedding_bwd(torch.ones((tokens, H), device="cuda"), words, T, out=torch.full((T, H), 9.0, device="cuda"))
    assert bool((dw[words] == 1).all())
    dw[words] = 0
    for lo in range(0, T, 1 << 26):
        assert not dw[lo:lo + (1 << 26)].any()


def test_dropout():
    M, N = 1_200_000_000, 9
    x = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    y = mx.mxtrain_dropout_fwd(x, 0.5, 21, 22)
    for r in (0, 7, 536_870_911, 1_073_741_824, M - 1):
        counter = np.zeros((2, 4), dtype=np.int64)
        counter[:, 0], counter[:, 1], counter[:, 2] = (0, 1), r, 22
        w = philox(counter, (21, 0)).astype(np.int64)
        keep = (np.stack([w & 0xFFFF, w >> 16], -1).reshape(16) >= 32768)[:N]
        assert np.array_equal(y[r].float().cpu().numpy(), keep * 2.0), r
