"""Layer norm at the ends of its range: more long rows than a launch has
workgroups for, and the backward with more columns than a launch of the column
sums' join has.

Backward: x, dy are -1, 0 or 1, the weight 1 or 2, mean and rstd 0 and 1 or 1 and 2:
every sum (of at most 2^25 terms of random sign, far below 2^24) is exact in
fp32 whatever its order, so dweight and dbias have to be equal.  dx's two means
lose three units of 2^-24 each (1 / N, the product, and the row's fma), its own
three operations as many: 8 units of the magnitudes cover them."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def test_backward_of_more_columns_than_the_join_has_workgroups():
    M, N = 5, (1 << 25) + 64
    print(f"case: layer norm backward {M}x{N}", flush=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, dy = (torch.randint(-1, 2, (M, N), generator=g, device="cuda").float() for _ in range(2))
    w = torch.randint(1, 3, (N,), generator=g, device="cuda").float()
    mean, rstd = torch.tensor([0.0, 1.0, 0.0, 1.0, 1.0], device="cuda"), torch.tensor([1.0, 2.0, 2.0, 1.0, 2.0], device="cuda")
    dx, dw, db = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    rw, rb = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    for i in range(M):
        xh, r = (x[i].double() - float(mean[i])) * float(rstd[i]), float(rstd[i])
        gd = dy[i].double() * w.double()
        c1, c2 = float(gd.mean()), float((gd * xh).mean())
        want = r * (gd - c1 - xh * c2)
        tol = 8 * U * r * (gd.abs() + abs(c1) + (xh * c2).abs())
        assert bool(((dx[i].double() - want).abs() <= tol).all())
        rw += (dy[i].double() * xh).float()
        rb += dy[i]
    assert torch.equal(dw, rw) and torch.equal(db, rb)


def test_forward_of_more_long_rows_than_a_launch_has_workgroups():
    """Rows of zeros (y is the bias, rstd 1 / sqrt(eps) to three fp32
    roundings) up to the last three, which are -1, 0 or 1: their sum is exact,
    their statistics and y are off by a few units of fp32 (64 cover the 17
    additions a thread makes and the joins) beside bf16's half unit, 2^-8."""
    M, N = (1 << 31) // 1024 + 9, 16385
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 140 GB")
    print(f"case: layer norm forward {M}x{N}", flush=True)
    x = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x[-3:] = torch.randint(-1, 2, (3, N), generator=g, device="cuda").to(torch.bfloat16)
    w, b = torch.randn(N, generator=g, device="cuda"), torch.randn(N, generator=g, device="cuda")
    mean, rstd = (torch.full((M,), float("nan"), device="cuda") for _ in range(2))
    y, _, _ = mx.mxtrain_layer_norm_fwd(x, w, b, eps=1.0, mean=mean, rstd=rstd)
    torch.cuda.synchronize()
    assert not mean[:-3].any() and bool(((rstd[:-3] - 1).abs() <= 3 * U).all())
    for row in (0, (1 << 21) - 2, (1 << 21) - 1, M - 4):
        assert torch.equal(y[row], b.to(torch.bfloat16))
    xd = x[-3:].double()
    m = xd.mean(1)
    r = (((xd - m[:, None]) ** 2).mean(1) + 1.0) ** -0.5
    xh = (xd - m[:, None]) * r[:, None]
    want = xh * w.double() + b.double()
    assert bool(((mean[-3:].double() - m).abs() <= 64 * U).all()) and bool(((rstd[-3:].double() - r).abs() <= 64 * U).all())
    tol = 2.0**-8 * want.abs() + 64 * U * ((1 + xh.abs()) * w.double().abs() + b.double().abs())
    assert bool(((y[-3:].double() - want).abs() <= tol).all())
    del x, y
    torch.cuda.empty_cache()
