"""Layer norm's backward with more columns than a launch of the column sums'
join has workgroups for.

x, dy are -1, 0 or 1, the weight 1 or 2, mean and rstd 0 and 1 or 1 and 2:
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
