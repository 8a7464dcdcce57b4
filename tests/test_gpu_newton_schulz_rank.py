"""Newton-Schulz updates of low-rank matrices (the gradient of an expert that
got few tokens), on the GPU against the definition in 64 bits.

For a wide G every step X' = P X keeps X's row space (for a tall one X' = X P
keeps the column space), so what a result holds outside G's space is the
arithmetic's own noise, and no rounding of S or P adds to it.  There a step
multiplies it by at most |P|_2 = max |p(s) / s| <= a, the quintic's 3.4445,
which over five steps makes hundreds of times of what X's storage loses early.
Bound (Frobenius norms, first order):

  noise <= out_u |X_5| + sum over steps k of
           a^(5 - k) (u |X_k| [k < 5] + gamma | |P_k| |X_k-1| |) + a^5 u_0 |X_0|

with u = 2^-21 (X between the steps in two fp16 parts: 2^-22, and as much
again for parts below fp16's normal range), gamma = (K / 16 + 16) 2^-23 for the
sums of a product whose K is the short side, taken twice (P times each part of
X) for a bf16 result and three times for an fp32 one, whose dropped product
of two low parts adds 2^-22, u_0 = 0 for bf16 G (exact in one part) and 2^-21
for fp32, and the result's own rounding out_u = 2^-8 for bf16, 2^-24 for fp32.
"""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MUON = (3.4445, -4.7750, 2.0315)


def low_rank(m, n, rank, seed, dtype):
    """A product of whole-number factors, scaled by a power of two: exact in
    either type as long as its entries stay below 2^8."""
    g = torch.Generator()
    g.manual_seed(seed)
    lo = 3 if rank <= 8 else 2
    t = (torch.randint(1 - lo, lo, (m, rank), generator=g).double() @ torch.randint(1 - lo, lo, (rank, n), generator=g).double())
    assert float(t.abs().max()) <= 256 and torch.linalg.matrix_rank(t) == rank
    return (t * 2.0**-10).to(dtype)


def noise_bound(g, dtype, out, steps=5, coeffs=MUON, eps=1e-7):
    """(the exact result, the bound) for one wide matrix."""
    a, b, c = coeffs
    u, out_u = 2.0**-21, 2.0**-8 if out == BF16 else 2.0**-24
    x = g.double()
    x = x / (x.norm() + eps)
    passes, dropped = (2, 0.0) if out == BF16 else (3, 2.0**-22)
    gamma = (passes * x.shape[0] / 16 + 16) * 2.0**-23 + dropped
    noise = 0.0 if dtype == BF16 else u * float(x.norm())
    for k in range(1, steps + 1):
        s = x @ x.T
        p = a * torch.eye(x.shape[0], dtype=x.dtype) + b * s + c * (s @ s)
        y = p @ x
        noise = a * noise + gamma * float((p.abs() @ x.abs()).norm()) + (u if k < steps else out_u) * float(y.norm())
        x = y
    return x, noise


@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F32, BF16), (F32, F32), (BF16, F32)])
@pytest.mark.parametrize("m,n,rank", [(128, 256, 1), (128, 256, 4), (97, 301, 8), (64, 3000, 4), (520, 1031, 4), (512, 1024, 32),
                                      (300, 300, 2)])
def test_no_noise_outside_the_matrix_own_space(m, n, rank, dtype, out):
    g = low_rank(m, n, rank, m + n + rank, dtype)
    want, tol = noise_bound(g, dtype, out)
    v = torch.linalg.svd(g.double(), full_matrices=False)[2][:rank]  # its row space
    # a tall matrix is the same problem transposed
    for h, back in ((g, lambda t: t), (g.T.contiguous(), lambda t: t.T)):
        print(f"case: newton-schulz {tuple(h.shape)} rank {rank} {dtype} -> {out}", flush=True)
        got = back(mx.mxtrain_newton_schulz(h.cuda(), out_dtype=out).cpu().double())
        outside = float((got - (got @ v.T) @ v).norm())
        assert outside <= tol, f"{outside:.3g} outside of the space, bound {tol:.3g}, |result| {float(want.norm()):.3g}"
