"""Newton-Schulz steps that run 256 x 256 tiles everywhere, and the longest
sides, pinned to the bit.

G is 0 and +-1 with 4^e entries that are not 0, so |G| = 2^e and X_0 are exact.
With (a, b, c) = (2^-4e, 2^-2e, 1) one step's p(S) holds whole numbers (I + S +
S^2 of G's own products) times 2^-4e, at most 2048 of them: S, p(S) and every sum
are exact in any of the formats (whole multiples of fp16's smallest number, of at
most 11 places), and the result is the exact one rounded once.  A wrong element
of S, p(S), a mirrored tile, a cut-off tile or a part of a cut-down round shows
as itself.
"""
import math

import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
CUS = 256


def sparse(batch, m, n, e, seed, near_end=0):
    """4^e entries of +-1 in each matrix, `near_end` of them in the last 4096 columns of rows as long as that."""
    g = torch.Generator()
    g.manual_seed(seed)
    out = torch.zeros((batch, m, n), device="cuda")
    for i in range(batch):
        at = torch.randperm(m * n, generator=g)[: 4**e]
        if near_end:
            last = torch.randperm(m * 4096, generator=g)
            last = (last // 4096) * n + (n - 4096) + last % 4096
            at = torch.cat([last[:near_end], at[at % n < n - 4096][: 4**e - near_end]])
        assert at.numel() == 4**e
        out[i].view(-1)[at.cuda()] = (2.0 * torch.randint(0, 2, (4**e,), generator=g) - 1.0).cuda()
    return out


def exact_step(g, e):
    """One step in whole numbers, in 64 bits; g wide."""
    x = g.double()
    s = x @ x.T.contiguous()
    p = torch.eye(x.shape[0], device=x.device, dtype=x.dtype) + s + s @ s
    assert float(p.abs().max()) <= 2048
    return (p @ x) * 2.0 ** (-5 * e)


def check_one_step(wide, e, tall, dtype):
    """`wide` [B, m, n], or each of its matrices transposed."""
    g = wide.transpose(1, 2).contiguous() if tall else wide
    out = mx.mxtrain_newton_schulz(g.to(dtype), steps=1, coeffs=(2.0 ** (-4 * e), 2.0 ** (-2 * e), 1.0), eps=0.0)
    for i in range(wide.shape[0]):
        want = exact_step(wide[i], e)
        assert torch.equal(out[i], (want.T if tall else want).to(dtype))


# the whole products' last round: quarters (up to 64 tiles), halves (up to 128), whole
CASES = [(1, 4000, 4104, 8, "quarters"), (1, 4500, 5000, 8, "halves"), (4, 2304, 2340, 7, "halves"),
         (1, 4100, 6044, 8, "whole")]


@pytest.mark.parametrize("batch,m,n,e,last", CASES)
def test_one_step_is_exact(batch, m, n, e, last):
    lower, all_ = batch * ((m + 255) // 256) * ((m + 255) // 256 + 1) // 2, batch * ((m + 255) // 256) * ((n + 255) // 256)
    tail = all_ % CUS
    assert CUS // 2 < lower <= CUS < all_  # the symmetric products in one round, the others in more
    assert last == ("quarters" if tail <= CUS // 4 else "halves" if tail <= CUS // 2 else "whole")
    g = sparse(batch, m, n, e, m + n)
    for dtype in (BF16, F32):
        for tall in (False, True):
            print(f"case: newton-schulz {batch}x{m}x{n} {dtype} tall {tall}", flush=True)
            check_one_step(g, e, tall, dtype)


@pytest.mark.parametrize("batch,m,n,e,last", CASES)
def test_steps_between_keep_every_element(batch, m, n, e, last):
    """With (1, 0, 0) every step's p(S) is I and X goes through unchanged."""
    e = int(math.log(m * n, 4))
    g = sparse(batch, m, n, e, m * n)
    for h in (g, g.transpose(1, 2).contiguous()):
        for dtype in (BF16, F32):
            print(f"case: newton-schulz {tuple(h.shape)} {dtype}, identity", flush=True)
            out = mx.mxtrain_newton_schulz(h.to(dtype), steps=3, coeffs=(1.0, 0.0, 0.0), eps=0.0)
            assert torch.equal(out, (h * 2.0**-e).to(dtype))


@pytest.mark.parametrize("batch,m,n,e,last", CASES)
def test_both_parts_of_x_reach_a_bf16_result(batch, m, n, e, last):
    """Entries 2^-13 to either side of a bf16 tie (1 + 2^-8): X's high part,
    fp16, is the tie itself, and the low part decides the rounding.  eps makes
    |G| + eps a power of two (to fp32's last place, which the scale's rounding to
    fp32 takes away)."""
    e = int(math.log(m * n, 4))
    near = torch.Generator(device="cuda")
    near.manual_seed(3)
    g = sparse(batch, m, n, e, m * n)
    g *= 1 + 2.0**-8 + 2.0**-13 * (2.0 * torch.randint(0, 2, g.shape, generator=near, device="cuda") - 1)
    for i in range(batch):
        for h in (g[i], g[i].T.contiguous()):
            eps = 2.0 ** (e + 1) - float(h.double().norm())
            assert eps > 0
            out = mx.mxtrain_newton_schulz(h, steps=3, coeffs=(1.0, 0.0, 0.0), eps=eps, out_dtype=BF16)
            assert torch.equal(out, (h.to(BF16).double() * 2.0 ** -(e + 1)).to(BF16))


def test_longest_sides():
    """Rows of 2^22 - 1 elements, which start off 16 bytes, and as many rows."""
    g = sparse(1, 40, 2**22 - 1, 5, 17, near_end=512)
    for dtype in (BF16, F32):
        for tall in (False, True):
            print(f"case: newton-schulz 40x{2**22 - 1} {dtype} tall {tall}", flush=True)
            check_one_step(g, 5, tall, dtype)


@pytest.mark.parametrize("batch,m,n,e", [(1, 250, 2621, 5), (2, 100, 2560, 5), (1, 60, 5003, 4), (1, 5, 40001, 3), (5, 64, 2564, 4)])
def test_long_thin_matrices_in_parts(batch, m, n, e):
    """At most 16 tiles of S and 40 stages of 64 or more along K: S's products
    dealt in parts, the last of them shorter or empty."""
    t = (m + 63) // 64
    assert batch * t * (t + 1) // 2 <= 16 and (n + 63) // 64 >= 40
    g = sparse(batch, m, n, e, m + n)
    for dtype in (BF16, F32):
        for tall in (False, True):
            check_one_step(g, e, tall, dtype)
