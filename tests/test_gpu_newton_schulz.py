"""Orthogonalised updates on the GPU against the definition in 64 bits.

Bound (Frobenius norms, first order).  One step X' = P X, P = a I + b S +
c S^2, S = X X^T (for a tall X the transposed) rounds S, P and X' to a
relative u entry by entry, and each product of depth K loses at most
gamma = (K / 16 + 16) 2^-23 of the magnitudes it adds, |A|_F |B|_F at most.
With s = |X|_2 this adds
  dS = u |S|_F + gamma |X|_F^2,
  dP = (|b| + 2 |c| s^2) dS + u |P|_F + |c| gamma |S|_F^2,
  dX' = s dP + u |X'|_F + gamma |P|_F |X|_F,
and an error that is there already grows by at most the largest |p'| or p(s)/s
over the singular values' range: a perturbation's components in the singular
bases grow by the divided differences of p, which p' and p(s) / s bound.
u is 2^-11 for a bf16 result (fp16 between the products), 2^-21 for fp32 (two
fp16 parts, the dropped low x low product within the same), and the output's
rounding adds 2^-8 or 2^-24 of |X'|_F.  X_0's own rounding: u |X_0|_F.
"""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MUON = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def matrix(batch, m, n, dtype, seed, scale=1.0):
    g = gen(seed)
    return (scale * torch.randn((batch, m, n), generator=g, device="cuda")).to(dtype)


def reference(g, steps, coeffs, eps, u, out_u):
    """(result, bound on the Frobenius error) of one matrix."""
    a, b, c = coeffs
    x = g.double()
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    x = x / (x.norm() + eps)
    err = u * float(x.norm())
    for _ in range(steps):
        s = x @ x.T
        p = a * torch.eye(s.shape[0], device=x.device, dtype=x.dtype) + b * s + c * (s @ s)
        y = p @ x
        sv = torch.linalg.svdvals(x)
        s2 = float(sv.max())
        t = torch.linspace(float(sv.min()), s2, 4097, device=x.device, dtype=x.dtype)
        grow = max(float((a + 3 * b * t**2 + 5 * c * t**4).abs().max()), float((a + b * t**2 + c * t**4).abs().max()))
        gl, gs = ((k / 16 + 16) * 2.0**-23 for k in (x.shape[1], x.shape[0]))
        fx, fs, fp = float(x.norm()), float(s.norm()), float(p.norm())
        ds = u * fs + gl * fx**2
        dp = (abs(b) + 2 * abs(c) * s2**2) * ds + u * fp + abs(c) * gs * fs**2
        err = grow * err + s2 * dp + u * float(y.norm()) + gs * fp * fx
        x = y
    return (x.T if tall else x), err + out_u * float(x.norm())


def check(got, g, steps, coeffs=MUON, eps=1e-7):
    u, out_u = (2.0**-11, 2.0**-8) if got.dtype == BF16 else (2.0**-21, 2.0**-24)
    for i in range(g.shape[0]):
        want, tol = reference(g[i], steps, coeffs, eps, u, out_u)
        off = float((got[i].double() - want).norm())
        assert off <= tol, f"matrix {i}: |error| {off:.3g} over {tol:.3g} (|result| {float(want.norm()):.3g})"


# single rows, columns and elements; sides around the tiles (64, 128, 256) and
# their chunks; odd ones; wide, tall and square
SHAPES = [(1, 1, 1), (2, 1, 9), (2, 9, 1), (3, 7, 5), (1, 63, 65), (2, 64, 64), (5, 100, 37), (1, 129, 300),
          (1, 300, 129), (2, 257, 255), (1, 520, 1031), (1, 1031, 520), (40, 130, 260)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,m,n", SHAPES)
def test_against_definition(batch, m, n, dtype):
    print(f"case: newton-schulz {batch}x{m}x{n} {dtype}", flush=True)
    g = matrix(batch, m, n, dtype, m + n, 0.02)
    for steps in (0, 1, 2, 5):
        check(mx.mxtrain_newton_schulz(g, steps=steps), g, steps)
    check(mx.mxtrain_newton_schulz(g, steps=3, coeffs=CUBIC, eps=0.1), g, 3, CUBIC, 0.1)
    other = F32 if dtype == BF16 else BF16
    out = mx.mxtrain_newton_schulz(g, steps=2, out_dtype=other)
    assert out.dtype == other
    check(out, g, 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("batch,m,n", [(2, 3001, 70), (1, 60, 5003), (1, 200, 1090), (3, 1024, 33), (1, 1, 4099), (20, 40, 1100)])
def test_long_thin_matrices(batch, m, n, dtype):
    """S's products dealt in parts of K, the last of them shorter or empty."""
    g = matrix(batch, m, n, dtype, m + 2 * n)
    for steps in (1, 3):
        out = mx.mxtrain_newton_schulz(g, steps=steps)
        check(out, g, steps)
    assert torch.equal(out, mx.mxtrain_newton_schulz(g, steps=3))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("m,n", [(2304, 4100), (4360, 2200)])
def test_large_tiles(m, n, dtype):
    """Sizes that run 256 x 256 tiles, cut off on every side."""
    g = matrix(1, m, n, dtype, 5)
    check(mx.mxtrain_newton_schulz(g, steps=2), g, 2)


def test_orthogonal():
    """Five steps bring the singular values of a well-conditioned matrix near
    1 (the quintic's fixed band is about 0.7 to 1.2)."""
    g = matrix(2, 96, 400, F32, 9)
    sv = torch.linalg.svdvals(mx.mxtrain_newton_schulz(g).double())
    assert float(sv.min()) > 0.6 and float(sv.max()) < 1.3


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_scale(dtype):
    """The result does not depend on G's scale beyond eps: powers of two give
    the same bits."""
    g = matrix(1, 70, 90, dtype, 10)
    base = mx.mxtrain_newton_schulz(g, eps=0.0)
    for e in (-60, -20, 20, 60):
        assert torch.equal(mx.mxtrain_newton_schulz((g.float() * 2.0**e).to(dtype), eps=0.0), base)


def test_zero_nan_and_infinite_matrices():
    g = matrix(4, 65, 130, F32, 11)
    alone = mx.mxtrain_newton_schulz(g[3:])
    g[0] = 0
    g[1, 3, 4] = float("nan")
    g[2, 64, 129] = float("inf")
    out = mx.mxtrain_newton_schulz(g)
    assert not out[0].any() and torch.isnan(out[1]).all() and torch.isnan(out[2]).all()
    assert torch.equal(out[3:], alone)
    assert not mx.mxtrain_newton_schulz(g[:1].to(BF16)).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_and_untouched_surroundings(dtype):
    g = matrix(3, 50, 77, dtype, 12)
    want = mx.mxtrain_newton_schulz(g)
    base = torch.full((3, 52, 81), 5.0, dtype=dtype, device="cuda")
    gin = torch.full((3, 51, 80), float("nan"), dtype=dtype, device="cuda")
    gin[:, :50, 1:78] = g
    out = base[:, 1:51, 3:80]
    mx.mxtrain_newton_schulz(gin[:, :50, 1:78], out=out)
    assert torch.equal(out, want)
    base[:, 1:51, 3:80] = 5.0
    assert bool((base == 5.0).all())
    # a matrix by itself, and one broadcast over the batch
    assert torch.equal(mx.mxtrain_newton_schulz(g[0]), want[0])
    assert torch.equal(mx.mxtrain_newton_schulz(g[:1].expand(3, 50, 77))[2], want[0])


def test_empty():
    for shape in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        assert mx.mxtrain_newton_schulz(torch.empty(shape, device="cuda")).shape == shape


def test_repeatable_and_on_another_stream():
    g = matrix(2, 300, 500, F32, 13)
    first = mx.mxtrain_newton_schulz(g)
    ws = torch.full((mx.train_lib().mxtrain_newton_schulz_workspace(2, 300, 500, 1),), 255, dtype=torch.uint8,
                    device="cuda")  # NaN everywhere: nothing unwritten is read
    assert torch.equal(mx.mxtrain_newton_schulz(g, workspace=ws), first)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = mx.mxtrain_newton_schulz(g, stream=side)
        junk = torch.full((1 << 22,), float("nan"), device="cuda")
        side.synchronize()
        assert torch.equal(got, first)
        del junk


def test_refusals():
    g = matrix(2, 8, 8, F32, 14)
    with pytest.raises(TypeError):
        mx.mxtrain_newton_schulz(g.half())
    with pytest.raises(TypeError):
        mx.mxtrain_newton_schulz(g, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.mxtrain_newton_schulz(g[0, 0])
    with pytest.raises(ValueError):
        mx.mxtrain_newton_schulz(g.cpu())
    with pytest.raises(ValueError):
        mx.mxtrain_newton_schulz(g, coeffs=(1.0, 2.0))
    with pytest.raises(ValueError):
        mx.mxtrain_newton_schulz(g, out=torch.empty((2, 8, 9), device="cuda"))
    with pytest.raises(ValueError, match="unit column stride"):
        mx.mxtrain_newton_schulz(g.transpose(1, 2))
    with pytest.raises(ValueError, match="workspace"):
        mx.mxtrain_newton_schulz(g, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for bad in (dict(steps=-1), dict(steps=101), dict(eps=float("inf")), dict(coeffs=(1.0, float("nan"), 0.0))):
        with pytest.raises(mx.MxtrainError):
            mx.mxtrain_newton_schulz(g, **bad)


def test_every_element_of_an_fp32_result():
    """No single element is off by much: a high and a low part that do not
    fit each other (one of them rounded twice) would be 2^-12 of it off, the
    rest of the bound is below 2^-16 of the entries' size."""
    g = matrix(2, 256, 512, F32, 15)
    out = mx.mxtrain_newton_schulz(g, steps=2)
    for i in range(2):
        want, _ = reference(g[i], 2, MUON, 1e-7, 0.0, 0.0)
        assert float((out[i].double() - want).abs().max()) < 2.0**-14 * float(want.square().mean().sqrt())
