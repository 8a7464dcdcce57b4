"""Layer norm on the GPU against its formulas in 64 bits.

Tolerances.  Every kernel computes in fp32 and rounds once.  With u = 2^-24
the row sums of N terms, taken in at most 32 serial additions a thread and a
tree over the threads, are off by a few tens of u relative to the sum of
magnitudes.  y and dx are O(|w| + |b|) resp. O(rstd |dy| |w|) per element;
64 u times that scale covers their fp32 evaluation (statistics, two
products, one sum), times (1 + |x_hat|) for the statistics' share, to which a
bf16 output adds half a unit in its last of eight places, 2^-8 of the value.  Column sums of M rows:
(M / 8 + 64) u of the sum of magnitudes at most (the serial length per
workgroup and the joins).
"""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def case(M, N, dtype, seed, shift=0.5, std=1.0):
    g = gen(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (std * r(M, N) + shift).to(dtype)
    dy = r(M, N).to(dtype)
    return x, dy, (1 + 0.3 * r(N)), 0.3 * r(N)


def ref_fwd(x, w, b, eps):
    x = x.double()
    mean = x.mean(1)
    var = ((x - mean[:, None]) ** 2).mean(1)
    rstd = (var + eps) ** -0.5
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * (1 if w is None else w.double()) + (0 if b is None else b.double())
    return y, mean, rstd, xh


def ref_bwd(dy, x, mean, rstd, w):
    dy = dy.double()
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    gd = dy if w is None else dy * w.double()
    dx = r * (gd - gd.mean(1, keepdim=True) - xh * (gd * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, gd


def close(got, want, tol):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((d - tol).max()):.3g} over its bound"


def half_unit(dtype, want):
    return want.abs() * 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


# every plan: 16 / 64 threads a row, one to sixteen wavefronts, the long rows;
# odd widths (by element), one column, one row, many rows
SHAPES = [(1, 1), (3, 1), (5, 7), (1, 128), (1030, 100), (1025, 128), (40, 512), (1027, 510), (1024, 1024), (9, 1000),
          (2, 2049), (1031, 2048), (1026, 3001), (7, 5120), (1100, 8192), (3, 16384), (5, 16391), (2, 32768),
          (2, 40001)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward_and_backward(M, N, dtype):
    print(f"case: layer norm {M}x{N} {dtype}", flush=True)
    x, dy, w, b = case(M, N, dtype, 100 * M + N)
    for pd in (torch.float32, torch.bfloat16):
        wp, bp = w.to(pd), b.to(pd)
        y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, wp, bp, eps=1e-5)
        wy, wm, wr, xh = ref_fwd(x, wp, bp, 1e-5)
        xmax = x.double().abs().amax(1)
        close(mean, wm, 64 * U * xmax)
        # the deviations' absolute error u |x| against their size 1 / rstd
        cond = 1 + wr * xmax
        close(rstd, wr, 64 * U * wr * cond)
        scale = wp.double().abs() * (1 + xh.abs()) * cond[:, None] + bp.double().abs()
        close(y, wy, 64 * U * scale + half_unit(dtype, wy))
        dx, dw, db = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, wp)
        rx, rw, rb, xh, gd = ref_bwd(dy, x, mean, rstd, wp)
        mag = gd.abs().mean(1, keepdim=True) + xh.abs() * (gd * xh).abs().mean(1, keepdim=True) + gd.abs()
        r = rstd.double()[:, None]
        close(dx, rx, 64 * U * r * mag * cond[:, None] + half_unit(dtype, rx))
        steps = (M / 8 + 64) * U
        close(dw, rw, steps * (dy.double() * xh).abs().sum(0) + 4 * U * (dy.double().abs() * cond[:, None]).sum(0))
        close(db, rb, steps * dy.double().abs().sum(0))
        assert dw.dtype == db.dtype == torch.float32


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_parameters_and_wanted_outputs_only(dtype):
    x, dy, w, b = case(33, 640, dtype, 1)
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x)
    one, zero = torch.ones_like(w), torch.zeros_like(b)
    assert torch.equal(y, mx.mxtrain_layer_norm_fwd(x, one, zero)[0])
    assert torch.equal(mx.mxtrain_layer_norm_fwd(x, None, b)[0], mx.mxtrain_layer_norm_fwd(x, one, b)[0])
    a = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd)
    c = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, one)
    assert all(torch.equal(p, q) for p, q in zip(a, c))
    # through the C entry: no statistics, no weight gradients
    lib = mx.train_lib()
    t = 0 if dtype == torch.bfloat16 else 1
    y2, dx2 = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.current_stream().cuda_stream
    assert lib.mxtrain_layer_norm_fwd(x.data_ptr(), 640, None, None, 0, 33, 640, t, 1e-5, y2.data_ptr(), 640, None,
                                      None, s) == 0
    assert lib.mxtrain_layer_norm_bwd(dy.data_ptr(), 640, x.data_ptr(), 640, mean.data_ptr(), rstd.data_ptr(), None, 0,
                                      33, 640, t, dx2.data_ptr(), 640, None, None, None, 0, s) == 0
    assert torch.equal(y2, y) and torch.equal(dx2, a[0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 0), (3, 1)])
def test_strides_and_alignment(dtype, pad, offset):
    """Padded rows and bases off 16 bytes give the contiguous result, and
    nothing outside the result is written."""
    M, N = 37, 1000
    x, dy, w, b = case(M, N, dtype, 3)
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, w, b)
    dx, dw, db = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w)

    def strided(t, fill=7.0):
        base = torch.full((M * (N + pad) + offset,), fill, dtype=dtype, device="cuda")
        v = base[offset:].view(M, N + pad)[:, :N]
        if t is not None:
            v.copy_(t)
        return base, v

    _, xs = strided(x)
    _, dys = strided(dy)
    yb, ys = strided(None)
    dxb, dxs = strided(None)
    _, m2, r2 = mx.mxtrain_layer_norm_fwd(xs, w, b, out=ys)
    g2 = mx.mxtrain_layer_norm_bwd(dys, xs, mean, rstd, w, out=dxs)
    # sums in another order where rows go by element: fp32 close, not equal;
    # two bf16 roundings of nearly equal values differ by up to a whole unit,
    # 2^-7 of the value
    torch.testing.assert_close(m2, mean, rtol=0, atol=1e-6)
    torch.testing.assert_close(r2, rstd, rtol=1e-5, atol=0)
    tol = dict(rtol=2.0 ** -7, atol=1e-5) if dtype == torch.bfloat16 else dict(rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(ys, y, **tol)
    torch.testing.assert_close(dxs, dx, **tol)
    torch.testing.assert_close(g2[1], dw, rtol=1e-5, atol=1e-4)
    torch.testing.assert_close(g2[2], db, rtol=1e-5, atol=1e-4)
    for base in (yb, dxb):
        outside = torch.ones_like(base, dtype=torch.bool)
        outside[offset:].view(M, N + pad)[:, :N] = False
        assert bool((base[outside] == 7.0).all())


def test_rows_of_equal_values_and_nonfinite_rows():
    x = torch.randn(6, 768, device="cuda")
    x[1] = 3.25          # no deviation: y is the bias
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    x[4] = 1e4 + 0.01 * torch.randn(768, device="cuda")  # far off centre
    w, b = torch.randn(768, device="cuda"), torch.randn(768, device="cuda")
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, w, b)
    assert torch.equal(y[1], b)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    wy, *_ = ref_fwd(x[[0, 4, 5]], w, b, 1e-5)
    assert torch.isfinite(y[[0, 1, 4, 5]]).all()
    close(y[[0, 5]], wy[[0, 2]], 1e-4)
    # the row's values themselves are 2^-24 * 1e4 = 6e-4 of 0.01 apart
    assert float((y[4].double() - wy[1]).abs().max()) < 0.1


def test_empty():
    x = torch.empty((0, 64), device="cuda")
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, torch.ones(64, device="cuda"))
    assert y.shape == (0, 64) and mean.shape == rstd.shape == (0,)
    dw = torch.full((64,), 5.0, device="cuda")
    dx, dw, db = mx.mxtrain_layer_norm_bwd(x, x, mean, rstd, torch.ones(64, device="cuda"), dweight=dw)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_gradient_against_differences():
    """d(sum y dy) along random directions, by central differences of the
    64-bit formula: step 1e-4, error O(step^2) and fp32 in the gradient."""
    x, dy, w, b = case(5, 300, torch.float32, 11)
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, w, b)
    dx, dw, db = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w)
    g = gen(12)
    for t, grad in ((0, dx), (1, dw), (2, db)):
        d = torch.randn(grad.shape, generator=g, device="cuda").double()
        h = 1e-4

        def loss(sign):
            a = [x.double(), w.double(), b.double()]
            a[t] = a[t] + sign * h * d
            return (ref_fwd(a[0], a[1], a[2], 1e-5)[0] * dy.double()).sum()

        num = (loss(1) - loss(-1)) / (2 * h)
        ana = (grad.double() * d).sum()
        assert abs(float(num - ana)) < 1e-4 * float((grad.double() * d).abs().sum()) + 1e-6


def test_repeatable_and_on_another_stream():
    x, dy, w, b = case(2000, 768, torch.bfloat16, 21)
    y, mean, rstd = mx.mxtrain_layer_norm_fwd(x, w, b)
    first = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        got = mx.mxtrain_layer_norm_bwd(dy, x, mean, rstd, w, stream=side)
        junk = torch.full((1 << 20,), float("nan"), device="cuda")  # would land in a workspace reused too early
        side.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, first))
        del junk


def test_refusals():
    x, dy, w, b = case(4, 64, torch.float32, 31)
    m = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        mx.mxtrain_layer_norm_fwd(x.half())
    with pytest.raises(ValueError):
        mx.mxtrain_layer_norm_fwd(x.cpu())
    with pytest.raises(ValueError):
        mx.mxtrain_layer_norm_fwd(x[0])
    with pytest.raises(ValueError, match="unit column stride"):
        mx.mxtrain_layer_norm_fwd(x.t())
    with pytest.raises(ValueError):
        mx.mxtrain_layer_norm_fwd(x, w[:32])
    with pytest.raises(TypeError):
        mx.mxtrain_layer_norm_fwd(x, w, b.bfloat16())
    with pytest.raises(TypeError):
        mx.mxtrain_layer_norm_bwd(dy.bfloat16(), x, m, m)
    with pytest.raises(ValueError):
        mx.mxtrain_layer_norm_bwd(dy[:2], x, m, m)
    with pytest.raises(ValueError, match="workspace"):
        big, stats = torch.zeros((2000, 64), device="cuda"), torch.zeros(2000, device="cuda")
        mx.mxtrain_layer_norm_bwd(big, big, stats, stats, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mx.MxtrainError):
        mx.mxtrain_layer_norm_fwd(x, eps=float("nan"))
