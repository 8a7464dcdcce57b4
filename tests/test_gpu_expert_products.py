"""The experts' bf16 products over ragged groups, against 64-bit products.

Two kinds of input.  Small whole numbers (|v| <= 8, |sum| < 2^24): every
product and every partial sum is exact in fp32 whatever the order, so an fp32
result has to be equal, and a bf16 result equal to its rounding.  That pins
every index, mask and tail.  Normal values: products of bf16 are exact in
fp32; adding K of them, 16 to a step, loses at most one fp32 unit (2^-23,
whether rounded or cut) of the magnitudes summed so far at each of the K / 16
steps and as much for each of the 16 terms within a step, so
(K / 16 + 16) 2^-23 sum |a b| bounds an fp32 result; a bf16 result adds half
a unit, 2^-8 of the value.
"""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def whole(shape, g):
    return torch.randint(-4, 5, shape, generator=g, device="cuda").to(BF16)


def bounds(ends, M):
    out, last = [], 0
    for e in ends:
        e = min(max(e, last, 0), M)
        out.append((last, e))
        last = e
    return out


def padded(t, pad, fill):
    """t with `pad` more elements per row that hold `fill`."""
    if not pad:
        return t
    big = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=t.device)
    big[..., : t.shape[-1]] = t
    return big[..., : t.shape[-1]]


def ref_m(a, b, ends, transpose_b):
    parts = []
    for g, (lo, hi) in enumerate(bounds(ends, a.shape[0])):
        w = b[g].double()
        parts.append(a[lo:hi].double() @ (w.T if transpose_b else w))
    return torch.cat(parts)


def ref_k(a, b, ends):
    return torch.stack([a[lo:hi].double().T @ b[lo:hi].double() for lo, hi in bounds(ends, a.shape[0])])


# tokens, ends, N, K: one token; tiles cut off everywhere; empty groups first,
# inside and last; unordered, negative and too large ends; rows past the last
# end; more groups than a wavefront; more rows than a tile; K below, at and
# across stages
CASES = [
    (1, [1], 8, 8), (1, [0, 1, 1], 1, 1), (5, [2, 5], 33, 70), (7, [0, 0, 7, 7], 130, 64), (300, [1, 300], 264, 65),
    (70, [40, 30, -5, 64, 900], 100, 200), (64, [10, 50], 72, 63), (513, [257, 258, 513], 257, 129),
    (200, list(range(2, 202, 2)), 48, 40), (130, [129] * 70 + [130], 40, 192), (1100, [1000, 1100], 1030, 256),
    (2000, [500, 700, 2000], 2304, 328), (17, [17], 4104, 1000), (0, [0, 0], 16, 16), (40, [0, 0], 24, 32),
]


@pytest.mark.parametrize("transpose_b", [True, False])
@pytest.mark.parametrize("T,ends,N,K", CASES)
def test_grouped_whole_numbers_are_exact(T, ends, N, K, transpose_b):
    print(f"case: grouped {T}x{N}x{K} ends {ends[:8]} transpose_b {transpose_b}", flush=True)
    g = gen(T + N + K)
    G = len(ends)
    # NaN between the rows: what is read past a row's end is not used
    a = padded(whole((T, K), g), -K % 8 + 8, float("nan"))
    b = padded(whole((G, N, K) if transpose_b else (G, K, N), g), (-K if transpose_b else -N) % 8 + 8, float("nan"))
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = ref_m(a, b, ends, transpose_b)
    for dtype in (F32, BF16):
        for pad in (0, 3):
            base = torch.full((T, N + pad), 77.0, dtype=dtype, device="cuda")
            out = base[:, :N]
            got = mx.mxtrain_grouped_gemm(a, b, e, transpose_b=transpose_b, out=out)
            assert got is out
            n = want.shape[0]
            assert torch.equal(out[:n], want.to(dtype))
            assert bool((out[n:] == 77.0).all()) and bool((base[:, N:] == 77.0).all())


@pytest.mark.parametrize("T,ends,N,K", CASES)
def test_grouped_k_whole_numbers_are_exact(T, ends, N, K):
    print(f"case: grouped over tokens {T}x{N}x{K} ends {ends[:8]}", flush=True)
    g = gen(T * 3 + N + K)
    a = padded(whole((T, N), g), -N % 8 + 8, float("nan"))
    b = padded(whole((T, K), g), -K % 8 + 8, float("nan"))
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    want = ref_k(a, b, ends)
    for dtype in (F32, BF16):
        got = mx.mxtrain_grouped_gemm_k(a, b, e, out_dtype=dtype)
        assert got.dtype == dtype and torch.equal(got, want.to(dtype))
        base = torch.full((len(ends), N + 1, K + 5), 77.0, dtype=dtype, device="cuda")
        mx.mxtrain_grouped_gemm_k(a, b, e, out=base[:, :N, :K])
        assert torch.equal(base[:, :N, :K], want.to(dtype))
        assert bool((base[:, N:] == 77.0).all()) and bool((base[:, :, K:] == 77.0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,ends,N,K", [(600, [13, 13, 400, 600], 520, 1096), (2100, [2000, 2100], 1536, 2048),
                                        (9, [3, 9], 2048, 5120)])
def test_normal_values(T, ends, N, K, dtype):
    g = gen(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)  # noqa: E731
    x, w, dy = r(T, K), r(len(ends), N, K), r(T, N)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")

    def check(got, want, mag, depth):
        tol = (depth / 16 + 16) * 2.0 ** -23 * mag + (want.abs() * 2.0 ** -8 if dtype == BF16 else 0)
        assert bool(((got.double() - want).abs() <= tol).all())

    check(mx.mxtrain_grouped_gemm(x, w, e, out_dtype=dtype), ref_m(x, w, ends, True),
          ref_m(x.abs(), w.abs(), ends, True), K)
    check(mx.mxtrain_grouped_gemm(dy, w, e, transpose_b=False, out_dtype=dtype), ref_m(dy, w, ends, False),
          ref_m(dy.abs(), w.abs(), ends, False), N)
    check(mx.mxtrain_grouped_gemm_k(dy, x, e, out_dtype=dtype), ref_k(dy, x, ends), ref_k(dy.abs(), x.abs(), ends), T)


def test_nonfinite_values_stay_in_their_group():
    """NaN and infinities of one group's tokens or weights reach that group's
    results only, and an infinity meets no zero that is not there."""
    g = gen(6)
    T, ends, N, K = 90, [37, 90], 72, 104
    x, w, dy = whole((T, K), g).abs() + 1, whole((2, N, K), g).abs() + 1, whole((T, N), g).abs() + 1
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    clean = mx.mxtrain_grouped_gemm_k(dy, x, e)
    x2 = x.clone()
    x2[37:] = float("nan")
    assert torch.equal(mx.mxtrain_grouped_gemm_k(dy, x2, e)[0], clean[0])
    x2 = x.clone()
    x2[36, 5] = float("inf")   # the last token of group 0: re-read past the group's end, never used
    got = mx.mxtrain_grouped_gemm_k(dy, x2, e)
    assert bool((got[0][:, 5] == float("inf")).all()) and torch.equal(got[1], clean[1])
    w2 = w.clone()
    w2[1] = float("inf")
    y = mx.mxtrain_grouped_gemm(x, w2, e)
    assert torch.equal(y[:37], mx.mxtrain_grouped_gemm(x, w, e)[:37]) and bool((y[37:] == float("inf")).all())


def test_backward_products_are_the_forwards_gradients():
    """sum(y dy) is bilinear in x and w: its change along a direction is the
    gradient times the direction, exactly on whole numbers."""
    g = gen(7)
    T, ends, N, K = 150, [60, 61, 150], 96, 80
    x, w, dy = whole((T, K), g), whole((3, N, K), g), whole((T, N), g)
    d, v = whole((T, K), g), whole((3, N, K), g)
    e = torch.tensor(ends, dtype=torch.int32, device="cuda")
    f = lambda x, w: (mx.mxtrain_grouped_gemm(x, w, e, out_dtype=F32).double() * dy.double()).sum()  # noqa: E731
    dx = mx.mxtrain_grouped_gemm(dy, w, e, transpose_b=False, out_dtype=F32)
    dw = mx.mxtrain_grouped_gemm_k(dy, x, e)
    assert float(f(x + d, w) - f(x - d, w)) == 2 * float((dx.double() * d.double()).sum())
    assert float(f(x, w + v) - f(x, w - v)) == 2 * float((dw.double() * v.double()).sum())


def test_repeatable_and_on_another_stream():
    g = gen(8)
    x, w = torch.randn(700, 1024, generator=g, device="cuda").to(BF16), torch.randn(4, 512, 1024, device="cuda").to(BF16)
    e = torch.tensor([100, 300, 300, 700], dtype=torch.int32, device="cuda")
    first = mx.mxtrain_grouped_gemm(x, w, e)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = mx.mxtrain_grouped_gemm(x, w, e, stream=side)
    side.synchronize()
    assert torch.equal(first, got)


def test_refusals():
    a = torch.zeros((16, 64), dtype=BF16, device="cuda")
    b = torch.zeros((2, 32, 64), dtype=BF16, device="cuda")
    e = torch.tensor([8, 16], dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        mx.mxtrain_grouped_gemm(a.float(), b, e)
    with pytest.raises(TypeError):
        mx.mxtrain_grouped_gemm(a, b, e.long())
    with pytest.raises(TypeError):
        mx.mxtrain_grouped_gemm(a, b, e, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        mx.mxtrain_grouped_gemm(a, b, e[:1])
    with pytest.raises(ValueError):
        mx.mxtrain_grouped_gemm(a, b, e, transpose_b=False)
    with pytest.raises(ValueError):
        mx.mxtrain_grouped_gemm(a, b, e, out=torch.zeros((16, 31), device="cuda"))
    with pytest.raises(ValueError, match="unit column stride"):
        mx.mxtrain_grouped_gemm(a.t()[:16, :16].contiguous().t(), b[..., :16], e)
    with pytest.raises(mx.MxtrainError):  # rows that start off 16 bytes
        mx.mxtrain_grouped_gemm(a[:, :60].contiguous(), b[..., :60].contiguous(), e)
    with pytest.raises(ValueError):
        mx.mxtrain_grouped_gemm_k(a, a[:8], e)
    with pytest.raises(ValueError):
        mx.mxtrain_grouped_gemm_k(a, a, e, out=torch.zeros((2, 64, 32), device="cuda"))
