"""Dropout on the GPU: its mask against the generator's definition in numpy (and
that against the published test vectors), its values in 64 bits.

A kept value is one fp32 product, the residual one addition: 2 u of their
magnitudes with u = 2^-24 (the scale itself is rounded to fp32, another u), and
half a step, 2^-8, of a bf16 result."""
import numpy as np
import pytest
import torch

import swiglu_activation_cast_amd as mx

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]
gpu = pytest.mark.gpu


def philox(counter, key):
    """Philox4x32-10 of Salmon, Moraes, Dror and Shaw (2011): counter [..., 4], key (k0, k1)."""
    c = [np.asarray(counter)[..., i].astype(object) for i in range(4)]
    k0, k1 = key
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k0, b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k1, a & 0xFFFFFFFF]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, -1)


def bits(M, N, seed, offset):
    """The 16 bits of each element of [M, N]."""
    seed, offset = seed % 2**64, offset % 2**64
    C = (N + 7) // 8
    counter = np.zeros((M, C, 4), dtype=np.int64)
    counter[..., 0] = np.arange(C)
    counter[..., 1] = np.arange(M)[:, None]
    counter[..., 2], counter[..., 3] = offset & 0xFFFFFFFF, offset >> 32
    w = philox(counter, (seed & 0xFFFFFFFF, seed >> 32)).astype(np.int64)
    return np.stack([w & 0xFFFF, w >> 16], -1).reshape(M, C * 8)[:, :N]


def test_generator_against_published_vectors():
    ones = 0xFFFFFFFF
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((ones,) * 4, (ones, ones), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
             (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        assert tuple(philox(np.array(counter), key)) == want


def randn(M, N, seed, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((M, N), generator=g, device="cuda").to(dtype)


def want(x, p, seed, offset, res):
    border = round(p * 65536)
    keep = torch.from_numpy(bits(*x.shape, seed, offset) >= border).cuda()
    y = torch.where(keep, x.double() * (65536 / max(1, 65536 - border)), 0.0)
    r = torch.zeros_like(y) if res is None else res.double()
    return y + r, 3 * U * (y.abs() + r.abs()), keep


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (3, 7), (1, 8), (5, 64), (129, 65), (64, 1000), (31, 2049), (2, 20011)])
def test_values_and_mask(M, N, dtype):
    print(f"case: dropout {M}x{N} {dtype}", flush=True)
    x, res = randn(M, N, 1, dtype), randn(M, N, 2, dtype)
    half = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for p, seed, offset in ((0.1, 1, 0), (0.5, 2**64 - 1, 2**64 - 1), (0.25, 0x123456789ABCDEF0, 2**32), (1 / 3, 0, 77)):
        for r in (None, res):
            y = mx.mxtrain_dropout_fwd(x, p, seed, offset, residual=r)
            ref, tol, keep = want(x, p, seed, offset, r)
            assert y.dtype == dtype and bool(((y.double() - ref).abs() <= tol + half * ref.abs()).all())
            if r is not None:
                assert torch.equal(y[~keep], r[~keep])
            else:
                assert not y[~keep].any()
                assert torch.equal(mx.mxtrain_dropout_bwd(x, p, seed, offset), y)


@gpu
def test_no_dropping_and_nothing_else():
    x = randn(20, 100, 3, torch.bfloat16)
    assert torch.equal(mx.mxtrain_dropout_fwd(x, 0.0, 5, 6), x)
    assert torch.equal(mx.mxtrain_dropout_fwd(x, 1e-6, 5, 6), x)  # below half of 1 / 65536
    x[0], x[1] = float("nan"), float("inf")
    assert not mx.mxtrain_dropout_fwd(x, 1.0, 5, 6).any()
    assert torch.equal(mx.mxtrain_dropout_fwd(x[2:], 1.0, 5, 6, residual=x[:18].nan_to_num(1.0, 2.0)), x[:18].nan_to_num(1.0, 2.0))
    y = mx.mxtrain_dropout_fwd(x, 0.5, 5, 6)
    _, _, keep = want(x, 0.5, 5, 6, None)
    assert bool(torch.isnan(y[0][keep[0]]).all()) and bool(torch.isinf(y[1][keep[1]]).all())
    assert not y[~keep].any()


@gpu
def test_the_mask_is_of_the_place_alone():
    """Type, strides, alignment and the number of rows do not enter."""
    M, N = 77, 203
    ones = torch.ones((M, N), device="cuda")
    keep = mx.mxtrain_dropout_fwd(ones, 0.4, 9, 10) != 0
    big = torch.full((M + 2, N + 7), 3.0, device="cuda", dtype=torch.bfloat16)
    out = torch.full((M + 2, N + 9), 3.0, device="cuda", dtype=torch.bfloat16)
    y = mx.mxtrain_dropout_fwd(big[1:-1, 3:3 + N], 0.4, 9, 10, residual=big[:M, 1:1 + N], out=out[1:-1, 5:5 + N])
    assert torch.equal(y != 3.0, keep)
    out[1:-1, 5:5 + N] = 3.0
    assert bool((out == 3.0).all())
    assert torch.equal(mx.mxtrain_dropout_fwd(ones[:13], 0.4, 9, 10) != 0, keep[:13])
    assert torch.equal(mx.mxtrain_dropout_fwd(ones[:, :8 * 3], 0.4, 9, 10) != 0, keep[:, :24])
    for other in ((8, 10), (9, 11), (9 + 2**32, 10), (9, 10 + 2**32)):
        assert not torch.equal(mx.mxtrain_dropout_fwd(ones, 0.4, *other) != 0, keep)


@gpu
def test_share_and_mean():
    """The share of 2^22 elements kept is within five standard deviations, and so
    are the products of neighbours, across columns, rows and calls."""
    x = torch.ones((2048, 2048), device="cuda")
    for p in (0.1, 0.5, 0.9):
        n, q = x.numel(), 1 - round(p * 65536) / 65536
        k = [(mx.mxtrain_dropout_fwd(x, p, 3, o) != 0).double() - q for o in (1, 2)]
        sd = (q * (1 - q) / n) ** 0.5
        assert abs(float(k[0].mean())) < 5 * sd
        for a, b in ((k[0][:, :-1], k[0][:, 1:]), (k[0][:-1], k[0][1:]), (k[0][:, :-8], k[0][:, 8:]), (k[0], k[1])):
            assert abs(float((a * b).mean())) < 5 * q * (1 - q) / (a.numel() ** 0.5)


@gpu
def test_state_on_the_device_adds_to_seed_and_offset():
    x = randn(30, 90, 4, torch.float32)
    state = torch.tensor([5, 2**40], device="cuda")
    assert torch.equal(mx.mxtrain_dropout_fwd(x, 0.3, 100, 7, state=state), mx.mxtrain_dropout_fwd(x, 0.3, 105, 2**40 + 7))
    state = torch.tensor([-1, -1], device="cuda")
    assert torch.equal(mx.mxtrain_dropout_bwd(x, 0.3, 0, 0, state=state),
                       mx.mxtrain_dropout_bwd(x, 0.3, 2**64 - 1, 2**64 - 1))


@gpu
def test_more_rows_than_2_to_the_31_elements():
    """Offsets past 32 bits, in bytes and in elements."""
    M, N = 300000, 8192
    x = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    y = mx.mxtrain_dropout_fwd(x, 0.5, 11, 12)
    for r in (0, 1, 262143, 262144, M - 1):
        counter = np.zeros((N // 8, 4), dtype=np.int64)
        counter[:, 0], counter[:, 1], counter[:, 2] = np.arange(N // 8), r, 12
        w = philox(counter, (11, 0)).astype(np.int64)
        keep = np.stack([w & 0xFFFF, w >> 16], -1).reshape(N) >= 32768
        assert np.array_equal(y[r].float().cpu().numpy(), keep * 2.0), r


@gpu
def test_empty_and_wrong_arguments():
    x = torch.randn((4, 8), device="cuda")
    assert mx.mxtrain_dropout_fwd(x[:0], 0.5, 1, 2).shape == (0, 8)
    assert mx.mxtrain_dropout_fwd(x[:, :0], 0.5, 1, 2).shape == (4, 0)
    for call, error in (
            (lambda: mx.mxtrain_dropout_fwd(x, 1.5, 1, 2), mx.MxtrainError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, -1, 2), ValueError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, 1, 2**64), ValueError),
            (lambda: mx.mxtrain_dropout_fwd(x.half(), 0.5, 1, 2), TypeError),
            (lambda: mx.mxtrain_dropout_fwd(x[0], 0.5, 1, 2), ValueError),
            (lambda: mx.mxtrain_dropout_fwd(x.t(), 0.5, 1, 2), ValueError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, 1, 2, residual=x[:3]), ValueError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, 1, 2, residual=x.bfloat16()), TypeError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, 1, 2, out=x.bfloat16()), TypeError),
            (lambda: mx.mxtrain_dropout_fwd(x, 0.5, 1, 2, state=torch.zeros(3, dtype=torch.int64, device="cuda")), ValueError),
            (lambda: mx.mxtrain_dropout_bwd(x, 0.5, 1, 2, state=torch.zeros(2, device="cuda")), TypeError)):
        with pytest.raises(error):
            call()


@gpu
@pytest.mark.parametrize("N", [8192, 8195])
def test_read_past_the_caches(N):
    """128 MB and more are read past the caches: the same bits as in two parts of columns, which are not."""
    M = 8300
    x, res = randn(M, N, 5, torch.bfloat16), randn(M, N, 6, torch.bfloat16)
    assert x.numel() * 2 >= 2**27
    y = mx.mxtrain_dropout_fwd(x, 0.3, 7, 8, residual=res)
    assert torch.equal(y[:, :4096], mx.mxtrain_dropout_fwd(x[:, :4096], 0.3, 7, 8, residual=res[:, :4096]))
    assert torch.equal(y[:4000], mx.mxtrain_dropout_fwd(x[:4000], 0.3, 7, 8, residual=res[:4000]))
    ref, tol, _ = want(x[:40], 0.3, 7, 8, res[:40])
    assert bool(((y[:40].double() - ref).abs() <= tol + 2.0 ** -8 * ref.abs()).all())
