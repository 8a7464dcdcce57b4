"""Embedding lookup and its gradient on the GPU against their formulas in 64 bits.

A looked-up value is one fp32 product rounded once: u = 2^-24 of it, and half a
step, 2^-8, in bf16.  A word's gradient sums n rows in parts of at most 64
serial additions, whose joining adds at most n / 8 + 1 more: (n + 2) u of the sum of
magnitudes bounds any order, and min(n, 64 + n / 8 + 4) this one; the scale's
product adds u, a running sum's addition another u of the result, a bf16 result
half a step."""
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float32]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def words(T, V, g, skew):
    if skew == "one":
        return torch.full((T,), V // 2, device="cuda")
    if skew == "zipf":
        p = 1.0 / (torch.arange(V, device="cuda") + 1.7)
        return torch.multinomial(p, T, replacement=True, generator=g)
    return torch.randint(0, V, (T,), generator=g, device="cuda")


@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("yt", TYPES)
@pytest.mark.parametrize("T,V,H", [(1, 1, 1), (1, 50, 8192), (7, 3, 5), (16, 1000, 64), (513, 77, 2049), (3000, 4099, 130)])
def test_lookup(T, V, H, wt, yt):
    print(f"case: lookup {T} of {V}x{H} {wt} {yt}", flush=True)
    g = gen(T + V + H)
    w = torch.randn((V, H), generator=g, device="cuda").to(wt)
    for dtype in (torch.int64, torch.int32):
        ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda").to(dtype)
        y = mx.mxtrain_embedding_fwd(w, ids, scale=1.7, out_dtype=yt)
        inside = (ids >= 0) & (ids < V)
        ref = torch.where(inside[:, None], w[ids.long().clamp(0, V - 1)].double() * torch.tensor(1.7).double().item(), 0.0)
        tol = ref.abs() * (2 * U + (2.0 ** -8 if yt == torch.bfloat16 else 0.0))
        assert y.dtype == yt and bool(((y.double() - ref).abs() <= tol).all())
    assert torch.equal(mx.mxtrain_embedding_fwd(w, ids), torch.where(inside[:, None], w[ids.long().clamp(0, V - 1)], 0))


def ref_grad(dy, ids, V, scale, first=0):
    key = ids.reshape(-1).long() - first
    ok = (key >= 0) & (key < V)
    dw, mag = (torch.zeros((V, dy.shape[-1]), dtype=torch.float64, device="cuda") for _ in range(2))
    d = dy.reshape(-1, dy.shape[-1]).double()[ok]
    dw.index_add_(0, key[ok], d)
    mag.index_add_(0, key[ok], d.abs())
    n = torch.bincount(key[ok], minlength=V).double()[:, None]
    s = torch.tensor(scale, dtype=torch.float32).double().item()
    return dw * s, mag * abs(s) * (torch.minimum(n, 64 + n / 8 + 4) + 4) * U


def check(got, want, tol):
    extra = want.abs() * 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    bad = (got.double() - want).abs() > tol + extra
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off"


# without a sort (up to 256 tokens); one chunk, several; sorts by comparing (up to 4096,
# or 8192), in tiles (up to 32768), by one, two and three digits; vocabularies smaller and larger than the
# tokens; odd widths
GRADS = [(1, 1, 1), (1, 1000, 5120), (5, 3, 7), (64, 64, 64), (65, 10, 513), (200, 600, 4), (256, 31, 520), (257, 30, 3), (1024, 700, 300), (1025, 600, 65), (700, 5000, 96), (3000, 40, 1000),
         (8192, 1024, 40), (8193, 1023, 40), (9001, 4099, 258), (20000, 1, 72), (30011, 70001, 33), (9000, 1100000, 24),
         (32768, 1500, 16), (32769, 1500, 24), (40007, 1100000, 8)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("wt", TYPES)
@pytest.mark.parametrize("T,V,H", GRADS)
def test_gradient(T, V, H, dt, wt):
    g = gen(T + V)
    dy = torch.randn((T, H), generator=g, device="cuda").to(dt)
    for skew in ("even", "zipf", "one"):
        print(f"case: gradient {T} of {V}x{H} {dt} {wt} {skew}", flush=True)
        ids = words(T, V, g, skew)
        want, tol = ref_grad(dy, ids, V, 0.7)
        dw = mx.mxtrain_embedding_bwd(dy, ids, V, scale=0.7, out_dtype=wt)
        assert dw.dtype == wt and dw.shape == (V, H)
        check(dw, want, tol)
        assert not dw[want.abs().sum(1) == 0].any()
        # added to a running gradient, with ids of the other type; other rows untouched to the bit
        run = torch.randn((V, H), generator=g, device="cuda").to(wt)
        got = mx.mxtrain_embedding_bwd(dy, ids.int(), V, scale=0.7, out=run.clone(), accumulate=True)
        check(got, run.double() + want, tol + (run.double().abs() + want.abs()) * 2 * U)
        idle = torch.bincount(ids, minlength=V) == 0
        assert torch.equal(got[idle], run[idle])


def test_words_outside_are_left_out():
    T, V, H, first = 5000, 300, 40, 1000
    g = gen(2)
    dy = torch.randn((T, H), generator=g, device="cuda")
    ids = torch.randint(first - 200, first + V + 200, (T,), generator=g, device="cuda")
    ids[::7] = -1
    ids[5], ids[6] = 2**63 - 1, -(2**63)
    want, tol = ref_grad(dy, ids, V, 1.0, first)
    check(mx.mxtrain_embedding_bwd(dy, ids, V, first=first), want, tol)
    dy[ids < first] = float("nan")
    check(mx.mxtrain_embedding_bwd(dy, ids, V, first=first), want, tol)
    none = mx.mxtrain_embedding_bwd(dy, torch.full_like(ids, -1), V)
    assert none.shape == (V, H) and not none.any()
    w = torch.randn((V, H), generator=g, device="cuda")
    y = mx.mxtrain_embedding_fwd(w, ids, first=first)
    ok = (ids >= first) & (ids < first + V)
    assert torch.equal(y[ok], w[ids[ok] - first]) and not y[~ok].any()


@pytest.mark.parametrize("dt", TYPES)
def test_strides_shapes_and_alignment(dt):
    V, H = 61, 75
    g = gen(3)
    big = torch.randint(0, V, (6, 50, 3), generator=g, device="cuda")
    ids = big[:, :, 0].contiguous()  # [6, 50]
    col = big.view(-1, 3)[:, 0]      # the same words, three apart
    table = torch.randn((V + 2, H + 9), generator=g, device="cuda").to(dt)
    w = table[1:-1, 3:3 + H]
    y = mx.mxtrain_embedding_fwd(w, ids)
    assert y.shape == (6, 50, H) and torch.equal(y, w[ids])
    assert torch.equal(mx.mxtrain_embedding_fwd(w, col), w[col])
    out = torch.full((300, H + 5), 4.0, device="cuda", dtype=dt)
    mx.mxtrain_embedding_fwd(w, col, out=out[:, 1:1 + H])
    assert torch.equal(out[:, 1:1 + H], w[col]) and bool((out[:, 0] == 4).all()) and bool((out[:, 1 + H:] == 4).all())
    dy = torch.randn((6, 50, H), generator=g, device="cuda").to(dt)
    want = mx.mxtrain_embedding_bwd(dy, ids, V)
    wide = torch.zeros((300, H + 5), device="cuda", dtype=dt)
    wide[:, 5:] = dy.view(300, H)
    assert torch.equal(mx.mxtrain_embedding_bwd(wide[:, 5:], col, V), want)
    grad = torch.full((V + 2, H + 9), 4.0, device="cuda")
    mx.mxtrain_embedding_bwd(dy, ids, V, out=grad[1:-1, 3:3 + H])
    assert torch.equal(grad[1:-1, 3:3 + H], want)
    grad[1:-1, 3:3 + H] = 4.0
    assert bool((grad == 4.0).all())
    one = mx.mxtrain_embedding_fwd(w, ids[2, 3])  # a single id of no dimensions
    assert one.shape == (H,) and torch.equal(one, w[ids[2, 3]])


def test_empty_sizes():
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    assert mx.mxtrain_embedding_fwd(torch.randn((4, 8), device="cuda"), ids).shape == (0, 8)
    dy = torch.zeros((0, 8), device="cuda")
    dw = mx.mxtrain_embedding_bwd(dy, ids, 70, out=torch.ones((70, 8), device="cuda"))
    assert not dw.any()
    same = mx.mxtrain_embedding_bwd(dy, ids, 70, out=torch.ones((70, 8), device="cuda"), accumulate=True)
    assert bool((same == 1).all())
    some = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert not mx.mxtrain_embedding_fwd(torch.zeros((0, 8), device="cuda"), some).any()
    assert mx.mxtrain_embedding_bwd(torch.ones((3, 8), device="cuda"), some, 0).shape == (0, 8)
    assert mx.mxtrain_embedding_bwd(torch.ones((3, 0), device="cuda"), some, 5).shape == (5, 0)


def test_equal_calls_give_equal_bits():
    g = gen(4)
    dy = torch.randn((20000, 520), generator=g, device="cuda").bfloat16()
    ids = words(20000, 900, g, "zipf")
    want = mx.mxtrain_embedding_bwd(dy, ids, 900)
    for _ in range(3):
        torch.full((1 << 24,), float("nan"), device="cuda")  # other contents where the workspace comes from
        assert torch.equal(mx.mxtrain_embedding_bwd(dy, ids, 900), want)


def test_table_past_32_bit_offsets():
    """Rows that lie more than 2^32 bytes from the first, looked up and written."""
    V, H = 600000, 4096
    ids = torch.tensor([V - 1, 0, V - 2, V - 1, 550000], device="cuda")
    w = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
    for i, v in enumerate((V - 1, V - 2, 550000)):
        w[v] = i + 1
    y = mx.mxtrain_embedding_fwd(w, ids)
    assert y[:, 0].tolist() == [1, 0, 2, 1, 3] and torch.equal(y[:, -1], y[:, 0])
    del w
    dw = mx.mxtrain_embedding_bwd(torch.ones((5, H), device="cuda"), ids, V, out_dtype=torch.bfloat16)
    assert dw[:, 0].nonzero()[:, 0].tolist() == [0, 550000, V - 2, V - 1] and float(dw.float().sum()) == 5 * H
    assert bool((dw[V - 1] == 2).all())


def test_gradient_against_differences():
    """<dw, v> against the difference of the lookup, which is linear in the table."""
    T, V, H = 300, 40, 56
    g = gen(6)
    w, v = (torch.randn((V, H), generator=g, device="cuda") for _ in range(2))
    dy = torch.randn((T, H), generator=g, device="cuda")
    ids = words(T, V, g, "zipf")
    f = lambda t: mx.mxtrain_embedding_fwd(t, ids, scale=1.5).double()  # noqa: E731
    lin = (mx.mxtrain_embedding_bwd(dy, ids, V, scale=1.5).double() * v.double()).sum()
    diff = (dy.double() * (f(w + v) - f(w))).sum()
    assert abs(float(lin - diff)) <= float(80 * U * (dy.double().abs() * (f(w.abs()) + f(v.abs()))).sum())


def test_wrong_arguments():
    w, ids = torch.randn((4, 8), device="cuda"), torch.zeros((3, 2), dtype=torch.int64, device="cuda")
    dy = torch.randn((3, 2, 8), device="cuda")
    many, more = torch.randn((1100, 8), device="cuda"), torch.zeros(1100, dtype=torch.int64, device="cuda")
    for call, error in (
            (lambda: mx.mxtrain_embedding_fwd(w, ids.float()), TypeError),
            (lambda: mx.mxtrain_embedding_fwd(w, [0, 1]), TypeError),
            (lambda: mx.mxtrain_embedding_fwd(w.half(), ids), TypeError),
            (lambda: mx.mxtrain_embedding_fwd(w, ids.cpu()), ValueError),
            (lambda: mx.mxtrain_embedding_fwd(w.t(), ids), ValueError),
            (lambda: mx.mxtrain_embedding_fwd(w, ids.t()), ValueError),
            (lambda: mx.mxtrain_embedding_fwd(w, ids, out_dtype=torch.float16), TypeError),
            (lambda: mx.mxtrain_embedding_fwd(w, ids, out=dy[:, :1]), ValueError),
            (lambda: mx.mxtrain_embedding_fwd(w, ids, scale=float("nan")), mx.MxtrainError),
            (lambda: mx.mxtrain_embedding_bwd(dy[:2], ids, 4), ValueError),
            (lambda: mx.mxtrain_embedding_bwd(dy.half(), ids, 4), TypeError),
            (lambda: mx.mxtrain_embedding_bwd(dy, ids, 4, accumulate=True), ValueError),
            (lambda: mx.mxtrain_embedding_bwd(dy, ids, 4, out=w[:3]), ValueError),
            (lambda: mx.mxtrain_embedding_bwd(many, more, 4, workspace=torch.zeros(4, device="cuda")), ValueError)):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("H", [2048, 2051])
def test_gradient_read_past_the_caches(H):
    """128 MB of dy and more are read past the caches."""
    T, V = 33000, 2000
    g = gen(8)
    dy = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    assert dy.numel() * 2 >= 2**27
    ids = words(T, V, g, "zipf")
    want, tol = ref_grad(dy, ids, V, 0.5)
    check(mx.mxtrain_embedding_bwd(dy, ids, V, scale=0.5), want, tol)
