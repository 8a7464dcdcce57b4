"""Tokens sorted by expert and back, on the GPU against the definitions.

Sorts are compared exactly with a stable sort on the host, moved rows to the
bit.  Sums of k fp32 products of 16- or 32-bit values: each of at most k + 1
fused or plain additions rounds once, at most u = 2^-24 of the running sum, itself at
most S = |residual| + sum |w y|; so (k + 2) u S covers them, to which a bf16
result adds half a step, 2^-8 of the value, and an fp32 one u of it.  A
weighted row is one product, rounded once: half a step of its type.  A weight's
gradient sums H products in chains of at most H / 16 + 8 serial additions and a tree
of six: (H / 16 + 16) u times the sum of magnitudes."""
import numpy as np
import pytest
import torch

import swiglu_activation_cast_amd as mx

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ref_sort(ids, E, first):
    """rank, ends, order by the definition, on the host (numpy)."""
    key = ids.cpu().numpy().astype(object).reshape(-1) - first if first else ids.cpu().numpy().astype(np.int64).reshape(-1)
    kept = np.array([(v >= 0) and (v < E) for v in key], dtype=bool) if first else (key >= 0) & (key < E)
    key = np.where(kept, key, E).astype(np.int64)
    by = np.argsort(key, kind="stable")
    n = int(kept.sum())
    rank = np.full(key.size, -1)
    rank[by[:n]] = np.arange(n)
    order = np.full(key.size, -1)
    order[:n] = by[:n]
    return rank.reshape(tuple(ids.shape)), np.cumsum(np.bincount(key, minlength=E + 1)[:E]), order


def check_sort(got, want):
    for g, w, name in zip(got, want, ("rank", "ends", "order")):
        assert g.dtype == torch.int32 and tuple(g.shape) == w.shape, name
        assert np.array_equal(g.cpu().numpy(), w), name


# up to 4096 pairs (8192 of more than 1023 experts, fewer of very many), compared in one
# launch, with 32 places a workgroup, or 128 from 16385 pairs and experts; up to 32768 of
# more than 1023 experts, in tiles of 1024; up to 16384 of fewer, where every workgroup counts all; more, by digits:
# one or two, with a tile of 8192 a workgroup and several; ranges that end inside a tile
SORTS = [(0, 2, 4), (1, 1, 1), (1, 8, 300), (5, 3, 7), (63, 1, 64), (200, 8, 64), (1021, 5, 33), (1024, 8, 255),
         (4096, 2, 1023), (4097, 2, 1024), (900, 9, 65535), (8193, 1, 2), (16640, 4, 16), (16384, 8, 64),
         (20011, 3, 1023), (20011, 3, 5000), (70001, 2, 65535), (300001, 2, 96), (2500003, 2, 40), (2300001, 1, 5000), (0, 1, 5000),
         (31, 1, 33), (65, 1, 3), (2731, 3, 9), (8192, 1, 17000), (3000, 1, 65535), (9, 1, 40000), (4107, 2, 6), (12289, 1, 3000),
         (8192, 2, 64), (16385, 1, 128), (10923, 3, 65535), (16384, 2, 7), (32769, 1, 7), (2048, 2, 64), (4097, 1, 1023), (16384, 2, 2000), (32769, 1, 1024), (5000, 1, 20000)]


@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort(T, k, E):
    print(f"case: sort {T}x{k} by {E}", flush=True)
    g = gen(T + k + E)
    for kind, dtype in (("even", torch.int64), ("one", torch.int32), ("dropped", torch.int64), ("wide", torch.int32)):
        ids = torch.randint(0, E, (T, k), generator=g, device="cuda")
        if kind == "one":
            ids.fill_(E - 1)
        elif kind == "dropped":  # one side, the other, the first past each end
            ids = torch.randint(-2, E + 2, (T, k), generator=g, device="cuda")
        elif kind == "wide":
            ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.3, -2**31, ids)
        ids = ids.to(dtype)
        check_sort(mx.mxtrain_expert_sort(ids, E), ref_sort(ids, E, 0))


def test_sort_of_a_shard_strides_and_one_dimension():
    ids = torch.randint(0, 64, (700, 6), generator=gen(1), device="cuda")
    for first, E in ((16, 16), (-5, 30), (60, 16), (1000, 4), (-(2**62), 3), (2**62, 3)):
        check_sort(mx.mxtrain_expert_sort(ids, E, first=first), ref_sort(ids, E, first))
    part = ids[::2, 1:4]  # rows 12 elements apart, off the first column
    check_sort(mx.mxtrain_expert_sort(part, 64), ref_sort(part.contiguous(), 64, 0))
    big = torch.randint(0, 64, (30000, 5), generator=gen(2), device="cuda").to(torch.int32)
    check_sort(mx.mxtrain_expert_sort(big[:, 2:], 64), ref_sort(big[:, 2:].contiguous(), 64, 0))
    col = big[:, 3]
    check_sort(mx.mxtrain_expert_sort(col, 64), ref_sort(col.contiguous(), 64, 0))
    check_sort(mx.mxtrain_expert_sort(ids[:0, 0], 5), ref_sort(ids[:0, 0], 5, 0))
    far = torch.tensor([[2**63 - 1, -(2**63)], [2**62 + 1, 2**62]], device="cuda")
    check_sort(mx.mxtrain_expert_sort(far, 9, first=2**62), ref_sort(far, 9, 2**62))
    check_sort(mx.mxtrain_expert_sort(far, 9, first=2**63 - 10), ref_sort(far, 9, 2**63 - 10))
    check_sort(mx.mxtrain_expert_sort(far, 9, first=-(2**63)), ref_sort(far, 9, -(2**63)))


def test_no_experts_drop_every_pair():
    ids = torch.randint(0, 4, (30, 2), generator=gen(1), device="cuda")
    rank, ends, order = mx.mxtrain_expert_sort(ids, 0)
    assert bool((rank == -1).all()) and bool((order == -1).all()) and ends.numel() == 0


def routed(T, k, E, H, dtype, seed, shards=1):
    g = gen(seed)
    ids = torch.topk(torch.rand((T, E), generator=g, device="cuda"), k, dim=1).indices
    local = E // shards
    first = local * (shards - 1)
    rank, ends, order = (torch.from_numpy(v).to(torch.int32).cuda() for v in ref_sort(ids, local, first))
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(ids=ids, rank=rank, ends=ends, order=order, local=local, first=first, x=r(T, H).to(dtype),
                rows=r(T * k, H).to(dtype), dy=r(T, H).to(dtype), w=torch.softmax(r(T, k), 1), res=r(T, H).to(dtype))


# widths: one element, under one piece, whole pieces, odd ones, rows of several
# thousand; tokens: one, few (one workgroup sorts), many
MOVES = [(1, 1, 1, 1), (1, 8, 16, 5120), (3, 2, 5, 7), (17, 2, 4, 8), (130, 3, 9, 65), (64, 8, 64, 1000), (700, 1, 4, 64),
         (5003, 3, 32, 129), (3001, 8, 40, 257), (1021, 2, 16, 2049), (2000, 12, 24, 96)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E,H", MOVES)
@pytest.mark.parametrize("shards", [1, 2])
def test_moves_and_gradients(T, k, E, H, dtype, shards):
    if E < shards:
        pytest.skip("fewer experts than shards")
    print(f"case: {T}x{k} of {E}, {H} {dtype} shards {shards}", flush=True)
    s = routed(T, k, E, H, dtype, T + H, shards)
    rank = s["rank"].long()
    kept = rank >= 0
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    # dispatch: in one call with the sort, and by rank; rows behind the last stay as they were
    want = torch.full((T * k, H), 7.0, dtype=dtype, device="cuda")
    want[rank[kept]] = s["x"][torch.nonzero(kept)[:, 0]]
    out = torch.full_like(want, 7.0)
    xs, got_rank, ends, order = mx.mxtrain_sort_dispatch(s["x"], s["ids"], s["local"], first=s["first"], out=out)
    assert xs is out and torch.equal(xs, want)
    assert torch.equal(got_rank, s["rank"]) and torch.equal(ends, s["ends"]) and torch.equal(order, s["order"])
    assert torch.equal(mx.mxtrain_dispatch_fwd(s["x"], s["rank"], out=torch.full_like(want, 7.0)), want)
    # combine and dispatch's gradient
    rows = torch.where(kept[:, :, None], s["rows"][rank.clamp(min=0)].double(), 0.0)
    for w in (s["w"], s["w"].bfloat16()):
        for res in (None, s["res"]):
            y = mx.mxtrain_combine_fwd(s["rows"], s["rank"], w, residual=res)
            terms = rows * w.double()[:, :, None]
            r = 0.0 if res is None else res.double()
            ref, mag = terms.sum(1) + r, terms.abs().sum(1) + (0.0 if res is None else r.abs())
            assert y.dtype == dtype and bool(((y.double() - ref).abs() <= (k + 2) * U * mag + half * ref.abs()).all())
    dx = mx.mxtrain_dispatch_bwd(s["rows"], s["rank"])
    ref, mag = rows.sum(1), rows.abs().sum(1)
    assert bool(((dx.double() - ref).abs() <= (k + 2) * U * mag + half * ref.abs()).all())
    # combine's gradients
    out = torch.full_like(want, 7.0)
    for w in (s["w"], s["w"].bfloat16()):
        dys, dw = mx.mxtrain_combine_bwd(s["dy"], s["rows"], s["rank"], w, out=out.clone())
        ref = out.double()
        ref[rank[kept]] = (w.double()[:, :, None] * s["dy"].double()[:, None, :])[kept]
        assert bool(((dys.double() - ref).abs() <= half * ref.abs()).all())
        prod = rows * s["dy"].double()[:, None, :]
        assert dw.dtype == torch.float32 and dw.shape == rank.shape
        assert bool(((dw.double() - prod.sum(2)).abs() <= (H / 16 + 16) * U * prod.abs().sum(2)).all())
        assert not dw[~kept].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(dtype):
    """Views whose rows start at odd elements, and rows around them left alone."""
    T, k, E, H = 301, 3, 8, 131
    s = routed(T, k, E, H, dtype, 5)

    def inside(t):
        big = torch.full((t.shape[0] + 2, t.shape[1] + 6), 9.0, dtype=dtype, device="cuda")
        view = big[1:-1, 3:-3]
        view.copy_(t)
        return big, view

    def rim(big):
        mask = torch.ones_like(big, dtype=torch.bool)
        mask[1:-1, 3:-3] = False
        return bool((big[mask] == 9.0).all())

    x, rows, dy, res = (inside(s[n])[1] for n in ("x", "rows", "dy", "res"))
    for name, plain, strided in (
            ("dispatch", lambda o: mx.mxtrain_dispatch_fwd(s["x"], s["rank"], out=o),
             lambda o: mx.mxtrain_dispatch_fwd(x, s["rank"], out=o)),
            ("sort_dispatch", lambda o: mx.mxtrain_sort_dispatch(s["x"], s["ids"], E, out=o)[0],
             lambda o: mx.mxtrain_sort_dispatch(x, s["ids"], E, out=o)[0]),
            ("combine_bwd", lambda o: mx.mxtrain_combine_bwd(s["dy"], s["rows"], s["rank"], s["w"], out=o)[0],
             lambda o: mx.mxtrain_combine_bwd(dy, rows, s["rank"], s["w"], out=o)[0])):
        big, view = inside(torch.zeros((T * k, H), dtype=dtype, device="cuda"))
        assert torch.equal(strided(view), plain(None)) and rim(big), name
    big, view = inside(torch.zeros((T, H), dtype=dtype, device="cuda"))
    mx.mxtrain_combine_fwd(rows, s["rank"], s["w"], residual=res, out=view)
    assert torch.equal(view, mx.mxtrain_combine_fwd(s["rows"], s["rank"], s["w"], residual=s["res"])) and rim(big)
    assert torch.equal(mx.mxtrain_combine_bwd(dy, rows, s["rank"], s["w"])[1],
                       mx.mxtrain_combine_bwd(s["dy"], s["rows"], s["rank"], s["w"])[1])
    big, view = inside(torch.zeros((T, H), dtype=dtype, device="cuda"))
    mx.mxtrain_dispatch_bwd(rows, s["rank"], out=view)
    assert torch.equal(view, mx.mxtrain_dispatch_bwd(s["rows"], s["rank"])) and rim(big)


def test_ranks_outside_the_rows_are_dropped():
    """Whatever rank holds, nothing outside the matrices is touched."""
    T, H, R = 40, 72, 50
    g = gen(3)
    rank = torch.stack([torch.randperm(R, generator=g, device="cuda")[:T],
                        torch.randint(R, 2**31 - 1, (T,), generator=g, device="cuda")], 1).to(torch.int32)
    rank[0, 1], rank[1, 1], rank[2, 1], rank[3, 1] = -1, R, -2**31, 2**31 - 1
    x, w = torch.randn((T, H), generator=g, device="cuda"), torch.rand((T, 2), generator=g, device="cuda")
    ys = torch.randn((R, H), generator=g, device="cuda")
    want = torch.full((R, H), 5.0, device="cuda")
    want[rank[:, 0].long()] = x
    assert torch.equal(mx.mxtrain_dispatch_fwd(x, rank, out=torch.full((R, H), 5.0, device="cuda")), want)
    first = ys[rank[:, 0].long()]
    assert torch.equal(mx.mxtrain_dispatch_bwd(ys, rank), first)
    assert torch.equal(mx.mxtrain_combine_fwd(ys, rank, w), first * w[:, :1])
    dys, dw = mx.mxtrain_combine_bwd(x, ys, rank, w, out=torch.full((R, H), 5.0, device="cuda"))
    want[rank[:, 0].long()] = x * w[:, :1]
    assert torch.equal(dys, want) and not dw[:, 1].any()


def test_dropped_rows_and_infinities():
    """A token without kept pairs gets its residual or zeros, NaN in rows that no
    pair names reach nothing, and those in kept rows reach their token only."""
    T, k, H = 33, 2, 40
    g = gen(4)
    ids = torch.randint(0, 4, (T, k), generator=g, device="cuda")
    ids[7] = -1
    rank, ends, order = mx.mxtrain_expert_sort(ids, 4)
    ys = torch.randn((T * k, H), generator=g, device="cuda").bfloat16()
    ys[-2:] = float("nan")
    w = torch.rand((T, k), generator=g, device="cuda")
    res = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    y = mx.mxtrain_combine_fwd(ys, rank, w, residual=res)
    assert torch.equal(y[7], res[7]) and bool(torch.isfinite(y).all())
    assert not mx.mxtrain_combine_fwd(ys, rank, w)[7].any() and not mx.mxtrain_dispatch_bwd(ys, rank)[7].any()
    ys[rank[9, 1].long()] = float("inf")
    y = mx.mxtrain_combine_fwd(ys, rank, w)
    assert bool(torch.isinf(y[9]).all()) and bool(torch.isfinite(y[torch.arange(T, device="cuda") != 9]).all())


def test_empty_sizes():
    x = torch.randn((0, 16), device="cuda")
    ids = torch.zeros((0, 2), dtype=torch.int64, device="cuda")
    xs, rank, ends, order = mx.mxtrain_sort_dispatch(x, ids, 3)
    assert xs.shape == (0, 16) and ends.tolist() == [0, 0, 0]
    assert mx.mxtrain_combine_fwd(xs, rank, torch.zeros((0, 2), device="cuda")).shape == (0, 16)
    none = torch.zeros((4, 0), dtype=torch.int32, device="cuda")
    res = torch.randn((4, 16), device="cuda")
    y = mx.mxtrain_combine_fwd(xs, none, torch.zeros((4, 0), device="cuda"), residual=res)
    assert torch.equal(y, res) and not mx.mxtrain_dispatch_bwd(xs, none).any()
    narrow = torch.zeros((4, 0), device="cuda")
    rank = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    dys, dw = mx.mxtrain_combine_bwd(narrow, torch.zeros((8, 0), device="cuda"), rank, torch.ones((4, 2), device="cuda"))
    assert dys.shape == (8, 0) and not dw.any()


def test_rows_past_32_bit_offsets():
    """Sorted rows that lie more than 2^32 bytes from the first."""
    T, k, H = 70000, 8, 4100
    ids = torch.topk(torch.rand((T, 16), generator=gen(1), device="cuda"), k, dim=1).indices
    x = (torch.arange(T, device="cuda") % 256).to(torch.bfloat16)[:, None] * torch.ones(H, dtype=torch.bfloat16, device="cuda")
    xs, rank, ends, order = mx.mxtrain_sort_dispatch(x, ids, 16)
    assert xs.numel() * 2 > 2**32
    assert torch.equal(xs[:, 0].float(), (order.long() // k % 256).float()) and torch.equal(xs[:, -1], xs[:, 0])
    y = mx.mxtrain_dispatch_bwd(xs, rank)
    assert torch.equal(y, x * 8)


def test_gradients_against_differences():
    """<dys, v> and <dw, u> against differences of the forward pass in fp32:
    it is linear in ys and in w, so a difference of size 1 has rounding alone, (k +
    2) u of each of the T H sums' magnitudes."""
    T, k, E, H = 50, 3, 6, 48
    s = routed(T, k, E, H, torch.float32, 8)
    g = gen(9)
    v, u = torch.randn((T * k, H), generator=g, device="cuda"), torch.randn((T, k), generator=g, device="cuda")
    f = lambda ys, w: mx.mxtrain_combine_fwd(ys, s["rank"], w).double()  # noqa: E731
    dys, dw = mx.mxtrain_combine_bwd(s["dy"], s["rows"], s["rank"], s["w"])
    dy = s["dy"].double()
    for diff, lin, mag in (((f(s["rows"] + v, s["w"]) - f(s["rows"], s["w"])), (dys.double() * v).sum(), f(s["rows"].abs() + v.abs(), s["w"])),
                           ((f(s["rows"], s["w"] + u) - f(s["rows"], s["w"])), (dw.double() * u).sum(), f(s["rows"].abs(), s["w"] + u.abs()))):
        assert abs(float((dy * diff).sum() - lin)) <= float(4 * (k + H) * U * (dy.abs() * mag).sum())


def test_wrong_arguments():
    x, ids = torch.randn((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int64, device="cuda")
    rank = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    w, rows = torch.ones((4, 2), device="cuda"), torch.randn((8, 8), device="cuda")
    for call, error in (
            (lambda: mx.mxtrain_expert_sort(ids.float(), 4), TypeError),
            (lambda: mx.mxtrain_expert_sort(ids.cpu(), 4), ValueError),
            (lambda: mx.mxtrain_expert_sort(ids[None], 4), ValueError),
            (lambda: mx.mxtrain_expert_sort(ids.t(), 4), ValueError),
            (lambda: mx.mxtrain_expert_sort(ids, 65536), mx.MxtrainError),
            (lambda: mx.mxtrain_expert_sort(ids, 4, order=torch.zeros(7, dtype=torch.int32, device="cuda")), ValueError),
            (lambda: mx.mxtrain_sort_dispatch(x[:3], ids, 4), ValueError),
            (lambda: mx.mxtrain_sort_dispatch(x.half(), ids, 4), TypeError),
            (lambda: mx.mxtrain_dispatch_fwd(x, ids), TypeError),
            (lambda: mx.mxtrain_dispatch_fwd(x, rank.t().contiguous().t()), ValueError),
            (lambda: mx.mxtrain_dispatch_fwd(x, rank[:3]), ValueError),
            (lambda: mx.mxtrain_combine_fwd(rows, rank, w[:, :1]), ValueError),
            (lambda: mx.mxtrain_combine_fwd(rows, rank, w.double()), TypeError),
            (lambda: mx.mxtrain_combine_fwd(rows, rank, w, residual=x.bfloat16()), TypeError),
            (lambda: mx.mxtrain_combine_fwd(rows, rank, w, residual=x[:3]), ValueError),
            (lambda: mx.mxtrain_combine_bwd(x[:, :7], rows, rank, w), ValueError),
            (lambda: mx.mxtrain_combine_bwd(x, rows, rank, w, dweights=w[:2]), ValueError),
            (lambda: mx.mxtrain_dispatch_bwd(rows.t(), rank, out=x.t()), ValueError)):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,k,E", [(64, 4, 255), (65, 4, 7), (128, 8, 64), (205, 5, 9), (512, 4, 200), (513, 4, 200), (100, 3, 256)])
def test_one_call_is_the_sort_and_the_move(T, k, E, dtype):
    """On both sides of every border of the form that sorts and moves in one launch (256, 1024 and 2048 pairs, 255
    experts): the same bits as the two calls."""
    g = gen(T)
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda")
    for H in (1, 3, 40, 1031):
        x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
        xs, *index = mx.mxtrain_sort_dispatch(x, ids, E, out=torch.zeros((T * k, H), dtype=dtype, device="cuda"))
        want = mx.mxtrain_expert_sort(ids, E)
        assert all(torch.equal(a, b) for a, b in zip(index, want))
        assert torch.equal(xs, mx.mxtrain_dispatch_fwd(x, want[0], out=torch.zeros_like(xs)))


@pytest.mark.parametrize("T,k,H", [(1024, 2, 4099), (2048, 1, 1030)])
def test_one_call_with_several_steps(T, k, H):
    """The form that sorts and moves in one launch, with more pieces than its workgroups take in one step."""
    g = gen(H)
    ids = torch.randint(-1, 12, (T, k), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda")
    assert T * ((H + 3) // 4) > 1024 * 256
    xs, rank, ends, order = mx.mxtrain_sort_dispatch(x, ids, 11)
    check_sort((rank, ends, order), ref_sort(ids, 11, 0))
    for j in range(k):
        kept = rank[:, j] >= 0
        assert torch.equal(xs[rank[kept, j].long()], x[kept])


@pytest.mark.parametrize("H", [2048, 2053])
def test_rows_read_past_the_caches(H):
    """128 MB of rows and more are read past the caches: the same bits as half of the tokens at a time, which is not."""
    T, k, E = 8300, 4, 16
    s = routed(T, k, E, H, torch.bfloat16, 11)
    assert T * k * H * 2 >= 2**27 > T * k * H
    y = mx.mxtrain_combine_fwd(s["rows"], s["rank"], s["w"], residual=s["res"])
    dx = mx.mxtrain_dispatch_bwd(s["rows"], s["rank"])
    dys, dw = mx.mxtrain_combine_bwd(s["dy"], s["rows"], s["rank"], s["w"])
    want = torch.empty_like(dys)
    for part in (slice(0, T // 2), slice(T // 2, T)):
        rank, w, dy = s["rank"][part], s["w"][part], s["dy"][part]
        assert torch.equal(y[part], mx.mxtrain_combine_fwd(s["rows"], rank, w, residual=s["res"][part]))
        assert torch.equal(dx[part], mx.mxtrain_dispatch_bwd(s["rows"], rank))
        assert torch.equal(dw[part], mx.mxtrain_combine_bwd(dy, s["rows"], rank, w, out=want)[1])
    assert torch.equal(dys, want)
