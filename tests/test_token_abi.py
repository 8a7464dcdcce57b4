"""The token operators' C ABI without a GPU: the library exports what the header
declares, and every argument check returns its status before any launch (every
call below is invalid or empty)."""
import os
import re

import pytest

import swiglu_activation_cast_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, STRIDE, ALIGN, TYPE, OVERFLOW, LAUNCH, WORKSPACE, VALUE = range(10)
BF16, F32 = 0, 1
I32, I64 = 0, 1
A = 1 << 20  # a fake, aligned "device address" (never dereferenced)
BIG = 1 << 31


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "mxtrain_tokens.h")).read()
    names = set(re.findall(r"\b(mxtrain_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"mxtrain_expert_sort_workspace", "mxtrain_expert_sort", "mxtrain_dispatch_fwd",
                     "mxtrain_sort_dispatch", "mxtrain_dispatch_bwd", "mxtrain_combine_fwd", "mxtrain_combine_bwd",
                     "mxtrain_embedding_fwd", "mxtrain_embedding_bwd_workspace", "mxtrain_embedding_bwd",
                     "mxtrain_dropout_fwd", "mxtrain_dropout_bwd"}
    for n in names:
        assert getattr(mx.train_lib(), n).argtypes is not None


def sort(**kw):
    a = dict(ids=A, ld=2, it=I64, T=8, k=2, first=0, G=4, rank=A, ends=A, order=A, ws=None, bytes=0)
    a.update(kw)
    return mx.train_lib().mxtrain_expert_sort(*a.values(), None)


def sort_dispatch(**kw):
    a = dict(x=A, ld_x=64, t=BF16, ids=A, ld=2, it=I64, T=8, k=2, first=0, G=4, H=64, xs=A, ld_xs=64, rank=A, ends=A,
             order=A, ws=None, bytes=0)
    a.update(kw)
    return mx.train_lib().mxtrain_sort_dispatch(*a.values(), None)


@pytest.mark.parametrize("call", [sort, sort_dispatch])
def test_sort_checks(call):
    assert call(it=2) == TYPE
    assert call(T=-1) == SHAPE and call(k=-1) == SHAPE and call(G=-1) == SHAPE and call(G=65536) == SHAPE
    assert call(T=1 << 16, k=1 << 15) == SHAPE  # 2^31 pairs
    assert call(first=2**63 - 1) == VALUE and call(first=2**63 - 4) == VALUE
    assert call(ids=None) == NULL and call(rank=None) == NULL and call(ends=None) == NULL
    assert call(ld=1) == STRIDE
    assert call(ids=A + 4) == ALIGN and call(rank=A + 2) == ALIGN and call(ends=A + 1) == ALIGN
    assert call(order=A + 2) == ALIGN and call(it=I32, ids=A + 2) == ALIGN
    assert call(T=1 << 15, ld=1 << 50, ws=A, bytes=1 << 40) == OVERFLOW
    need = mx.train_lib().mxtrain_expert_sort_workspace(40000, 4)
    assert need > 0
    assert call(T=20000, bytes=need) == NULL and call(T=20000, ws=A + 2, bytes=need) == ALIGN
    assert call(T=20000, ws=A, bytes=need - 1) == WORKSPACE


def test_sort_sizes():
    ws = mx.train_lib().mxtrain_expert_sort_workspace
    assert ws(16, 4) == 0 and ws(-1, 4) == 0 and ws(1 << 20, 65536) == 0 and ws(BIG, 4) == 0
    assert ws(1 << 20, 65535) > ws(1 << 20, 64) > 0
    assert sort(T=0, G=0, ids=None, rank=None, ends=None, order=None) == OK
    assert sort(k=0, G=0, ids=None, rank=None, ends=None, order=None) == OK


def dispatch(**kw):
    a = dict(tokens=A, ld_t=64, t=BF16, rank=A, T=8, k=2, H=64, R=16, rows=A, ld_r=64)
    a.update(kw)
    return mx.train_lib().mxtrain_dispatch_fwd(*a.values(), None)


def dispatch_bwd(**kw):
    a = dict(rows=A, ld_r=64, t=BF16, rank=A, T=8, k=2, H=64, R=16, tokens=A, ld_t=64)
    a.update(kw)
    return mx.train_lib().mxtrain_dispatch_bwd(*a.values(), None)


def combine(**kw):
    a = dict(rows=A, ld_r=64, t=BF16, rank=A, w=A, wt=F32, res=A, ld_res=64, T=8, k=2, H=64, R=16, tokens=A, ld_t=64)
    a.update(kw)
    return mx.train_lib().mxtrain_combine_fwd(*a.values(), None)


def combine_bwd(**kw):
    a = dict(tokens=A, ld_t=64, rows=A, ld_r=64, t=BF16, rank=A, w=A, wt=F32, T=8, k=2, H=64, R=16, dys=A, ld_d=64,
             dw=A)
    a.update(kw)
    return mx.train_lib().mxtrain_combine_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [dispatch, dispatch_bwd, combine, combine_bwd])
def test_move_checks(call):
    assert call(t=2) == TYPE and call(t=-1) == TYPE
    for name in ("T", "k", "H", "R"):
        assert call(**{name: -1}) == SHAPE and call(**{name: BIG}) == SHAPE
    assert call(T=1 << 16, k=1 << 15) == SHAPE
    assert call(tokens=None) == NULL and call(rows=None) == NULL and call(rank=None) == NULL
    assert call(ld_t=63) == STRIDE and call(ld_r=63) == STRIDE
    assert call(tokens=A + 1) == ALIGN and call(rows=A + 1) == ALIGN and call(rank=A + 2) == ALIGN
    assert call(t=F32, rows=A + 2) == ALIGN and call(t=F32, tokens=A + 2) == ALIGN
    assert call(ld_r=1 << 60) == OVERFLOW and call(ld_t=1 << 60) == OVERFLOW
    assert call(T=0, tokens=None, rank=None) == OK


def test_move_own_checks():
    assert dispatch(k=0, rank=None) == OK and dispatch(H=0, tokens=None, rows=None) == OK
    assert dispatch(R=0, rows=None) == OK
    assert dispatch_bwd(H=0, tokens=None, rows=None) == OK and combine(H=0, tokens=None, rows=None) == OK
    assert combine(wt=2) == TYPE and combine_bwd(wt=-1) == TYPE
    assert combine(w=None) == NULL and combine_bwd(w=None) == NULL and combine_bwd(dw=None) == NULL
    assert combine(w=A + 2) == ALIGN and combine(wt=BF16, w=A + 1) == ALIGN
    assert combine_bwd(w=A + 2) == ALIGN and combine_bwd(dw=A + 2) == ALIGN
    assert combine(ld_res=63) == STRIDE and combine(res=A + 1) == ALIGN and combine(ld_res=1 << 60) == OVERFLOW
    assert combine_bwd(dys=None) == NULL and combine_bwd(ld_d=63) == STRIDE and combine_bwd(dys=A + 1) == ALIGN
    assert combine_bwd(ld_d=1 << 60) == OVERFLOW and combine_bwd(k=0, rank=None, w=None, dw=None) == OK


def test_sort_dispatch_checks_the_move_too():
    assert sort_dispatch(t=2) == TYPE and sort_dispatch(H=-1) == SHAPE and sort_dispatch(H=BIG) == SHAPE
    assert sort_dispatch(x=None) == NULL and sort_dispatch(xs=None) == NULL
    assert sort_dispatch(ld_x=63) == STRIDE and sort_dispatch(ld_xs=63) == STRIDE
    assert sort_dispatch(x=A + 1) == ALIGN and sort_dispatch(xs=A + 1) == ALIGN
    assert sort_dispatch(ld_x=1 << 60) == OVERFLOW and sort_dispatch(ld_xs=1 << 60) == OVERFLOW


def embed(**kw):
    a = dict(table=A, ld_w=64, wt=BF16, V=100, H=64, ids=A, step=1, it=I64, T=8, first=0, scale=1.0, tokens=A, ld_t=64,
             tt=BF16)
    a.update(kw)
    return mx.train_lib().mxtrain_embedding_fwd(*a.values(), None)


def embed_bwd(**kw):
    a = dict(tokens=A, ld_t=64, tt=BF16, ids=A, step=1, it=I64, T=8, first=0, scale=1.0, V=100, H=64, table=A, ld_w=64,
             wt=F32, acc=0, ws=A, bytes=1 << 40)
    a.update(kw)
    return mx.train_lib().mxtrain_embedding_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [embed, embed_bwd])
def test_embedding_checks(call):
    assert call(wt=2) == TYPE and call(tt=2) == TYPE and call(it=2) == TYPE
    for scale in (float("nan"), float("inf"), -float("inf")):
        assert call(scale=scale) == VALUE
    for name in ("T", "V", "H"):
        assert call(**{name: -1}) == SHAPE and call(**{name: BIG}) == SHAPE
    assert call(first=2**63 - 1) == VALUE
    assert call(table=None) == NULL and call(tokens=None) == NULL and call(ids=None) == NULL
    assert call(ld_w=63) == STRIDE and call(ld_t=63) == STRIDE and call(step=-1) == STRIDE
    assert call(table=A + 1) == ALIGN and call(tokens=A + 1) == ALIGN and call(ids=A + 4) == ALIGN
    assert call(ld_w=1 << 60) == OVERFLOW and call(ld_t=1 << 60) == OVERFLOW and call(step=1 << 60) == OVERFLOW
    assert call(H=0, table=None, tokens=None) == OK


def test_embedding_own_checks():
    assert embed(T=0, tokens=None, ids=None) == OK
    assert embed_bwd(acc=2) == VALUE
    assert embed_bwd(T=5000, ws=None) == NULL and embed_bwd(T=5000, ws=A + 8) == ALIGN
    for wt, tt in ((BF16, BF16), (F32, BF16), (BF16, F32), (F32, F32)):
        need = mx.train_lib().mxtrain_embedding_bwd_workspace(5000, 100, 64, tt, wt)
        assert need > 0 and embed_bwd(T=5000, wt=wt, tt=tt, bytes=need - 1) == WORKSPACE
        assert mx.train_lib().mxtrain_embedding_bwd_workspace(256, 100, 64, tt, wt) == 0
    big = dict(T=1 << 29, H=513, ld_w=513, ld_t=513, bytes=1 << 62)
    assert embed_bwd(**big) == OVERFLOW and embed_bwd(wt=F32, tt=F32, **{**big, "H": 257}) == OVERFLOW
    assert embed_bwd(V=0, table=None) == OK and embed_bwd(T=0, acc=1, ids=None, tokens=None, ws=None) == OK
    ws = mx.train_lib().mxtrain_embedding_bwd_workspace
    assert ws(0, 100, 64, 0, 0) == 0 and ws(8, 0, 64, 0, 0) == 0 and ws(8, 100, 0, 0, 0) == 0
    assert ws(5000, 100, 64, 2, 0) == 0 and ws(5000, 100, 64, 0, 2) == 0 and ws(BIG, 100, 64, 0, 0) == 0


def dropout(**kw):
    a = dict(x=A, ld_x=64, res=A, ld_res=64, t=BF16, M=8, N=64, p=0.1, seed=1, offset=2, state=None, y=A, ld_y=64)
    a.update(kw)
    return mx.train_lib().mxtrain_dropout_fwd(*a.values(), None)


def dropout_bwd(**kw):
    a = dict(x=A, ld_x=64, t=BF16, M=8, N=64, p=0.1, seed=1, offset=2, state=None, y=A, ld_y=64)
    a.update(kw)
    return mx.train_lib().mxtrain_dropout_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [dropout, dropout_bwd])
def test_dropout_checks(call):
    assert call(t=2) == TYPE
    for p in (-0.1, 1.0001, float("nan"), float("inf")):
        assert call(p=p) == VALUE
    for name in ("M", "N"):
        assert call(**{name: -1}) == SHAPE and call(**{name: BIG}) == SHAPE and call(**{name: 0}) == OK
    assert call(x=None) == NULL and call(y=None) == NULL
    assert call(ld_x=63) == STRIDE and call(ld_y=63) == STRIDE
    assert call(x=A + 1) == ALIGN and call(y=A + 1) == ALIGN and call(state=A + 4) == ALIGN
    assert call(ld_x=1 << 60) == OVERFLOW and call(ld_y=1 << 60) == OVERFLOW


def test_dropout_residual_checks():
    assert dropout(ld_res=63) == STRIDE and dropout(res=A + 1) == ALIGN and dropout(ld_res=1 << 60) == OVERFLOW
