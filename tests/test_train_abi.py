"""The training operators' C ABI without a GPU: the library exports what its
header declares, and every argument check returns its status before any launch
(every call below is invalid or empty)."""
import ctypes
import os
import re

import pytest

import swiglu_activation_cast_amd as mx

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, STRIDE, ALIGN, TYPE, OVERFLOW, LAUNCH, WORKSPACE, VALUE = range(10)
BF16, F32 = 0, 1
A = 1 << 20  # a fake, aligned "device address" (never dereferenced)


def test_library_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "mxtrain.h")).read()
    names = set(re.findall(r"\b(mxtrain_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"mxtrain_layer_norm_fwd", "mxtrain_layer_norm_bwd", "mxtrain_layer_norm_bwd_workspace",
                     "mxtrain_grouped_gemm", "mxtrain_grouped_gemm_k", "mxtrain_newton_schulz",
                     "mxtrain_newton_schulz_workspace", "mxtrain_status_str"}
    for n in names:
        assert getattr(mx.train_lib(), n) is not None


def test_status_strings():
    texts = [mx.train_status_str(st) for st in range(10)]
    assert len(set(texts)) == 10 and mx.train_status_str(99) == "unknown status"


def ln_fwd(**kw):
    a = dict(x=A, ld_x=64, w=A, b=A, pt=F32, M=4, N=64, t=BF16, eps=1e-5, y=A, ld_y=64, mean=A, rstd=A)
    a.update(kw)
    return mx.train_lib().mxtrain_layer_norm_fwd(*a.values(), None)


def ln_bwd(**kw):
    a = dict(dy=A, ld_dy=64, x=A, ld_x=64, mean=A, rstd=A, w=A, pt=F32, M=4, N=64, t=BF16, dx=A, ld_dx=64, dw=A, db=A,
             ws=A, bytes=1 << 20)
    a.update(kw)
    return mx.train_lib().mxtrain_layer_norm_bwd(*a.values(), None)


@pytest.mark.parametrize("call", [ln_fwd, ln_bwd])
def test_layer_norm_checks(call):
    assert call(t=2) == TYPE and call(pt=-1) == TYPE
    assert call(M=-1) == SHAPE and call(N=-1) == SHAPE and call(N=0) == SHAPE and call(M=1 << 31) == SHAPE
    assert call(x=None) == NULL
    assert call(ld_x=63) == STRIDE
    assert call(x=A + 1) == ALIGN and call(w=A + 2) == ALIGN and call(t=F32, x=A + 2) == ALIGN
    assert call(mean=A + 2) == ALIGN
    assert call(M=1 << 30, ld_x=1 << 40) == OVERFLOW


def test_layer_norm_own_checks():
    for eps in (-1e-5, float("nan"), float("inf")):
        assert ln_fwd(eps=eps) == VALUE
    assert ln_fwd(y=None) == NULL and ln_fwd(ld_y=1) == STRIDE and ln_fwd(y=A + 1) == ALIGN
    assert ln_fwd(M=0, x=None, y=None) == OK
    assert ln_bwd(mean=None) == NULL and ln_bwd(rstd=None) == NULL and ln_bwd(dy=None) == NULL
    assert ln_bwd(M=2000, ws=None) == NULL and ln_bwd(M=2000, ws=A + 2) == ALIGN and ln_bwd(dw=A + 1) == ALIGN
    need = mx.train_lib().mxtrain_layer_norm_bwd_workspace(2000, 64)
    assert need > 0 and ln_bwd(M=2000, bytes=need - 1) == WORKSPACE
    assert mx.train_lib().mxtrain_layer_norm_bwd_workspace(4, 64) == 0
    assert ln_bwd(M=0, N=0) == OK
    assert ln_bwd(M=0, dw=None, db=None, ws=None, dy=None, x=None, mean=None, rstd=None, dx=None) == OK
    assert mx.train_lib().mxtrain_layer_norm_bwd_workspace(0, 64) == 0


def gemm(**kw):
    a = dict(a=A, lda=64, b=A, ldb=64, sb=64 * 32, tb=1, ends=A, G=2, M=16, N=32, K=64, c=A, ldc=32, ct=BF16)
    a.update(kw)
    return mx.train_lib().mxtrain_grouped_gemm(*a.values(), None)


def gemm_k(**kw):
    a = dict(a=A, lda=64, b=A, ldb=32, ends=A, G=2, M=64, N=32, T=16, c=A, ldc=32, sc=64 * 32, ct=F32)
    a.update(kw)
    return mx.train_lib().mxtrain_grouped_gemm_k(*a.values(), None)


@pytest.mark.parametrize("call", [gemm, gemm_k])
def test_product_checks(call):
    assert call(ct=2) == TYPE
    assert call(G=-1) == SHAPE and call(M=-1) == SHAPE and call(G=65536) == SHAPE and call(N=1 << 31) == SHAPE
    assert call(G=0) == OK and call(M=0) == OK and call(N=0) == OK
    assert call(a=None) == NULL and call(b=None) == NULL and call(c=None) == NULL and call(ends=None) == NULL
    assert call(lda=60) == STRIDE and call(lda=68) == STRIDE and call(ldc=31) == STRIDE
    assert call(a=A + 8) == ALIGN and call(b=A + 2) == ALIGN and call(c=A + 1) == ALIGN and call(ends=A + 2) == ALIGN
    assert call(lda=1 << 22) == OVERFLOW and call(ldc=1 << 58) == OVERFLOW


def test_product_own_checks():
    assert gemm(tb=2) == VALUE
    assert gemm(sb=64 * 32 - 8) == STRIDE and gemm(sb=64 * 32 + 4) == STRIDE and gemm(sb=-8) == STRIDE
    assert gemm(tb=0, ldb=24) == STRIDE            # [K, N]: rows of N
    assert gemm(sb=1 << 60, G=65535) == OVERFLOW
    assert gemm_k(sc=64 * 32 - 1) == STRIDE and gemm_k(ldb=24) == STRIDE


def ortho(**kw):
    a = dict(g=A, ld_g=40, sg=30 * 40, t=F32, B=2, m=30, n=40, steps=5, co=(ctypes.c_float * 3)(3.4445, -4.775, 2.0315),
             eps=1e-7, out=A, ld_o=40, so=30 * 40, ot=F32, ws=A, bytes=1 << 40)
    a.update(kw)
    return mx.train_lib().mxtrain_newton_schulz(*a.values(), None)


def test_newton_schulz_checks():
    assert ortho(t=2) == TYPE and ortho(ot=3) == TYPE
    assert ortho(co=None) == NULL and ortho(g=None) == NULL and ortho(out=None) == NULL and ortho(ws=None) == NULL
    assert ortho(steps=-1) == VALUE and ortho(steps=101) == VALUE and ortho(eps=-1.0) == VALUE
    assert ortho(co=(ctypes.c_float * 3)(1, float("inf"), 0)) == VALUE
    assert ortho(B=-1) == SHAPE and ortho(m=1 << 22) == SHAPE and ortho(B=65536) == SHAPE
    assert ortho(B=0) == OK and ortho(m=0) == OK and ortho(n=0) == OK
    assert ortho(ld_g=39) == STRIDE and ortho(ld_o=39) == STRIDE and ortho(so=30 * 40 - 1) == STRIDE
    assert ortho(g=A + 2) == ALIGN and ortho(out=A + 1) == ALIGN and ortho(ws=A + 16) == ALIGN
    assert ortho(ld_g=1 << 58) == OVERFLOW
    for ot in (BF16, F32):
        need = mx.train_lib().mxtrain_newton_schulz_workspace(2, 30, 40, ot)
        assert need > 0 and ortho(ot=ot, bytes=need - 1) == WORKSPACE
    assert mx.train_lib().mxtrain_newton_schulz_workspace(2, 0, 40, F32) == 0
    assert mx.train_lib().mxtrain_newton_schulz_workspace(2, 30, 40, 7) == 0
