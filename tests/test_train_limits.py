"""Argument checks that must not refuse what the header allows: every call
below is wrong in its last argument checked, so that nothing is ever launched,
and the status says how far the checks went."""
import ctypes

import swiglu_activation_cast_amd as mx

OK, NULL, SHAPE, STRIDE, ALIGN, TYPE, OVERFLOW, LAUNCH, WORKSPACE, VALUE = range(10)
BF16, F32 = 0, 1
A = 1 << 20  # a fake, aligned "device address" (never dereferenced)


def gemm(**kw):
    a = dict(a=A, lda=64, b=A, ldb=64, sb=64 * 32, tb=1, ends=A, G=2, M=16, N=32, K=64, c=A + 1, ldc=64, ct=BF16)
    a.update(kw)
    return mx.train_lib().mxtrain_grouped_gemm(*a.values(), None)


def gemm_k(**kw):
    a = dict(a=A, lda=64, b=A, ldb=32, ends=A, G=2, M=64, N=32, T=16, c=A + 1, ldc=64, sc=64 * 64, ct=F32)
    a.update(kw)
    return mx.train_lib().mxtrain_grouped_gemm_k(*a.values(), None)


def test_operands_without_elements_have_no_strides():
    """torch gives a tensor without elements strides of one and two."""
    assert gemm() == ALIGN
    assert gemm(K=0, a=None, lda=1, b=None, ldb=1, N=33, sb=33) == ALIGN
    assert gemm(K=0, tb=0, lda=1, ldb=33, N=33, sb=33) == ALIGN
    assert gemm_k(T=0, a=None, b=None, M=33, lda=33, N=31, ldb=31) == ALIGN


def test_a_single_row_has_no_row_stride():
    assert gemm(M=1, K=60, lda=60, ldb=64) == ALIGN
    assert gemm(N=1, G=1, K=60, lda=64, ldb=60, sb=0) == ALIGN
    assert gemm(N=1, G=2, K=60, lda=64, ldb=60, sb=64) == ALIGN
    assert gemm(N=1, G=2, K=60, lda=64, ldb=60, sb=60) == STRIDE  # the second expert would start off 16 bytes
    assert gemm(tb=0, K=1, N=33, lda=8, ldb=33, G=1, sb=0) == ALIGN
    assert gemm_k(T=1, M=60, lda=60, N=33, ldb=33) == ALIGN
    assert gemm(M=1, K=60, lda=59) == STRIDE  # still no shorter than the row


def test_layer_norm_takes_every_width_below_2_to_the_31():
    last = 2**31 - 1
    lib = mx.train_lib()
    # a row stride shorter than the row, checked after the sizes
    assert lib.mxtrain_layer_norm_fwd(A, 64, A, A, F32, 4, last, BF16, 1e-5, A, 64, A, A, None) == STRIDE
    assert lib.mxtrain_layer_norm_bwd(A, 64, A, 64, A, A, A, F32, 4, last, BF16, A, 64, A, A, A, 1 << 20, None) == STRIDE
    assert lib.mxtrain_layer_norm_bwd_workspace(4, last) == 2 * last * 4
    assert lib.mxtrain_layer_norm_fwd(A, 64, A, A, F32, 4, last + 1, BF16, 1e-5, A, 64, A, A, None) == SHAPE


def test_newton_schulz_takes_every_side_below_2_to_the_22():
    lib, co, last = mx.train_lib(), (ctypes.c_float * 3)(3.4445, -4.775, 2.0315), 2**22 - 1
    for m, n in ((last, 40), (40, last)):
        need = lib.mxtrain_newton_schulz_workspace(1, m, n, BF16)
        args = (A, n, 0, F32, 1, m, n, 5, co, 1e-7, A, n, 0, BF16, A)
        assert need > 0 and lib.mxtrain_newton_schulz(*args, need - 1, None) == WORKSPACE
    assert lib.mxtrain_newton_schulz(A, 40, 0, F32, 1, last + 1, 40, 5, co, 1e-7, A, 40, 0, BF16, A, 1 << 40, None) == SHAPE
