"""The vocabulary-head operators refuse bad arguments before anything reaches
the GPU.  No GPU needed."""
import ctypes as ct

import pytest
import torch

import rns_emulated_fp64_gb300 as os2
from rns_emulated_fp64_gb300 import binding as b

P = ct.c_void_p(0x1000)       # never dereferenced: every case fails validation first
ODD = ct.c_void_p(0x1001)
F32, F16, BF16 = 0, 1, 2


def test_quantize_rows_refusals():
    f = os2.load().os2_quantize_rows
    assert f(-1, 4, F32, P, 4, P, 4, P, None) == b.ERR_INVALID_ARG
    assert f(4, 4, F32, P, 3, P, 4, P, None) == b.ERR_INVALID_ARG       # ldx < k
    assert f(4, 4, F32, P, 4, P, 3, P, None) == b.ERR_INVALID_ARG       # ldq < k
    assert f(4, 4, 3, P, 4, P, 4, P, None) == b.ERR_INVALID_ARG         # type
    assert f(4, 4, F32, None, 4, P, 4, P, None) == b.ERR_INVALID_ARG
    assert f(4, 4, F32, P, 4, P, 4, None, None) == b.ERR_INVALID_ARG
    assert f(4, 4, BF16, ODD, 4, P, 4, P, None) == b.ERR_INVALID_ARG
    assert f(0, 4, F32, None, 4, None, 4, None, None) == b.OK


def test_i8_refusals():
    lib = os2.load()
    g, l = lib.os2_i8gemm, lib.os2_i8linear
    big = 1 << 30

    def gemm(m=4, n=4, k=4, A=P, lda=4, sa=P, B=P, ldb=4, sb=P, bias=None, C=P, ldc=4, dt=F32, ws=P, nb=big):
        return g(m, n, k, A, lda, sa, B, ldb, sb, bias, C, ldc, dt, ws, nb, None)

    def linear(m=4, n=4, k=4, xt=BF16, X=P, ldx=4, B=P, ldb=4, sb=P, bias=None, C=P, ldc=4, dt=F32, ws=P, nb=big):
        return l(m, n, k, xt, X, ldx, B, ldb, sb, bias, C, ldc, dt, ws, nb, None)

    bad = [dict(m=-1), dict(n=-1), dict(k=-1), dict(ldb=3), dict(ldc=3), dict(dt=3), dict(B=None),
           dict(sb=None), dict(C=None), dict(C=ODD), dict(bias=ODD)]
    for kw in bad + [dict(lda=3), dict(A=None), dict(sa=None)]:
        assert gemm(**kw) == b.ERR_INVALID_ARG, kw
    for kw in bad + [dict(ldx=3), dict(X=None), dict(X=ODD), dict(xt=3)]:
        assert linear(**kw) == b.ERR_INVALID_ARG, kw
    for f, ld in ((gemm, "lda"), (linear, "ldx")):
        assert f(k=1 << 17, ldb=1 << 17, **{ld: 1 << 17}) == b.ERR_UNSUPPORTED
        assert f(ws=None) == b.ERR_WORKSPACE
        assert f(nb=1) == b.ERR_WORKSPACE
        assert f(ws=ODD) == b.ERR_WORKSPACE
        assert f(m=0, A=None) == b.OK if f is gemm else f(m=0, X=None) == b.OK
    size = lib.os2_i8gemm_workspace_size
    assert size(-1, 4, 4, P, 4) == 0 and size(4, 4, 1 << 17, P, 1 << 17) == 0 and size(4, 4, 4, P, 3) == 0
    assert size(4, 4, 4, P, 16) > 0


def test_xent_refusals():
    lib = os2.load()
    big = 1 << 40

    def fwd(n=4, k=8, v=4, dt=BF16, H=P, ldh=8, W=P, ldw=8, y=P, loss=P, lse=P, ws=P, nb=big):
        return lib.os2_xent(n, k, v, dt, H, ldh, W, ldw, y, -100, loss, lse, ws, nb, None)

    def bwd(n=4, k=8, v=4, dt=BF16, H=P, ldh=8, W=P, ldw=8, y=P, lse=P, grad=P, dH=P, lddh=8, dW=P, lddw=8, ws=P, nb=big):
        return lib.os2_xent_backward(n, k, v, dt, H, ldh, W, ldw, y, -100, lse, grad, dH, lddh, dW, lddw, ws, nb, None)

    bad = [dict(n=-1), dict(k=0), dict(v=0), dict(ldh=7), dict(ldw=7), dict(dt=3), dict(H=None), dict(W=None),
           dict(y=None), dict(H=ODD), dict(W=ODD), dict(y=ODD), dict(lse=None)]
    for kw in bad + [dict(loss=None)]:
        assert fwd(**kw) == b.ERR_INVALID_ARG, kw
    for kw in bad + [dict(grad=None), dict(lddh=7), dict(lddw=7), dict(dH=ODD), dict(dW=ODD)]:
        assert bwd(**kw) == b.ERR_INVALID_ARG, kw
    for f in (fwd, bwd):
        assert f(dt=F32) == b.ERR_UNSUPPORTED
        assert f(v=(1 << 22) + 1) == b.ERR_UNSUPPORTED
        assert f(n=(1 << 22) + 1) == b.ERR_UNSUPPORTED
        assert f(ws=None) == b.ERR_WORKSPACE
        assert f(nb=256) == b.ERR_WORKSPACE
        assert f(ws=ODD) == b.ERR_WORKSPACE
    assert fwd(n=0) == b.OK
    assert bwd(dH=None, dW=None) == b.OK
    size = lib.os2_xent_workspace_size
    assert size(4, 0, 4, P, 8, 0) == 0 and size(-1, 8, 4, P, 8, 1) == 0 and size(4, 8, 4, P, 7, 1) == 0
    # a head whose rows TMA cannot take is copied: its size is in the workspace
    assert size(4, 8, 1 << 20, ODD, 8, 0) >= size(4, 8, 1 << 20, P, 8, 0) + (1 << 20) * 8 * 2
    # the logits of a long batch over a large vocabulary are never there as a whole
    n, k, v = 1 << 15, 1024, 1 << 18
    assert size(n, k, v, P, k, 0) < n * v // 4
    assert size(n, k, v, P, k, 1) < n * v // 4


def test_adamw_refusals():
    lib = os2.load()
    ptrs = (ct.c_void_p * 1)(0x1000)
    odd = (ct.c_void_p * 1)(0x1001)
    null = (ct.c_void_p * 1)(None)

    def f(count=1, numel=4, p=ptrs, g=ptrs, m=ptrs, v=ptrs, ms=None, vs=None, pt=F32, gt=F32, bits=32, lr=1e-3,
          b1=0.9, b2=0.95, eps=1e-8, wd=0.1, step=1):
        return lib.os2_adamw(count, (ct.c_longlong * 1)(numel), p, g, m, v, ms, vs, pt, gt, bits, lr, b1, b2, eps, wd,
                             step, None)

    for kw in [dict(count=-1), dict(numel=-1), dict(p=None), dict(p=null), dict(p=odd), dict(g=odd), dict(m=odd),
               dict(v=null), dict(pt=3), dict(gt=-1), dict(bits=16), dict(bits=8), dict(bits=8, ms=null, vs=null),
               dict(lr=-1.0), dict(lr=float("nan")), dict(b1=1.0), dict(b2=-0.1), dict(eps=-1.0), dict(eps=float("inf")),
               dict(wd=float("nan")), dict(step=0)]:
        assert f(**kw) == b.ERR_INVALID_ARG, kw
    assert f(numel=(1 << 40) + 1) == b.ERR_UNSUPPORTED
    assert f(count=0) == b.OK
    mo = lib.os2_adamw_moments
    assert mo(-1, P, P, P, P, P, P, None) == b.ERR_INVALID_ARG
    assert mo(4, P, P, P, P, None, P, None) == b.ERR_INVALID_ARG
    assert mo(4, P, ODD, P, P, P, P, None) == b.ERR_INVALID_ARG
    assert mo(0, None, None, None, None, None, None, None) == b.OK


def test_python_refusals():
    x = torch.zeros(4, 8)
    for f in (lambda: os2.quantize_rows(x), lambda: os2.i8linear(x, x.to(torch.int8), x[:, 0]),
              lambda: os2.i8gemm(x.to(torch.int8), x[:, 0], x.to(torch.int8), x[:, 0]),
              lambda: os2.xent(x.half(), x.half(), torch.zeros(4, dtype=torch.int64)),
              lambda: os2.adamw([x], [x], [x], [x], step=1, lr=1e-3),
              lambda: os2.adamw_moments(x.to(torch.int8), x[0, :1], x.to(torch.uint8), x[0, :1])):
        with pytest.raises(ValueError):
            f()                                    # host tensors
    os2.adamw([], [], [], [], step=1, lr=1e-3)      # nothing to do
