"""Host-side checks of the dense entry points and the distillation loss (no GPU
needed): bad calls are refused before anything is enqueued."""
import ctypes

import pytest

from bit_ptq_looped_b200 import build as B
from bit_ptq_looped_b200 import lq

X, W, Y, Z, R, WS = ((i + 1) << 40 for i in range(6))  # never dereferenced
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    B.build()
    return lq.lib()


def dense(L, x=X, w=W, b=None, r=None, dt=lq.LQ_BF16, M=4, N=8, K=16, act=0, y=Y, z=None):
    return L.lq_dense_linear(x, w, b, r, dt, M, N, K, act, y, z, None)


def dense_bwd(L, dy=X, z=None, x=W, w=Z, dt=lq.LQ_BF16, M=4, N=8, K=16, act=0, dx=Y, dw=R,
              db=None, g=lq.LQ_BF16, acc=0, ws=WS, n=BIG):
    return L.lq_dense_linear_bwd(dy, z, x, w, dt, M, N, K, act, dx, dw, db, g, acc, ws, n, None)


def distill(L, z=X, dt=lq.LQ_BF16, M=4, V=100, t=W, tdt=lq.LQ_F32, i=Z, ib=8, k=5, lse=None,
            w=None, temp=1.0, loss=Y, grad=None):
    return L.lq_distill_loss(z, dt, M, V, t, tdt, i, ib, k, lse, w, temp, loss, grad, None)


def test_dense_linear_refusals(L):
    for dt in (lq.LQ_F32, 3, -1):
        assert dense(L, dt=dt) == lq.LQ_ERR_UNSUPPORTED
    for act in (-1, 5):
        assert dense(L, act=act) == lq.LQ_ERR_UNSUPPORTED
    assert dense(L, K=12) == lq.LQ_ERR_SHAPE and "multiple of 8" in L.lq_last_error().decode()
    for kw in (dict(M=-1), dict(N=0), dict(K=0), dict(N=-8), dict(x=None), dict(w=None),
               dict(y=None)):
        assert dense(L, **kw) == lq.LQ_ERR_ARG
    for kw in (dict(M=1 << 31), dict(N=1 << 31), dict(K=1 << 31), dict(M=1 << 30, N=1 << 30)):
        assert dense(L, **kw) == lq.LQ_ERR_SHAPE
    for kw in (dict(x=X + 8), dict(w=W + 2), dict(b=R + 4), dict(r=R + 2), dict(y=Y + 8),
               dict(z=Z + 8)):
        assert dense(L, **kw) == lq.LQ_ERR_ALIGN
    # outputs over inputs or over each other
    for kw in (dict(y=X), dict(y=X + 16), dict(y=W + 16), dict(b=Y), dict(r=Y + 16), dict(z=Y),
               dict(z=W), dict(y=X - 16)):
        assert dense(L, **kw) == lq.LQ_ERR_ARG, kw
        assert "overlaps" in L.lq_last_error().decode()
    assert dense(L, M=0, x=None, y=None) == lq.LQ_OK


def test_gated_linear_refusals(L):
    def gated(x=X, wg=W, wu=R, dt=lq.LQ_F16, M=4, N=8, K=16, act=2, h=Y, g=None, u=None, b=None):
        return L.lq_gated_linear(x, wg, wu, b, b, dt, M, N, K, act, h, g, u, None)

    assert gated(dt=lq.LQ_F32) == lq.LQ_ERR_UNSUPPORTED
    assert gated(K=20) == lq.LQ_ERR_SHAPE
    assert gated(g=Z) == lq.LQ_ERR_ARG  # u missing
    assert gated(g=Z, u=Z) == lq.LQ_ERR_ARG
    assert gated(h=R) == lq.LQ_ERR_ARG and gated(wu=None) == lq.LQ_ERR_ARG
    assert gated(wu=R + 2) == lq.LQ_ERR_ALIGN
    assert gated(M=0, x=None, h=None) == lq.LQ_OK


def test_backward_refusals(L):
    assert dense_bwd(L, g=lq.LQ_F16) == lq.LQ_ERR_UNSUPPORTED
    assert dense_bwd(L, acc=1) == lq.LQ_ERR_UNSUPPORTED
    assert dense_bwd(L, act=lq.LQ_ACT_SILU) == lq.LQ_ERR_ARG  # z missing
    for kw in (dict(dy=None), dict(x=None), dict(w=None)):
        assert dense_bwd(L, **kw) == lq.LQ_ERR_ARG
    need = L.lq_dense_linear_bwd_workspace_bytes(40, 8, 16, lq.LQ_ACT_SILU)
    assert need > 0 and need % 256 == 0
    assert dense_bwd(L, M=40, z=5 << 44, act=2, n=need - 1) == lq.LQ_ERR_WORKSPACE
    assert dense_bwd(L, M=40, z=5 << 44, act=2, ws=None) == lq.LQ_ERR_ARG
    assert dense_bwd(L, M=40, z=5 << 44, act=2, ws=WS + 16) == lq.LQ_ERR_ALIGN
    for kw in (dict(dx=X), dict(dw=Y), dict(db=Z), dict(dx=WS), dict(dw=WS)):
        assert dense_bwd(L, M=40, **kw) == lq.LQ_ERR_ARG, kw
    # nothing wanted, or no rows to add: nothing is enqueued
    assert dense_bwd(L, dx=None, dw=None) == lq.LQ_OK
    assert dense_bwd(L, M=0, dy=None, x=None, acc=1, g=lq.LQ_F32, ws=None, n=0) == lq.LQ_OK

    def gated_bwd(dh=X, g=1 << 45, u=2 << 45, x=3 << 45, wg=4 << 45, wu=5 << 45, dx=6 << 45,
                  dwg=7 << 45, dwu=8 << 45, gd=lq.LQ_BF16, acc=0, n=BIG):
        return L.lq_gated_linear_bwd(dh, g, u, x, wg, wu, lq.LQ_BF16, 40, 8, 16, 2, dx, dwg, dwu,
                                     None, None, gd, acc, WS, n, None)

    for kw in (dict(dh=None), dict(g=None), dict(u=None), dict(wg=None), dict(wu=None),
               dict(x=None), dict(dwu=7 << 45), dict(dx=1 << 45)):
        assert gated_bwd(**kw) == lq.LQ_ERR_ARG, kw
    assert gated_bwd(n=0) == lq.LQ_ERR_WORKSPACE
    assert gated_bwd(gd=lq.LQ_F16) == lq.LQ_ERR_UNSUPPORTED
    assert gated_bwd(acc=1) == lq.LQ_ERR_UNSUPPORTED


def test_workspace_sizes(L):
    for f in (L.lq_gated_linear_bwd_workspace_bytes,
              lambda M, N, K: L.lq_dense_linear_bwd_workspace_bytes(M, N, K, 2)):
        for bad in ((-1, 8, 8), (4, 0, 8), (4, 8, -8), (1 << 31, 8, 8), (1 << 30, 1 << 30, 8)):
            assert f(*bad) == -1
        for ok in ((0, 1, 8), (1, 1, 8), (4096, 5632, 2048)):
            n = f(*ok)
            assert n >= 0 and n % 256 == 0
    # a few rows need none; an aligned output gradient without an activation is
    # used as it is
    assert L.lq_gated_linear_bwd_workspace_bytes(4, 5632, 2048) == 0
    assert L.lq_dense_linear_bwd_workspace_bytes(4096, 2048, 2048, 0) < 4096 * 2048
    assert L.lq_dense_linear_bwd_workspace_bytes(4096, 2047, 2048, 0) >= 4096 * 2047 * 2
    assert L.lq_gated_linear_bwd_workspace_bytes(4096, 2048, 64) >= 4096 * 2048 * 4


def test_distill_refusals(L):
    for kw in (dict(dt=3), dict(tdt=7), dict(ib=2), dict(ib=16)):
        assert distill(L, **kw) == lq.LQ_ERR_UNSUPPORTED
    for kw in (dict(M=-1), dict(V=0), dict(k=0), dict(temp=0.0), dict(temp=-1.0),
               dict(temp=float("nan")), dict(temp=float("inf")), dict(temp=1e-45), dict(z=None),
               dict(t=None), dict(i=None), dict(loss=None)):
        assert distill(L, **kw) == lq.LQ_ERR_ARG, kw
    for kw in (dict(k=101), dict(k=8193, V=20000), dict(V=512 * 1024 + 1), dict(M=1 << 30)):
        assert distill(L, **kw) == lq.LQ_ERR_SHAPE, kw
    for kw in (dict(z=X + 2), dict(t=W + 4), dict(i=Z + 8), dict(loss=Y + 4), dict(grad=R + 2),
               dict(lse=R + 4), dict(w=R + 4)):
        assert distill(L, **kw) == lq.LQ_ERR_ALIGN, kw
    for kw in (dict(grad=X + 16), dict(grad=W), dict(loss=X), dict(grad=Y)):
        assert distill(L, **kw) == lq.LQ_ERR_ARG, kw
    assert distill(L, M=0, z=None, t=None, i=None, loss=None) == lq.LQ_OK


def test_header_limit_matches():
    text = open(B.INCLUDE + "/lq.h").read()
    assert "#define LQ_DISTILL_MAX_V (512 * 1024)" in text
    assert "#define LQ_DISTILL_MAX_K 8192" in text
    for name, code in (("NONE", 0), ("RELU", 1), ("SILU", 2), ("GELU", 3), ("GELU_TANH", 4)):
        assert getattr(lq, "LQ_ACT_" + name) == code == lq.LQ_ACTS[name.lower()]
        assert any(line.split()[:3] == ["#define", "LQ_ACT_" + name, str(code)]
                   for line in text.splitlines())
    assert ctypes.sizeof(ctypes.c_void_p) == 8
