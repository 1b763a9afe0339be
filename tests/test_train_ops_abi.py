"""Host-side argument checks of the training operators, without a GPU: every
call below is refused, or is an empty no-op, before any CUDA call."""
import ctypes as C

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6


@pytest.fixture(scope="module")
def L():
    import quantized_gnn_message_gb300 as q
    from quantized_gnn_message_gb300 import build
    build.build()
    return q.lib()


FAKE = C.c_void_p(0x1000)
ODD = C.c_void_p(0x1002)


def _drop(L, X=FAKE, ty=0, n=10, d=16, ldx=16, p=0.5, Y=FAKE, ldy=16):
    return L.gq_dropout(X, ty, n, d, ldx, p, 1, Y, ldy, None)


@pytest.mark.parametrize("kw", [dict(ty=3), dict(ty=-1), dict(n=-1), dict(n=1 << 32), dict(d=0), dict(ldx=15),
                                dict(ldy=15), dict(p=-0.1), dict(p=1.01), dict(p=float("nan")), dict(X=None),
                                dict(Y=None), dict(X=ODD), dict(Y=ODD), dict(ty=1, Y=C.c_void_p(0x1001))])
def test_dropout_refuses(L, kw):
    assert _drop(L, **kw) == INVALID


def test_empty_calls_are_no_ops(L):
    assert _drop(L, n=0, X=None, Y=None) == 0
    assert _fwd(L, n=0, X=None, Y=None) == 0
    assert _bwd(L, n=0, dY=None, X=None, dX=None, mean=None, rstd=None, dg=None, db=None, ws=None) == 0


def _fwd(L, X=FAKE, ty=0, n=10, d=16, ldx=16, ga=None, be=None, eps=1e-5, act=0, p=0.0, Y=FAKE, ldy=16, mean=None,
         rstd=None, bits=None, ldrb=0):
    return L.gq_layer_norm_fwd(X, ty, n, d, ldx, ga, be, eps, act, p, 0, Y, ldy, mean, rstd, bits, ldrb, None)


@pytest.mark.parametrize("kw", [dict(ty=9), dict(n=-5), dict(n=1 << 32), dict(d=0), dict(ldx=8), dict(ldy=8),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(act=2),
                                dict(p=2.0), dict(X=None), dict(Y=None), dict(bits=FAKE, ldrb=1),
                                dict(act=1, bits=FAKE, ldrb=0), dict(act=1, bits=ODD, ldrb=1), dict(ga=ODD),
                                dict(mean=ODD)])
def test_layer_norm_fwd_refuses(L, kw):
    assert _fwd(L, **kw) == INVALID


def test_layer_norm_limits(L):
    assert _fwd(L, d=16385, ldx=16385, ldy=16385) == UNSUPPORTED
    assert _bwd(L, d=16385, ldx=16385, lddy=16385, lddx=16385) == UNSUPPORTED
    assert L.gq_layer_norm_bwd_workspace_bytes(10, 16385) == 0 and L.gq_layer_norm_bwd_workspace_bytes(-1, 8) == 0


def _bwd(L, dY=FAKE, lddy=16, X=FAKE, ldx=16, ty=0, n=10, d=16, mean=FAKE, rstd=FAKE, ga=None, act=0, p=0.0,
         bits=None, ldrb=0, dX=FAKE, dxt=None, lddx=16, dg=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30):
    return L.gq_layer_norm_bwd(dY, lddy, X, ldx, ty, n, d, mean, rstd, ga, act, p, 0, bits, ldrb, dX,
                               ty if dxt is None else dxt, lddx, dg, db, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(ty=5), dict(dxt=2), dict(ty=1, dxt=0), dict(ty=2, dxt=1), dict(n=-1), dict(d=0),
                                dict(ldx=2), dict(lddy=2), dict(lddx=2), dict(act=1), dict(act=-1), dict(p=-1.0),
                                dict(act=1, bits=FAKE, ldrb=0), dict(mean=None), dict(rstd=None), dict(dY=None),
                                dict(X=None), dict(dX=None), dict(dg=ODD)])
def test_layer_norm_bwd_refuses(L, kw):
    assert _bwd(L, **kw) == INVALID


def test_layer_norm_bwd_workspace(L):
    assert _bwd(L, ws=None) == WORKSPACE
    assert _bwd(L, wsb=L.gq_layer_norm_bwd_workspace_bytes(10, 16) - 1) == WORKSPACE


def _xent(L, X=FAKE, n=10, k=16, ldx=16, W=FAKE, C=30, ldw=16, lab=FAKE, dX=FAKE, lddx=16, dW=FAKE, lddw=16,
          ws=FAKE, wsb=1 << 40, loss=FAKE):
    return L.gq_linear_xent(X, n, k, ldx, W, C, ldw, lab, None, 1.0, loss, None, dX, lddx, dW, lddw, ws, wsb, None,
                            None)


@pytest.mark.parametrize("kw", [dict(X=None), dict(W=None), dict(lab=None), dict(n=-1), dict(k=0), dict(C=0),
                                dict(ldx=8), dict(ldx=17), dict(ldw=8), dict(ldw=20), dict(lddx=8), dict(lddx=18),
                                dict(lddw=8), dict(lddw=18), dict(X=C.c_void_p(0x1008)), dict(W=C.c_void_p(0x1008)),
                                dict(dX=C.c_void_p(0x1008)), dict(dW=C.c_void_p(0x1008)), dict(lab=ODD),
                                dict(loss=ODD)])
def test_linear_xent_refuses(L, kw):
    assert _xent(L, **kw) == INVALID


def test_linear_xent_limits(L):
    assert _xent(L, k=16392, ldx=16392, ldw=16392, lddx=16392, lddw=16392) == UNSUPPORTED
    assert _xent(L, n=1 << 31) == UNSUPPORTED and _xent(L, C=(1 << 30) + 1) == UNSUPPORTED
    assert _xent(L, n=1 << 30, C=1 << 20) == UNSUPPORTED
    assert _xent(L, ws=None) == WORKSPACE and _xent(L, ws=C.c_void_p(0x1010)) == WORKSPACE
    need = L.gq_linear_xent_workspace_bytes(10, 16, 30, 1)
    assert need > L.gq_linear_xent_workspace_bytes(10, 16, 30, 0) > 0
    assert _xent(L, wsb=need - 1) == WORKSPACE
    assert L.gq_linear_xent_workspace_bytes(10, 0, 30, 1) == 0
    assert _xent(L, n=0, X=None, W=None, lab=None, dX=None, dW=None, ws=None) == 0
