"""Host-side argument checks of AdamW, the 8-bit integer products and group
normalization, without a GPU: every call below is refused, or is an empty
no-op, before any CUDA call."""
import ctypes as C

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 6
FAKE = C.c_void_p(0x1000)
ODD = C.c_void_p(0x1002)
BYTE = C.c_void_p(0x1001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def q():
    import quantized_gnn_message_gb300 as q
    from quantized_gnn_message_gb300 import build
    build.build()
    return q


@pytest.fixture(scope="module")
def L(q):
    return q.lib()


# ------------------------------------------------------------------ adamw --


def _adamw(q, L, pt=0, gt=0, bits=32, count=1, args=None, **kw):
    t = dict(p=0x1000, g=0x1000, m=0x1000, v=0x1000, m_exp=0x1000, v_exp=0x1000, n=10, cols=0, ldp=0, ldg=0, block0=0)
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.0, step=1, seed=0, grad_scale=None, dev=None,
             advance=0)
    t.update({k: v for k, v in kw.items() if k in t})
    a.update({k: v for k, v in kw.items() if k in a})
    arr = (q.AdamwTensor_t * 1)()
    for k, v in t.items():
        setattr(arr[0], k, v)
    c = q.AdamwArgs_t()
    for k, v in a.items():
        setattr(c, k, v)
    return L.gq_adamw_step(arr, count, pt, gt, bits, C.byref(c), None)


@pytest.mark.parametrize("kw", [dict(pt=3), dict(gt=-1), dict(bits=16), dict(count=-1), dict(p=None), dict(g=None),
                                dict(m=None), dict(v=None), dict(p=0x1002), dict(g=0x1002), dict(m=0x1002), dict(v=0x1001),
                                dict(pt=1, p=0x1001), dict(gt=2, g=0x1001), dict(bits=8, m_exp=None),
                                dict(bits=8, v_exp=None), dict(n=-1), dict(cols=-1), dict(cols=3, ldp=3, ldg=3),
                                dict(cols=5, ldp=4, ldg=5), dict(cols=5, ldp=5, ldg=4), dict(block0=-1),
                                dict(block0=1 << 32), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=NAN), dict(beta2=1.0),
                                dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF), dict(lr=INF), dict(lr=NAN),
                                dict(weight_decay=NAN), dict(step=0), dict(step=-3), dict(dev=0x1004),
                                dict(grad_scale=0x1002)])
def test_adamw_refuses(q, L, kw):
    assert _adamw(q, L, **kw) == INVALID


def test_adamw_limits_and_empty(q, L):
    assert _adamw(q, L, n=(1 << 40) + 1) == UNSUPPORTED
    assert _adamw(q, L, count=0) == 0
    assert _adamw(q, L, n=0, p=None, g=None, m=None, v=None) == 0
    assert L.gq_adamw_step(None, 1, 0, 0, 32, None, None) == INVALID
    assert L.gq_adamw_dev_bytes() >= 16


@pytest.mark.parametrize("args", [(None, FAKE, 10, 0, FAKE, 0), (FAKE, None, 10, 0, FAKE, 0), (FAKE, FAKE, 10, 0, None, 0),
                                  (FAKE, FAKE, -1, 0, FAKE, 0), (FAKE, FAKE, 10, 0, FAKE, 3), (FAKE, FAKE, 10, 0, ODD, 0),
                                  (FAKE, FAKE, 10, 1, BYTE, 1)])
def test_adam_moment_refuses(L, args):
    assert L.gq_adam_moment(*args, None) == INVALID


def test_adam_moment_empty(L):
    assert L.gq_adam_moment(None, None, 0, 0, None, 0, None) == 0


# -------------------------------------------------------------------- int8 --


def _quant(L, X=FAKE, ty=0, n=10, d=20, ldx=20, tr=0, Q=FAKE, ldq=32, S=FAKE, ws=FAKE, wsb=1 << 30):
    return L.gq_quantize_i8(X, ty, n, d, ldx, tr, Q, ldq, S, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(ty=3), dict(n=-1), dict(d=0), dict(ldx=19), dict(ldq=16), dict(ldq=24),
                                dict(tr=1, n=40, ldq=32), dict(X=None), dict(Q=None), dict(S=None), dict(X=ODD),
                                dict(ty=1, X=BYTE), dict(Q=C.c_void_p(0x1008)), dict(S=ODD)])
def test_quantize_refuses(L, kw):
    assert _quant(L, **kw) == INVALID


def test_quantize_limits(L):
    assert _quant(L, n=(1 << 30) + 1) == UNSUPPORTED
    assert _quant(L, d=1 << 22, ldx=1 << 22, ldq=1 << 22) == UNSUPPORTED
    assert _quant(L, tr=1, ws=None) == WORKSPACE and _quant(L, tr=1, ws=C.c_void_p(0x1004)) == WORKSPACE
    need = L.gq_quantize_i8_workspace_bytes(10, 20, 1)
    assert need >= 80 and _quant(L, tr=1, wsb=need - 1) == WORKSPACE
    assert L.gq_quantize_i8_workspace_bytes(10, 20, 0) == 0
    assert _quant(L, n=0, X=None, Q=None, S=None) == 0


def _gemm(L, A=FAKE, m=10, lda=32, sa=FAKE, B=FAKE, n=20, ldb=32, sb=FAKE, k=30, bias=None, act=0, Cp=FAKE, ty=0,
          ldc=20, ws=FAKE, wsb=1 << 40, err=None):
    return L.gq_gemm_i8(A, m, lda, sa, B, n, ldb, sb, k, bias, act, Cp, ty, ldc, ws, wsb, err, None)


@pytest.mark.parametrize("kw", [dict(m=-1), dict(n=0), dict(k=0), dict(ty=5), dict(act=2), dict(act=-1), dict(lda=16),
                                dict(lda=40), dict(ldb=16), dict(ldb=33), dict(ldc=19), dict(A=None), dict(B=None),
                                dict(Cp=None), dict(sa=None), dict(sb=None), dict(A=C.c_void_p(0x1008)),
                                dict(B=C.c_void_p(0x1004)), dict(Cp=ODD), dict(ty=1, Cp=BYTE), dict(sa=ODD), dict(sb=ODD),
                                dict(bias=ODD), dict(err=ODD)])
def test_gemm_refuses(L, kw):
    assert _gemm(L, **kw) == INVALID


def test_gemm_limits(L):
    big = (1 << 30) + 16
    assert _gemm(L, m=big) == UNSUPPORTED and _gemm(L, n=big, ldc=big) == UNSUPPORTED
    assert _gemm(L, k=big, lda=big, ldb=big) == UNSUPPORTED
    assert _gemm(L, m=0, A=None, B=None, Cp=None) == 0
    need = L.gq_gemm_i8_workspace_bytes(100, 100, 1 << 20)
    assert need >= 16 * 100 * 100 * 4  # sums of at most 65,536 products
    big = dict(m=100, n=100, k=1 << 20, lda=1 << 20, ldb=1 << 20, ldc=100)
    assert _gemm(L, **big, wsb=need - 1) == WORKSPACE and _gemm(L, **big, ws=None) == WORKSPACE
    assert L.gq_gemm_i8_workspace_bytes(0, 5, 5) == 0 and L.gq_gemm_i8_workspace_bytes(5, 5, 0) == 0


def _linear(L, X=FAKE, ty=0, n=10, k=30, ldx=30, W=FAKE, out=20, ldw=32, sw=FAKE, bias=None, act=0, Y=FAKE, yt=0,
            ldy=20, ws=FAKE, wsb=1 << 40, err=None):
    return L.gq_linear_i8(X, ty, n, k, ldx, W, out, ldw, sw, bias, act, Y, yt, ldy, ws, wsb, err, None)


@pytest.mark.parametrize("kw", [dict(ty=3), dict(yt=3), dict(n=-1), dict(k=0), dict(out=0), dict(ldx=29), dict(ldw=16),
                                dict(ldw=36), dict(ldy=19), dict(act=2), dict(X=None), dict(W=None), dict(Y=None),
                                dict(sw=None), dict(X=ODD), dict(W=C.c_void_p(0x1008)), dict(Y=ODD), dict(sw=ODD),
                                dict(bias=ODD), dict(err=ODD)])
def test_linear_refuses(L, kw):
    assert _linear(L, **kw) == INVALID


def test_linear_workspace(L):
    need = L.gq_linear_i8_workspace_bytes(10, 30, 20)
    assert need > 0
    assert _linear(L, ws=None) == WORKSPACE and _linear(L, ws=C.c_void_p(0x1010)) == WORKSPACE
    assert _linear(L, wsb=need - 1) == WORKSPACE
    assert _linear(L, n=0, X=None, W=None, Y=None, ws=None) == 0
    assert L.gq_linear_i8_workspace_bytes(0, 30, 20) == 0


def _bwd(L, dY=FAKE, lddy=20, X=FAKE, ldx=30, ty=0, n=10, k=30, out=20, W=FAKE, wt=0, ldw=30, dX=FAKE, dxt=0, lddx=30,
         dW=FAKE, dwt=0, lddw=30, db=FAKE, ws=FAKE, wsb=1 << 40, err=None):
    return L.gq_linear_i8_bwd(dY, lddy, X, ldx, ty, n, k, out, W, wt, ldw, dX, dxt, lddx, dW, dwt, lddw, db, ws, wsb, err,
                              None)


@pytest.mark.parametrize("kw", [dict(ty=4), dict(n=-1), dict(k=0), dict(out=0), dict(lddy=19), dict(ldx=29), dict(ldw=29),
                                dict(lddx=29), dict(lddw=29), dict(wt=3), dict(dxt=3), dict(dwt=-1), dict(dY=None),
                                dict(X=None), dict(W=None), dict(dY=ODD), dict(X=ODD), dict(W=ODD), dict(dX=ODD),
                                dict(dW=ODD), dict(db=ODD), dict(err=ODD), dict(dW=None)])
def test_linear_bwd_refuses(L, kw):
    assert _bwd(L, **kw) == INVALID


def test_linear_bwd_workspace(L):
    need = L.gq_linear_i8_bwd_workspace_bytes(10, 30, 20, 1, 1)
    assert need >= L.gq_linear_i8_bwd_workspace_bytes(10, 30, 20, 0, 1) > 0
    assert _bwd(L, wsb=need - 1) == WORKSPACE and _bwd(L, ws=None) == WORKSPACE
    assert _bwd(L, n=0, dY=None, X=None, dX=None, dW=None, db=None, ws=None) == 0
    assert _bwd(L, dX=None, dW=None, db=None, ws=None) == 0


# -------------------------------------------------------------- group norm --


def _fwd(L, X=FAKE, ty=0, n=10, d=12, ldx=12, groups=3, ptr=FAKE, s=2, mr=0, ga=None, be=None, eps=1e-5, act=0, Y=FAKE,
         ldy=12, mean=FAKE, rstd=FAKE, ws=FAKE, wsb=1 << 40):
    return L.gq_group_norm_fwd(X, ty, n, d, ldx, groups, ptr, s, mr, ga, be, eps, act, Y, ldy, mean, rstd, ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(ty=3), dict(n=-1), dict(d=0), dict(groups=0), dict(groups=5), dict(s=-1),
                                dict(mr=-1), dict(act=3), dict(act=-1), dict(ptr=None), dict(ptr=C.c_void_p(0x1004)),
                                dict(ldx=11), dict(ldy=11), dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(X=None),
                                dict(Y=None), dict(mean=None), dict(rstd=None), dict(X=ODD), dict(Y=ODD), dict(mean=ODD),
                                dict(ga=ODD), dict(be=ODD), dict(ty=1, X=BYTE)])
def test_group_norm_fwd_refuses(L, kw):
    assert _fwd(L, **kw) == INVALID


def test_group_norm_limits(L):
    assert _fwd(L, d=16386, ldx=16386, ldy=16386) == UNSUPPORTED
    assert _fwd(L, n=(1 << 31) + 1) == UNSUPPORTED and _fwd(L, s=(1 << 30) + 1) == UNSUPPORTED
    assert _fwd(L, s=1 << 30, groups=3) == UNSUPPORTED
    assert _fwd(L, s=0) == 0
    long = dict(n=1 << 20, d=12, groups=3)
    need = L.gq_group_norm_workspace_bytes(1 << 20, 12, 3, 0, 2, 0, 0)
    assert need > 0 and _fwd(L, **long, wsb=need - 1) == WORKSPACE and _fwd(L, **long, ws=None) == WORKSPACE
    assert L.gq_group_norm_workspace_bytes(10, 16385, 1, 0, 1, 0, 0) == 0


def _gbwd(L, dY=FAKE, lddy=12, X=FAKE, ldx=12, ty=0, n=10, d=12, groups=3, ptr=FAKE, s=2, mr=0, mean=FAKE, rstd=FAKE,
          ga=None, be=None, act=0, dX=FAKE, lddx=12, dg=FAKE, db=FAKE, ws=FAKE, wsb=1 << 40):
    return L.gq_group_norm_bwd(dY, lddy, X, ldx, ty, n, d, groups, ptr, s, mr, mean, rstd, ga, be, act, dX, lddx, dg, db,
                               ws, wsb, None)


@pytest.mark.parametrize("kw", [dict(ty=3), dict(n=-1), dict(d=0), dict(groups=7), dict(act=4), dict(ptr=None),
                                dict(lddy=11), dict(ldx=11), dict(lddx=11), dict(dY=None), dict(X=None), dict(dX=None),
                                dict(mean=None), dict(rstd=None), dict(dY=ODD), dict(dX=ODD), dict(dg=ODD), dict(db=ODD),
                                dict(ga=ODD), dict(be=ODD)])
def test_group_norm_bwd_refuses(L, kw):
    assert _gbwd(L, **kw) == INVALID


def test_group_norm_bwd_workspace(L):
    need = L.gq_group_norm_workspace_bytes(10, 12, 3, 0, 2, 0, 1)
    assert need > 0 and _gbwd(L, wsb=need - 1) == WORKSPACE and _gbwd(L, ws=None) == WORKSPACE
    assert _gbwd(L, n=0, dY=None, X=None, dX=None, dg=None, db=None, ws=None) == 0
