"""Layer normalization and dropout on the GPU against the oracle's float64
forms.  u = 2^-24 is half a step of fp32; a stored result is off by at most
half a step of its type relative to its value (eps_t / 2).

The kernels add at most 16 values of a lane in sequence and then combine 32
lanes and up to 32 warps pairwise: at most 16 + 5 + 5 roundings per row sum,
27 with the division by d.  With A = max|x| of a row:
  mean:  27 u A
  rstd:  relative 27 u A rstd + 18 u  (the variance is off by 2 * 27 u A sd
         from the mean's error, 27 + 2 roundings of its own sum, halved by the
         root; two more for root and division)
  y:     u |gamma| A rstd 27 (1 + |xhat|) + 24 u |xhat gamma| + 2 u |y|
  dx:    rstd u (6 |g| + 34 mean|g| + 40 |xhat| mean|g xhat|)
  dgamma, dbeta: the chain of a lane's rows, then shuffles, warps and blocks:
         (rows of a lane + 100) u sum|dz xhat|, sum|dz|"""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _mat(n, d, pad, dtype, seed, mul=1.0, off=0.0):
    buf = torch.full((n, d + pad), 77.0, dtype=dtype, device="cuda")
    x = synth.normal_matrix(n, d, seed=seed, device="cuda") * mul
    x = x + off * synth.normal_matrix(n, 1, seed=seed + 1, device="cuda")
    buf[:, :d] = x.to(dtype)
    return buf, buf[:, :d]


def _np(t):
    return t.double().cpu().numpy()


def _half_step(dtype, ref):
    # types below the smallest normal number have an absolute step
    return torch.finfo(dtype).eps / 2 * np.maximum(np.abs(ref), torch.finfo(dtype).tiny)


def _within(got, ref, tol, what):
    e = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and e.max() <= 0, f"{what}: {e.max()} over the bound at " \
        f"{np.unravel_index(np.argmax(e), e.shape)}"


def _fwd_tol(f, X, gamma, scale, dtype):
    A = np.abs(X).max(1, keepdims=True)
    r = f["rstd"][:, None]
    xh = (X - f["mean"][:, None]) * r
    g = np.abs(np.ones(X.shape[1]) if gamma is None else gamma)
    t = U * (g * A * r * 27 * (1 + np.abs(xh)) + 24 * np.abs(xh * g) + 2 * np.abs(f["z"]))
    return scale * t + 2 * U * np.abs(f["Y"]) + _half_step(dtype, f["Y"]) * (1 + 1e-3)


def _unpack(bits, n, d):
    w = bits.cpu().numpy().view(np.uint32)
    c = np.arange(d)
    return ((w[:, c // 32] >> (c % 32).astype(np.uint32)) & 1).astype(bool)


WIDTHS = [1, 2, 7, 31, 32, 33, 47, 64, 100, 128, 129, 256, 257, 300, 512, 513, 1000, 2048, 4099, 8192, 16384]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_layer_norm_forward_and_backward(orc, d, dtype, pad):
    q = gq()
    t = TYPES[dtype]
    n = 1 if d == 31 else (37 if d > 600 else 333)
    p, seed, eps = (0.3, 0xABCDEF0123456789, 1e-5) if d % 2 else (0.0, 0, 1e-3)
    relu = d % 3 != 0
    xb, x = _mat(n, d, pad, t, seed=d, mul=0.7, off=1.0)
    _, dy = _mat(n, d, pad, t, seed=d + 5)
    gamma = 1 + 0.3 * synth.normal_matrix(1, d, seed=d + 7, device="cuda")[0]
    beta = 0.3 * synth.normal_matrix(1, d, seed=d + 8, device="cuda")[0]
    act = q.ACT_RELU if relu else q.ACT_NONE
    bits = torch.full((n, (d + 31) // 32), -1, dtype=torch.int32, device="cuda") if relu else None
    yb = torch.full((n, d + pad), 55.0, dtype=t, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(x, gamma, beta, eps, act=act, p=p, seed=seed, out=yb[:, :d], relu_bits=bits)
    assert (yb[:, d:] == 55).all(), "columns past d are not written"
    X, G, B = _np(x), _np(gamma), _np(beta)
    f = orc.layer_norm_fwd(X, G, B, eps, relu, p, seed)
    A = np.abs(X).max(1)
    _within(_np(mean), f["mean"], 27 * U * A + U * np.abs(f["mean"]), "mean")
    # the bound is first order in the error of the variance; a variance far
    # below eps leaves rstd at 1 / sqrt(eps)
    r_tol = np.minimum(27 * U * A * f["rstd"], 0.5) + 18 * U
    _within(_np(rstd), f["rstd"], r_tol * f["rstd"], "rstd")
    tol = _fwd_tol(f, X, G, 1.0 / (1.0 - p), t)
    _within(_np(y), f["Y"], tol, "y")
    if relu:
        on = _unpack(bits, n, d)
        z_tol = _fwd_tol(dict(f, Y=0 * f["Y"]), X, G, 1.0, torch.float32)
        wrong = (on != f["on"]) & (np.abs(f["z"]) > z_tol)
        assert not wrong.any()
        assert (bits.cpu().numpy().view(np.uint32)[:, -1] >> np.uint64((d - 1) % 32) >> np.uint64(1) == 0).all()
    # backward, from the statistics and bits the forward pass wrote
    dxb = torch.full((n, d + pad), 33.0, dtype=t, device="cuda")
    dx, dgamma, dbeta = q.layer_norm_bwd(dy, x, mean, rstd, gamma, act=act, p=p, seed=seed, relu_bits=bits,
                                         dX=dxb[:, :d])
    assert (dxb[:, d:] == 33).all()
    b = orc.layer_norm_bwd(_np(dy), X, _np(mean), _np(rstd), G, on if relu else None, p, seed)
    g, xh, R = np.abs(b["g"]), np.abs(b["xhat"]), _np(rstd)[:, None]
    tol = R * U * (6 * g + 34 * g.mean(1, keepdims=True) + 40 * xh * (g * xh).mean(1, keepdims=True))
    _within(_np(dx), b["dX"], tol + _half_step(t, b["dX"]) * (1 + 1e-3), "dx")
    rows = n + 100
    _within(_np(dgamma), b["dgamma"], rows * U * (np.abs(b["dz"]) * xh).sum(0), "dgamma")
    _within(_np(dbeta), b["dbeta"], rows * U * np.abs(b["dz"]).sum(0), "dbeta")


@pytest.mark.parametrize("n,d", [(100_003, 64), (70_001, 256), (5000, 1024), (20_011, 47)])
def test_many_rows_per_lane(orc, n, d):
    """More rows than the grid has groups, and the bf16 gradient of fp32 rows."""
    q = gq()
    _, x = _mat(n, d, 0, torch.float32, seed=3, off=0.5)
    _, dy = _mat(n, d, 0, torch.float32, seed=4)
    gamma = 1 + 0.2 * synth.normal_matrix(1, d, seed=5, device="cuda")[0]
    y, mean, rstd = q.layer_norm_fwd(x, gamma, None, p=0.5, seed=9)
    f = orc.layer_norm_fwd(_np(x), _np(gamma), None, 1e-5, False, 0.5, 9)
    _within(_np(y), f["Y"], _fwd_tol(f, _np(x), _np(gamma), 2.0, torch.float32), "y")
    dx, dgamma, dbeta = q.layer_norm_bwd(dy, x, mean, rstd, gamma, p=0.5, seed=9)
    ld8 = (d + 7) // 8 * 8
    dz = torch.zeros(n, ld8, dtype=torch.bfloat16, device="cuda")
    q.layer_norm_bwd(dy, x, mean, rstd, gamma, p=0.5, seed=9, dX=dz[:, :d])
    assert torch.equal(dz[:, :d], dx.to(torch.bfloat16)) and not dz[:, d:].any()
    b = orc.layer_norm_bwd(_np(dy), _np(x), _np(mean), _np(rstd), _np(gamma), None, 0.5, 9)
    rows = n // 100 + 100  # 152 SMs x 4 blocks x 8 warps take more than 100 rows at a time
    _within(_np(dgamma), b["dgamma"], rows * U * np.abs(b["dz"] * b["xhat"]).sum(0), "dgamma")
    _within(_np(dbeta), b["dbeta"], rows * U * np.abs(b["dz"]).sum(0), "dbeta")
    again = q.layer_norm_bwd(dy, x, mean, rstd, gamma, p=0.5, seed=9)
    assert all(torch.equal(s, t) for s, t in zip((dx, dgamma, dbeta), again))


def test_large_mean_small_spread(orc):
    # the variance is summed over the centred row: a mean 1000 times the
    # spread costs the digits of x itself only
    q = gq()
    x = 1000.0 + synth.normal_matrix(64, 256, seed=1, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(x)
    f = orc.layer_norm_fwd(_np(x))
    _within(_np(y), f["Y"], _fwd_tol(f, _np(x), None, 1.0, torch.float32), "y")
    assert np.abs(_np(rstd) / f["rstd"] - 1).max() < 1e-4


def test_constant_and_empty_rows():
    q = gq()
    x = torch.full((5, 40), 2.5, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(x, None, torch.arange(40.0, device="cuda"))
    assert torch.equal(y, torch.arange(40.0, device="cuda").expand(5, 40)) and (mean == 2.5).all()
    dx, dg, db = q.layer_norm_bwd(torch.ones_like(x), x, mean, rstd)
    assert not dx.any() and not dg.any() and (db == 5).all()
    e = torch.empty(0, 40, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(e)
    dg = torch.full((40,), 9.0, device="cuda")
    dx, dg, db = q.layer_norm_bwd(e, e, mean, rstd, dgamma=dg)
    assert y.shape == (0, 40) and not dg.any() and not db.any()
    assert q.dropout(e, 0.5, 1).shape == (0, 40)


def test_rows_with_nan_stay_to_themselves():
    q = gq()
    x = synth.normal_matrix(9, 100, seed=1, device="cuda")
    ref = q.layer_norm_fwd(x)[0]
    x[4, 50] = float("nan")
    y = q.layer_norm_fwd(x)[0]
    keep = torch.arange(9, device="cuda") != 4
    assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[4]).all()


def test_in_place(orc):
    q = gq()
    x = synth.normal_matrix(50, 96, seed=2, device="cuda")
    ref, mean, rstd = q.layer_norm_fwd(x, p=0.2, seed=4)
    dy = synth.normal_matrix(50, 96, seed=3, device="cuda")
    dref = q.layer_norm_bwd(dy, x, mean, rstd, p=0.2, seed=4)[0]
    assert torch.equal(q.layer_norm_bwd(dy, x, mean, rstd, p=0.2, seed=4, dX=dy)[0], dref)
    assert torch.equal(q.layer_norm_fwd(x, p=0.2, seed=4, out=x)[0], ref)
    z = q.dropout(ref, 0.5, 8)
    assert torch.equal(q.dropout(ref, 0.5, 8, out=ref), z)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (1000, 1, 0), (333, 4, 0), (77, 47, 1), (77, 47, 0), (65, 256, 0),
                                     (10, 1000, 3), (3, 4099, 5), (2, 20000, 0)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.6, 1.0])
def test_dropout(orc, n, d, pad, dtype, p):
    q = gq()
    t = TYPES[dtype]
    _, x = _mat(n, d, pad, t, seed=n + d)
    seed = 0x9876543210FEDCBA
    yb = torch.full((n, d + pad), 5.0, dtype=t, device="cuda")
    y = q.dropout(x, p, seed, out=yb[:, :d])
    assert (yb[:, d:] == 5).all()
    # one fp32 product with the fp32 scale, rounded once: exact
    s = np.float32(1.0 / (1.0 - p)) if p < 1 else np.float32(0)
    keep = torch.from_numpy(orc.kept(seed, n, d, p)).cuda()
    ref = torch.where(keep, x.float() * float(s), torch.zeros((), device="cuda")).to(t)
    assert torch.equal(y, ref)


def test_dropout_hides_nan_and_rate():
    q = gq()
    x = torch.full((200, 500), float("nan"), device="cuda")
    y = q.dropout(x, 0.5, 3)
    dropped = ~torch.isnan(y)
    assert (y[dropped] == 0).all() and not torch.signbit(y[dropped]).any()
    assert abs(dropped.float().mean().item() - 0.5) < 6 * 0.5 / np.sqrt(x.numel())
    # another seed, another mask
    assert not torch.equal(torch.isnan(q.dropout(x, 0.5, 4)), torch.isnan(y))


def test_offsets_past_32_bits():
    # the last rows of a matrix of more than 2^32 elements
    q = gq()
    n, d = (1 << 24) + 70, 260
    x = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda")
    x[-1].fill_(1.0)
    x[-1, 0] = 3.0
    y = q.dropout(x, 0.25, 6, out=x)
    tail = y[-1].float().cpu()
    assert set(tail[1:].unique().tolist()) == {0.0, float(torch.tensor(4 / 3).bfloat16())}
    z, mean, _ = q.layer_norm_fwd(y, out=y)
    assert torch.isfinite(z[-1].float()).all() and abs(mean[-1].item() - tail.mean().item()) < 1e-6
    del x, y, z
    torch.cuda.empty_cache()


def test_captured_and_replayed():
    q = gq()
    x = synth.normal_matrix(1000, 200, seed=1, device="cuda")
    dy = synth.normal_matrix(1000, 200, seed=2, device="cuda")
    ws = q.Workspace()
    side = torch.cuda.Stream()

    def step():
        y, mean, rstd = q.layer_norm_fwd(x, p=0.5, seed=2)
        return (y, *q.layer_norm_bwd(dy, x, mean, rstd, p=0.5, seed=2, ws=ws), q.dropout(y, 0.1, 7))

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(synth.normal_matrix(1000, 200, seed=5, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, step()))


def test_refusals_of_the_binding():
    q = gq()
    x = torch.zeros(4, 8, device="cuda")
    m = torch.zeros(4, device="cuda")
    for call in (lambda: q.dropout(x, 1.5, 0), lambda: q.dropout(x, float("nan"), 0), lambda: q.dropout(x.int(), 0.5, 0),
                 lambda: q.dropout(x.t(), 0.5, 0), lambda: q.dropout(x, 0.5, 0, out=x.bfloat16()),
                 lambda: q.dropout(x.cpu(), 0.5, 0), lambda: q.layer_norm_fwd(x, gamma=m),
                 lambda: q.layer_norm_fwd(x, eps=-1.0), lambda: q.layer_norm_fwd(x, act=7),
                 lambda: q.layer_norm_fwd(x, relu_bits=torch.zeros(4, 1, dtype=torch.int32, device="cuda")),
                 lambda: q.layer_norm_fwd(torch.zeros(1, 16385, device="cuda")),
                 lambda: q.layer_norm_bwd(x, x, m, m, act=q.ACT_RELU),
                 lambda: q.layer_norm_bwd(x[:3], x, m, m), lambda: q.layer_norm_bwd(x, x, m[:3], m),
                 lambda: q.layer_norm_bwd(x, x, m, m, dX=x.half())):
        with pytest.raises(q.GQError):
            call()


def test_overflowing_variance_is_not_nan():
    # squares beyond fp32: the variance is infinite, 1 / sqrt of it 0
    q = gq()
    for d in (64, 100, 1000):
        x = synth.normal_matrix(3, d, seed=1, device="cuda") * 1e25
        beta = torch.ones(d, device="cuda")
        y, mean, rstd = q.layer_norm_fwd(x, None, beta)
        assert (rstd == 0).all() and (y == 1).all() and torch.isfinite(mean).all()


@pytest.mark.parametrize("d", [17, 64, 300, 700, 2000])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_that_start_anywhere(d, dtype):
    """Column slices, whose rows start off the 16-byte grid, give bit for bit
    what aligned copies give (sums run over the same lanes' columns in another
    order: only what is elementwise is compared exactly, the rest by norm)."""
    q = gq()
    t = TYPES[dtype]
    buf, _ = _mat(45, d + 9, 0, t, seed=d, off=0.5)
    dbuf, _ = _mat(45, d + 9, 0, t, seed=d + 1)
    x, dy = buf[:, 3:3 + d], dbuf[:, 5:5 + d]
    assert torch.equal(q.dropout(x, 0.3, 5), q.dropout(x.contiguous(), 0.3, 5))
    a = q.layer_norm_fwd(x, p=0.3, seed=5)
    b = q.layer_norm_fwd(x.contiguous(), p=0.3, seed=5)
    ga = q.layer_norm_bwd(dy, x, a[1], a[2], p=0.3, seed=5)
    gb = q.layer_norm_bwd(dy.contiguous(), x.contiguous(), a[1], a[2], p=0.3, seed=5)
    # one rounding of the type, and 40 of fp32 (the row sums' orders differ)
    tol = torch.finfo(t).eps + 40 * U
    for u, v in zip(a + ga, b + gb):
        u, v = u.double(), v.double()
        assert torch.linalg.norm(u - v) <= tol * torch.linalg.norm(v)


@pytest.mark.parametrize("d", [40, 600, 9000])
def test_everything_dropped_and_one_row(d):
    q = gq()
    x = synth.normal_matrix(1, d, seed=1, device="cuda")
    dy = synth.normal_matrix(1, d, seed=2, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(x, beta=torch.ones(d, device="cuda"), p=1.0, seed=3)
    assert not y.any() and abs(mean.item() - x.double().mean().item()) < 1e-6
    dx, dg, db = q.layer_norm_bwd(dy, x, mean, rstd, p=1.0, seed=3)
    assert not dx.any() and not dg.any() and not db.any()
    # one row: dgamma and dbeta are the row's own terms
    dx, dg, db = q.layer_norm_bwd(dy, x, mean, rstd)
    assert torch.equal(db, dy[0])
    xh = ((x.double() - mean.double()) * rstd.double())[0]
    assert (dg.double() - dy[0].double() * xh).abs().max() <= 4 * U * (dy[0].double() * xh).abs().max()


@pytest.mark.parametrize("d", [64, 100, 2000, 10000])
def test_without_weight_gradients(d):
    """gq_layer_norm_bwd with NULL dgamma and dbeta needs no workspace."""
    q = gq()
    x = synth.normal_matrix(70, d, seed=1, device="cuda")
    dy = synth.normal_matrix(70, d, seed=2, device="cuda")
    _, mean, rstd = q.layer_norm_fwd(x)
    ref, dg, db = q.layer_norm_bwd(dy, x, mean, rstd)
    dx = torch.empty_like(x)
    p = q._ptr
    q._check(q.lib().gq_layer_norm_bwd(p(dy), d, p(x), d, q.F32, 70, d, p(mean), p(rstd), None, q.ACT_NONE, 0.0, 0,
                                       None, 0, p(dx), q.F32, d, None, None, None, 0, q._stream()), "bwd")
    assert torch.equal(dx, ref)
    # one of the two
    only = torch.empty(d, device="cuda")
    ws = torch.empty(int(q.lib().gq_layer_norm_bwd_workspace_bytes(70, d)), dtype=torch.uint8, device="cuda")
    q._check(q.lib().gq_layer_norm_bwd(p(dy), d, p(x), d, q.F32, 70, d, p(mean), p(rstd), None, q.ACT_NONE, 0.0, 0,
                                       None, 0, p(dx), q.F32, d, None, p(only), p(ws), ws.numel(), q._stream()), "bwd")
    assert torch.equal(only, db)


def test_two_streams_at_once():
    q = gq()
    x = synth.normal_matrix(20000, 256, seed=1, device="cuda")
    dy = synth.normal_matrix(20000, 256, seed=2, device="cuda")
    y, mean, rstd = q.layer_norm_fwd(x, p=0.2, seed=1)
    ref = q.layer_norm_bwd(dy, x, mean, rstd, p=0.2, seed=1)
    torch.cuda.synchronize()
    outs = []
    for st in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(st):
            for _ in range(3):
                a = q.layer_norm_fwd(x, p=0.2, seed=1)
                outs.append((a[0], *q.layer_norm_bwd(dy, x, a[1], a[2], p=0.2, seed=1)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, (y, *ref)))
