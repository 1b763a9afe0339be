"""Group normalization of segments of rows against the formulas in 64 bits.
u = 2^-24.  For a segment and group with mean m, D = max |x - m|:

  K   the roundings that a value meets on its way through the sums of a segment:
      its thread's rows, the threads of its channel and the group's channels:
      at most rows + K2 for a segment that one block takes; for one cut into
      chunks rows / 2,368 (16 chunks for each of 148 SMs) + 5 of a thread,
      5 channels-of-a-group + 21 where they are combined
  K2  threads of a channel (256 threads of at least one channel each; 4096 / d + 1
      is more) and the lanes' sum over a group's channels: + cg / 32 + 48
  mean:  e_m = u (2 K D + (2 K2 + 8) (|m| + D))    (shifted values, then parts' means)
  var:   e_v = 4 u (K + K2 + 20) D^2 + 2 D e_m + e_m^2
  rstd:  e_r = e_v / (2 (var + eps)) + 3u, relative
  z:     |gamma| rstd e_m + |gamma xhat| (e_r + 4u) + 2u |z|
  y:     SiLU has slope <= 1.1 and costs u (8 + 2 |z|) |y| itself; half a step of the type
backward, from the stored statistics:
  xhat 2u, z_e = 2u |xhat gamma| + u |z|, act' off by z_e / 2 + u (10 + 4 |z|)
  dz_e = |dy| of that + u |dz|;  h_e = |gamma| dz_e + u |h|
  dx:  rstd (h_e + mean(h_e) + K u mean|h| + |xhat| (mean(h_e |xhat|) + (K + 3) u mean|h xhat|)
       + 4u (|h| + |mean h| + |xhat mean(h xhat)|)), half a step of the type
  dgamma, dbeta: sums of dz_e |xhat| and dz_e, and (K + 2 + 300) u of the absolute sums
       (300: the blocks' or chunks' sums, at most 2,432 / 32 + 32 in a row, segments
       of a block among them)"""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = {"none": 0, "relu": 1, "silu": 2}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _matrix(n, d, pad, t, seed, off=0.0, fill=7.0):
    buf = torch.full((n, d + pad), fill, dtype=t, device="cuda")
    x = torch.randn(n, d, device="cuda", generator=_gen(seed))
    buf[:, :d] = x * (0.5 + torch.rand(n, 1, device="cuda", generator=_gen(seed + 1))) + off
    return buf[:, :d]


def _half(t, x):
    return torch.finfo(t).eps / 2 * x.abs().clamp(min=torch.finfo(t).tiny) * 1.01


def _within(got, want, tol, what):
    if got.numel() == 0:
        return
    bad = (got.double() - want).abs() - tol
    assert torch.isfinite(got).all() and bad.max() <= 0, f"{what}: {bad.max().item()} over the bound at {bad.argmax().item()}"


def _check(q, x, dy, ptr, groups, gamma, beta, act, eps=1e-5, max_rows=0, long_=False, inplace=False):
    """Both passes, every segment."""
    n, d = x.shape
    cg = d // groups
    t = x.dtype
    s = 1 if ptr is None else ptr.numel() - 1
    a = ACTS[act]
    y0 = None
    if inplace:
        y0 = x.clone() if x.is_contiguous() else torch.empty_strided(x.shape, x.stride(), dtype=t, device="cuda").copy_(x)
    y, mean, rstd = q.group_norm_fwd(x if not inplace else y0, groups, ptr, gamma, beta, eps, act=a, max_rows=max_rows,
                                     out=y0)
    g0 = dy.clone() if inplace else None
    dx, dgamma, dbeta = q.group_norm_bwd(dy if not inplace else g0, x, groups, mean, rstd, ptr, gamma, beta, act=a,
                                         max_rows=max_rows, dX=g0)
    assert mean.shape == (s, groups)
    G = (torch.ones(d, device="cuda") if gamma is None else gamma).double()
    B = (torch.zeros(d, device="cuda") if beta is None else beta).double()
    DG, DB, GT, BT = (torch.zeros(d, dtype=torch.float64, device="cuda") for _ in range(4))
    edges = [0, n] if ptr is None else ptr.tolist()
    K2 = min(512, 4096 // d + 1) + cg / 32 + 48
    for j in range(s):
        r0, r1 = edges[j], edges[j + 1]
        if r1 == r0:
            assert not mean[j].any() and torch.allclose(rstd[j], torch.full_like(rstd[j], eps ** -0.5), rtol=4 * U)
            continue
        rows = r1 - r0
        K = rows / 2368 + 26 + 5 * cg + K2 if long_ else rows + K2
        X = x[r0:r1].double().view(rows, groups, cg)
        m = X.mean((0, 2), keepdim=True)
        var = (X - m).square().mean((0, 2), keepdim=True)
        D = (X - m).abs().amax((0, 2), keepdim=True)
        r = 1 / torch.sqrt(var + eps)
        e_m = U * (2 * K * D + (2 * K2 + 8) * (m.abs() + D))
        e_v = 4 * U * (K + K2 + 20) * D * D + 2 * D * e_m + e_m * e_m
        e_r = e_v / (2 * (var + eps)) + 3 * U
        _within(mean[j], m.view(-1), e_m.view(-1), f"mean {j}")
        _within(rstd[j], r.view(-1), (e_r * r).view(-1), f"rstd {j}")
        Gv, Bv = G.view(1, groups, cg), B.view(1, groups, cg)
        xh = (X - m) * r
        z = xh * Gv + Bv
        z_e = Gv.abs() * r * e_m + (Gv * xh).abs() * (e_r + 4 * U) + 2 * U * z.abs()
        Y = z if act == "none" else z.clamp(min=0) if act == "relu" else z * torch.sigmoid(z)
        _within(y[r0:r1].reshape(X.shape), Y, 1.1 * z_e + U * (8 + 2 * z.abs()) * Y.abs() + _half(t, Y), f"y {j}")
        # backward from the stored statistics
        m, r = mean[j].double().view(1, groups, 1), rstd[j].double().view(1, groups, 1)
        xh = (X - m) * r
        z = xh * Gv + Bv
        z_e = 2 * U * (xh * Gv).abs() + U * z.abs()
        dY = dy[r0:r1].double().view(X.shape)
        sg = torch.sigmoid(z)
        slope = torch.ones_like(z) if act == "none" else (z > 0).double() if act == "relu" else sg * (1 + z * (1 - sg))
        if act == "relu":
            dY = dY.clone()
            assert not (z.abs() <= z_e).any(), "an input at the ReLU's edge decides nothing"
        dz = dY * slope
        dz_e = U * dz.abs() + (dY.abs() * (z_e / 2 + U * (10 + 4 * z.abs())) if act == "silu" else 0)
        h, h_e = dz * Gv, Gv.abs() * dz_e + U * (dz * Gv).abs()
        mn = lambda v: v.mean((0, 2), keepdim=True)
        h1, h2 = mn(h), mn(h * xh)
        dX = r * (h - h1 - xh * h2)
        tol = r * (h_e + mn(h_e) + K * U * mn(h.abs()) + xh.abs() * (mn(h_e * xh.abs()) + (K + 3) * U * mn((h * xh).abs()))
                   + 4 * U * (h.abs() + h1.abs() + (xh * h2).abs()))
        _within(dx[r0:r1].reshape(X.shape), dX, tol + _half(t, dX), f"dx {j}")
        DG += (dz * xh).sum(0).view(-1)
        DB += dz.sum(0).view(-1)
        GT += ((dz_e * xh.abs()) + (K + 302) * U * (dz * xh).abs()).sum(0).view(-1)
        BT += (dz_e + (K + 302) * U * dz.abs()).sum(0).view(-1)
    _within(dgamma, DG, GT, "dgamma")
    _within(dbeta, DB, BT, "dbeta")
    return y, dx


def _weights(d):
    return (1 + 0.3 * torch.randn(d, device="cuda", generator=_gen(91)),
            0.3 * torch.randn(d, device="cuda", generator=_gen(92)))


def _ptr(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("d,groups,pad,act", [(1, 1, 0, "none"), (8, 8, 0, "silu"), (47, 1, 1, "relu"), (64, 8, 0, "silu"),
                                              (255, 5, 2, "none"), (256, 32, 0, "silu"), (96, 3, 8, "relu"),
                                              (1000, 4, 0, "silu"), (2048, 2, 0, "none"), (4100, 41, 0, "silu"),
                                              (6000, 1, 3, "silu")])
def test_short_segments(d, groups, pad, act, t):
    """Graphs of 0 to 90 rows, one block each."""
    q = gq()
    lengths = [0, 1, 2, 31, 90, 0, 0, 17, 64, 5, 0]
    n = sum(lengths)
    x, dy = _matrix(n, d, pad, TYPES[t], d, off=1.5), _matrix(n, d, pad, TYPES[t], d + 7)
    _check(q, x, dy, _ptr(lengths), groups, *_weights(d), act, max_rows=90)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("d,groups,pad,act", [(16, 2, 0, "silu"), (47, 47, 1, "none"), (256, 16, 0, "silu"),
                                              (256, 1, 0, "relu"), (1100, 11, 0, "silu"), (2304, 3, 1, "none")])
def test_one_long_segment(d, groups, pad, act, t):
    q = gq()
    n = 2 * (1 << 20) // d + 1000  # more than a block takes
    x, dy = _matrix(n, d, pad, TYPES[t], d, off=-0.7), _matrix(n, d, pad, TYPES[t], d + 3)
    slabs = -(-d // (256 if d % 8 or pad % 8 else 1024))
    _check(q, x, dy, None, groups, *_weights(d), act, long_=slabs == 1)


@pytest.mark.parametrize("hint", [0, 20000, 7])
@pytest.mark.parametrize("d,groups,t", [(64, 4, "f32"), (72, 9, "bf16"), (33, 3, "f16")])
def test_uneven_segments(d, groups, t, hint):
    """Long, short and empty segments in one call, with each hint: none, the
    right one, and one that is far too small."""
    q = gq()
    lengths = [3, 0, 20000, 1, 0, 0, 500, 2, 9000, 1, 1, 1, 0, 64]
    n = sum(lengths)
    x, dy = _matrix(n, d, 0, TYPES[t], 5, off=0.3), _matrix(n, d, 0, TYPES[t], 6)
    _check(q, x, dy, _ptr(lengths), groups, *_weights(d), "silu", max_rows=hint)


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_many_segments(t):
    q = gq()
    lengths = [(i * 7) % 13 for i in range(3000)]
    n = sum(lengths)
    x, dy = _matrix(n, 32, 0, TYPES[t], 1), _matrix(n, 32, 0, TYPES[t], 2)
    ptr = _ptr(lengths)
    _check(q, x, dy, ptr[:400].contiguous(), 4, *_weights(32), "silu", max_rows=12)
    # all of them, against those of a single call's first ones and a second order of blocks
    a = q.group_norm_fwd(x, 4, ptr, act=q.ACT_SILU, max_rows=12)
    b = q.group_norm_fwd(x, 4, ptr, act=q.ACT_SILU, max_rows=12)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_rows_outside_segments_stay():
    q = gq()
    for n, hint in ((5000, 0), (300, 50)):
        x = _matrix(n, 40, 0, torch.float32, 3)
        ptr = torch.tensor([10, 10 + n // 3, n - 20], device="cuda")
        out = torch.full_like(x, 9.0)
        _, mean, rstd = q.group_norm_fwd(x, 5, ptr, out=out, max_rows=hint)
        assert (out[:10] == 9).all() and (out[n - 20:] == 9).all()
        dx = torch.full_like(x, 4.0)
        x2 = x.clone()
        x2[:10] = float("nan")
        x2[n - 20:] = float("inf")
        _, dg, db = q.group_norm_bwd(x2, x2, 5, mean, rstd, ptr, dX=dx, max_rows=hint)
        assert (dx[:10] == 4).all() and (dx[n - 20:] == 4).all() and torch.isfinite(dg).all() and torch.isfinite(db).all()


def test_offsets_that_are_not_rising_stay_inside():
    """Offsets outside the rows or falling: something finite or not, but inside the buffers."""
    q = gq()
    buf = torch.full((130, 16), 5.0, device="cuda")
    x = buf[10:120]
    x.copy_(_matrix(110, 16, 0, torch.float32, 3))
    out = torch.full((130, 16), 6.0, device="cuda")
    for hint in (0, 8, 1 << 20):
        q.group_norm_fwd(x, 2, torch.tensor([-50, 30, 20, 5000, 1 << 40], device="cuda"), out=out[10:120], max_rows=hint)
        assert (out[:10] == 6).all() and (out[120:] == 6).all()


@pytest.mark.parametrize("n,d,groups", [(300, 64, 4), (30000, 64, 4)])
def test_in_place_and_without_weights(n, d, groups):
    q = gq()
    x, dy = _matrix(n, d, 0, torch.float32, 1), _matrix(n, d, 0, torch.float32, 2)
    _check(q, x, dy, None, groups, None, None, "silu", long_=n > 1000, inplace=True)


def test_large_offset_and_constant_rows():
    """A mean of a thousand spreads; segments of equal values (variance 0)."""
    q = gq()
    for n in (200, 40000):
        x = _matrix(n, 32, 0, torch.float32, 1, off=3000.0)
        _check(q, x, _matrix(n, 32, 0, torch.float32, 2), None, 4, *_weights(32), "none", long_=n > 1000)
        x = torch.full((n, 32), 123.25, device="cuda")
        y, mean, rstd = q.group_norm_fwd(x, 4)
        assert torch.equal(y, torch.zeros_like(y)) and (mean == 123.25).all()
        dx, dg, _ = q.group_norm_bwd(torch.ones_like(x), x, 4, mean, rstd)
        assert (dx.abs() <= rstd.max() * 1e-4).all() and not dg.any()


@pytest.mark.parametrize("n", [50, 20000])
def test_nan_and_infinity_stay_in_their_group(n):
    q = gq()
    x = _matrix(n, 24, 0, torch.float32, 8)
    x[7, 3], x[9, 13] = float("nan"), float("inf")
    for act in ("none", "silu"):
        y, mean, _ = q.group_norm_fwd(x, 3, act=ACTS[act])
        assert torch.isnan(y[:, :8]).all() and torch.isnan(y[:, 8:16]).any() and torch.isfinite(y[:, 16:]).all()
    y, _, _ = q.group_norm_fwd(x, 3, act=q.ACT_RELU)
    assert (y[:, :8] == 0).all()


def test_gradient_by_differences():
    """d/dx, d/dgamma, d/dbeta of sum(y * w) by central differences in 64 bits
    (step 1e-4: truncation about 1e-8 of the third derivative)."""
    q = gq()
    n, d, groups = 30, 12, 3
    x = _matrix(n, d, 0, torch.float32, 1)
    w = _matrix(n, d, 0, torch.float32, 2)
    gamma, beta = _weights(d)
    ptr = _ptr([11, 0, 19])

    def loss(x, gamma, beta):
        total = 0
        for r0, r1 in ((0, 11), (11, 30)):
            v = x[r0:r1].view(r1 - r0, groups, -1)
            m = v.mean((0, 2), keepdim=True)
            z = ((v - m) / torch.sqrt((v - m).square().mean((0, 2), keepdim=True) + 1e-5)).reshape(r1 - r0, d) * gamma + beta
            total = total + (z * torch.sigmoid(z) * w[r0:r1].double()).sum()
        return total

    _, mean, rstd = q.group_norm_fwd(x, groups, ptr, gamma, beta, act=q.ACT_SILU)
    got = q.group_norm_bwd(w, x, groups, mean, rstd, ptr, gamma, beta, act=q.ACT_SILU)
    args = [x.double(), gamma.double(), beta.double()]
    for k, places in ((0, [(0, 0), (10, 11), (11, 5), (29, 7)]), (1, [(0,), (11,)]), (2, [(3,), (8,)])):
        for at in places:
            e = torch.zeros_like(args[k])
            e[at] = 1e-4
            lo, hi = list(args), list(args)
            lo[k], hi[k] = args[k] - e, args[k] + e
            diff = ((loss(*hi) - loss(*lo)) / 2e-4).item()
            assert abs(got[k][at].item() - diff) <= 2e-5 * (1 + abs(diff)), (k, at)


def test_captured_and_on_a_stream():
    q = gq()
    x, dy = _matrix(9000, 64, 0, torch.bfloat16, 1), _matrix(9000, 64, 0, torch.bfloat16, 2)
    ptr = _ptr([100, 8000, 900])
    ws = q.Workspace()
    want = q.group_norm_fwd(x, 4, ptr, act=q.ACT_SILU, ws=ws)
    wb = q.group_norm_bwd(dy, x, 4, want[1], want[2], ptr, act=q.ACT_SILU, ws=ws)
    out = [torch.empty_like(t) for t in (*want, *wb)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.group_norm_fwd(x, 4, ptr, act=q.ACT_SILU, out=out[0], mean=out[1], rstd=out[2], ws=ws)
        q.group_norm_bwd(dy, x, 4, out[1], out[2], ptr, act=q.ACT_SILU, dX=out[3], dgamma=out[4], dbeta=out[5], ws=ws)
    for _ in range(2):
        for t in out:
            t.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, (*want, *wb)))


def test_empty():
    q = gq()
    x = torch.zeros(0, 12, device="cuda")
    y, mean, rstd = q.group_norm_fwd(x, 3, torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert y.shape == (0, 12) and mean.shape == (2, 3) and not mean.any() and (rstd > 300).all()
    dx, dg, db = q.group_norm_bwd(x, x, 3, mean, rstd, torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert dx.shape == (0, 12) and not dg.any() and not db.any()
    y, mean, _ = q.group_norm_fwd(torch.ones(4, 12, device="cuda"), 3, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert mean.shape == (0, 3)


def test_refusals():
    q = gq()
    x = torch.zeros(10, 12, device="cuda")
    ptr = torch.tensor([0, 4, 10], device="cuda")
    y, mean, rstd = q.group_norm_fwd(x, 3, ptr)
    for kw in (dict(groups=5), dict(groups=0), dict(ptr=ptr.int()), dict(ptr=ptr.cpu()), dict(ptr=ptr[:0]),
               dict(gamma=torch.ones(11, device="cuda")), dict(eps=-1.0), dict(eps=float("inf")), dict(act=3),
               dict(max_rows=-1), dict(out=torch.zeros(10, 13, device="cuda")), dict(mean=torch.zeros(3, 2, device="cuda"))):
        with pytest.raises(q.GQError):
            q.group_norm_fwd(x, **{**dict(groups=3, ptr=ptr), **kw})
    for kw in (dict(mean=None), dict(mean=mean[:1]), dict(dY=x[:9]), dict(ptr=None), dict(dX=x.double())):
        with pytest.raises(q.GQError):
            q.group_norm_bwd(**{**dict(dY=x, X=x, groups=3, mean=mean, rstd=rstd, ptr=ptr), **kw})
