"""Products of 8-bit integers with row and channel scales, their quantizers and
the linear layer, against whole-number and 64-bit arithmetic.  u = 2^-24.

Codes are exact: round(x / s), ties to even, with s the fp32 value of max / 127.
Sums are exact, so with scales of 1 a product is the sum rounded once to fp32.
With scales: (float)sum u, a product u, then a fused product and sum u: with
t = sum sa sb, |C - (t + bias)| <= 2.1u |t| + u |t + bias|, half a step of the type
on top of it."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _matrix(n, d, pad, t, seed):
    buf = torch.full((n, d + pad), 7.0, dtype=t, device="cuda")
    buf[:, :d] = torch.randn(n, d, device="cuda", generator=_gen(seed)) * torch.exp(
        torch.randn(n, 1, device="cuda", generator=_gen(seed + 1)))
    return buf[:, :d]


def _codes64(x):
    """(codes, scale) of rows by the definition."""
    x = x.double()
    s = (x.abs().amax(1) / 127).float().double()  # a quotient of fp32 values, rounded once
    s = torch.where(x.abs().amax(1) < 2.0 ** -100, torch.zeros_like(s), s)
    q = torch.round(torch.where(s[:, None] > 0, x / s[:, None], torch.zeros_like(x)))
    return q, s


def _half(t, x):
    return torch.finfo(t).eps / 2 * x.abs().clamp(min=torch.finfo(t).tiny) * 1.01 if t != torch.float32 else 0.0


def _within(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert torch.isfinite(got).all() and bad.max() <= 0, f"{what}: {bad.max().item()} over the bound"


# ------------------------------------------------------------- quantizers --


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (5, 3, 1), (33, 16, 0), (64, 255, 1), (130, 256, 0), (7, 1000, 8),
                                     (9, 4096, 0), (3, 4097, 3), (2, 20000, 0), (1000, 47, 1)])
def test_quantize(n, d, pad, t):
    q = gq()
    x = _matrix(n, d, pad, TYPES[t], n + d)
    x[n // 2] = 0
    for transpose in (False, True):
        codes, scale = q.quantize_i8(x, transpose)
        want, s = _codes64(x.t() if transpose else x)
        assert torch.equal(scale.double(), s), (t, transpose)
        assert torch.equal(codes.double(), want), (t, transpose)


def test_ties_go_to_even():
    """x / s is a whole number and a half: max = 127 gives s = 1."""
    q = gq()
    x = (torch.arange(-127, 127, device="cuda") + 0.5).repeat(4, 1)
    x = torch.cat([x, torch.full((4, 1), 127.0, device="cuda")], 1) * torch.tensor([[1.0], [2.0], [0.25], [2 ** -60]],
                                                                                    device="cuda")
    want = torch.round((torch.arange(-127, 127, device="cuda") + 0.5).double())
    for transpose in (False, True):
        codes, _ = q.quantize_i8(x.t().contiguous() if transpose else x, transpose)
        assert all(torch.equal(codes[i, :-1].double(), want) for i in range(4))
    # scales that are not whole: values one step either side of a half
    m = torch.rand(64, 1, device="cuda", generator=_gen(1)) + 0.5
    s = (m.double() / 127).float()
    k = torch.arange(-126, 127, device="cuda")
    half = ((k + 0.5).double() * s.double()).float()
    x = torch.cat([m, half, torch.nextafter(half, half + 1), torch.nextafter(half, half - 1)], 1)
    codes, _ = q.quantize_i8(x)
    assert torch.equal(codes.double(), _codes64(x)[0])


def test_rows_that_are_not_finite():
    q = gq()
    x = torch.randn(6, 100, device="cuda", generator=_gen(2))
    x[1, 7] = float("nan")
    x[2, 99] = float("inf")
    x[3] = 1e-38
    x[4] = 3e38
    for transpose in (False, True):
        codes, scale = q.quantize_i8(x.t().contiguous() if transpose else x, transpose)
        assert torch.isnan(scale[1:3]).all() and not codes[1:4].any() and scale[3] == 0
        assert torch.equal(codes[4], torch.full((100,), 127, dtype=torch.int8, device="cuda"))
        y = q.gemm_i8(codes, scale, codes[5:], scale[5:])
        assert torch.isnan(y[1:3]).all() and torch.isfinite(y[[0, 3, 5]]).all() and (y[3] == 0).all()
        assert (q.gemm_i8(codes, scale, codes[5:], scale[5:], act=q.ACT_RELU)[1:3] == 0).all()


def test_quantize_leaves_other_memory_alone():
    q = gq()
    x = _matrix(50, 77, 0, torch.float32, 3)
    buf = torch.full((52, 96), 55, dtype=torch.int8, device="cuda")
    q.quantize_i8(x, out=buf[1:51, :77])
    assert (buf[0] == 55).all() and (buf[51] == 55).all() and (buf[:, 80:] == 55).all()
    buf.fill_(55)
    xt = _matrix(77, 50, 0, torch.float32, 3)
    q.quantize_i8(xt, True, out=buf[1:51, :77])
    assert (buf[0] == 55).all() and (buf[51] == 55).all() and (buf[:, 80:] == 55).all()


# ---------------------------------------------------------------- products --


def _int8(n, k, seed, lo=-128, hi=128):
    buf = torch.full((n, (k + 15) // 16 * 16 + 16), 99, dtype=torch.int8, device="cuda")
    buf[:, :k] = torch.randint(lo, hi, (n, k), device="cuda", generator=_gen(seed), dtype=torch.int32).to(torch.int8)
    return buf[:, :k]


def _sum64(a, b):
    """Whole sums; every one is below 2^53."""
    return a.double() @ b.double().t()


SHAPES = [(1, 1, 1), (1, 10007, 1024), (1, 33, 17), (2, 100, 64), (3, 50, 1000), (5, 5, 5), (8, 333, 4096), (7, 64, 20000),
          (9, 33, 100), (17, 500, 777), (40, 40, 40), (64, 1024, 1024), (256, 256, 64), (257, 255, 65), (300, 1000, 1024),
          (1000, 300, 1025), (128, 64, 5000), (513, 2000, 2048), (2000, 47, 256), (70, 70, 70000), (32, 20, 140000),
          (5000, 5000, 128), (20000, 256, 256), (255, 20001, 1056), (9, 9, 16), (1, 3, 70001), (60000, 20, 256), (50001, 1, 100), (80000, 32, 64), (40000, 33, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sums_are_exact(m, n, k):
    q = gq()
    a, b = _int8(m, k, m + k), _int8(n, k, n + k + 1)
    one = lambda c: torch.ones(c, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c = q.gemm_i8(a, one(m), b, one(n), dev_err=err)
    assert err.item() == 0
    assert torch.equal(c, _sum64(a, b).float())


@pytest.mark.parametrize("m,n,k", [(4, 100, 65536), (300, 300, 1024), (300, 300, 1040), (300, 260, 8192), (40, 40, 66000),
                                   (600, 300, 3000)])
@pytest.mark.parametrize("va,vb", [(-128, -128), (127, 127), (-128, 127)])
def test_largest_sums(m, n, k, va, vb):
    """Equal values of the largest magnitude: partial sums of one sign up to 2^30
    and beyond, odd ones among them where a value differs."""
    q = gq()
    a = torch.full((m, (k + 15) // 16 * 16), va, dtype=torch.int8, device="cuda")[:, :k]
    b = torch.full((n, (k + 15) // 16 * 16), vb, dtype=torch.int8, device="cuda")[:, :k]
    a[:, k // 2] = 1
    b[:, k // 3] = 3
    one = lambda c: torch.ones(c, device="cuda")
    assert torch.equal(q.gemm_i8(a, one(m), b, one(n)), _sum64(a, b).float())


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("m,n,k,pad", [(1, 777, 300, 0), (6, 100, 96, 1), (50, 90, 512, 0), (90, 50, 512, 3),
                                       (700, 1030, 1500, 0), (1030, 700, 200, 5), (513, 264, 128, 8), (40, 30, 9000, 0)])
def test_scales_bias_activation(m, n, k, pad, out):
    q = gq()
    a, b = _int8(m, k, 1), _int8(n, k, 2)
    sa = torch.exp(torch.randn(m, device="cuda", generator=_gen(3))) / 100
    sb = torch.exp(torch.randn(n, device="cuda", generator=_gen(4))) / 100
    bias = torch.randn(n, device="cuda", generator=_gen(5))
    t = TYPES[out]
    want = _sum64(a, b) * sa.double()[:, None] * sb.double()
    for use_bias, act in ((True, q.ACT_NONE), (True, q.ACT_RELU), (False, q.ACT_RELU)):
        buf = torch.full((m + 1, n + pad), 3.0, dtype=t, device="cuda")
        c = q.gemm_i8(a, sa, b, sb, bias if use_bias else None, act, out=buf[:m, :n])
        ref = want + bias.double() if use_bias else want
        tol = 2.1 * U * want.abs() + U * ref.abs() + _half(t, ref)
        if act == q.ACT_RELU:
            ref = ref.clamp(min=0)
        _within(c, ref, tol, "C")
        assert (buf[m] == 3.0).all() and (buf[:, n:] == 3.0).all()


def test_values_behind_a_row_do_not_count():
    q = gq()
    a, b = _int8(5, 33, 1), _int8(70, 33, 2)
    one = lambda c: torch.ones(c, device="cuda")
    for m in (5, 1):
        c = q.gemm_i8(a[:m], one(m), b, one(70))
        assert torch.equal(c, _sum64(a[:m], b).float())


def test_two_captured_graphs_and_a_stream():
    """Graphs with workspaces of their own, replayed on two streams; a third call between."""
    q = gq()
    one = lambda c: torch.ones(c, device="cuda")
    cases = [(300, 300, 20000), (64, 500, 9000)]
    made = []
    for i, (m, n, k) in enumerate(cases):
        a, b = _int8(m, k, i), _int8(n, k, i + 9)
        ws = q.Workspace()
        out = torch.empty(m, n, device="cuda")
        q.gemm_i8(a, one(m), b, one(n), out=out, ws=ws)
        sa, sb = one(m), one(n)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.gemm_i8(a, sa, b, sb, out=out, ws=ws)
        made.append((g, a, b, out, sa, sb, ws))
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for (g, a, b, out, *_), s in zip(made, streams):
            with torch.cuda.stream(s):
                out.zero_()
                g.replay()
    torch.cuda.synchronize()
    for g, a, b, out, *_ in made:
        assert torch.equal(out, _sum64(a, b).float())


# ------------------------------------------------------------------ layer --


def _prod64(a, b):
    (qa, sa), (qb, sb) = _codes64(a), _codes64(b)
    return (qa @ qb.t()) * sa[:, None] * sb


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,out,pad", [(1, 64, 100, 0), (8, 100, 30, 1), (9, 100, 30, 1), (300, 256, 256, 0),
                                         (1000, 77, 513, 3), (3000, 1000, 47, 8), (4097, 64, 64, 0), (20, 1100, 1300, 0)])
def test_linear(n, k, out, pad, t):
    q = gq()
    T = TYPES[t]
    x, w, dy = _matrix(n, k, pad, T, 1), _matrix(out, k, 0, torch.float32, 2), _matrix(n, out, pad, T, 3)
    w = w / k ** 0.5
    bias = torch.randn(out, device="cuda", generator=_gen(4))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = q.linear_i8(x, *q.quantize_i8(w), bias, act=q.ACT_RELU, dev_err=err)
    prod = _prod64(x, w)
    ref = prod + bias.double()
    _within(y, ref.clamp(min=0), 2.1 * U * prod.abs() + U * ref.abs() + _half(T, ref), "y")
    dx, dw, db = q.linear_i8_bwd(dy, x, w, dev_err=err)
    ref = _prod64(dy, w.t())
    _within(dx, ref, 3.2 * U * ref.abs() + _half(T, ref), "dx")
    ref = _prod64(dy.t(), x.t())
    _within(dw, ref, 3.2 * U * ref.abs(), "dw")
    # a thread's rows, the block's and the parts' partial sums: at most n roundings of the running sum
    _within(db, dy.double().sum(0), n * U * dy.double().abs().sum(0), "dbias")
    assert err.item() == 0
    only_x, none, nb = q.linear_i8_bwd(dy, x, w, need_dW=False)
    assert none is None and nb is None and torch.equal(only_x, dx)
    none, only_w, _ = q.linear_i8_bwd(dy, x, w, need_dX=False)
    assert none is None and torch.equal(only_w, dw)


@pytest.mark.parametrize("t", list(TYPES))
@pytest.mark.parametrize("n,k,out", [(9, 8, 1), (40, 16, 32), (128, 64, 33), (257, 100, 47), (30000, 256, 256),
                                     (100001, 200, 20), (60000, 72, 160), (50000, 4, 256)])
def test_rows_quantized_on_the_way_equal_codes(n, k, out, t):
    """Aligned rows of up to 256 values are quantized inside the product, others
    before it: the same result, bit for bit, and the rows behind the last untouched."""
    q = gq()
    T = TYPES[t]
    a = torch.zeros(n, (k + 7) // 8 * 8, dtype=T, device="cuda")[:, :k]
    a.copy_(_matrix(n, k, 0, T, 5))
    a[n // 2] = 0
    a[n // 3, k // 2] = float("inf")
    w, s = q.quantize_i8(_matrix(out, k, 0, torch.float32, 6))
    bias = torch.randn(out, device="cuda", generator=_gen(7))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    buf = torch.full((n + 1, (out + 7) // 8 * 8), 3.0, dtype=T, device="cuda")
    y = q.linear_i8(a, w, s, bias, out=buf[:n, :out], dev_err=err)
    x, sx = q.quantize_i8(a)
    want = q.gemm_i8(x, sx, w, s, bias, dtype=T)
    assert err.item() == 0 and torch.equal(torch.isnan(y), torch.isnan(want)) and torch.isnan(y[n // 3]).all()
    assert torch.equal(y.nan_to_num(7.0), want.nan_to_num(7.0))
    assert (buf[n] == 3.0).all() and (buf[:, out:] == 3.0).all()


def test_linear_is_the_product_it_approximates():
    """The gradients' products against central differences of the layer in full
    precision: within the quantization's own error.  Both operands are off by
    at most half a step, s / 2 per element: |C - C_exact| <= sum_k (|a| sb / 2 +
    |b| sa / 2 + sa sb / 4)."""
    q = gq()
    n, k, out = 60, 50, 40
    x, w, dy = (_matrix(*s, 0, torch.float32, i) for i, s in enumerate(((n, k), (out, k), (n, out))))
    dx, dw, db = q.linear_i8_bwd(dy, x, w)
    h = 0.5

    def loss(x, w, b):  # linear in each of them: central differences are exact
        return ((x.double() @ w.double().t() + b) * dy.double()).sum()

    def bound(a, b):
        sa, sb = (t.abs().amax(1).double() / 127 for t in (a, b))
        return (a.double().abs().sum(1)[:, None] * sb + sa[:, None] * b.double().abs().sum(1)) / 2 + a.shape[1] * torch.outer(
            sa, sb) / 4

    zero = torch.zeros(out, dtype=torch.float64, device="cuda")
    bx, bw = bound(dy, w.t()), bound(dy.t(), x.t())
    for i, j in ((0, 0), (17, 33), (59, 49)):
        e = torch.zeros_like(x)
        e[i, j] = h
        d = (loss(x + e, w, zero) - loss(x - e, w, zero)) / (2 * h)
        assert (dx[i, j].double() - d).abs() <= 1.001 * bx[i, j] + 1e-5
    for i, j in ((0, 0), (17, 33), (39, 49)):
        e = torch.zeros_like(w)
        e[i, j] = h
        d = (loss(x, w + e, zero) - loss(x, w - e, zero)) / (2 * h)
        assert (dw[i, j].double() - d).abs() <= 1.001 * bw[i, j] + 1e-5
        z = zero.clone()
        z[i] = h
        assert (db[i].double() - (loss(x, w, z) - loss(x, w, -z)) / (2 * h)).abs() <= 1e-3


def test_empty():
    q = gq()
    w, s = q.quantize_i8(torch.randn(30, 20, device="cuda"))
    x = torch.zeros(0, 20, device="cuda")
    assert q.linear_i8(x, w, s).shape == (0, 30)
    dx, dw, db = q.linear_i8_bwd(torch.zeros(0, 30, device="cuda"), x, torch.randn(30, 20, device="cuda"))
    assert dx.shape == (0, 20) and not dw.any() and not db.any()
    c, sc = q.quantize_i8(x, True)
    assert c.shape == (20, 0) and not sc.any()


def test_refusals():
    q = gq()
    a, b = _int8(4, 32, 1), _int8(6, 32, 2)
    sa, sb = torch.ones(4, device="cuda"), torch.ones(6, device="cuda")
    bad = torch.zeros(4, 36, dtype=torch.int8, device="cuda")
    for args in ((a, sa, b[:, :16], sb), (a, sb, b, sb), (a, sa, b, None), (a.int(), sa, b, sb), (bad[:, 1:33], sa, b, sb),
                 (bad[:, :32], sa, b, sb), (a.cpu(), sa, b, sb), (a, sa, b, sb, sa)):
        with pytest.raises(q.GQError):
            q.gemm_i8(*args)
    with pytest.raises(q.GQError):
        q.gemm_i8(a, sa, b, sb, dtype=torch.float64)
    with pytest.raises(q.GQError):
        q.gemm_i8(a, sa, b, sb, out=torch.zeros(4, 7, device="cuda"))
    with pytest.raises(q.GQError):
        q.gemm_i8(a, sa, b, sb, act=7)
    with pytest.raises(q.GQError):  # the last row ends with its allocation, short of 16 bytes
        q.gemm_i8(torch.zeros(1 * 17, dtype=torch.int8, device="cuda").as_strided((1, 17), (32, 1)), sa[:1],
                  torch.zeros(2, 32, dtype=torch.int8, device="cuda")[:, :17], sa[:2])
    with pytest.raises(q.GQError):
        q.quantize_i8(a)
    with pytest.raises(q.GQError):
        q.quantize_i8(torch.zeros(4, 4, device="cuda"), out=torch.zeros(4, 4, dtype=torch.int8, device="cuda"))
    x = torch.zeros(4, 32, device="cuda")
    with pytest.raises(q.GQError):
        q.linear_i8(x, b, sa)
    with pytest.raises(q.GQError):
        q.linear_i8(x[:, :31], b, sb)
    with pytest.raises(q.GQError):
        q.linear_i8_bwd(x, x, torch.zeros(6, 32, device="cuda"))
