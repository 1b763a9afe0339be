"""Layer normalization where a block or a group takes many rows one after the
other, in every vector width and type, and the rows' ragged ends, against the
formulas in 64 bits.  u = 2^-24 is half a step of fp32, eps_t / 2 half a
step of the type t that a result is stored in, relative to its value.

Row sums: at most 16 values of a lane in sequence, then 5 shuffles and 5 steps
across the warps: 26 roundings and the division by d.  With A = max|x|,
xhat and rstd of the row:
  y:   u |gamma| A rstd 27 (1 + |xhat|) + 24 u |xhat gamma| + 2 u |y|
  dx:  rstd u (6 |g| + 34 mean|g| + 40 |xhat| mean|g xhat|)
  dgamma, dbeta: the chain of a lane's rows (n / rows at a time), then at most
       100 roundings of shuffles, warps and blocks:
       (n / rows at a time + 100) u sum|dz xhat|, sum|dz|"""
import pytest
import torch

import synth
from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _mat(n, d, pad, dtype, seed, off=0.0):
    buf = torch.full((n, d + pad), 77.0, dtype=dtype, device="cuda")
    x = synth.normal_matrix(n, d, seed=seed, device="cuda")
    buf[:, :d] = (x + off * synth.normal_matrix(n, 1, seed=seed + 1, device="cuda")).to(dtype)
    return buf[:, :d]


def _half_step(t, ref):
    return torch.finfo(t).eps / 2 * ref.abs().clamp(min=torch.finfo(t).tiny) * (1 + 1e-3)


def _within(got, ref, tol, what):
    e = (got.double() - ref).abs() - tol
    assert torch.isfinite(got).all() and e.max() <= 0, f"{what}: {e.max().item()} over the bound at {e.argmax().item()}"


def _both_ways(q, orc, n, d, pad, t, relu, p, seed, at_a_time):
    """Both passes in 64 bits by the definition, on the GPU; the mask is the oracle's."""
    x, dy = _mat(n, d, pad, t, seed=d, off=0.5), _mat(n, d, pad, t, seed=d + 5)
    gamma = 1 + 0.3 * synth.normal_matrix(1, d, seed=d + 7, device="cuda")[0]
    beta = 0.3 * synth.normal_matrix(1, d, seed=d + 8, device="cuda")[0]
    act = q.ACT_RELU if relu else q.ACT_NONE
    bits = torch.full((n, (d + 31) // 32), -1, dtype=torch.int32, device="cuda") if relu else None
    y, mean, rstd = q.layer_norm_fwd(x, gamma, beta, act=act, p=p, seed=seed, relu_bits=bits)
    dx, dgamma, dbeta = q.layer_norm_bwd(dy, x, mean, rstd, gamma, act=act, p=p, seed=seed, relu_bits=bits)
    factor = torch.from_numpy(orc.kept(seed, n, d, p)).cuda().double() / (1 - p) if p > 0 else 1.0
    X, G = x.double(), gamma.double()
    m = X.sum(1, keepdim=True) / d
    xc = X - m
    r = 1 / torch.sqrt((xc * xc).sum(1, keepdim=True) / d + 1e-5)
    xh = xc * r
    z = xh * G + beta.double()
    Y = (z.clamp(min=0) if relu else z) * factor
    A = X.abs().amax(1, keepdim=True)
    z_tol = U * (G.abs() * A * r * 27 * (1 + xh.abs()) + 24 * (xh * G).abs() + 2 * z.abs())
    _within(y, Y, z_tol / (1 - p) + 2 * U * Y.abs() + _half_step(t, Y), "y")
    dz = dy.double() * factor
    if relu:
        c = torch.arange(d, device="cuda")
        on = (bits[:, c // 32] >> (c % 32).to(torch.int32)) & 1
        assert not ((on.bool() != (z > 0)) & (z.abs() > z_tol)).any()
        dz = dz * on
    m, r = mean.double()[:, None], rstd.double()[:, None]  # the backward pass is given the stored ones
    xh = (X - m) * r
    g = dz * G
    dX = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    tol = r * U * (6 * g.abs() + 34 * g.abs().mean(1, keepdim=True)
                   + 40 * xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    _within(dx, dX, tol + _half_step(t, dX), "dx")
    rows = n // at_a_time + 100
    _within(dgamma, (dz * xh).sum(0), rows * U * (dz * xh).abs().sum(0), "dgamma")
    _within(dbeta, dz.sum(0), rows * U * dz.abs().sum(0), "dbeta")


# Rows of a block (d > 512), with a ragged end: pitches that are a multiple of
# 8 make the vectors 16 bytes, even ones pairs of 16-bit elements, odd ones
# single elements.  A block has 16 elements of a row per thread (8 in some
# backward passes) and an SM about 1,024 threads, so 152 SMs hold at most
# 152 x 1,024 x 16 elements at a time: eight rows of a block each.
@pytest.mark.parametrize("dtype,pitch", [("f32", 8), ("f32", 1), ("bf16", 8), ("bf16", 2), ("bf16", 1), ("f16", 8),
                                         ("f16", 2), ("f16", 1)])
@pytest.mark.parametrize("n,d", [(20_000, 533), (9_000, 2_051), (4_000, 4_603), (1_300, 8_203)])
def test_many_rows_of_a_block(orc, n, d, dtype, pitch):
    _both_ways(gq(), orc, n, d, (pitch - d) % 8, TYPES[dtype], d != 533, 0.25 if pitch != 2 else 0.0, d * 3, 100)


# Rows of a group of 8, 16 or 32 lanes, 16-bit: 152 SMs x 8 blocks x 8 warps
# hold 9,728 warps of up to four rows; at least 1,000 rows go at a time.
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n,d", [(200_003, 8), (120_001, 64), (80_001, 120), (60_001, 256), (40_003, 504)])
@pytest.mark.parametrize("pad", [0, 1])
def test_many_rows_of_a_group(orc, n, d, dtype, pad):
    _both_ways(gq(), orc, n, d, pad, TYPES[dtype], d > 64, 0.25, d, 1000)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [5, 21, 47, 133, 301, 515, 2_051, 9_001])
def test_constant_rows_of_huge_values(d, dtype):
    """A constant row has xhat = 0: dx = rstd (g - mean g), dgamma = 0.  The
    lanes past its end must add nothing either, although (0 - mean) rstd is
    beyond fp32 there: mean 2^113 and rstd = 1 / sqrt(1e-10) = 1e5.  (Sums of
    d times a power of two are exact, and the longest is within fp32.)"""
    q = gq()
    t, n, eps = TYPES[dtype], 70, 1e-10
    ld = (d + 7) // 8 * 8 + 8
    buf = torch.full((n, ld), 2.0 ** 113, dtype=t, device="cuda")
    dbuf = synth.normal_matrix(n, ld, seed=d, device="cuda").to(t)
    for first in (0, 1):  # whole vectors, single elements
        x, dy = buf[:, first:first + d], dbuf[:, first:first + d]
        y, mean, rstd = q.layer_norm_fwd(x, eps=eps)
        assert not y.any() and torch.equal(mean, x[:, 0].float())
        dx, dgamma, dbeta = q.layer_norm_bwd(dy, x, mean, rstd)
        assert torch.isfinite(dx).all() and not dgamma.any()
        g = dy.double()
        ref = rstd.double()[:, None] * (g - g.mean(1, keepdim=True))
        tol = rstd.double()[:, None] * U * (6 * g.abs() + 34 * g.abs().mean(1, keepdim=True))
        assert ((dx.double() - ref).abs() <= tol + torch.finfo(t).eps / 2 * ref.abs() * (1 + 1e-3)).all()
        assert ((dbeta.double() - g.sum(0)).abs() <= (n + 100) * U * g.abs().sum(0)).all()


@pytest.mark.parametrize("d", [40, 300, 1000])
def test_relu_gives_zero_for_nan(d):
    q = gq()
    x = synth.normal_matrix(5, d, seed=1, device="cuda")
    x[2, d // 2] = float("nan")
    bits = torch.full((5, (d + 31) // 32), -1, dtype=torch.int32, device="cuda")
    y = q.layer_norm_fwd(x, act=q.ACT_RELU, relu_bits=bits)[0]
    assert torch.isfinite(y).all() and not y[2].any() and not bits[2].any() and y[1].any()
    assert torch.isnan(q.layer_norm_fwd(x)[0][2]).all()


@pytest.mark.parametrize("d", [64, 300, 2000])
def test_forward_without_statistics(d):
    """gq_layer_norm_fwd with NULL mean and rstd."""
    q = gq()
    x = synth.normal_matrix(50, d, seed=1, device="cuda")
    ref, y, p = q.layer_norm_fwd(x)[0], torch.empty_like(x), q._ptr
    q._check(q.lib().gq_layer_norm_fwd(p(x), q.F32, 50, d, d, None, None, 1e-5, q.ACT_NONE, 0.0, 0, p(y), d, None,
                                       None, None, 0, q._stream()), "fwd")
    assert torch.equal(y, ref)
