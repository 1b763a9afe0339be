"""Group normalization of one huge segment under a hint that says it is short:
one block takes it alone, and its sums are those of pieces of 1,024 rows a
thread, so that the hint costs time and no accuracy.  u = 2^-24.

Every value is C but for the first eight of each thread (0), so that the shift is
0, every running sum grows by the same step, and its roundings go the same way
for long stretches.  With N rows a thread in pieces of 1,024:
  a thread's piece: 8 values added up (exact: C has 8 bits), 128 running sums
  of a piece's threads R sums, N / 1,024 pieces put together, the lanes' 48
  K = 128 + R + N / 1,024 + 48 + 16 roundings, each of at most u of the sum
  mean: K u |mean| + u;  variance: sums of squares the same way, differences of
  means by 2 K u C, and the last operations: 4 K u C^2
  backward (dY = 1, no activation) adds rows one by one: B = 1,024 + R + N / 1,024 + 48
  + 16, dbeta B u n, dgamma (B + 4) u sum |xhat|"""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("d,t", [(64, torch.float32), (256, torch.bfloat16), (63, torch.float32)])
def test_a_hint_far_too_small_costs_no_accuracy(d, t):
    q = gq()
    v = 4 if d % 4 == 0 else 1
    R = 256 // (d // v)               # threads of a channel
    N = 30000                         # rows of each
    n, C = N * R, 1.4140625
    x = torch.full((n, d), C, dtype=t, device="cuda")
    x[:8 * R] = 0
    y, mean, rstd = q.group_norm_fwd(x, 1, max_rows=7)
    K = 128 + R + N / 1024 + 48 + 16
    m = C * (N - 8) / N
    var = m * (C - m)
    assert abs(mean.item() - m) <= K * U * m + U
    assert abs(rstd.item() * (var + 1e-5) ** 0.5 - 1) <= (4 * K * U * C * C) / (2 * var) + 4 * U
    _, dgamma, dbeta = q.group_norm_bwd(torch.ones_like(x), x, 1, mean, rstd, max_rows=7)
    xh = (x[:, :1].double() - mean.item()) * rstd.item()
    B = K + 1024 - 128
    assert (dbeta.double() - n).abs().max() <= B * U * n
    assert (dgamma.double() - xh.sum()).abs().max() <= (B + 4) * U * xh.abs().sum()


def test_one_huge_segment_among_many_small_ones():
    """A warp a segment: the same with the 2 threads that a warp has for a channel of 64."""
    q = gq()
    R, N, C, d = 2, 30000, 1.4140625, 64
    n = N * R
    x = torch.full((n + 4000, d), 1.0, device="cuda")
    x[1000:1000 + n] = C
    x[1000:1000 + 8 * R] = 0
    cuts = torch.cat([torch.arange(0, 1000, 2), torch.tensor([1000]), torch.arange(1000 + n, n + 4001, 2)]).cuda()
    y, mean, rstd = q.group_norm_fwd(x, 1, cuts, max_rows=7)
    K = 128 + R + N / 1024 + 48 + 16
    m = C * (N - 8) / N
    var = m * (C - m)
    assert cuts.numel() - 1 > 4 * 152 and (mean[:500] == 1).all() and (mean[501:] == 1).all()
    assert abs(mean[500].item() - m) <= K * U * m + U
    assert abs(rstd[500].item() * (var + 1e-5) ** 0.5 - 1) <= (4 * K * U * C * C) / (2 * var) + 4 * U
    _, dgamma, dbeta = q.group_norm_bwd(torch.ones_like(x), x, 1, mean, rstd, cuts, max_rows=7)
    B = K + 1024 - 128
    assert (dbeta.double() - (n + 4000)).abs().max() <= (B + 100) * U * (n + 4000)
