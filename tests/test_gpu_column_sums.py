"""Sums over very many rows: dbeta of group normalization, dbias of the 8-bit linear
layer.  The parts that threads and blocks add up are joined with what each
addition loses, so with whole values, whose parts stay below 2^24 and are
exact, the result is the exact sum, rounded once."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


def _whole(n, d, t, seed, lo, hi):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return torch.randint(lo, hi, (n, d), device="cuda", generator=gen).to(t)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d,lo,hi", [(300001, 47, 100, 256), (600000, 64, 200, 256), (4097, 300, -255, 256),
                                       (1, 5, -255, 256), (2449029, 8, 0, 33)])
def test_dbias_is_the_sum(n, d, lo, hi, t):
    q = gq()
    dy, x = _whole(n, d, t, 1, lo, hi), _whole(n, 16, t, 2, -9, 9)
    w = torch.ones(d, 16, device="cuda")
    _, _, db = q.linear_i8_bwd(dy, x, w, need_dX=False)
    assert torch.equal(db, dy.double().sum(0).float())


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,d,lo,hi", [(300001, 47, 100, 256), (600000, 64, 200, 256), (2449029, 8, 0, 33)])
def test_dbeta_is_the_sum(n, d, lo, hi, t):
    q = gq()
    dy, x = _whole(n, d, t, 1, lo, hi), _whole(n, d, t, 2, -9, 9)
    ptr = torch.tensor([0, n // 3, n], device="cuda")
    _, mean, rstd = q.group_norm_fwd(x, 1, ptr, max_rows=n - n // 3)
    _, _, dbeta = q.group_norm_bwd(dy, x, 1, mean, rstd, ptr, max_rows=n - n // 3)
    assert torch.equal(dbeta, dy.double().sum(0).float())


def test_sums_that_are_not_finite():
    q = gq()
    for n in (300, 300001):
        x, dy = _whole(n, 32, torch.float32, 1, -9, 9), _whole(n, 32, torch.float32, 2, -9, 9)
        dy[n // 2, 3], dy[n - 1, 5], dy[0, 7] = float("inf"), float("nan"), -float("inf")
        _, mean, rstd = q.group_norm_fwd(x, 32)
        _, _, dbeta = q.group_norm_bwd(dy, x, 32, mean, rstd)
        assert dbeta[3] == float("inf") and dbeta[7] == -float("inf") and torch.isnan(dbeta[5])
        rest = [c for c in range(32) if c not in (3, 5, 7)]
        assert torch.equal(dbeta[rest], dy.double().sum(0).float()[rest])
