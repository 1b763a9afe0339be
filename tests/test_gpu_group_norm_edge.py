"""Group normalization at ReLU's edge: an element passes its gradient exactly
where forward let it through, also where z is a rounding error away from 0."""
import pytest
import torch

from gpu_helpers import gq

pytestmark = pytest.mark.gpu


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("s,n,d,groups", [(1, 300, 256, 8), (3, 260, 255, 5), (1500, 6000, 64, 4), (1, 40000, 256, 16),
                                          (2, 50000, 63, 3)])
def test_gradient_passes_where_forward_did(s, n, d, groups, t):
    """A block, a warp and several launches a segment, four channels and one a thread.
    beta is minus the product of one element of each channel, so that its z is
    the product's rounding error, of either sign.  dY is 1: dbeta counts the
    elements that passed, a whole number below 2^24, which has no rounding."""
    q = gq()
    x = torch.randn(n, d, device="cuda", generator=_gen(n)).to(t)
    gamma = 1 + 0.3 * torch.randn(d, device="cuda", generator=_gen(d))
    ptr = torch.arange(s + 1, device="cuda") * n // s
    rows = int((ptr[1:] - ptr[:-1]).max())
    _, mean, rstd = q.group_norm_fwd(x, groups, ptr, gamma, max_rows=rows)
    c = torch.arange(d, device="cuda")
    r = (c * 37 + 11) % n
    at = (torch.searchsorted(ptr, r, right=True) - 1, c // (d // groups))
    beta = -((x[r, c].float() - mean[at]) * (rstd[at] * gamma))
    y, mean, rstd = q.group_norm_fwd(x, groups, ptr, gamma, beta, act=q.ACT_RELU, max_rows=rows)
    _, _, dbeta = q.group_norm_bwd(torch.ones_like(x), x, groups, mean, rstd, ptr, gamma, beta, act=q.ACT_RELU,
                                   max_rows=rows)
    assert torch.equal(dbeta.double(), (y > 0).sum(0).double())
    # the elements at the edge are there: some passed, some did not
    assert 0.1 * d < (y[r, c] > 0).sum() < 0.9 * d
