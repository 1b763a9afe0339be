"""gq_linear_xent where the label decides: rows whose label's logit is far above
the others, so that loss and gradient vanish, at ordinary and at large logits.

The label's logit and the sum of exponentials come from the same products, so
a logit's own rounding drops out of their difference.  The scaled logit is
x = z log2(e) - r with |x| <= 1 for the largest one; 2^x is off by 2^-22
relative, log2 of it by 2^-22 absolute, x itself is rounded once (2^-24): the
loss is off by at most 2^-20, and so is the label's p - 1."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq

pytestmark = pytest.mark.gpu

E = 2.0 ** -20


def _bf(rows, k, seed, scale):
    return (synth.normal_matrix(rows, k, seed=seed, device="cuda") * scale).to(torch.bfloat16)


# the logits' spread: 40 (a usual confident head), 5,000, 500,000
@pytest.mark.parametrize("spread", [40.0, 5e3, 5e5])
@pytest.mark.parametrize("n,k,C", [(500, 64, 40), (500, 256, 300), (700, 1024, 1000), (300, 72, 5003)])
def test_certain_rows(n, k, C, spread):
    q = gq()
    s = (spread / k ** 0.5) ** 0.5
    X, W = _bf(n, k, 1, s), _bf(C, k, 2, s)
    z = X.double() @ W.double().T
    top, lab = z.max(1)
    gap = top - z.scatter(1, lab[:, None], -np.inf).max(1)[0]
    sure = gap > 40.0  # the other classes have less than C e^-40 together
    assert sure.any()
    lab = torch.where(sure, lab, -1).to(torch.int32)
    loss, dX, dW = q.linear_xent(X, W, lab)
    assert (loss.abs() <= E).all(), f"loss of a certain row: {loss.abs().max().item()}"
    Wy = W.double()[lab.clamp(min=0).long()].abs()
    assert (dX.double().abs() <= E * Wy * 1.01).all(), f"{(dX.double().abs() / Wy).max().item()} of the label's row"
    assert (dW.double().abs() <= E * 1.01 * X.double().abs().sum(0)).all()
    # the losses alone are the same
    assert torch.equal(q.linear_xent(X, W, lab, grad=False)[0], loss)


# a single feature: every logit is exact.  log2(e) z is beyond 2^31 from 2e9
# on, where a step of it is 256
@pytest.mark.parametrize("size", [1e8, 1.2e9, 2e9, 3e10, 1e20, 1e38])
@pytest.mark.parametrize("C", [5, 256, 300, 5000])
def test_huge_logits(C, size):
    """Logits are apart by more than any exponential holds: the top class has
    probability 1, the loss is the difference to it."""
    q = gq()
    X = torch.zeros(6, 8, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = 1.0
    W = torch.zeros(C, 8, dtype=torch.bfloat16, device="cuda")
    top, low, mid = C - 1, 0, C // 2
    W[:, 0] = -1e6
    W[top, 0], W[low, 0], W[mid, 0] = size, -size / 2, size / 2
    lab = torch.tensor([top, low, mid, -1, 1, top], dtype=torch.int32, device="cuda")
    lse = torch.empty(6, device="cuda")
    loss, dX, dW = q.linear_xent(X, W, lab, lse=lse)
    w = W[:, 0].double()
    ref = torch.where(lab >= 0, w[top] - w[lab.long()], 0.0)
    # the scaled logits, their difference, ln 2 and the product: one rounding each
    assert ((loss.double() - ref).abs() <= 8 * 2.0 ** -24 * size + E).all() and (loss[[0, 5]].abs() <= E).all()
    assert ((lse.double() - torch.where(lab >= 0, w[top], 0.0)).abs() <= 8 * 2.0 ** -24 * size).all()
    # G = onehot(top) - onehot(label); half a step of bf16
    ref = torch.where(lab >= 0, w[top] - w[lab.long()], 0.0)
    assert ((dX[:, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + E * size).all() and not dX[:, 1:].any()
    G = torch.zeros(6, C, dtype=torch.float64, device="cuda")
    on = torch.nonzero(lab >= 0)[:, 0]
    G[on, top] = 1.0
    G[on, lab[on].long()] -= 1.0
    ref = G.T @ X.double()
    assert ((dW.double() - ref).abs() <= 2.0 ** -8 * ref.abs() * 1.01 + 6 * E).all()
