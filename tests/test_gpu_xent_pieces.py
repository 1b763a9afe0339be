"""gq_linear_xent where G takes several pieces of 1 GB (sums carried from piece
to piece, two buffers of G, a shorter last piece, split sums) and over the
longest contraction, against the formulas in 64 bits.

Bounds, h = 2^-8 half a step of bf16, relative:
  a sum of m products on the tensor cores takes m / 16 additions, each off by
  at most 2^-23 of what has been summed up, and 16 products of one addition
  are off by at most 2^-20 of their absolute sum;
  logits z:  dz = (k / 16) 2^-23 P + 2^-20 Zm, P the largest partial sum of
             blocks of 16, Zm = sum_k |x_k w_ck|;
  an exponential: relative 2^-22 + dz + (|z| + 1) 2^-22 from its scaled
             argument; a sum of C of them, chains of C / 32 and then 64 terms
             with errors of both signs: + (sqrt(C / 32) + 64) 2^-24
             =: d for an entry of G, twice that for loss and lse (in absolute
             terms), plus 2^-22 (|lse| + |z|);
  dX, dW:    each entry of G is rounded to bf16 once, so is the result:
             (h (1 + h) + 2 d + (m / 16 + 16) 2^-23) sum|G||W| + h |dX|, and
             2 (d + 2^-21) weight scale |W_y| (|x_i|) for the label's entry,
             whose p - 1 is off by p's error;
  dX, dW as a whole: the roundings of G's entries are independent of one
             another, at most h each: ||error|| <= h (||dX|| + sqrt(sum G^2
             W^2)) + the norm of the rest of the bound above.
A bound that is not far below the result itself would show nothing: its norm
is checked against the result's."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq

pytestmark = pytest.mark.gpu

H = 2.0 ** -8


def _bf(rows, k, seed, scale=1.0):
    buf = torch.full((rows, (k + 7) // 8 * 8), 99.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :k] = (synth.normal_matrix(rows, k, seed=seed, device="cuda") * scale).to(torch.bfloat16)
    return buf[:, :k]


def _labels(n, C, frac, seed):
    rng = np.random.default_rng(seed)
    lab = rng.integers(0, C, n)
    lab[rng.random(n) >= frac] = -1
    return torch.from_numpy(lab.astype(np.int32)).cuda()


def _logit_error(x, w):
    """dz of a few rows and all classes (the largest of them)."""
    k = x.shape[1]
    worst = 0.0
    for c in range(0, w.shape[0], 4096):
        t = torch.zeros(x.shape[0], len(w[c:c + 4096]), dtype=torch.float64, device="cuda")
        top, zm = t.clone(), t.clone()
        for i in range(0, k, 16):
            t += x[:, i:i + 16] @ w[c:c + 4096, i:i + 16].T
            zm += x[:, i:i + 16].abs() @ w[c:c + 4096, i:i + 16].abs().T
            top = torch.maximum(top, t.abs())
        worst = max(worst, (k / 16 * 2.0 ** -23 * top + 2.0 ** -20 * zm).max().item())
    return worst


def _close(got, ref, absref, root2, rel, label, m, what):
    rest = (rel + (m / 16 + 16) * 2.0 ** -23) * absref + label
    tol = H * (1 + H) * absref + H * ref.abs() + rest
    e = (got.double() - ref).abs()
    norm = torch.linalg.norm
    assert norm(tol) < 0.1 * norm(ref), f"{what}: the bound says nothing"
    assert torch.isfinite(got).all() and (e <= tol).all(), \
        f"{what}: {(e - tol).max().item()} over the bound, {(e > tol).sum().item()} of {e.numel()}"
    assert norm(e) <= H * (norm(ref) + root2) + norm(rest), f"{what}: norm of the error"


def _check(q, X, W, lab, weight=None, scale=1.0):
    n, k = X.shape
    C = W.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((n,), 7.0, device="cuda")
    loss, dX, dW = q.linear_xent(X, W, lab, weight, scale, lse=lse, dev_err=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    f64 = dict(dtype=torch.float64, device="cuda")
    x, w = X.double(), W.double()
    step = max(1, (1 << 26) // C)
    rdX, adX, label_X = (torch.zeros(n, k, **f64) for _ in range(3))
    rdW, adW, label_W = (torch.zeros(C, k, **f64) for _ in range(3))
    sqX = sqW = 0.0
    on = (lab >= 0) & (lab < C)
    rows = torch.nonzero(on)[:, 0]
    few = rows[:: max(1, len(rows) // 64)][:64]
    dz = 2 * _logit_error(x[few], w)  # rows of one distribution: twice the largest of 64
    zmax = 0.0
    worst = torch.zeros(2, **f64)
    for r in range(0, n, step):
        at = rows[(rows >= r) & (rows < r + step)]
        if not len(at):
            continue
        y = lab[at].long()
        z = x[at] @ w.T
        zmax = max(zmax, z.abs().max().item())
        e_lse = torch.logsumexp(z, 1)
        e_loss = e_lse - z[torch.arange(len(at), device="cuda"), y]
        d = dz + (zmax + 2) * 2.0 ** -22 + ((C / 32) ** 0.5 + 64) * 2.0 ** -24
        bound = 2 * d + 2.0 ** -22 * (e_lse.abs() + zmax)
        worst = torch.maximum(worst, torch.stack([((loss[at].double() - e_loss).abs() - bound).max(),
                                                  ((lse[at].double() - e_lse).abs() - bound).max()]))
        g = torch.exp(z - e_lse[:, None])
        g[torch.arange(len(at), device="cuda"), y] -= 1.0
        wt = torch.ones(len(at), **f64) if weight is None else weight[at].double()
        g *= (scale * wt)[:, None]
        rdX[at], adX[at] = g @ w, g.abs() @ w.abs()
        rdW += g.T @ x[at]
        adW += g.abs().T @ x[at].abs()
        one = 2 * (d + 2.0 ** -21) * scale * wt[:, None]
        label_X[at] = one * w[y].abs()
        label_W.index_add_(0, y, one * x[at].abs())
        g.square_()
        sqX += (g @ w.square()).sum().item()
        sqW += (g.T @ x[at].square()).sum().item()
    assert worst.max() <= 0, f"loss, lse over the bound by {worst.tolist()}"
    assert not loss[~on].any() and not lse[~on].any() and not dX[~on].any()
    _close(dX, rdX, adX, sqX ** 0.5, 2 * d, label_X, C, "dX")
    _close(dW, rdW, adW, sqW ** 0.5, 2 * d, label_W, n, "dW")


# classes per piece: 192 of 520 (its last 256-class tile of dW reaches into the
# next piece), 256 of 600, 92, 92 and 90 tiles of 256, 10 tiles of 256 with the
# sums of dW split, 4,493 tiles with the sums of dX split, three column tiles
# of the gradients
@pytest.mark.parametrize("n,k,C", [(1_500_000, 8, 520), (1_200_000, 24, 600), (20_000, 72, 70_001),
                                   (200_000, 16, 30_000), (250, 16, 2_300_000), (20_000, 520, 30_000)])
@pytest.mark.parametrize("frac", [1.0, 0.5])
def test_several_pieces(n, k, C, frac):
    assert 2 * n * C > 1 << 30, "G fits one piece"
    q = gq()
    weight = torch.rand(n, device="cuda") + 0.5 if frac < 1 else None
    _check(q, _bf(n, k, 1), _bf(C, k, 2, 2 / k ** 0.5), _labels(n, C, frac, 3), weight, 1.0)
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n,k,C", [(5, 16384, 70), (300, 16384, 300), (300, 8192, 47)])
def test_longest_contraction(n, k, C):
    q = gq()
    _check(q, _bf(n, k, 1), _bf(C, k, 2, 2 / k ** 0.5), _labels(n, C, 0.9, 3))


@pytest.mark.parametrize("n,k,C", [(1_500_000, 8, 520), (1_200_000, 24, 600)])
def test_short_tiles_of_several_pieces_are_the_same_every_time(n, k, C):
    """Tiles of three or four steps whose epilogues move more than their
    products take: the units posted ahead are read late.  Nothing may be left
    unwritten (NaN in every buffer beforehand) and nothing done twice."""
    q = gq()
    X, W, lab = _bf(n, k, 1), _bf(C, k, 2, 2 / k ** 0.5), _labels(n, C, 1.0, 3)
    ws, first = q.Workspace(), None
    dX, dW = torch.empty(n, k, dtype=torch.bfloat16, device="cuda"), torch.empty(C, k, dtype=torch.bfloat16, device="cuda")
    loss = torch.empty(n, device="cuda")
    ws.get(int(q.lib().gq_linear_xent_workspace_bytes(n, k, C, 1)))
    for _ in range(12):
        for t in (ws.buf, dX.view(torch.uint8), dW.view(torch.uint8), loss.view(torch.uint8)):
            t.fill_(255)
        q.linear_xent(X, W, lab, ws=ws, loss=loss, dX=dX, dW=dW)
        if first is None:
            first = [t.clone() for t in (loss, dX, dW)]
            assert all(torch.isfinite(t).all() for t in first)
        assert all(torch.equal(a, b) for a, b in zip(first, (loss, dX, dW)))
    del ws, dX
    torch.cuda.empty_cache()


def test_one_gradient_of_several_pieces():
    q = gq()
    n, k, C = 1_200_000, 24, 600
    X, W, lab = _bf(n, k, 1), _bf(C, k, 2, 2 / k ** 0.5), _labels(n, C, 0.7, 3)
    loss, dX, dW = q.linear_xent(X, W, lab)
    a, b = q.linear_xent(X, W, lab, need_dW=False), q.linear_xent(X, W, lab, need_dX=False)
    assert torch.equal(a[0], loss) and torch.equal(a[1], dX) and a[2] is None
    assert torch.equal(b[0], loss) and torch.equal(b[2], dW) and b[1] is None
    torch.cuda.empty_cache()
