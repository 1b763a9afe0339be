"""The class head's cross entropy and gradients (gq_linear_xent) against the
oracle's float64 form on the same bf16 inputs.

Bounds, u = 2^-24, Zm = max_c sum_k |x_k w_ck| of a row:
  logits: at most k roundings of the products' fp32 sum, each at most u Zm
          (the tensor cores add 16 products at a time; k bounds any order);
  loss:   the label's logit and lse are both off by at most k u Zm; an
          exponential is off by 2^-22 relative plus u |z| log2(e) from its
          scaled argument, the sum of C of them by (C / 32 + 64) u, the
          logarithm and the final sums by 4 u (|lse| + Zm):
          2 k u Zm + (8 + 6 Zm + C / 32 + 64) u + 4 u (|lse| + Zm)
  dX, dW: each G entry is rounded to bf16 once: bf16 has 8 significant bits,
          neighbours at 1 are eps = 2^-7 apart, so half a step is eps / 2 =
          2^-8 relative; on top of the relative error d of its exponential,
          d = the bound of lse; sums are exact to (terms) u; the result is
          rounded to bf16: with h = 2^-8
          (h (1 + h) + 2 d + terms u) sum|G||W| + h |dX|;
          the label's G is a difference p - 1, so its error counts against 1:
          2 (d + 8 u) weight scale |W_y| more (|x_i| for dW's row y)"""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
H = 2.0 ** -8


def _bf(rows, k, seed, scale=1.0, ld=None):
    ld = ld or (k + 7) // 8 * 8
    buf = torch.full((rows, ld), 99.0, dtype=torch.bfloat16, device="cuda")
    buf[:, :k] = (synth.normal_matrix(rows, k, seed=seed, device="cuda") * scale).to(torch.bfloat16)
    return buf[:, :k]


def _labels(n, C, frac, seed):
    rng = np.random.default_rng(seed)
    lab = rng.integers(0, C, n)
    lab[rng.random(n) >= frac] = rng.choice([-1, -100, C, 2 ** 31 - 1])
    return torch.from_numpy(lab.astype(np.int32)).cuda()


def _np(t):
    return t.double().cpu().numpy()


def _check(q, orc, X, W, lab, weight=None, scale=1.0, **kw):
    n, k = X.shape
    C = W.shape[0]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.full((n,), 7.0, device="cuda")
    loss, dX, dW = q.linear_xent(X, W, lab, weight, scale, lse=lse, dev_err=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    o = orc.linear_xent(_np(X), _np(W), lab.cpu().numpy(), None if weight is None else _np(weight), scale)
    rows = o["rows"]
    zm = o["absZ"]
    t = np.zeros(n)
    t[rows] = 2 * k * U * zm + (72 + 6 * zm + C / 32) * U + 4 * U * (np.abs(o["lse"][rows]) + zm)
    for got, name in ((loss, "loss"), (lse, "lse")):
        e = np.abs(_np(got) - o[name]) - t
        assert e.max(initial=-1) <= 0, f"{name}: {e.max()} over the bound at {e.argmax()}"
    d = 2 * t[rows].max(initial=0)
    y = lab.cpu().numpy()[rows]
    one = np.zeros((n, C))
    one[rows, y] = 2 * (d + 8 * U) * scale * (1.0 if weight is None else _np(weight)[rows])
    label = {"dX": one @ np.abs(_np(W)), "dW": one[rows].T @ np.abs(_np(X)[rows])}
    for got, name, terms in ((dX, "dX", C), (dW, "dW", n)):
        if got is None:
            continue
        tol = (H * (1 + H) + 2 * d + terms * U) * o["abs" + name] + H * np.abs(o[name]) * (1 + d)
        tol = tol + label[name] * (1 + H)
        g = _np(got)
        e = np.abs(g - o[name]) - tol
        ok = bool(np.isfinite(g).all() and e.max(initial=-1) <= 1e-30)
        assert ok, f"{name}: {e.max()} over the bound at {np.unravel_index(e.argmax(), e.shape)}"
    return loss, dX, dW


@pytest.mark.parametrize("n,k,C", [(1, 1, 1), (1, 8, 2), (5, 16, 47), (64, 64, 64), (127, 100, 65), (128, 128, 128),
                                   (129, 136, 255), (256, 256, 256), (257, 264, 257), (300, 72, 1000),
                                   (1000, 256, 47), (513, 520, 2049), (37, 1024, 5003), (2050, 40, 513),
                                   (3, 2000, 30)])
@pytest.mark.parametrize("frac", [1.0, 0.6])
def test_loss_and_gradients(orc, n, k, C, frac):
    q = gq()
    X, W = _bf(n, k, n + k), _bf(C, k, C + 1, 2.0 / np.sqrt(k))
    weight = torch.rand(n, device="cuda") + 0.5 if C % 2 else None
    _check(q, orc, X, W, _labels(n, C, frac, n + C), weight, 1.0 / n)


def test_single_column_strides_and_padding(orc):
    # wider pitches; what stands past column k is neither used nor written
    q = gq()
    X, W = _bf(70, 50, 1, ld=64), _bf(90, 50, 2, 0.3, ld=72)
    lab = _labels(70, 90, 0.8, 3)
    dXb = torch.full((70, 80), 5.0, dtype=torch.bfloat16, device="cuda")
    dWb = torch.full((90, 56), 6.0, dtype=torch.bfloat16, device="cuda")
    _check(q, orc, X, W, lab, dX=dXb[:, :50], dW=dWb[:, :50])
    assert (dXb[:, 50:] == 5).all() and (dWb[:, 50:] == 6).all()


def test_many_pieces_of_the_classes(orc):
    # G larger than one piece: sums carried from piece to piece
    q = gq()
    n, k, C = 70_000, 24, 1500
    X, W = _bf(n, k, 1), _bf(C, k, 2, 0.5)
    _check(q, orc, X, W, _labels(n, C, 0.9, 5), None, 1.0 / n)


def test_long_sums_are_split(orc):
    # few output tiles over a long contraction, both ways round
    q = gq()
    _check(q, orc, _bf(60_000, 64, 1), _bf(47, 64, 2, 0.4), _labels(60_000, 47, 0.5, 1), None, 1e-3)
    _check(q, orc, _bf(40, 64, 3), _bf(60_000, 64, 4, 0.4), _labels(40, 60_000, 1.0, 2))


def test_few_classes_many_rows(orc):
    # tiles that hold every class, by turns to two warps; every row labelled,
    # so that gradients leave in whole boxes
    q = gq()
    _check(q, orc, _bf(40_003, 72, 5), _bf(200, 72, 6, 0.4), _labels(40_003, 200, 1.0, 3), None, 1e-3)
    _check(q, orc, _bf(20_481, 64, 7), _bf(3, 64, 8, 0.4), _labels(20_481, 3, 0.9, 4))


def test_no_labelled_row():
    q = gq()
    X, W = _bf(300, 64, 1), _bf(500, 64, 2)
    X.fill_(float("nan"))
    lse = torch.full((300,), 3.0, device="cuda")
    loss, dX, dW = q.linear_xent(X, W, torch.full((300,), -1, dtype=torch.int32, device="cuda"), lse=lse)
    assert not loss.any() and not lse.any() and not dX.any() and not dW.any()
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    loss, dX, dW = q.linear_xent(e, W, torch.empty(0, dtype=torch.int32, device="cuda"))
    assert loss.numel() == 0 and dX.shape == (0, 64) and not dW.any()


def test_unlabelled_rows_may_hold_anything(orc):
    q = gq()
    X, W = _bf(600, 96, 1), _bf(300, 96, 2, 0.3)
    lab = _labels(600, 300, 0.5, 4)
    clean = _check(q, orc, X, W, lab)
    off = (lab < 0) | (lab >= 300)
    Y = X.clone()
    Y[off] = float("inf")
    Y[off, 3] = float("nan")
    w = torch.ones(600, device="cuda")
    w[off] = float("nan")
    dirty = q.linear_xent(Y, W, lab, w)
    assert all(torch.equal(a, b) for a, b in zip(clean, dirty))


def test_extreme_logits(orc):
    q = gq()
    X = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(64, 8, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = 1.0
    W[:, 0] = torch.linspace(-30000, 30000, 64).bfloat16()
    lab = torch.tensor([63, 0, 31, -1], dtype=torch.int32, device="cuda")
    loss, dX, dW = _check(q, orc, X, W, lab)
    # a certain row: loss 0 and no gradient beyond the exponential's 2^-20
    assert loss[0].abs() < 2.0 ** -20 and dX[0].abs().max() < 2.0 ** -20 * 30000
    # z L - r, the final product and ln 2 are rounded once each
    assert abs(loss[1].item() / (2 * W[63, 0].item()) - 1) < 4 * U
    # a logit of -inf has probability zero and does not spoil the others
    W[5, 0] = float("-inf")
    loss, _, _ = q.linear_xent(X, W, lab, grad=False)
    assert torch.isfinite(loss).all() and loss[0].abs() < 2.0 ** -20
    # a run of classes that are all -inf
    W[:, 0] = float("-inf")
    W[60, 0] = 2.0
    loss, _, _ = q.linear_xent(X, W, torch.full((4,), 60, dtype=torch.int32, device="cuda"), grad=False)
    assert loss.abs().max() < 2.0 ** -20


def test_one_gradient_only():
    q = gq()
    X, W, lab = _bf(200, 64, 1), _bf(333, 64, 2, 0.3), _labels(200, 333, 0.7, 1)
    loss, dX, dW = q.linear_xent(X, W, lab)
    a = q.linear_xent(X, W, lab, need_dW=False)
    b = q.linear_xent(X, W, lab, need_dX=False)
    c = q.linear_xent(X, W, lab, grad=False)
    assert torch.equal(a[1], dX) and a[2] is None and torch.equal(b[2], dW) and b[1] is None
    assert c[1] is None and c[2] is None and all(torch.equal(t[0], loss) for t in (a, b, c))


def test_same_results_every_time():
    q = gq()
    X, W, lab = _bf(3000, 200, 1), _bf(7000, 200, 2, 0.2), _labels(3000, 7000, 0.9, 1)
    ws = q.Workspace()
    first = q.linear_xent(X, W, lab, ws=ws)
    ws.buf.fill_(255)  # NaN in every float of the workspace
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, q.linear_xent(X, W, lab, ws=ws)))


def test_gradients_are_differences(orc):
    """dX and dW against central differences of the library's own loss."""
    q = gq()
    n, k, C = 6, 16, 40
    X, W = _bf(n, k, 1, 0.5), _bf(C, k, 2, 0.5)
    lab = torch.tensor([0, 5, 39, -1, 7, 7], dtype=torch.int32, device="cuda")
    _, dX, dW = q.linear_xent(X, W, lab)
    h = 2.0 ** -2
    for M, D, at in ((X, dX, [(0, 0), (1, 7), (5, 15), (3, 2)]), (W, dW, [(0, 1), (39, 3), (7, 8), (20, 0)])):
        for i, j in at:
            old = M[i, j].item()
            f = []
            for s in (+1, -1):
                M[i, j] = old + s * h
                f.append((q.linear_xent(X, W, lab, grad=False)[0].double().sum().item(), M[i, j].item()))
            M[i, j] = old
            slope = (f[0][0] - f[1][0]) / (f[0][1] - f[1][1])
            # the difference is off by h^2 / 6 times the third derivative: at
            # most |entry|^3 / 10 a row, entries below 2, six rows at most
            assert abs(slope - D[i, j].item()) < 0.05 + 2.0 ** -8 * abs(slope)


def test_two_streams_and_captured(orc):
    q = gq()
    X, W, lab = _bf(900, 128, 1), _bf(2000, 128, 2, 0.2), _labels(900, 2000, 0.8, 1)
    ref = q.linear_xent(X, W, lab)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:
        with torch.cuda.stream(st):
            outs.append([q.linear_xent(X, W, lab, ws=q.Workspace()) for _ in range(3)])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for r in o for a, b in zip(ref, r))
    ws = q.Workspace()
    q.linear_xent(X, W, lab, ws=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = q.linear_xent(X, W, lab, ws=ws)
    lab.copy_(_labels(900, 2000, 0.3, 9))  # another number of labelled rows
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, q.linear_xent(X, W, lab)))


def test_refusals_of_the_binding():
    q = gq()
    X, W, lab = _bf(20, 16, 1), _bf(30, 16, 2), torch.zeros(20, dtype=torch.int32, device="cuda")
    odd = torch.zeros(20, 17, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: q.linear_xent(X.float(), W, lab), lambda: q.linear_xent(X, W[:, :8], lab),
                 lambda: q.linear_xent(X, W, lab.long()), lambda: q.linear_xent(X, W, lab[:-1]),
                 lambda: q.linear_xent(odd[:, :16], W, lab), lambda: q.linear_xent(X, W, lab, lab.float()[:3]),
                 lambda: q.linear_xent(X, W, lab, dX=torch.empty(20, 16, device="cuda")),
                 lambda: q.linear_xent(X.t(), W, lab), lambda: q.linear_xent(X, W.cpu(), lab)):
        with pytest.raises(q.GQError):
            call()


def test_rows_and_classes_off_the_grid_are_refused():
    q = gq()
    buf = torch.zeros(20, 32, dtype=torch.bfloat16, device="cuda")
    lab = torch.zeros(20, dtype=torch.int32, device="cuda")
    for X, W in ((buf[:, 1:17], buf[:, :16]), (buf[:, :16], buf[:, 4:20])):
        with pytest.raises(q.GQError):
            q.linear_xent(X, W, lab)


def test_weights_and_the_same_class_everywhere(orc):
    # one class takes every label; weights of both signs and zero
    q = gq()
    X, W = _bf(700, 48, 1), _bf(600, 48, 2, 0.3)
    w = torch.linspace(-1.0, 1.0, 700, device="cuda")
    w[100:200] = 0.0
    _check(q, orc, X, W, torch.full((700,), 599, dtype=torch.int32, device="cuda"), w.abs(), 0.125)
    a = q.linear_xent(X, W, torch.full((700,), 599, dtype=torch.int32, device="cuda"), w, 1.0)
    b = q.linear_xent(X, W, torch.full((700,), 599, dtype=torch.int32, device="cuda"), -w, -1.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert not a[1][100:200].any()


@pytest.mark.parametrize("n,k,C,frac", [(5, 16384, 70, 1.0), (2, 64, 200_000, 1.0), (70_000, 8, 3000, 0.3),
                                        (1, 256, 131_072, 1.0)])
def test_long_axes(orc, n, k, C, frac):
    q = gq()
    _check(q, orc, _bf(n, k, 1), _bf(C, k, 2, 2.0 / np.sqrt(k)), _labels(n, C, frac, 3), None, 1.0 / n)


def test_offsets_past_32_bits():
    """X and dX of more than 2^32 elements: the last rows' losses and gradients
    are those of a call on them alone (a row's depend on the row and W only)."""
    q = gq()
    n, k, C, last = (1 << 24) + 300, 264, 70, 333
    X = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    X[-last:] = _bf(last, k, 1)
    W = _bf(C, k, 2, 0.2)
    lab = torch.zeros(n, dtype=torch.int32, device="cuda")
    lab[-last:] = torch.arange(last, dtype=torch.int32, device="cuda") % C
    few = q.linear_xent(X[-last:], W, lab[-last:].contiguous())
    loss, dX, _ = q.linear_xent(X, W, lab)  # every row labelled
    assert torch.equal(loss[-last:], few[0]) and torch.equal(dX[-last:], few[1])
    del dX
    lab[:-last] = -1                        # none but the last
    loss, dX, dW = q.linear_xent(X, W, lab)
    assert torch.equal(loss[-last:], few[0]) and torch.equal(dX[-last:], few[1]) and not dX[:-last].any()
    assert torch.linalg.norm((dW - few[2]).double()) <= 2.0 ** -7 * torch.linalg.norm(few[2].double())
    del X, dX
    torch.cuda.empty_cache()
