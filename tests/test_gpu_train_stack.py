"""model.GCNStack with normalization, dropout and a class head: the chain a
training step runs, against the oracle's layers chained in float64 with the
GPU's own ReLU bits (a gate of a value within rounding of zero may fall either
way; every other value of the chain is the oracle's own).

The chain rounds A, dZ, W and the head's operands to bf16: half a step is 2^-8
relative, at most four such roundings lie on a path through one layer (A, W
forward; dZ, W backward), and three layers and the head make sixteen.
Independent roundings add up as their root sum of squares, uniform ones have a
standard deviation of 2^-8 / sqrt(3): sqrt(16) 2^-8 / sqrt(3) = 0.9% of the
norm; normalization's backward pass takes the mean out and can double what is
left relative to it.  Bound: 3% of each result's 2-norm."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq, rmat_small

pytestmark = pytest.mark.gpu


def _setup(widths, classes, n=3000, seed=0):
    q = gq()
    g = rmat_small(scale=12, n=n, deg=12, seed=seed + 1)
    G = q.graph_prepare(g.rowptr.cuda(), g.col.cuda())
    X = synth.normal_matrix(g.n, widths[0], seed=seed + 2).cuda()
    L = len(widths) - 1
    Ws = [synth.glorot(widths[l], widths[l + 1], seed=seed + 3 + l).cuda() for l in range(L)]
    norms = [(1 + 0.2 * synth.normal_matrix(1, widths[l + 1], seed=seed + 30 + l).cuda()[0],
              0.2 * synth.normal_matrix(1, widths[l + 1], seed=seed + 40 + l).cuda()[0]) for l in range(L - 1)]
    Wc = torch.zeros(classes, (widths[L] + 7) // 8 * 8, dtype=torch.bfloat16, device="cuda")[:, :widths[L]]
    Wc.copy_(synth.normal_matrix(classes, widths[L], seed=seed + 50).cuda() * 0.3)
    rng = np.random.default_rng(seed)
    lab = rng.integers(0, classes, g.n)
    lab[rng.random(g.n) < 0.4] = -1
    return q, g, G, X, Ws, norms, Wc, torch.from_numpy(lab.astype(np.int32)).cuda()


def _near(got, ref, what):
    got = got.double().cpu().numpy()
    e = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert np.isfinite(got).all() and e < 0.03, f"{what}: {e}"


def _unpack(bits, d):
    w = bits.cpu().numpy().view(np.uint32)
    c = np.arange(d)
    return ((w[:, c // 32] >> (c % 32).astype(np.uint32)) & 1).astype(bool)


@pytest.mark.parametrize("widths,classes,p", [((100, 128, 256, 64), 47, 0.5), ((64, 44, 33), 1000, 0.25),
                                              ((40, 64), 10, 0.0)])
def test_normalized_stack_with_head_matches_chained_oracle(orc, widths, classes, p):
    from quantized_gnn_message_gb300.model import GCNStack
    q, g, G, X, Ws, norms, Wc, lab = _setup(widths, classes)
    L = len(widths) - 1
    model = GCNStack(G, widths, None, norm=True, p=p, classes=classes)
    sf = [synth.layer_seed(0, l, False) for l in range(L)]
    sb = [synth.layer_seed(0, l, True) for l in range(L)]
    out = model.forward(X, Ws, 32, sf, norms=norms)
    loss = model.loss_and_grad(Wc, lab, 1.0)
    model.backward(None, Ws, 32, sb, need_input_grad=True, norms=norms)
    torch.cuda.synchronize()
    assert int(model.err.item()) == 0 and int(G.status.cpu()[0]) == 0

    rp, co = g.rowptr.numpy(), g.col.numpy()
    np64 = lambda t: t.double().cpu().numpy()
    H, saved = np64(X), []
    for l in range(L):
        o = orc.gcn_layer_fwd(rp, co, orc.COEF_GCN, H.astype(np.float32), Ws[l].cpu().numpy(), None, 32, 0, relu=False)
        H = o["H_out"]
        if l < L - 1:
            ga, be = np64(norms[l][0]), np64(norms[l][1])
            f = orc.layer_norm_fwd(H, ga, be)
            on = _unpack(model.Rb[l], widths[l + 1])
            o.update(f, on=on, H=H)
            H = orc.dropout(np.where(on, f["z"], 0.0), p, sf[l] ^ q.DROPOUT_SEED_TAG)
        saved.append(o)
    _near(out, H, "output")
    o = orc.linear_xent(H, np64(Wc), lab.cpu().numpy())
    _near(loss, o["loss"], "loss")
    _near(model.dWc, o["dW"], "head gradient")
    D = o["dX"]
    for l in reversed(range(L)):
        b = orc.gcn_layer_bwd(rp, co, orc.COEF_GCN, D.astype(np.float32), saved[l]["A"], saved[l]["Z"],
                              Ws[l].cpu().numpy(), None, 32, 0, relu=False, need_dinput=True)
        _near(model.dW[l], b["dW"], f"layer {l} dW")
        D = b["dH_in"]
        if l > 0:
            s = saved[l - 1]
            b = orc.layer_norm_bwd(D, s["H"], s["mean"], s["rstd"], np64(norms[l - 1][0]), s["on"], p,
                                   sf[l - 1] ^ q.DROPOUT_SEED_TAG)
            _near(model.dgamma[l - 1], b["dgamma"], f"layer {l - 1} dgamma")
            _near(model.dbeta[l - 1], b["dbeta"], f"layer {l - 1} dbeta")
            D = b["dX"]
    _near(model.dH[0], D, "input gradient")


@pytest.mark.parametrize("bits", [2, 32])
def test_stack_step_is_its_calls(bits):
    """The stack's quantized training step, bit for bit the sequence of the
    library's calls that it stands for."""
    from quantized_gnn_message_gb300.model import GCNStack
    widths, classes, p = (64, 96, 40), 30, 0.5
    q, g, G, X, Ws, norms, Wc, lab = _setup(widths, classes, seed=5)
    mask = synth.bernoulli_mask(g.n, 0.5, seed=6).cuda()
    model = GCNStack(G, widths, mask, norm=True, p=p, classes=classes)
    loss = None
    for _ in range(2):  # the second step finds the first one's buffers
        model.forward(X, Ws, bits, [11, 12], norms=norms)
        loss = model.loss_and_grad(Wc, lab, 0.5)
        model.backward(None, Ws, bits, [21, 22], norms=norms)
    A0, H0 = q.gcn_layer_fwd(G, X, Ws[0], mask, bits, 11, q.ACT_NONE)
    rb = torch.empty(g.n, 3, dtype=torch.int32, device="cuda")
    s = 11 ^ q.DROPOUT_SEED_TAG
    N0, m0, r0 = q.layer_norm_fwd(H0, *norms[0], act=q.ACT_RELU, p=p, seed=s, relu_bits=rb)
    A1, H1 = q.gcn_layer_fwd(G, N0, Ws[1], mask, bits, 12, q.ACT_NONE)
    loss2, dX, dWc = q.linear_xent(q.to_bf16(H1), Wc, lab, scale=0.5)
    dW1, dN = q.gcn_layer_bwd(G, None, A1, None, Ws[1], mask, bits, 22, q.ACT_NONE, dZ_in=dX)
    dz = torch.empty(g.n, 96, dtype=torch.bfloat16, device="cuda")
    _, dga, dbe = q.layer_norm_bwd(dN, H0, m0, r0, norms[0][0], act=q.ACT_RELU, p=p, seed=s, relu_bits=rb, dX=dz)
    dW0, _ = q.gcn_layer_bwd(G, None, A0, None, Ws[0], mask, bits, 21, q.ACT_NONE, need_dinput=False, dZ_in=dz)
    torch.cuda.synchronize()
    assert int(model.err.item()) == 0
    for a, b in ((loss, loss2), (model.dWc, dWc), (model.dW[1], dW1), (model.dgamma[0], dga), (model.dbeta[0], dbe),
                 (model.dW[0], dW0)):
        assert torch.equal(a, b)


def test_dropout_without_norm_and_evaluation(orc):
    from quantized_gnn_message_gb300.model import GCNStack
    widths = (64, 48, 24)
    q, g, G, X, Ws, _, _, _ = _setup(widths, 5, seed=9)
    dY = synth.normal_matrix(g.n, 24, seed=3).cuda()
    model = GCNStack(G, widths, None, p=0.4)
    model.forward(X, Ws, 32, [1, 2])
    H0, N0 = model.H[0].clone(), model.N[0].clone()
    assert torch.equal(N0, q.dropout(H0, 0.4, 1 ^ q.DROPOUT_SEED_TAG))
    model.backward(dY, Ws, 32, [3, 4])
    # by hand: the unfused stack's layer calls around the same dropout
    A1, _ = q.gcn_layer_fwd(G, N0, Ws[1], None, 32, 2, q.ACT_NONE)
    dW1, dN = q.gcn_layer_bwd(G, dY, A1, None, Ws[1], None, 32, 4, q.ACT_NONE)
    q.dropout(dN, 0.4, 1 ^ q.DROPOUT_SEED_TAG, out=dN)
    dW0, _ = q.gcn_layer_bwd(G, dN, model.A[0], H0, Ws[0], None, 32, 3, q.ACT_RELU, need_dinput=False)
    assert torch.equal(model.dW[1], dW1) and torch.equal(model.dW[0], dW0)
    # evaluation: no dropout, the plain stack's output; no backward pass from it
    y = model.forward(X, Ws, 32, [1, 2], training=False)
    plain = GCNStack(G, widths, None)
    assert torch.equal(y, plain.forward(X, Ws, 32, [1, 2]))
    with pytest.raises(q.GQError):
        model.backward(dY, Ws, 32, [3, 4])


def test_head_on_the_plain_stack(orc):
    """A head on a stack without norm or dropout: the fused hand-off below it
    gives the weight gradients of the same stack fed with the head's dX."""
    from quantized_gnn_message_gb300.model import GCNStack
    widths, classes = (64, 128, 64, 32), 300
    q, g, G, X, Ws, _, Wc, lab = _setup(widths, classes, seed=13)
    a = GCNStack(G, widths, None, classes=classes)
    a.forward(X, Ws, 32, [1, 2, 3])
    la = a.loss_and_grad(Wc, lab, 1e-2).clone()
    a.backward(None, Ws, 32, [4, 5, 6])
    assert torch.equal(a.loss(Wc, lab), la)
    b = GCNStack(G, widths, None, fuse_dz=False)
    out = b.forward(X, Ws, 32, [1, 2, 3])
    lb, dX, dWc = q.linear_xent(q.to_bf16(out), Wc, lab, scale=1e-2)
    b.backward(dX.float(), Ws, 32, [4, 5, 6])
    assert torch.equal(la, lb) and torch.equal(a.dWc, dWc)
    for l in range(3):
        assert torch.equal(a.dW[l], b.dW[l])


def test_refusals():
    from quantized_gnn_message_gb300.model import GCNStack
    q, g, G, X, Ws, norms, Wc, lab = _setup((16, 16, 8), 5, n=200)
    with pytest.raises(q.GQError):
        GCNStack(G, (16, 16, 8), None, p=1.5)
    m = GCNStack(G, (16, 16, 8), None, norm=True)
    with pytest.raises(q.GQError):
        m.forward(X, Ws, 32, [1, 2], norms=norms + norms)
    m.forward(X, Ws, 32, [1, 2], norms=norms)
    with pytest.raises(q.GQError):
        m.backward(None, Ws, 32, [1, 2], norms=norms)
    with pytest.raises(q.GQError):
        m.loss(Wc, lab)
