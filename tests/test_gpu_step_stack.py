"""model.GCNStack with group normalization over a batch of graphs, class scores
from 8-bit integers and AdamW on its gradients: whole training steps, bit for
bit the sequence of calls they stand for, and against the layers chained in 64
bits.

The chain's bound is that of the other chained test: A, dZ, W and the head's
operands are rounded to bf16 (2^-8 relative, standard deviation 2^-8 / sqrt(3)),
sixteen roundings on a path give 0.9% of a result's 2-norm, and normalization's
backward pass can double what is left: 3%."""
import numpy as np
import pytest
import torch

import synth
from gpu_helpers import gq, rmat_small

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


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
    lab = np.random.default_rng(seed).integers(-classes // 2, classes, g.n).astype(np.int32)
    ptr = torch.tensor([0, 100, 100, 1200, 1201, g.n], device="cuda")
    return q, g, G, X, Ws, norms, Wc, torch.from_numpy(lab).cuda(), ptr


@pytest.mark.parametrize("state_bits", [8, 32])
@pytest.mark.parametrize("p", [0.0, 0.5])
def test_training_steps_are_their_calls(state_bits, p):
    from quantized_gnn_message_gb300.model import GCNStack
    widths, classes, groups, bits = (64, 96, 44), 30, 12, 2
    q, g, G, X, Ws, norms, Wc, lab, ptr = _setup(widths, classes, seed=5)
    mask = synth.bernoulli_mask(g.n, 0.5, seed=6).cuda()
    W2, n2 = [w.clone() for w in Ws], [tuple(t.clone() for t in pr) for pr in norms]
    Wc2 = torch.zeros(classes, 48, dtype=torch.bfloat16, device="cuda")[:, :44]
    Wc2.copy_(Wc)
    kw = dict(lr=1e-2, state_bits=state_bits, seed=9)
    model = GCNStack(G, widths, mask, norm="group", groups=groups, ptr=ptr, max_rows=1799, p=p, classes=classes)
    opt = model.optimizer(Ws, norms, Wc, **kw)
    by_hand = q.AdamW([*W2, *n2[0], Wc2], **kw)
    for step in range(2):
        model.forward(X, Ws, bits, [11, 12], norms=norms)
        loss = model.loss_and_grad(Wc, lab, 0.5)
        model.backward(None, Ws, bits, [21, 22], norms=norms)
        opt.step()
        s = 11 ^ q.DROPOUT_SEED_TAG
        A0, H0 = q.gcn_layer_fwd(G, X, W2[0], mask, bits, 11, q.ACT_NONE)
        N0, m0, r0 = q.group_norm_fwd(H0, groups, ptr, *n2[0], act=q.ACT_RELU, max_rows=1799)
        N0 = q.dropout(N0, p, s) if p else N0
        A1, H1 = q.gcn_layer_fwd(G, N0, W2[1], mask, bits, 12, q.ACT_NONE)
        loss2, dX, dWc = q.linear_xent(q.to_bf16(H1), Wc2, lab, scale=0.5)
        dW1, dN = q.gcn_layer_bwd(G, None, A1, None, W2[1], mask, bits, 22, q.ACT_NONE, dZ_in=dX)
        dN = q.dropout(dN, p, s) if p else dN
        dH0, dga, dbe = q.group_norm_bwd(dN, H0, groups, m0, r0, ptr, *n2[0], act=q.ACT_RELU, max_rows=1799)
        dW0, _ = q.gcn_layer_bwd(G, dH0, A0, H0, W2[0], mask, bits, 21, q.ACT_NONE, need_dinput=False)
        assert torch.equal(loss, loss2)
        for a, b in ((model.dWc, dWc), (model.dW[1], dW1), (model.dgamma[0], dga), (model.dbeta[0], dbe),
                     (model.dW[0], dW0)):
            assert torch.equal(a, b)
        by_hand.step([dW0, dW1, dga, dbe, dWc])
        for a, b in zip([*Ws, *norms[0], Wc], [*W2, *n2[0], Wc2]):
            assert torch.equal(a, b)
    assert int(model.err.item()) == 0
    codes, scale = q.quantize_i8(Wc)
    y = model.scores(codes, scale)
    qh, sh = q.quantize_i8(model.H[1])
    assert torch.equal(y, q.gemm_i8(qh, sh, codes, scale)) and y.shape == (g.n, classes)


def test_chain_in_64_bits(orc):
    """Two hidden layers with group normalization, without quantization or dropout."""
    from quantized_gnn_message_gb300.model import GCNStack
    widths, classes, groups = (40, 64, 48, 32), 20, 4
    q, g, G, X, Ws, norms, Wc, lab, ptr = _setup(widths, classes, seed=3)
    L = 3
    model = GCNStack(G, widths, None, norm="group", groups=groups, ptr=ptr, classes=classes)
    out = model.forward(X, Ws, 32, [1, 2, 3], norms=norms)
    loss = model.loss_and_grad(Wc, lab, 1.0)
    model.backward(None, Ws, 32, [4, 5, 6], need_input_grad=True, norms=norms)
    assert int(model.err.item()) == 0
    np64 = lambda t: t.double().cpu().numpy()
    rp, co = g.rowptr.numpy(), g.col.numpy()
    edges = ptr.tolist()

    def per_segment(x, fn):
        res = np.zeros_like(x)
        for a, b in zip(edges, edges[1:]):
            if b > a:
                res[a:b] = fn(x[a:b].reshape(b - a, groups, -1)).reshape(b - a, -1)
        return res

    def spread(x):
        m = per_segment(x, lambda v: np.broadcast_to(v.mean((0, 2), keepdims=True), v.shape))
        return m

    H, saved = np64(X), []
    for l in range(L):
        o = orc.gcn_layer_fwd(rp, co, orc.COEF_GCN, H.astype(np.float32), Ws[l].cpu().numpy(), None, 32, 0, relu=False)
        H = o["H_out"].astype(np.float64)
        if l < L - 1:
            ga, be = np64(norms[l][0]), np64(norms[l][1])
            xc = H - spread(H)
            r = 1 / np.sqrt(spread(xc * xc) + 1e-5)
            on = np64(model.N[l]) > 0  # a value within rounding of zero may fall either way
            o.update(xh=xc * r, r=r, on=on)
            H = np.where(on, xc * r * ga + be, 0.0)
        saved.append(o)

    def near(got, ref, what):
        e = np.linalg.norm(np64(got) - ref) / np.linalg.norm(ref)
        assert np.isfinite(np64(got)).all() and e < 0.03, f"{what}: {e}"

    near(out, H, "output")
    o = orc.linear_xent(H, np64(Wc), lab.cpu().numpy())
    near(loss, o["loss"], "loss")
    D = o["dX"]
    for l in reversed(range(L)):
        b = orc.gcn_layer_bwd(rp, co, orc.COEF_GCN, D.astype(np.float32), saved[l]["A"], saved[l]["Z"],
                              Ws[l].cpu().numpy(), None, 32, 0, relu=False, need_dinput=True)
        near(model.dW[l], b["dW"], f"layer {l} dW")
        D = b["dH_in"].astype(np.float64)
        if l > 0:
            s = saved[l - 1]
            dz = np.where(s["on"], D, 0.0)
            near(model.dgamma[l - 1], (dz * s["xh"]).sum(0), f"layer {l - 1} dgamma")
            near(model.dbeta[l - 1], dz.sum(0), f"layer {l - 1} dbeta")
            h = dz * np64(norms[l - 1][0])
            D = s["r"] * (h - spread(h) - s["xh"] * spread(h * s["xh"]))
    near(model.dH[0], D, "input gradient")


def test_captured_training_step():
    """Forward, loss, backward and a step that counts on the device as one graph."""
    from quantized_gnn_message_gb300.model import GCNStack
    widths, classes = (32, 64, 32), 10
    q, g, G, X, Ws, norms, Wc, lab, ptr = _setup(widths, classes, n=1500, seed=8)
    ptr = torch.tensor([0, 700, g.n], device="cuda")
    params = [*Ws, *norms[0], Wc]
    start = [t.clone() for t in params]
    model = GCNStack(G, widths, None, norm="group", groups=8, ptr=ptr, max_rows=800, classes=classes)
    opt = model.optimizer(Ws, norms, Wc, lr=1e-2, state_bits=8, seed=4, capturable=True)

    def step():
        model.forward(X, Ws, 32, [1, 2], norms=norms)
        model.loss_and_grad(Wc, lab, 1e-3)
        model.backward(None, Ws, 32, [3, 4], norms=norms)
        opt.step()

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in params]
    assert opt.device_steps().item() == 3
    for t, a in zip(params, start):
        t.copy_(a)
    eager = model.optimizer(Ws, norms, Wc, lr=1e-2, state_bits=8, seed=4, capturable=True)
    opt = eager
    for _ in range(3):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, params))


def test_refusals():
    from quantized_gnn_message_gb300.model import GCNStack
    q, g, G, X, Ws, norms, Wc, lab, ptr = _setup((16, 16, 8), 5, n=2000)
    for kw in (dict(norm="batch"), dict(norm="group", groups=3), dict(groups=2), dict(ptr=ptr),
               dict(norm="group", ptr=ptr.int())):
        with pytest.raises(q.GQError):
            GCNStack(G, (16, 16, 8), None, **kw)
    m = GCNStack(G, (16, 16, 8), None, norm="group", groups=4, ptr=ptr)
    for args in ((Ws[:1],), (Ws, norms + norms), (Ws, None, Wc)):
        with pytest.raises(q.GQError):
            m.optimizer(*args)
    with pytest.raises(q.GQError):
        GCNStack(G, (16, 16, 8), None).optimizer(Ws, norms)
