"""The order of model.GCNStack's calls, on the host: the library's calls are
replaced by records of their arguments, so nothing is launched."""
import pytest
import torch


@pytest.fixture
def stack(monkeypatch):
    """(GQError, make): make(**options) builds a stack over 5 nodes whose
    library calls are recorded in stack.calls."""
    import quantized_gnn_message_gb300 as q
    from quantized_gnn_message_gb300 import build, model
    build.build()
    c = q.Graph_t()
    c.n = 5
    empty = torch.empty(0, dtype=torch.int32)
    g = q.Graph(5, 0, empty, empty, empty, c)

    def make(widths=(8, 8, 8), **kw):
        st = model.GCNStack(g, widths, None, device="cpu", **kw)
        st.calls = []
        for name in ("gcn_layer_fwd", "gcn_layer_bwd", "layer_norm_fwd", "layer_norm_bwd", "dropout", "to_bf16",
                     "linear_xent"):
            def record(*a, _name=name, **k):
                st.calls.append((_name, a, k))
                return (st.node_loss,) if _name == "linear_xent" else a[0]
            monkeypatch.setattr(model, name, record)
        return st

    return q.GQError, make


X = torch.zeros(5, 8)
WS = [torch.zeros(8, 8)] * 2
WC = torch.zeros(3, 8, dtype=torch.bfloat16)
LAB = torch.zeros(5, dtype=torch.int32)


def test_backward_from_the_head_follows_loss_and_grad(stack):
    err, make = stack
    m = make(classes=3)
    with pytest.raises(err):
        m.backward(None, WS, 32, [1, 2])       # before any pass
    m.forward(X, WS, 32, [1, 2])
    with pytest.raises(err):
        m.backward(None, WS, 32, [1, 2])       # no gradient yet
    m.loss(WC, LAB)
    with pytest.raises(err):
        m.backward(None, WS, 32, [1, 2])       # losses only
    assert not any(c[0] == "gcn_layer_bwd" for c in m.calls)
    m.loss_and_grad(WC, LAB, 1.0)
    m.loss(WC, LAB)                            # leaves the gradient as it is
    m.backward(None, WS, 32, [1, 2])
    m.backward(None, WS, 32, [1, 2])           # the same step again
    assert sum(c[0] == "gcn_layer_bwd" for c in m.calls) == 4
    m.forward(X, WS, 32, [3, 4])
    with pytest.raises(err):
        m.backward(None, WS, 32, [3, 4])       # the gradient is the last step's
    m.backward(torch.zeros(5, 8), WS, 32, [3, 4])  # a gradient of the caller's own


def test_normalized_stack_without_dropout_goes_backward_from_an_evaluation_pass(stack):
    # with p = 0 the evaluation pass is the training pass
    err, make = stack
    m = make(norm=True)
    m.forward(X, WS, 32, [1, 2], training=False)
    m.backward(torch.zeros(5, 8), WS, 32, [3, 4])
    (call,) = [c for c in m.calls if c[0] == "layer_norm_bwd"]
    (fwd,) = [c for c in m.calls if c[0] == "layer_norm_fwd"]
    assert call[2]["p"] == fwd[2]["p"] == 0.0 and call[2]["seed"] == fwd[2]["seed"]
    m = make(norm=True, p=0.5)
    m.forward(X, WS, 32, [1, 2], training=False)
    with pytest.raises(err):
        m.backward(torch.zeros(5, 8), WS, 32, [3, 4])


def test_backward_takes_the_weights_that_forward_took(stack):
    err, make = stack
    pair = [(torch.ones(8), torch.zeros(8))]
    m = make(norm=True)
    for given, missing in ((pair, None), (None, pair)):
        m.forward(X, WS, 32, [1, 2], norms=given)
        with pytest.raises(err):
            m.backward(torch.zeros(5, 8), WS, 32, [3, 4], norms=missing)
        m.backward(torch.zeros(5, 8), WS, 32, [3, 4], norms=given)
    gammas = [c[1][4] for c in m.calls if c[0] == "layer_norm_bwd"]
    assert len(gammas) == 2 and gammas[0] is pair[0][0] and gammas[1] is None
