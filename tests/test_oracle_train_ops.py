"""The oracle's dropout, layer normalization and class-head cross entropy
against closed forms and central differences (CPU only)."""
import numpy as np
import pytest


def _diff(f, X, h=1e-6):
    """Central differences of the scalar f at every entry of X."""
    g = np.zeros(X.shape)
    for i in np.ndindex(X.shape):
        a, b = X.copy(), X.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_noise_codes_are_the_library_hash(orc):
    c = orc.noise_codes(0x123456789ABCDEF, 7, 9)
    for r in range(7):
        for j in range(9):
            assert c[r, j] == orc.hash32(0x123456789ABCDEF, r, j) >> 9


def test_dropout_rate_and_scale(orc):
    X = np.ones((400, 250))
    for p in (0.1, 0.5, 0.9):
        Y = orc.dropout(X, p, 11)
        assert set(np.unique(Y)) == {0.0, 1.0 / (1.0 - p)}
        # kept elements: binomial, 6 standard deviations
        assert abs((Y > 0).mean() - (1 - p)) < 6 * np.sqrt(p * (1 - p) / Y.size)
    assert (orc.dropout(X, 1.0, 3) == 0).all() and (orc.dropout(X, 0.0, 3) == X).all()


@pytest.mark.parametrize("relu,p", [(False, 0.0), (True, 0.0), (True, 0.4)])
def test_layer_norm_gradients(orc, relu, p):
    rng = np.random.default_rng(1)
    X, dY = rng.normal(size=(4, 6)) + 0.3, rng.normal(size=(4, 6))
    ga, be = 1 + 0.3 * rng.normal(size=6), 0.3 * rng.normal(size=6)
    f = orc.layer_norm_fwd(X, ga, be, 1e-5, relu, p, 5)
    assert abs((X - f["mean"][:, None]).sum()) < 1e-12
    b = orc.layer_norm_bwd(dY, X, f["mean"], f["rstd"], ga, f["on"] if relu else None, p, 5)
    val = lambda X, ga, be: float((orc.layer_norm_fwd(X, ga, be, 1e-5, relu, p, 5)["Y"] * dY).sum())
    np.testing.assert_allclose(b["dX"], _diff(lambda x: val(x, ga, be), X), atol=1e-7)
    np.testing.assert_allclose(b["dgamma"], _diff(lambda x: val(X, x, be), ga), atol=1e-7)
    np.testing.assert_allclose(b["dbeta"], _diff(lambda x: val(X, ga, x), be), atol=1e-7)


def test_linear_xent_gradients_and_unlabelled_rows(orc):
    rng = np.random.default_rng(2)
    X, W = rng.normal(size=(5, 4)), rng.normal(size=(7, 4))
    lab = np.array([3, -1, 0, 7, 6])
    w = np.array([1.0, 2.0, 0.5, 3.0, 1.5])
    o = orc.linear_xent(X, W, lab, w, 0.25)
    assert o["loss"][1] == o["loss"][3] == 0 and not o["dX"][[1, 3]].any()
    val = lambda X, W: float((orc.linear_xent(X, W, lab)["loss"] * w * 0.25).sum())
    np.testing.assert_allclose(o["dX"], _diff(lambda x: val(x, W), X), atol=1e-8)
    np.testing.assert_allclose(o["dW"], _diff(lambda x: val(X, x), W), atol=1e-8)
    # uniform logits: loss = log C
    assert abs(orc.linear_xent(np.zeros((1, 4)), W, np.array([2]))["loss"][0] - np.log(7)) < 1e-14
