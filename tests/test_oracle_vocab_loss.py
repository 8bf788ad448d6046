"""CPU pins of the vocabulary loss's oracle: the definition, ignored rows, a
nearly certain target, and the gradient against differences."""

import numpy as np

from oracle import vocab_loss


def test_definition_by_loops():
    rng = np.random.default_rng(0)
    X, W = rng.standard_normal((4, 6)), rng.standard_normal((9, 6))
    t = np.array([3, -100, 0, 8])
    o = vocab_loss.loss(X, W, t)
    for i in range(4):
        l = np.array([sum(X[i] * W[v]) for v in range(9)])
        ref = 0.0 if t[i] < 0 else np.log(np.exp(l).sum()) - l[t[i]]
        np.testing.assert_allclose(o["loss"][i], ref, rtol=1e-12, atol=1e-15)
    np.testing.assert_allclose(o["total"], o["loss"].sum() / 3, rtol=1e-13)
    assert (o["dX"][1] == 0).all() and o["lse"][1] == 0


def test_one_word_and_a_certain_target():
    o = vocab_loss.loss(np.ones((2, 3)), np.ones((1, 3)), np.array([0, 0]))
    assert (o["loss"] == 0).all() and (o["dX"] == 0).all()
    o = vocab_loss.loss(np.array([[1.0]]), np.array([[60.0], [0.0]]), np.array([0]))
    np.testing.assert_allclose(o["loss"][0], np.exp(-60.0), rtol=1e-12)
    np.testing.assert_allclose(o["dX"][0, 0], -60.0 * np.exp(-60.0), rtol=1e-12)
    o = vocab_loss.loss(np.array([[1.0]]), np.array([[-900.0], [0.0]]), np.array([0]))
    np.testing.assert_allclose(o["loss"][0], 900.0)


def test_gradient_against_differences():
    rng = np.random.default_rng(1)
    X, W = rng.standard_normal((5, 7)), rng.standard_normal((11, 7))
    t, w = np.array([1, 2, -100, 10, 0]), rng.standard_normal(5)
    g = vocab_loss.loss(X, W, t, w)["dX"]
    d = rng.standard_normal(X.shape)
    f = lambda x: vocab_loss.loss(x, W, t, w)["total"]
    num = (f(X + 1e-5 * d) - f(X - 1e-5 * d)) / 2e-5
    assert abs(num - (g * d).sum()) <= 1e-8 * np.abs(g * d).sum()
