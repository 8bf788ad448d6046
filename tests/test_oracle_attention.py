"""CPU pins of the attention oracle: the softmax's definition, packing, cache
lengths, empty rows, and the gradients against differences."""

import numpy as np
import pytest

from oracle import attention


def _case(seed, Lq, Lk, Hq, Hkv, D):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    return n(Lq, Hq, D), n(Lk, Hkv, D), n(Lk, Hkv, D), n(Lq, Hq, D)


def test_one_key_is_the_value_itself():
    Q, K, V, _ = _case(0, 1, 1, 4, 2, 8)
    o = attention.forward(Q, K, V, 0.3, [(0, 1)], [(0, 1)])
    for h in range(4):
        np.testing.assert_allclose(o["O"][0, h], V[0, h // 2], rtol=1e-15)
        np.testing.assert_allclose(o["lse"][0, h], 0.3 * Q[0, h] @ K[0, h // 2], rtol=1e-14)


def test_weights_by_loops():
    Q, K, V, _ = _case(1, 5, 9, 2, 1, 4)
    o = attention.forward(Q, K, V, 0.7, [(0, 5)], [(0, 9)])
    for h in range(2):
        for i in range(5):
            s = [0.7 * sum(Q[i, h, e] * K[j, 0, e] for e in range(4)) for j in range(i + 9 - 5 + 1)]
            w = np.exp(s)
            ref = sum(w[j] * V[j, 0] for j in range(len(s))) / w.sum()
            np.testing.assert_allclose(o["O"][i, h], ref, rtol=1e-13)
            np.testing.assert_allclose(o["lse"][i, h], np.log(w.sum()), rtol=1e-13)


def test_packing_equals_separate_calls_and_rows_outside_are_untouched():
    Q, K, V, dO = _case(2, 12, 12, 4, 2, 8)
    r = [(0, 3), (3, 3), (3, 10)]
    o = attention.forward(Q, K, V, 0.4, r, r)
    b = attention.backward(Q, K, V, o["O"], dO, 0.4, r, r)
    for x, y in r:
        s = attention.forward(Q[x:y], K[x:y], V[x:y], 0.4, [(0, y - x)], [(0, y - x)])
        np.testing.assert_array_equal(o["O"][x:y], s["O"])
    for n in ("dQ", "dK", "dV"):
        assert np.isnan(b[n][10:]).all() and np.isfinite(b[n][:10]).all()
    assert np.isnan(o["O"][10:]).all()


def test_rows_that_see_nothing():
    Q, K, V, dO = _case(3, 6, 2, 2, 2, 8)
    o = attention.forward(Q, K, V, 0.4, [(0, 6)], [(0, 2)])
    assert (o["O"][:4] == 0).all() and (o["lse"][:4] == -np.inf).all() and np.isfinite(o["lse"][4:]).all()
    b = attention.backward(Q, K, V, o["O"], dO, 0.4, [(0, 6)], [(0, 2)])
    assert (b["dQ"][:4] == 0).all() and np.isfinite(b["dK"]).all()
    e = attention.forward(Q, K, V, 0.4, [(0, 6)], [(0, 0)])
    assert (e["O"] == 0).all() and (e["lse"] == -np.inf).all()


@pytest.mark.parametrize("Lq,Lk", [(5, 5), (3, 7), (6, 4)])
def test_gradients_against_differences(Lq, Lk):
    Q, K, V, dO = _case(4, Lq, Lk, 4, 2, 6)
    r = ([(0, Lq)], [(0, Lk)])
    f = lambda q, k, v: float((attention.forward(q, k, v, 0.5, *r)["O"] * dO).sum())
    g = attention.backward(Q, K, V, attention.forward(Q, K, V, 0.5, *r)["O"], dO, 0.5, *r)
    rng = np.random.default_rng(5)
    eps = 1e-5
    for i, n in enumerate(("dQ", "dK", "dV")):
        d = rng.standard_normal(g[n].shape)
        x = [Q, K, V]
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + eps * d, x[i] - eps * d
        num = (f(*up) - f(*dn)) / (2 * eps)
        assert abs(num - (g[n] * d).sum()) <= 1e-8 * max(1.0, np.abs(g[n] * d).sum())


def test_rows_of_few_keys_do_not_take_delta_from_the_given_output():
    Q, K, V, dO = _case(6, 40, 40, 2, 1, 8)
    r = [(0, 40)]
    O = attention.forward(Q, K, V, 0.5, r, r)["O"]
    g, w = (attention.backward(Q, K, V, o, dO, 0.5, r, r) for o in (O, O * (1 + 2.0 ** -9)))
    n = attention.EXACT
    np.testing.assert_array_equal(g["dQ"][:n], w["dQ"][:n])
    assert (g["dQ"][n:] != w["dQ"][n:]).any(axis=(1, 2)).all()
    for k in ("dK", "dV"):
        np.testing.assert_array_equal(g[k], w[k])
    # where O is exact both forms are the same
    for x in (g, w):
        x["dQ"][n:] = 0
    P, _ = attention._weights(Q[:, 0], K[:, 0], 0.5)
    dP = dO[:, 0] @ V[:, 0].T
    for delta in ((dO[:, 0] * O[:, 0]).sum(axis=1), (P * dP).sum(axis=1)):
        d = (P * (dP - delta[:, None])) @ K[:, 0] * 0.5
        np.testing.assert_allclose(d[:n], g["dQ"][:n, 0], rtol=1e-9, atol=1e-12)
