"""CPU pins of the attention oracle's dQ by the definition alone: against differences,
and what an O of fewer bits costs an implementation that takes delta from it."""

import numpy as np
import pytest

from oracle import attention

U = 2.0 ** -8


def _case(seed, Lq, Lk, Hq, Hkv, D, std=1.0):
    rng = np.random.default_rng(seed)
    n = lambda *s: rng.standard_normal(s)
    return std * n(Lq, Hq, D), std * n(Lk, Hkv, D), n(Lk, Hkv, D), n(Lq, Hq, D)


@pytest.mark.parametrize("Lq,Lk", [(5, 5), (40, 70), (6, 4)])
def test_differences(Lq, Lk):
    Q, K, V, dO = _case(0, Lq, Lk, 4, 2, 6)
    r = ([(0, Lq)], [(0, Lk)])
    g = attention.dq(Q, K, V, dO, 0.5, *r, U)["dQ"]
    d = np.random.default_rng(1).standard_normal(Q.shape)
    f = lambda q: float((attention.forward(q, K, V, 0.5, *r)["O"] * dO).sum())
    assert abs((f(Q + 1e-5 * d) - f(Q - 1e-5 * d)) / 2e-5 - (g * d).sum()) <= 1e-8 * max(1.0, np.abs(g * d).sum())


@pytest.mark.parametrize("std", [1.0, 3.0])
def test_what_a_rounded_output_costs(std):
    """O off by a uniform error within u of each element: dQ of delta = dO O stays
    within D_dQ element by element, and all of it within N_dQ; neither is idle."""
    Q, K, V, dO = _case(2, 300, 300, 2, 1, 16, std)
    r = [(0, 300)]
    t = attention.dq(Q, K, V, dO, 0.25, r, r, U)
    O = attention.forward(Q, K, V, 0.25, r, r)["O"]
    O = O * (1 + U * np.random.default_rng(3).uniform(-1, 1, O.shape))
    n = attention.EXACT
    err = np.abs(attention.backward(Q, K, V, O, dO, 0.25, r, r)["dQ"] - t["dQ"])[n:]
    assert np.all(err <= t["D_dQ"][n:] + 1e-12)
    assert 0.1 * np.linalg.norm(t["N_dQ"][n:]) <= np.linalg.norm(err) <= np.linalg.norm(t["N_dQ"][n:])
