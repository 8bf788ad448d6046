"""GPU tests of views that start off 16 bytes where a user has them: the targets and
weights of the next-token loss, and rows of a table of offsets."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
from gpu_util import DEV, to_dev
from test_gpu_attention import normal, offsets

pytestmark = pytest.mark.gpu


def test_next_token_loss():
    rng = np.random.default_rng(0)
    T, K, V = 71, 64, 500
    X, W = to_dev(normal(rng, (T, K))), to_dev(normal(rng, (V, K)))
    ids = torch.from_numpy(rng.integers(0, V, T)).to(DEV)
    w = torch.rand(T, device=DEV)
    assert (ids[1:].data_ptr() % 16, w[1:].data_ptr() % 16) == (8, 4)
    for a, b in ((1, None), (2, 9), (3, 4), (1, 1)):
        t, v = ids[a:b], w[a:b]
        x = X[:t.numel()]
        got = L.head_loss(x, W, t, weights=v)
        ref = L.head_loss(x, W, t.clone(), weights=v.clone())
        mean, mean_ref = L.head_loss(x, W, t), L.head_loss(x, W, t.clone())
        for n in ("loss", "total", "dX"):
            assert torch.equal(got[n], ref[n]) and torch.equal(mean[n], mean_ref[n]), (a, b, n)


def test_rows_of_a_table_of_offsets():
    rng = np.random.default_rng(1)
    T, Hq, Hkv, D = 60, 4, 2, 64
    q, k, v, do = (to_dev(normal(rng, (T, h, D))) for h in (Hq, Hkv, Hkv, Hq))
    table = torch.stack([offsets([20, 40]), offsets([1, 59]), offsets([59, 1])])
    lens = torch.tensor([[7, 20, 40], [7, 1, 33]], device=DEV)
    assert table[1].data_ptr() % 16 == 8 and lens[0, 1:].data_ptr() % 16 == 8
    for qo, ko, kl in ((table[1], None, None), (table[1], table[1], None), (table[0], table[1], lens[0, 1:]),
                       (table[2], table[1], lens[1, 1:])):
        kw = dict(q_offsets=qo, k_offsets=ko, k_lengths=kl)
        ref = {n: None if x is None else x.clone() for n, x in kw.items()}
        o, r = L.attention(q, k, v, 0.125, **kw), L.attention(q, k, v, 0.125, **ref)
        # (keys past the filled ones have no gradient: zeros on both sides)
        new = lambda: {n: torch.zeros_like(x) for n, x in (("dQ", q), ("dK", k), ("dV", v))}
        g = L.attention_backward(q, k, v, o["O"], o["lse"], do, 0.125, out=new(), **kw)
        h = L.attention_backward(q, k, v, r["O"], r["lse"], do, 0.125, out=new(), **ref)
        for a, b in ((o, r), (g, h)):
            assert all(torch.equal(a[n], b[n]) for n in a)


def test_captured():
    """The views are read when the graph is replayed."""
    rng = np.random.default_rng(2)
    T, H, D, K, V = 40, 2, 64, 128, 300
    q, k, v = (to_dev(normal(rng, (T, H, D))) for _ in range(3))
    X, W = to_dev(normal(rng, (T, K))), to_dev(normal(rng, (V, K)))
    ids = torch.from_numpy(rng.integers(0, V, T + 1)).to(DEV)
    table = torch.stack([offsets([20, 20]), offsets([10, 30])])

    def step():
        return {**L.attention(q, k, v, 0.125, q_offsets=table[1]), **L.head_loss(X, W, ids[1:])}

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for n in (10, 33, 0, 10):
        ids.copy_(torch.from_numpy(rng.integers(0, V, T + 1)))
        table[1].copy_(offsets([n, 40 - n]))
        g.replay()
        torch.cuda.synchronize()
        ref = step()
        for name in ("O", "loss", "total", "dX"):
            assert torch.equal(out[name], ref[name]), (n, name)
