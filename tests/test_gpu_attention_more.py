"""More GPU tests of attention: offsets past 32 bits, two calls at once, old
workspace contents, gradients against differences, many sequences."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
from gpu_util import DEV, f64, print_case, to_dev, to_host
from oracle import attention, lora
from test_gpu_attention import compare, normal, offsets, run_case

pytestmark = pytest.mark.gpu


def strided(rng, T, H, D, ld):
    """[T, H, D] with token stride ld in a buffer of its own, and its values."""
    buf = torch.empty((T - 1) * ld + H * D, dtype=torch.bfloat16, device=DEV)
    x = normal(rng, (T, H, D))
    t = torch.as_strided(buf, (T, H, D), (ld, D, 1))
    t.copy_(to_dev(x))
    return t, x


def test_a_cache_past_32_bit_offsets():
    """Keys, values and their gradients 5 GB apart: 600 tokens of 4 million elements."""
    rng = np.random.default_rng(0)
    T, Hq, Hkv, D, ld = 600, 4, 2, 128, 1 << 22
    print_case("long strides", T, ld)
    k, fk = strided(rng, T, Hkv, D, ld)
    v, fv = strided(rng, T, Hkv, D, ld)
    assert k[-1].data_ptr() - k.data_ptr() > 1 << 32
    for Lq in (1, 40):
        q = normal(rng, (Lq, Hq, D))
        o = L.attention(to_dev(q), k, v, 0.09)
        ref = attention.forward(f64(q), f64(fk), f64(fv), 0.09, [(0, Lq)], [(0, T)])
        compare("O", to_host(o["O"]), ref, "O", np.ones(Lq, bool))
    dk, dv = torch.empty_strided(k.shape, k.stride(), dtype=k.dtype, device=DEV), torch.empty_strided(
        k.shape, k.stride(), dtype=k.dtype, device=DEV)
    do = normal(rng, (Lq, Hq, D))
    b = L.attention_backward(to_dev(q), k, v, o["O"], o["lse"], to_dev(do), 0.09, out={"dK": dk, "dV": dv})
    ref = attention.backward(f64(q), f64(fk), f64(fv), f64(to_host(o["O"])), f64(do), 0.09, [(0, Lq)], [(0, T)])
    for n in ("dQ", "dK", "dV"):
        compare(n, to_host(b[n]), ref, n, np.ones(ref[n].shape[0], bool))


def test_two_calls_at_once():
    rng = np.random.default_rng(1)
    jobs = []
    for i, (nq, cap) in enumerate([([300, 40], None), ([1, 1, 1], 4000)]):
        Hq, Hkv, D = 8, 2, 128
        T, Tk = sum(nq), sum(nq) if cap is None else cap * len(nq)
        q, k, v = to_dev(normal(rng, (T, Hq, D))), to_dev(normal(rng, (Tk, Hkv, D))), to_dev(normal(rng, (Tk, Hkv, D)))
        kw = dict(q_offsets=offsets(nq))
        if cap is not None:
            kw["k_offsets"] = offsets([cap] * len(nq))
        jobs.append((q, k, v, kw, L.attention(q, k, v, 0.1, **kw)["O"].clone()))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    for _ in range(5):
        for i, (s, (q, k, v, kw, _)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i].append(L.attention(q, k, v, 0.1, **kw)["O"])
    torch.cuda.synchronize()
    for g, j in zip(got, jobs):
        assert all(torch.equal(x, j[4]) for x in g)


def test_old_workspace_contents_do_not_matter():
    rng = np.random.default_rng(2)
    Hq, Hkv, D, cap = 8, 2, 64, 3000
    q, k, v, do = (to_dev(normal(rng, s)) for s in ((2, Hq, D), (2 * cap, Hkv, D), (2 * cap, Hkv, D), (2, Hq, D)))
    kw = dict(q_offsets=offsets([1, 1]), k_offsets=offsets([cap, cap]), k_lengths=torch.tensor([2900, 0], device=DEV))
    w = [L.attention_workspace(i, 2, 2 * cap, 2, Hq, Hkv, D, DEV) for i in (0, 1)]
    res = []
    for fill in (0, 0x7F, 0xFF):
        for t in w:
            t.fill_(fill)
        o = L.attention(q, k, v, 0.125, workspace=w[0], **kw)
        b = L.attention_backward(q, k, v, o["O"], o["lse"], do, 0.125, workspace=w[1],
                                 out={n: torch.zeros_like(x) for n, x in (("dK", k), ("dV", v))}, **kw)
        res.append({**o, **b})
    assert not res[0]["O"][1].any() and torch.isneginf(res[0]["lse"][1]).all()
    for r in res[1:]:
        assert all(torch.equal(r[n], res[0][n]) for n in r)


def test_a_workspace_that_is_too_small():
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        L.attention(q, q, q, 0.1, workspace=ws)
    with pytest.raises(ValueError):
        L.attention_backward(q, q, q, q, torch.zeros(4, 2, device=DEV), q, 0.1, workspace=ws)


def test_gradients_against_differences():
    """Directional derivatives of sum(O dO), by the float64 forward around the bf16
    inputs: each gradient's product with a direction is off by at most 2^-8 of the
    sum of its terms (every element by u of itself, and as much again by the
    roundings inside)."""
    rng = np.random.default_rng(3)
    r = [(0, 70), (70, 75)]
    Q, K, V, dO = (normal(rng, (75, h, 64)) for h in (6, 2, 2, 6))
    q, k, v, do = map(to_dev, (Q, K, V, dO))
    o = L.attention(q, k, v, 0.125, q_offsets=offsets([70, 5]))
    g = L.attention_backward(q, k, v, o["O"], o["lse"], do, 0.125, q_offsets=offsets([70, 5]))
    x = [f64(Q), f64(K), f64(V)]
    f = lambda y: float((attention.forward(*y, 0.125, r, r)["O"] * f64(dO)).sum())
    for i, n in enumerate(("dQ", "dK", "dV")):
        d = rng.standard_normal(x[i].shape)
        up, dn = list(x), list(x)
        up[i], dn[i] = x[i] + 1e-5 * d, x[i] - 1e-5 * d
        gd = f64(to_host(g[n])) * d
        assert abs((f(up) - f(dn)) / 2e-5 - gd.sum()) <= 2 * 2.0 ** -8 * np.abs(gd).sum(), n


def test_many_sequences():
    rng = np.random.default_rng(4)
    run_case(list(rng.integers(0, 9, 300)), None, 2, 1, 32, seed=5, tail=4)
    run_case([1] * 200, list(rng.integers(0, 40, 200)), 4, 1, 64, seed=6, cap=40)


@pytest.mark.parametrize("G", [1, 3, 64])
def test_groups(G):
    run_case([67, 3], None, 2 * G, 2, 32, seed=G)


@pytest.mark.parametrize("D", [8, 24, 40, 56, 104, 112])
def test_head_sizes(D):
    run_case([50, 90], None, 4, 2, D, seed=D)
