"""A whole training step of a pre-norm block over packed sequences, every operator
of the library in its place: norm, q/k/v projection (one base), attention, output
projection with the residual, norm, gated projections, down projection with the
residual, norm, loss over the vocabulary, and all of it backwards. Compared with
the oracles chained in float64, and the oracles' chain with differences of its own
loss.

Tolerance: a bf16 rounding moves a tensor by at most u = 2^-8 of its norm, and
between two of them every operator here passes a relative change on with a gain of
about one (norms and residuals keep scales). There are 12 roundings from the input
to the loss (Y of three norms, qkv, O and its P, two residual sums, H with G and U,
codes aside, and s Z and Z of the adapters with them) and as many on the way back,
so results may be off by 24 u = 0.094 of their norm; a wrong term shows as about 1.
"""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import DEV, f64, oracle_dequant, oracle_pack, pack_gpu, to_dev, to_host
from oracle import attention, ffn, lora, vocab_loss

pytestmark = pytest.mark.gpu

LENS, HQ, HKV, HD, K, F, V, R, S = [37, 0, 90, 1, 72], 4, 2, 64, 256, 320, 1000, 8, 2.0
T = sum(LENS)
SCALE, EPS = HD ** -0.5, 1e-5
BOUND = 24 * 2.0 ** -8


def normal(rng, shape, std=1.0):
    return synth.to_bf16((rng.standard_normal(shape) * std).astype(np.float32))


@pytest.fixture(scope="module")
def data():
    rng = np.random.default_rng(21)
    d = {"x": normal(rng, (T, K))}
    for n in ("w1", "w2", "w3"):
        d[n] = synth.to_bf16((1 + 0.1 * rng.standard_normal(K)).astype(np.float32))
    shapes = {"qkv": ((HQ + 2 * HKV) * HD, K), "o": (K, HQ * HD), "gate": (F, K), "up": (F, K), "down": (K, F)}
    for n, (N, k) in shapes.items():
        d["W" + n] = normal(rng, (N, k), 1.5 / np.sqrt(k))
        d["A" + n], d["B" + n] = normal(rng, (R, k), 1 / np.sqrt(k)), normal(rng, (N, R), 0.1)
    d["head"] = normal(rng, (V, K), 0.1)
    d["t"] = rng.integers(0, V, T)
    d["t"][rng.random(T) < 0.3] = -100
    return d


def ranges():
    e = np.concatenate([[0], np.cumsum(LENS)])
    return [(int(a), int(b)) for a, b in zip(e[:-1], e[1:])]


def oracle_step(d, fmt, par=None):
    """(total, gradients) of the chain; par: adapters and input in float64."""
    p = {n: f64(v) for n, v in d.items() if n != "t"} if par is None else par
    W = {n: f64(oracle_dequant(oracle_pack(d["W" + n], fmt), fmt)) for n in ("qkv", "o", "gate", "up", "down")}
    r = ranges()
    n1 = ffn.rmsnorm(p["x"], p["w1"], EPS)["Y"]
    qkv = lora.forward(n1, W["qkv"], p["Aqkv"], p["Bqkv"], S)["Y"].reshape(T, HQ + 2 * HKV, HD)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    O = attention.forward(q, k, v, SCALE, r, r)["O"]
    o = O.reshape(T, -1)
    x1 = ffn.epilogue_forward(o, W["o"], p["Ao"], p["Bo"], S, "none", R=p["x"])["Y"]
    n2 = ffn.rmsnorm(x1, p["w2"], EPS)["Y"]
    A, B = np.stack([p["Agate"], p["Aup"]]), np.stack([p["Bgate"], p["Bup"]])
    g = ffn.gated_forward(n2, W["gate"], W["up"], A, B, S, "silu")
    x2 = ffn.epilogue_forward(g["H"], W["down"], p["Adown"], p["Bdown"], S, "none", R=x1)["Y"]
    n3 = ffn.rmsnorm(x2, p["w3"], EPS)["Y"]
    ls = vocab_loss.loss(n3, p["head"], d["t"])
    G = {}
    b = ffn.rmsnorm_backward(ls["dX"], x2, p["w3"], EPS)
    G["w3"], dx2 = b["dW"], b["dX"]
    b = ffn.epilogue_backward(g["H"], W["down"], p["Adown"], p["Bdown"], S, "none", dx2)
    G["Adown"], G["Bdown"] = b["dA"], b["dB"]
    b = ffn.gated_backward(n2, W["gate"], W["up"], A, B, S, "silu", b["dX"], g["G"], g["U"])
    (G["Agate"], G["Aup"]), (G["Bgate"], G["Bup"]) = b["dA"], b["dB"]
    b = ffn.rmsnorm_backward(b["dX"], x1, p["w2"], EPS, dx2)
    G["w2"], dx1 = b["dW"], b["dX"]
    b = ffn.epilogue_backward(o, W["o"], p["Ao"], p["Bo"], S, "none", dx1)
    G["Ao"], G["Bo"] = b["dA"], b["dB"]
    a = attention.backward(q, k, v, O, b["dX"].reshape(O.shape), SCALE, r, r)
    dqkv = np.concatenate([a["dQ"], a["dK"], a["dV"]], axis=1).reshape(T, -1)
    b = lora.backward(n1, W["qkv"], p["Aqkv"], p["Bqkv"], S, dqkv)
    G["Aqkv"], G["Bqkv"] = b["dA"], b["dB"]
    b = ffn.rmsnorm_backward(b["dX"], p["x"], p["w1"], EPS, dx1)
    G["w1"], G["x"] = b["dW"], b["dX"]
    return ls["total"], G


def gpu_step(d, fmt):
    bases = {n: pack_gpu(d["W" + n], fmt) for n in ("qkv", "o", "down")}
    gate_up = pack_gpu(np.stack([d["Wgate"], d["Wup"]]), fmt)
    p = {n: to_dev(v) for n, v in d.items() if n != "t" and n[0] != "W"}
    t = torch.from_numpy(d["t"]).to(DEV)
    qo = torch.tensor(np.concatenate([[0], np.cumsum(LENS)]), dtype=torch.int64, device=DEV)
    A, B = torch.stack([p["Agate"], p["Aup"]]), torch.stack([p["Bgate"], p["Bup"]])
    cut = lambda x: (x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:])

    n1 = L.rmsnorm(p["x"], p["w1"], EPS)["Y"]
    f1 = L.forward(bases["qkv"], n1, p["Aqkv"], p["Bqkv"], S)
    qkv = f1["Y"].view(T, HQ + 2 * HKV, HD)
    at = L.attention(*cut(qkv), SCALE, q_offsets=qo)
    o = at["O"].view(T, -1)
    f2 = L.forward_epilogue(bases["o"], o, p["Ao"], p["Bo"], S, residual=p["x"])
    n2 = L.rmsnorm(f2["Y"], p["w2"], EPS)["Y"]
    g = L.gated_forward(gate_up, n2, A, B, S)
    f3 = L.forward_epilogue(bases["down"], g["H"], p["Adown"], p["Bdown"], S, residual=f2["Y"])
    n3 = L.rmsnorm(f3["Y"], p["w3"], EPS)["Y"]
    ls = L.head_loss(n3, p["head"], t)

    G = {}
    b = L.rmsnorm_backward(ls["dX"], f3["Y"], p["w3"], EPS)
    G["w3"], dx2 = b["dW"], b["dX"]
    b = L.backward_epilogue(bases["down"], g["H"], dx2, p["Adown"], p["Bdown"], S, Z=f3["Z"])
    G["Adown"], G["Bdown"] = b["dA"], b["dB"]
    b = L.gated_backward(gate_up, n2, b["dX"], g["GU"], A, B, S, Z=g["Z"])
    (G["Agate"], G["Aup"]), (G["Bgate"], G["Bup"]) = b["dA"], b["dB"]
    b = L.rmsnorm_backward(b["dX"], f2["Y"], p["w2"], EPS, dH=dx2)
    G["w2"], dx1 = b["dW"], b["dX"]
    b = L.backward_epilogue(bases["o"], o, dx1, p["Ao"], p["Bo"], S, Z=f2["Z"])
    G["Ao"], G["Bo"] = b["dA"], b["dB"]
    dqkv = torch.empty_like(qkv)
    L.attention_backward(*cut(qkv), at["O"], at["lse"], b["dX"].view(at["O"].shape), SCALE, q_offsets=qo,
                         out=dict(zip(("dQ", "dK", "dV"), cut(dqkv))))
    b = L.backward(bases["qkv"], n1, dqkv.view(T, -1), p["Aqkv"], p["Bqkv"], S, Z=f1["Z"])
    G["Aqkv"], G["Bqkv"] = b["dA"], b["dB"]
    b = L.rmsnorm_backward(b["dX"], p["x"], p["w1"], EPS, dH=dx1)
    G["w1"], G["x"] = b["dW"], b["dX"]
    return ls["total"], G


@pytest.mark.parametrize("fmt", [synth.NF4, synth.MXFP4])
def test_training_step(data, fmt):
    total, G = gpu_step(data, fmt)
    torch.cuda.synchronize()
    ref_total, ref = oracle_step(data, fmt)
    assert abs(float(total) - ref_total) <= BOUND * abs(ref_total)
    for n, r in ref.items():
        assert lora.rel_frobenius(f64(to_host(G[n])), r) <= BOUND, n


def test_the_oracles_chain_against_differences(data):
    rng = np.random.default_rng(22)
    _, G = oracle_step(data, synth.NF4)
    base = {n: f64(v) for n, v in data.items() if n != "t"}
    for names in (["x"], ["Aqkv", "Bqkv"], ["Ao", "Bo", "w2"], ["Agate", "Aup", "Bgate", "Bup", "Adown", "Bdown"]):
        d = {n: rng.standard_normal(base[n].shape) * 1e-5 for n in names}
        up = oracle_step(data, synth.NF4, {**base, **{n: base[n] + d[n] for n in names}})[0]
        dn = oracle_step(data, synth.NF4, {**base, **{n: base[n] - d[n] for n in names}})[0]
        want = sum((G[n] * d[n]).sum() for n in names)
        size = sum(np.abs(G[n] * d[n]).sum() for n in names)
        assert abs((up - dn) / 2 - want) <= 1e-5 * size, names


def test_training_step_twice_and_captured(data):
    """The same bits on every step, and from a captured one replayed."""
    t1, g1 = gpu_step(data, synth.NF4)
    t2, g2 = gpu_step(data, synth.NF4)
    assert torch.equal(t1, t2) and all(torch.equal(g1[n], g2[n]) for n in g1)
