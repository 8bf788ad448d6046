"""GPU test of a whole training step of a pre-norm block (the one of test_gpu_block)
captured into a HIP graph: replayed with other tokens, targets and sequence lengths,
every replay gives the eager step's bits."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import DEV, pack_gpu, to_dev
from test_gpu_block import EPS, HD, HKV, HQ, K, S, SCALE, T, V, data, normal  # noqa: F401 (data: a fixture)

pytestmark = pytest.mark.gpu


def prepare(d, fmt):
    s = {n: to_dev(v) for n, v in d.items() if n != "t" and n[0] != "W"}
    for n in ("qkv", "o", "down"):
        s["W" + n] = pack_gpu(d["W" + n], fmt)
    s["Wgate_up"] = pack_gpu(np.stack([d["Wgate"], d["Wup"]]), fmt)
    s["A"], s["B"] = torch.stack([s["Agate"], s["Aup"]]), torch.stack([s["Bgate"], s["Bup"]])
    s["t"] = torch.from_numpy(d["t"]).to(DEV)
    s["q_offsets"] = torch.zeros(6, dtype=torch.int64, device=DEV)
    return s


def step(s):
    """Forward and backward of the block; the loss and all gradients."""
    cut = lambda x: (x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:])
    n1 = L.rmsnorm(s["x"], s["w1"], EPS)["Y"]
    f1 = L.forward(s["Wqkv"], n1, s["Aqkv"], s["Bqkv"], S)
    qkv = f1["Y"].view(T, HQ + 2 * HKV, HD)
    at = L.attention(*cut(qkv), SCALE, q_offsets=s["q_offsets"])
    o = at["O"].view(T, -1)
    f2 = L.forward_epilogue(s["Wo"], o, s["Ao"], s["Bo"], S, residual=s["x"])
    n2 = L.rmsnorm(f2["Y"], s["w2"], EPS)["Y"]
    g = L.gated_forward(s["Wgate_up"], n2, s["A"], s["B"], S)
    f3 = L.forward_epilogue(s["Wdown"], g["H"], s["Adown"], s["Bdown"], S, residual=f2["Y"])
    n3 = L.rmsnorm(f3["Y"], s["w3"], EPS)["Y"]
    loss = L.head_loss(n3, s["head"], s["t"])

    out = {"total": loss["total"], "loss": loss["loss"]}
    b3 = L.rmsnorm_backward(loss["dX"], f3["Y"], s["w3"], EPS)
    down = L.backward_epilogue(s["Wdown"], g["H"], b3["dX"], s["Adown"], s["Bdown"], S, Z=f3["Z"])
    gated = L.gated_backward(s["Wgate_up"], n2, down["dX"], g["GU"], s["A"], s["B"], S, Z=g["Z"])
    b2 = L.rmsnorm_backward(gated["dX"], f2["Y"], s["w2"], EPS, dH=b3["dX"])
    proj = L.backward_epilogue(s["Wo"], o, b2["dX"], s["Ao"], s["Bo"], S, Z=f2["Z"])
    dqkv = torch.empty_like(qkv)
    L.attention_backward(*cut(qkv), at["O"], at["lse"], proj["dX"].view(at["O"].shape), SCALE,
                         q_offsets=s["q_offsets"], out=dict(zip(("dQ", "dK", "dV"), cut(dqkv))))
    lin = L.backward(s["Wqkv"], n1, dqkv.view(T, -1), s["Aqkv"], s["Bqkv"], S, Z=f1["Z"])
    b1 = L.rmsnorm_backward(lin["dX"], s["x"], s["w1"], EPS, dH=b2["dX"])
    for n, b in (("w3", b3), ("w2", b2), ("w1", b1)):
        out["d" + n] = b["dW"]
    for n, b in (("down", down), ("gate_up", gated), ("o", proj), ("qkv", lin)):
        out["dA" + n], out["dB" + n] = b["dA"], b["dB"]
    out["dx"] = b1["dX"]
    return out


@pytest.mark.parametrize("fmt", [synth.NF4, synth.MXFP4])
def test_training_step_captured(data, fmt):  # noqa: F811
    rng = np.random.default_rng(31)
    s = prepare(data, fmt)

    def batch(lens, ignored):
        """Other tokens, targets and lengths (together T rows), where the step finds them."""
        s["x"].copy_(to_dev(normal(rng, (T, K))))
        t = rng.integers(0, V, T)
        t[rng.random(T) < ignored] = -100
        s["t"].copy_(torch.from_numpy(t))
        s["q_offsets"].copy_(torch.from_numpy(np.concatenate([[0], np.cumsum(lens)])))

    batch([37, 0, 90, 1, 72], 0.3)
    step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(s)
    for lens, ignored in (([37, 0, 90, 1, 72], 0.3), ([200, 0, 0, 0, 0], 0.0), ([1, 1, 1, 1, 196], 0.9),
                          ([50, 50, 50, 49, 1], 0.5)):
        batch(lens, ignored)
        for x in out.values():
            x.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        eager = step(s)
        for n, x in eager.items():
            assert torch.isfinite(x.float()).all() and x.float().abs().max() > 0, n
            assert torch.equal(x, out[n]), (lens, n)
