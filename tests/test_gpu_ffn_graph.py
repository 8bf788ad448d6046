"""GPU tests of captured feed-forward calls: experts whose row offsets change
between the replays (they are read on the device), with bias, activation,
residual and a bias gradient, and graphs captured before anything else ran."""

import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import print_case
from test_gpu_ffn import Case

pytestmark = pytest.mark.gpu

OFFSETS = [[0, 0, 37, 100], [0, 100, 100, 100], [0, 1, 2, 100], [0, 33, 66, 100], [0, 0, 0, 100]]


def step(g, w):
    """A gated and a fused layer over the same experts, forward and backward."""
    X, A, B, dY = g.args
    f = L.gated_forward(g.base, X, A, B, g.s, group_offsets=g.offsets)
    b = L.gated_backward(g.base, X, dY, f["GU"], A, B, g.s, Z=f["Z"], group_offsets=g.offsets)
    X, A, B, dY, bias, R = w.args
    e = L.forward_epilogue(w.base, X, A, B, w.s, bias=bias, activation="gelu", residual=R, group_offsets=w.offsets)
    d = L.backward_epilogue(w.base, X, dY, A, B, w.s, P=e["P"], activation="gelu", Z=None, want_dbias=True,
                            group_offsets=w.offsets)
    n = L.backward_epilogue(w.base, X, dY, A, B, w.s, Z=e["Z"], want_dbias=True, group_offsets=w.offsets)
    return [t for o in (f, b, e, d, n) for t in o.values() if t is not None]


@pytest.mark.parametrize("fmt", [synth.NF4_DQ, synth.NVFP4])
@pytest.mark.parametrize("M", [100, 9])
def test_offsets_change_between_replays(fmt, M):
    print_case("graph offsets", fmt, M)
    rows = [[min(o, M) for o in offs] for offs in OFFSETS]
    g, w = Case(M, 256, 130, 8, fmt, 2, rows[0], seed=30), Case(M, 256, 130, 8, fmt, 1, rows[0], seed=31)
    g.args, w.args = g.dev("X", "A", "B", "dY"), w.dev("X", "A", "B", "dY", "bias", "R")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):        # (the first calls of these kernels in the process, if run alone)
        got = step(g, w)
    for offs in rows + rows[::-1]:
        new = torch.tensor(offs, dtype=torch.int64, device=g.offsets.device)
        g.offsets.copy_(new)
        w.offsets.copy_(new)
        want = step(g, w)             # eager, with the same offsets
        for t in got:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)), offs
