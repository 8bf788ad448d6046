"""GPU tests that what belongs to one projection stays out of the other: the gate's
and the up projection's rank columns lie side by side in one operand."""

import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import print_case
from test_gpu_ffn import POLICIES, Case

pytestmark = pytest.mark.gpu


CASES = [(M, r, policy) for M, r in [(3, 8), (40, 12), (130, 24), (300, 128), (70, 3), (1100, 16)]
         for policy in POLICIES if not (policy in ("4", "8") and M > 130)]


@pytest.mark.parametrize("M,r,policy", CASES)
def test_infinite_adapter_of_one_projection(M, r, policy, monkeypatch):
    """An infinite element in one projection's A makes that projection's Z and
    outputs non-finite, one in its B the column of its outputs, and both leave the
    other's bits as they were."""
    print_case("apart", M, r, policy)
    monkeypatch.setenv("LORA4_FFN_ROWS", policy)
    c = Case(M, 256, 200, r, synth.MXFP4, 2)
    X, A, B = c.dev("X", "A", "B")
    want = L.gated_forward(c.base, X, A, B, c.s)
    for j in (0, 1):
        halves = lambda t, n: (t[:, :n], t[:, n:])
        bad = B.clone()
        bad[j, 7, r - 1] = float("inf")
        got = L.gated_forward(c.base, X, A, bad, c.s)
        gu, clean = halves(got["GU"], c.N), halves(want["GU"], c.N)
        assert torch.equal(gu[1 - j], clean[1 - j]) and torch.equal(got["Z"], want["Z"])
        others = [n for n in range(c.N) if n != 7]
        assert torch.equal(gu[j][:, others], clean[j][:, others]) and not gu[j][:, 7].isfinite().any()
        bad = A.clone()
        bad[j, r - 1, 5] = float("inf")
        got = L.gated_forward(c.base, X, bad, B, c.s)
        gu, z = halves(got["GU"], c.N), halves(got["Z"], r)
        assert torch.equal(gu[1 - j], halves(want["GU"], c.N)[1 - j])
        assert torch.equal(z[1 - j], halves(want["Z"], r)[1 - j])
        assert not gu[j].isfinite().any() and not z[j][:, r - 1].isfinite().any()
