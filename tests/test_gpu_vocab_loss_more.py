"""More GPU tests of the loss over the vocabulary: one workspace for batches of
different lengths."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
from gpu_util import DEV, guarded, to_dev
from test_gpu_vocab_loss import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("grad,K,V,lengths", [(True, 2080, 50021, (260, 253, 70, 1)), (False, 512, 30000, (134, 127, 3)),
                                              (True, 64, 700, (4100, 4096, 300, 64, 0))])
def test_the_longest_batchs_workspace_does_for_all(grad, K, V, lengths):
    """Batches of up to the first length in one workspace, in any order: the bits that
    each has with one of its own."""
    rng = np.random.default_rng(K)
    M = max(lengths)
    X, W = to_dev(normal(rng, (M, K))), to_dev(normal(rng, (V, K), 0.2))
    t = torch.from_numpy(np.where(rng.random(M) < 0.2, -100, rng.integers(0, V, M))).to(DEV)
    ws, check = guarded((L.head_loss_workspace(grad, M, K, V, DEV).numel(),), torch.uint8)
    for m in (*lengths, *lengths[::-1]):
        a = L.head_loss(X[:m], W, t[:m], want_grad=grad, want_lse=True, workspace=ws)
        b = L.head_loss(X[:m], W, t[:m], want_grad=grad, want_lse=True)
        torch.cuda.synchronize()
        check("workspace")
        for n in a:
            assert (a[n] is None and b[n] is None) or torch.equal(a[n], b[n]), (m, n)
