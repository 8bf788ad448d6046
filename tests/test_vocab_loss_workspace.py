"""CPU tests of the vocabulary loss's workspace: what is enough for a batch is enough
for every shorter one, whatever tiles the shorter one takes."""

import numpy as np
import pytest

import lora_fine_tuning_amd as L

ESHAPE, EWS = -2, -5
P = 4096


def size(grad, M, K, V):
    n = L.lora4_head_loss_workspace_bytes(grad, M, K, V)
    assert n > 0
    return n


@pytest.mark.parametrize("K,V", [(4096, 128256), (2080, 50021), (4600, 2070), (24632, 1024), (792, 5813), (64, 100),
                                 (8, 1), (104, 3000000), (1 << 20, 9)])
@pytest.mark.parametrize("grad", [0, 1])
@pytest.mark.parametrize("tiles", [None, "small", "big"])
def test_a_longer_batch_never_needs_less(monkeypatch, grad, K, V, tiles):
    if tiles:
        monkeypatch.setenv("LORA4_LOSS_TILES", tiles)
    sizes = np.array([size(grad, M, K, V) for M in [*range(0, 1500), *range(1500, 4200, 7), 8192, 40000]])
    assert np.all(np.diff(sizes) >= 0), int(np.argmax(np.diff(sizes) < 0))


def test_random_sizes():
    rng = np.random.default_rng(0)
    for _ in range(300):
        K, V = 8 * int(np.exp(rng.uniform(0, np.log(2048)))), int(np.exp(rng.uniform(0, np.log(300000))))
        grad = int(rng.integers(2))
        sizes = np.array([size(grad, M, K, V) for M in sorted(rng.integers(0, 4400, 60))])
        assert np.all(np.diff(sizes) >= 0), (grad, K, V)


@pytest.mark.parametrize("M", [1, 64, 127, 134, 253, 260, 4096, 5000])
def test_one_byte_less_is_refused(M):
    for grad, dX in ((0, None), (1, P)):
        n = size(grad, M, 2080, 50021)
        assert L.lora4_head_loss(P, P, P, None, M, 2080, 50021, -100, P, None, None, dX, P, n - 1, None) == EWS
