"""CPU tests of the vocabulary loss's refusals."""

import pytest
import torch

import lora_fine_tuning_amd as L

OK, ENULL, ESHAPE, EALIGN, EWS = 0, -1, -2, -3, -5
P = 4096


def call(X=P, W=P, t=P, w=None, M=16, K=64, V=100, loss=P, lse=None, total=None, dX=None, ws=P, n=1 << 40):
    return L.lora4_head_loss(X, W, t, w, M, K, V, -100, loss, lse, total, dX, ws, n, None)


def test_statuses():
    for kw in (dict(M=-1), dict(M=1 << 31), dict(K=0), dict(K=60), dict(K=1 << 21), dict(V=0), dict(V=1 << 31)):
        assert call(**kw) == ESHAPE, kw
    for n in ("X", "W", "t", "loss"):
        assert call(**{n: None}) == ENULL
    for n in ("X", "W", "t", "w", "loss", "lse", "total", "dX", "ws"):
        assert call(**{n: P + 8}) == EALIGN
    assert call(ws=None) == EWS
    a, g = (L.lora4_head_loss_workspace_bytes(x, 16, 64, 100) for x in (0, 1))
    assert g > a > 0
    assert call(n=a - 1) == EWS and call(dX=P, n=g - 1) == EWS
    f = L.lora4_head_loss_workspace_bytes
    for bad in [(2, 16, 64, 100), (-1, 16, 64, 100), (0, -1, 64, 100), (1, 16, 60, 100), (1, 16, 64, 0)]:
        assert f(*bad) == 0


def test_the_workspace_does_not_hold_the_logits():
    M, K, V = 32768, 4096, 128256
    assert L.lora4_head_loss_workspace_bytes(1, M, K, V) < M * V * 2 // 8


def test_binding():
    bf = torch.bfloat16
    X, W, t = torch.zeros(4, 16, dtype=bf), torch.zeros(9, 16, dtype=bf), torch.zeros(4, dtype=torch.int64)
    for args, kw in [
        ((X[0], W, t), {}), ((X.float(), W, t), {}), ((X, W[:, :8], t), {}), ((X, W.float(), t), {}),
        ((X, W, t[:3]), {}), ((X, W, t.int()), {}), ((X, W, t), dict(weights=torch.zeros(4, dtype=bf))),
        ((X, W, t), dict(weights=torch.zeros(3))), ((X, W, t), dict(out={"dX": torch.zeros(4, 8, dtype=bf)})),
        ((X, W, t), dict(out={"loss": torch.zeros(4, dtype=bf)})), ((X, W, t), {}),     # not on a GPU
    ]:
        with pytest.raises(ValueError):
            L.head_loss(*args, **kw)
