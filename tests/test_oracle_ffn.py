"""Pins of the feed-forward oracle (CPU): activations against torch's own,
every gradient against central differences, the norm's closed forms, and the
refusals of the binding and the C ABI for the feed-forward operators."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
from oracle import ffn

rng = np.random.default_rng(5)


@pytest.mark.parametrize("name", ffn.ACTIVATIONS)
def test_activation_matches_torch(name):
    x = np.concatenate([rng.standard_normal(200) * 4, [0.0, -30.0, 30.0, -1e-3, 1e-3]])
    t = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    y = {"none": lambda v: v * 1.0, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name](t)
    y.sum().backward()
    v, d = ffn.act(x, name)
    assert np.allclose(v, y.detach().numpy(), rtol=1e-12, atol=1e-14)
    assert np.allclose(d, t.grad.numpy(), rtol=1e-10, atol=1e-14)


def _numeric(f, x, h=1e-6):
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


def test_norm_gradients_by_differences():
    X, R, w = rng.standard_normal((3, 7)), rng.standard_normal((3, 7)), rng.standard_normal(7)
    dY, dH = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    loss = lambda X_, w_: float((ffn.rmsnorm(X_, w_, 1e-3, R)["Y"] * dY).sum() + ((X_ + R) * dH).sum())
    g = ffn.rmsnorm_backward(dY, X + R, w, 1e-3, dH)
    assert np.allclose(g["dX"], _numeric(lambda v: loss(v, w), X), atol=1e-7)
    assert np.allclose(g["dW"], _numeric(lambda v: loss(X, v), w), atol=1e-7)


def test_norm_closed_forms():
    # a row of equal magnitudes has rstd 1 / |a|; a zero row gives zeros
    y = ffn.rmsnorm(np.array([[2.0, -2.0, 2.0, -2.0], [0, 0, 0, 0]]), np.array([1.0, 2, 3, 4]), 0.25)["Y"]
    assert np.allclose(y[0], np.array([1, -2, 3, -4]) * 2 / np.sqrt(4.25))
    assert np.all(y[1] == 0)


def _layer(M=4, K=5, N=6, r=2):
    z = lambda *s: rng.standard_normal(s)
    return z(M, K), z(N, K), z(N, K), z(2, r, K), z(2, N, r)


@pytest.mark.parametrize("name", ffn.ACTIVATIONS)
def test_gated_gradients_by_differences(name):
    X, Wg, Wu, A, B = _layer()
    dH = rng.standard_normal((4, 6))
    f = ffn.gated_forward(X, Wg, Wu, A, B, 0.7, name)
    g = ffn.gated_backward(X, Wg, Wu, A, B, 0.7, name, dH, f["G"], f["U"], f["Z"])
    loss = lambda X_, A_, B_: float((ffn.gated_forward(X_, Wg, Wu, A_, B_, 0.7, name)["H"] * dH).sum())
    assert np.allclose(g["dX"], _numeric(lambda v: loss(v, A, B), X), atol=1e-5)
    assert np.allclose(g["dA"], _numeric(lambda v: loss(X, v, B), A), atol=1e-5)
    assert np.allclose(g["dB"], _numeric(lambda v: loss(X, A, v), B), atol=1e-5)


@pytest.mark.parametrize("name", ffn.ACTIVATIONS)
def test_epilogue_gradients_by_differences(name):
    X, W, _, A, B = _layer()
    A, B = A[0], B[0]
    bias, R, dY = rng.standard_normal(6), rng.standard_normal((4, 6)), rng.standard_normal((4, 6))
    f = ffn.epilogue_forward(X, W, A, B, 0.7, name, bias, R)
    g = ffn.epilogue_backward(X, W, A, B, 0.7, name, dY, f["P"], f["Z"])
    loss = lambda X_, A_, B_, b_: float((ffn.epilogue_forward(X_, W, A_, B_, 0.7, name, b_, R)["Y"] * dY).sum())
    assert np.allclose(g["dX"], _numeric(lambda v: loss(v, A, B, bias), X), atol=1e-5)
    assert np.allclose(g["dA"], _numeric(lambda v: loss(X, v, B, bias), A), atol=1e-5)
    assert np.allclose(g["dB"], _numeric(lambda v: loss(X, A, v, bias), B), atol=1e-5)
    assert np.allclose(g["dbias"], _numeric(lambda v: loss(X, A, B, v), bias), atol=1e-5)


# ---------------------------------------------------------------------------
# Refusals (no GPU: the argument checks come before any HIP call)
# ---------------------------------------------------------------------------

OK, ENULL, ESHAPE, EALIGN, EFORMAT, EWS = 0, -1, -2, -3, -4, -5


def test_norm_abi_refusals():
    def fwd(X=4096, R=4096, w=4096, M=8, D=256, eps=1e-5, H=8192, Y=8192, c=None, s=None):
        return L.lora4_rmsnorm_forward(X, R, w, M, D, eps, H, Y, c, s, None)
    assert fwd(M=-1) == ESHAPE and fwd(D=0) == ESHAPE and fwd(D=16385) == ESHAPE and fwd(D=16377) == ESHAPE
    assert fwd(eps=float("nan")) == ESHAPE and fwd(eps=-1.0) == ESHAPE
    assert fwd(X=None) == ENULL and fwd(w=None) == ENULL and fwd(Y=None) == ENULL
    assert fwd(R=None) == ENULL                        # H without a residual
    assert fwd(c=4096) == ENULL and fwd(s=4096) == ENULL
    assert fwd(D=40, c=4096, s=4096) == ESHAPE         # D % 32 for MXFP8
    assert fwd(X=4104) == EALIGN and fwd(D=256, c=4104, s=4096) == EALIGN
    assert fwd(M=0) == OK

    def bwd(dY=4096, H=4096, w=4096, dH=None, M=8, D=256, eps=1e-5, dX=8192, dW=8192, ws=4096, n=1 << 30):
        return L.lora4_rmsnorm_backward(dY, H, w, dH, M, D, eps, dX, dW, ws, n, None)
    assert bwd(D=0) == ESHAPE and bwd(dX=None) == ENULL and bwd(H=None) == ENULL and bwd(dH=4100) == EALIGN
    assert bwd(ws=None) == EWS and bwd(n=64) == EWS and bwd(ws=4100) == EALIGN
    assert L.lora4_rmsnorm_workspace_bytes(8, 256) >= 256 * 4
    assert L.lora4_rmsnorm_workspace_bytes(8, 0) == 0 and L.lora4_rmsnorm_workspace_bytes(-1, 8) == 0


def _W(fmt=1, block=64, N=1000, K=512, groups=2, codes=256, scales=512, scales2=None):
    return L.lora4_W(fmt, block, N, K, groups, codes, scales, scales2)


def test_gated_abi_refusals():
    def fwd(W=None, act=1, X=4096, M=16, A=4096, B=4096, r=16, s=1.0, offs=None, H=8192, GU=8192, Z=8192, ws=4096,
            n=1 << 40):
        return L.lora4_gated_forward(W or _W(), act, X, M, A, B, r, s, offs, H, GU, Z, ws, n, None)

    def bwd(W=None, act=1, X=4096, dH=4096, GU=4096, M=16, A=4096, B=4096, r=16, s=1.0, offs=None, Z=None, dX=8192,
            dA=8192, dB=8192, ws=4096, n=1 << 40):
        return L.lora4_gated_backward(W or _W(), act, X, dH, GU, M, A, B, r, s, offs, Z, dX, dA, dB, ws, n, None)
    for call in (fwd, bwd):
        assert call(W=_W(groups=1)) == ESHAPE and call(W=_W(groups=3)) == ESHAPE
        assert call(W=_W(fmt=9)) == EFORMAT and call(act=4) == EFORMAT and call(act=-1) == EFORMAT
        assert call(r=0) == ESHAPE and call(r=129) == ESHAPE and call(M=-1) == ESHAPE
        assert call(s=float("inf")) == ESHAPE
        assert call(W=_W(groups=4)) == ENULL            # experts need offsets
        assert call(offs=4096) == ESHAPE
        assert call(X=None) == ENULL and call(A=None) == ENULL and call(X=4100) == EALIGN
        assert call(ws=None) == EWS and call(n=16) == EWS and call(ws=4104) == EALIGN
    assert fwd(H=None) == ENULL and fwd(GU=4104) == EALIGN and fwd(M=0) == OK
    assert bwd(GU=None) == ENULL and bwd(dH=None) == ENULL and bwd(dX=None) == ENULL and bwd(dB=None) == ENULL
    assert L.lora4_gated_workspace_bytes(0, _W(), 16, 16) > 0 and L.lora4_gated_workspace_bytes(1, _W(), 16, 16) > 0
    assert L.lora4_gated_workspace_bytes(2, _W(), 16, 16) == 0
    assert L.lora4_gated_workspace_bytes(0, _W(groups=1), 16, 16) == 0
    assert L.lora4_gated_workspace_bytes(0, _W(groups=6), 16, 16) > 0


def test_epilogue_abi_refusals():
    W1 = _W(groups=1)

    def fwd(W=None, act=2, X=4096, M=16, A=4096, B=4096, r=16, s=1.0, offs=None, bias=4096, R=4096, Y=8192, P=8192,
            Z=8192, ws=4096, n=1 << 40):
        return L.lora4_forward_epilogue(W or W1, act, X, M, A, B, r, s, offs, bias, R, Y, P, Z, ws, n, None)

    def bwd(W=None, act=2, X=4096, dY=4096, P=4096, M=16, A=4096, B=4096, r=16, s=1.0, offs=None, Z=None, dX=8192,
            dA=8192, dB=8192, db=8192, ws=4096, n=1 << 40):
        return L.lora4_backward_epilogue(W or W1, act, X, dY, P, M, A, B, r, s, offs, Z, dX, dA, dB, db, ws, n, None)
    for call in (fwd, bwd):
        assert call(act=7) == EFORMAT and call(r=257) == ESHAPE and call(M=-5) == ESHAPE
        assert call(W=_W(groups=2)) == ENULL and call(offs=4096) == ESHAPE
        assert call(X=None) == ENULL and call(B=None) == ENULL and call(A=4100) == EALIGN
        assert call(ws=None) == EWS and call(n=16) == EWS
    assert fwd(Y=None) == ENULL and fwd(bias=4100) == EALIGN and fwd(R=4100) == EALIGN and fwd(M=0) == OK
    assert bwd(P=None) == ENULL and bwd(dA=None) == ENULL and bwd(db=4100) == EALIGN
    assert L.lora4_epilogue_workspace_bytes(1, W1, 16, 16) > 0
    assert L.lora4_epilogue_workspace_bytes(3, W1, 16, 16) == 0


def _base(N=96, K=128, groups=2):
    return L.PackedBase(L.LORA4_NF4, N, K, groups, torch.zeros((groups, 16), dtype=torch.uint8),
                        torch.zeros((groups, 16)), None)


def test_binding_refusals():
    bf = torch.bfloat16
    z = lambda *s: torch.zeros(s, dtype=bf)
    X, A, B = z(40, 128), z(2, 8, 128), z(2, 96, 8)
    assert L.check_gated_args(_base(), X, A, B) == (40, 8, 1)
    offs = torch.tensor([0, 10, 40])
    assert L.check_gated_args(_base(groups=4), X, z(4, 8, 128), z(4, 96, 8), offs) == (40, 8, 2)
    bad = [dict(base=_base(groups=3)), dict(A=z(8, 128)), dict(A=z(2, 8, 64)), dict(B=z(2, 95, 8)), dict(B=z(96, 8)),
           dict(X=z(40, 64)), dict(X=X.float()), dict(offsets=offs), dict(tensors=[("H", z(40, 95), (40, 96))]),
           dict(base=_base(groups=4), A=z(4, 8, 128), B=z(4, 96, 8)),
           dict(base=_base(groups=4), A=z(4, 8, 128), B=z(4, 96, 8), offsets=offs.int())]
    for kw in bad:
        with pytest.raises(ValueError):
            L.check_gated_args(**{**dict(base=_base(), X=X, A=A, B=B), **kw})
    w = z(128)
    for args, kw in [((X, w[:64], 1e-5), {}), ((X.float(), w, 1e-5), {}), ((X.t(), w, 1e-5), {}),
                     ((X, w, 1e-5), dict(residual=z(40, 64))), ((X, w, 1e-5), dict(out={"H": z(40, 128)})),
                     ((z(4, 40), z(40), 1e-5), dict(mx=True)), ((X, w, 1e-5), dict(want_y=False)),
                     ((X, w, 1e-5), dict(out={"Y": z(40, 127)})),
                     ((X, w, 1e-5), {})]:                # (the last: CPU tensors)
        with pytest.raises(ValueError):
            L.rmsnorm(*args, **kw)
    for kw in [dict(dY=z(40, 64)), dict(dH=z(4, 128)), dict(workspace=torch.zeros(8, dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            L.rmsnorm_backward(**{**dict(dY=X, H=X, weight=w, eps=1e-5), **kw})
    b1, A1, B1 = _base(groups=1), z(8, 128), z(96, 8)
    for kw in [dict(activation="relu"), dict(bias=z(95)), dict(residual=z(40, 95)), dict(bias=torch.zeros(96)),
               dict(out={"Y": z(39, 96)})]:
        with pytest.raises(ValueError):
            L.forward_epilogue(b1, X, A1, B1, 1.0, **kw)
    for kw in [dict(activation="gelu"), dict(activation="gelu", P=z(40, 95)), dict(Z=z(40, 7)),
               dict(out={"dbias": z(95)})]:
        with pytest.raises(ValueError):
            L.backward_epilogue(b1, X, z(40, 96), A1, B1, 1.0, **kw)
    for kw in [dict(GU=z(40, 96)), dict(dH=z(40, 95)), dict(Z=z(40, 8)), dict(activation="tanh")]:
        with pytest.raises(ValueError):
            L.gated_backward(**{**dict(base=_base(), X=X, dH=z(40, 96), GU=z(40, 192), A=A, B=B, s=1.0), **kw})
