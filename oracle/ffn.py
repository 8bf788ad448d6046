"""The feed-forward half of a pre-norm block, plain float64.

Test infrastructure only (see the package docstring). The definitions:

* RMS norm with the residual's addition: ``h = x + res``,
  ``y = h w / sqrt(mean(h^2) + eps)`` per row; with ``n = h rstd`` and
  ``t = dy w`` its gradients are ``dx = rstd (t - n mean(t n)) + dh`` (dh reaches
  h past the norm) and ``dw = sum over rows of dy n``.
* The activations ``silu(x) = x / (1 + e^-x)``, ``gelu(x) = x Phi(x)`` and its
  tanh form, with their derivatives.
* Gated projections: ``H = act(G) * U`` of two unmerged-LoRA projections of one
  X; the gradients by the chain rule.
* The linear with an epilogue: ``P = Y_lora_linear + bias``,
  ``Y = act(P) + residual``.

All products and sums are float64; the linear parts are ``lora.forward`` and
``lora.backward``.
"""

import math

import numpy as np

from . import lora

_erfc = np.vectorize(math.erfc, otypes=[np.float64])

ACTIVATIONS = ("none", "silu", "gelu", "gelu_tanh")


def act(x, name):
    """The activation and its derivative at x: (value, slope)."""
    x = np.asarray(x, dtype=np.float64)
    if name == "none":
        return x.copy(), np.ones_like(x)
    if name == "silu":
        p = 1.0 / (1.0 + np.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    if name == "gelu":
        cdf = 0.5 * _erfc(-x / math.sqrt(2.0))
        return x * cdf, cdf + x * np.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (x + 0.044715 * x ** 3))
        return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * x * x)
    raise ValueError(name)


def rmsnorm(X, w, eps, R=None):
    """{"H", "Y"} of rows X [M, D] (+ R)."""
    h = np.asarray(X, np.float64) + (0.0 if R is None else np.asarray(R, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    return {"H": h, "Y": h * rstd * np.asarray(w, np.float64)}


def rmsnorm_backward(dY, H, w, eps, dH=None):
    """{"dX", "dW"} at H."""
    dY, h, w = (np.asarray(t, np.float64) for t in (dY, H, w))
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    n, t = h * rstd, dY * w
    dX = rstd * (t - n * np.mean(t * n, axis=1, keepdims=True))
    return {"dX": dX if dH is None else dX + np.asarray(dH, np.float64), "dW": np.sum(dY * n, axis=0)}


def gated_forward(X, Wg, Wu, A, B, s, activation):
    """{"H", "G", "U", "Z"} for A [2, r, K], B [2, N, r] (gate, up)."""
    g = lora.forward(X, Wg, A[0], B[0], s)
    u = lora.forward(X, Wu, A[1], B[1], s)
    return {"H": act(g["Y"], activation)[0] * u["Y"], "G": g["Y"], "U": u["Y"],
            "Z": np.concatenate([g["Z"], u["Z"]], axis=1)}


def gated_backward(X, Wg, Wu, A, B, s, activation, dH, G, U, Z=None):
    """{"dX", "dA" [2, r, K], "dB" [2, N, r], "dG", "dU"} at the given G, U
    (and Z [M, 2 r])."""
    v, d = act(G, activation)
    dH = np.asarray(dH, np.float64)
    dG, dU = dH * np.asarray(U, np.float64) * d, dH * v
    r = A[0].shape[0]
    g = lora.backward(X, Wg, A[0], B[0], s, dG, None if Z is None else Z[:, :r])
    u = lora.backward(X, Wu, A[1], B[1], s, dU, None if Z is None else Z[:, r:])
    return {"dX": g["dX"] + u["dX"], "dA": np.stack([g["dA"], u["dA"]]), "dB": np.stack([g["dB"], u["dB"]]),
            "dG": dG, "dU": dU, "dZ": np.concatenate([g["dZ"], u["dZ"]], axis=1)}


def epilogue_forward(X, W, A, B, s, activation, bias=None, R=None):
    """{"Y", "P", "Z"}."""
    f = lora.forward(X, W, A, B, s)
    P = f["Y"] + (0.0 if bias is None else np.asarray(bias, np.float64))
    Y = act(P, activation)[0]
    return {"Y": Y if R is None else Y + np.asarray(R, np.float64), "P": P, "Z": f["Z"]}


def epilogue_backward(X, W, A, B, s, activation, dY, P=None, Z=None):
    """{"dX", "dA", "dB", "dbias", "dP"} at the given pre-activation P."""
    dP = np.asarray(dY, np.float64)
    if activation != "none":
        dP = dP * act(P, activation)[1]
    b = lora.backward(X, W, A, B, s, dP, Z)
    return {**b, "dbias": dP.sum(axis=0), "dP": dP}
