"""Oracle of the softmax cross entropy behind a frozen head, with the gradient of
its input, in float64 (test infrastructure; no code shared with the HIP path).
"""

import numpy as np


def loss(X, W, targets, weights=None, ignore=-100):
    """{"loss", "lse", "total", "dX", "I_dX"}: I_dX = w sum over the other words of
    p |W|, the scale of what rounding their exponentials costs; "size" [M] bounds
    the sums of absolute values of the rows' logits."""
    M = X.shape[0]
    counts = targets != ignore
    w = np.where(counts, 1.0 / max(1, counts.sum()) if weights is None else weights, 0.0)
    l = X @ W.T
    at = np.where(counts, targets, 0)
    lt = l[np.arange(M), at]
    top = l.max(axis=1)
    lse = top + np.log(np.exp(l - top[:, None]).sum(axis=1))
    p = np.exp(l - lse[:, None])
    p[np.arange(M), at] = 0.0
    # log of 1 + the others over the target, which keeps its digits
    with np.errstate(over="ignore"):
        rest = np.exp(l - lt[:, None])
        rest[np.arange(M), at] = 0.0
        rest = rest.sum(axis=1)
    value = np.where(np.isfinite(rest), np.log1p(np.where(np.isfinite(rest), rest, 0.0)), lse - lt)
    value = np.where(counts, value, 0.0)
    dX = w[:, None] * (p @ W - p.sum(axis=1, keepdims=True) * W[at])
    return {"loss": value, "lse": np.where(counts, lse, 0.0), "total": float((w * value).sum()), "dX": dX,
            "I_dX": np.abs(w)[:, None] * (p @ np.abs(W)), "I_t": np.abs(w)[:, None] * p.sum(axis=1, keepdims=True) * np.abs(W[at]),
            "size": (np.abs(X) @ np.abs(W).T).max(axis=1)}
