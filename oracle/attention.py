"""Oracle of causal attention over packed sequences with grouped heads, forward
and backward, in float64 (test infrastructure; no code shared with the HIP path).

Sequence i has queries q_ranges[i] = (first, end) and keys k_ranges[i] likewise;
its query a sees the keys b <= a + Lk - Lq. A query that sees none has O = 0,
lse = -inf and no gradient.
"""

import numpy as np


def _weights(q, k, scale):
    """P [Lq, Lk] and lse [Lq] of one head."""
    Lq, Lk = q.shape[0], k.shape[0]
    seen = np.arange(Lk)[None, :] <= np.arange(Lq)[:, None] + (Lk - Lq)
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    top = s.max(axis=1, initial=-np.inf, keepdims=True)
    e = np.where(seen, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
    n = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(top), top, 0.0) + np.log(n))[:, 0]
    return e / np.where(n > 0, n, 1.0), lse


# A value below the smallest normal number of fp32 and bf16 may be flushed to
# zero: it is off by at most this, absolutely.
TINY = 2.0 ** -126

EXACT = 32   # keys of a row whose delta dQ takes from P and dP


def weight_error(q, k, lse, scale):
    """[Lq]: how far a weight P computed in fp32 may be off, relative to itself.
    A score is D exact products summed in fp32, off by at most D 2^-24 of the sum of
    their sizes; its multiple of log2 e and lse (which is fp32 itself) by 2^-24 each;
    exp2 of a number of size x by 2^-24 x and one unit."""
    if k.shape[0] == 0:
        return np.zeros(q.shape[0])
    size = scale * (np.abs(q) @ np.abs(k).T).max(axis=1)
    return 2.0 ** -24 * ((q.shape[1] + 4) * size + 4 * np.abs(np.where(np.isfinite(lse), lse, 0.0))) + 2.0 ** -20


def forward(Q, K, V, scale, q_ranges, k_ranges):
    """{"O", "lse", "I_O", "E_O"}; I_O = sum over the keys of P |V|, the scale of
    what rounding P costs; E_O: what fp32 arithmetic may cost. Rows of no sequence
    are NaN."""
    Hq, Hkv = Q.shape[1], K.shape[1]
    O, I, E = (np.full(Q.shape, np.nan) for _ in range(3))
    lse = np.full(Q.shape[:2], np.nan)
    for (a, b), (c, d) in zip(q_ranges, k_ranges):
        for h in range(Hq):
            g = h // (Hq // Hkv)
            P, lse[a:b, h] = _weights(Q[a:b, h], K[c:d, g], scale)
            O[a:b, h] = P @ V[c:d, g]
            I[a:b, h] = P @ np.abs(V[c:d, g])
            # the weights, and their sum that divides
            E[a:b, h] = 2 * weight_error(Q[a:b, h], K[c:d, g], lse[a:b, h], scale)[:, None] * I[a:b, h]
            E[a:b, h] += TINY * (1 + np.abs(V[c:d, g]).sum(axis=0))
    return {"O": O, "lse": lse, "I_O": I, "E_O": E}


def backward(Q, K, V, O, dO, scale, q_ranges, k_ranges):
    """{"dQ", "dK", "dV"}: delta = sum dO O of the given O for dQ of rows that see
    more than EXACT keys, and for all others and dK what it stands for, the sum of
    P (dO V^T) over the keys (the two differ by O's rounding, where the given O is
    rounded). I_dQ, I_dK, I_dV: the
    sums of absolute values that the roundings of dS and P enter; E_dQ, E_dK, E_dV:
    what fp32 arithmetic may cost (the weights' error, and that of dP and delta,
    sums of D exact products each, whose difference may cancel)."""
    Hq, Hkv = Q.shape[1], K.shape[1]
    o = {p + n: np.full(x.shape, np.nan) for n, x in (("dQ", Q), ("dK", K), ("dV", V)) for p in ("", "I_", "E_")}
    for (a, b), (c, d) in zip(q_ranges, k_ranges):
        for n in ("dK", "dV", "I_dK", "I_dV", "E_dK", "E_dV"):
            o[n][c:d] = 0.0
        for h in range(Hq):
            g = h // (Hq // Hkv)
            q, k, do = Q[a:b, h], K[c:d, g], dO[a:b, h]
            P, lse = _weights(q, k, scale)
            dP = do @ V[c:d, g].T
            few = (np.arange(b - a) + (d - c) - (b - a) < EXACT)[:, None]
            exact = (P * dP).sum(axis=1, keepdims=True)
            dS = P * (dP - np.where(few, exact, (do * O[a:b, h]).sum(axis=1, keepdims=True))) * scale
            dSk = P * (dP - exact) * scale
            r = weight_error(q, k, lse, scale)[:, None]
            terms = np.abs(do) @ np.abs(V[c:d, g]).T + np.abs(do * O[a:b, h]).sum(axis=1, keepdims=True)
            e = r * np.abs(dS) + P * terms * scale * Q.shape[2] * 2.0 ** -24 + TINY * (1 + scale * (1 + terms))
            # (the exact delta: weights off by r each, which do not sum to 1 then, and n terms)
            ek = e + P * scale * ((r + (d - c) * 2.0 ** -24) * (P * terms).sum(axis=1, keepdims=True))
            o["E_dQ"][a:b, h] = np.where(few, ek, e) @ np.abs(k) + TINY
            e = ek
            o["E_dK"][c:d, g] += e.T @ np.abs(q) + TINY
            o["E_dV"][c:d, g] += (r * P + TINY).T @ np.abs(do) + TINY
            o["dQ"][a:b, h] = dS @ k
            o["dK"][c:d, g] += dSk.T @ q
            o["dV"][c:d, g] += P.T @ do
            o["I_dQ"][a:b, h] = np.abs(dS) @ np.abs(k)
            o["I_dK"][c:d, g] += np.abs(dSk).T @ np.abs(q)
            o["I_dV"][c:d, g] += P.T @ np.abs(do)
    return o


def dq(Q, K, V, dO, scale, q_ranges, k_ranges, u):
    """{"dQ", "I_dQ", "E_dQ", "D_dQ", "N_dQ"} of the definition alone: delta is the sum
    of P (dO V^T) in all rows, whatever O a caller holds. An implementation that takes
    delta from an O of unit roundoff u has it off by d = sum dO (the error of O), and
    dQ by d scale P K, in D_dQ at most (each element of O off by 1.01 u (|O| + I_O) +
    E_O, as forward states) and in N_dQ [rows] the root of the mean square of the row's
    norm: the roundings of O's elements and P's are independent, uniform within u at
    most, of variance below u^2 of their terms' squares."""
    f = forward(Q, K, V, scale, q_ranges, k_ranges)
    o = {n: np.full(Q.shape, np.nan) for n in ("dQ", "I_dQ", "E_dQ", "D_dQ")}
    o["N_dQ"] = np.full(Q.shape[:2], np.nan)
    G = Q.shape[1] // K.shape[1]
    for (a, b), (c, d) in zip(q_ranges, k_ranges):
        for h in range(Q.shape[1]):
            q, k, v, do = Q[a:b, h], K[c:d, h // G], V[c:d, h // G], dO[a:b, h]
            P, lse = _weights(q, k, scale)
            dP = do @ v.T
            dS = P * (dP - (P * dP).sum(axis=1, keepdims=True)) * scale
            O, I, E = (f[n][a:b, h] for n in ("O", "I_O", "E_O"))
            off = (np.abs(do) * (1.01 * u * (np.abs(O) + I) + E)).sum(axis=1, keepdims=True)
            rms = u * np.sqrt((do ** 2 * (O ** 2 + I ** 2)).sum(axis=1))
            r = weight_error(q, k, lse, scale)[:, None]
            terms = np.abs(do) @ np.abs(v).T + (np.abs(do) * I).sum(axis=1, keepdims=True)
            e = r * np.abs(dS) + P * terms * scale * Q.shape[2] * 2.0 ** -24 + TINY * (1 + scale * (1 + terms))
            e += P * scale * ((r + (d - c) * 2.0 ** -24) * (P * terms).sum(axis=1, keepdims=True))
            o["dQ"][a:b, h] = dS @ k
            o["I_dQ"][a:b, h] = np.abs(dS) @ np.abs(k)
            o["E_dQ"][a:b, h] = e @ np.abs(k) + TINY
            # (dS is rounded with delta's error in it)
            o["D_dQ"][a:b, h] = scale * off * (np.abs(P @ k) + 2 * u * (P @ np.abs(k)))
            o["N_dQ"][a:b, h] = scale * rms * np.linalg.norm(P @ k, axis=1)
    return o
