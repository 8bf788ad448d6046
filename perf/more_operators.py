"""Measured cases of the operators around the projections of a fine-tuning step:
causal attention over packed sequences with grouped heads (forward, single tokens
over a cache, backward), and the softmax cross entropy over a large vocabulary
behind a frozen head (loss, and loss with the gradient of its input).

With ``own`` false, ``run`` computes an operator in its plain form (elementary
torch operations in float32, rounded once at the end); with ``own`` true it
makes the calls a user makes of the library.

A case's ``op`` is one of attn, attn_bwd, loss, loss_grad. Attention: Hq query
heads over Hkv key heads of D elements; kind "packed": S sequences of together T
tokens that attend to themselves; kind "cache": S sequences of Lq new tokens each
over their own slab of ``cap`` cache rows, part of it filled (the new tokens'
keys among them). ``mix`` fixes the lengths. fused: q, k and v are columns of one
projection's output. Loss: M tokens, hidden size K, V words.
"""

import math
import random

import torch

own = False

BF = torch.bfloat16
DEV = "cuda"
IGNORE = -100


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _attn(name, **kw):
    c = dict(name=name, op="attn", kind="packed", Hq=32, Hkv=8, D=128, mix=1, fused=False, lse=False)
    c.update(kw)
    return c


def _loss(name, **kw):
    c = dict(name=name, op="loss", M=4096, K=4096, V=128256, weights=False, ignored=0.0)
    c.update(kw)
    return c


def listed():
    return [
        # one token of one sequence over its cache: latency
        _attn("attn_decode", kind="cache", S=1, Lq=1, cap=4096),
        # a serving batch, one token per sequence, caches of very different fill
        _attn("attn_decode_batch", kind="cache", S=24, Lq=1, cap=32768, Hq=64, mix=2),
        # the training forward of a packed batch, q, k and v from one projection
        _attn("attn_train", S=6, T=4096, fused=True, lse=True, mix=3),
        # one long prompt, as many key heads as query heads
        _attn("attn_prompt", S=1, T=32768, Hq=40, Hkv=40),
        # chunks of new tokens behind caches, odd lengths, seven query heads to a key head
        _attn("attn_chunk_odd", kind="cache", S=3, Lq=333, cap=5003, Hq=14, Hkv=2, D=80, mix=4),
        # backward of the packed training batch
        _attn("attn_train_bwd", op="attn_bwd", S=6, T=4096, fused=True, mix=3),
        # backward over one long sequence, eight query heads to a key head
        _attn("attn_long_bwd", op="attn_bwd", S=1, T=8192, Hq=64),
        # backward of short ragged sequences, ungrouped heads of 96
        _attn("attn_odd_bwd", op="attn_bwd", S=9, T=2081, Hq=12, Hkv=12, D=96, mix=5),
        # a few tokens scored against the vocabulary: the head is read once
        _loss("loss_score", M=8),
        # evaluation: loss alone, wide hidden size, odd vocabulary
        _loss("loss_eval", M=2048, K=5120, V=32003),
        # the end of the training forward and the start of its backward
        _loss("loss_train", op="loss_grad", ignored=0.1),
        # the same on a ragged batch with weights of its own per token
        _loss("loss_train_odd", op="loss_grad", M=1333, K=2080, V=50021, weights=True, ignored=0.3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn_bwd", "loss", "loss_grad"])
    if op.startswith("attn"):
        D = rng.choice([128, 128, 64, 8 * rng.randint(2, 16)])
        Hkv = rng.choice([1, 2, 4, 8, 8, rng.randint(1, 12)])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
        c = dict(op=op, Hq=Hq, Hkv=Hkv, D=D, mix=rng.randint(1, 1 << 20), fused=False, lse=rng.random() < 0.5)
        if op == "attn" and rng.random() < 0.5:
            c["kind"] = "cache"
            c["S"] = _log_int(rng, 1, 32)
            c["cap"] = _log_int(rng, 16, 32768)
            c["Lq"] = min(c["cap"], rng.choice([1, 1, 2, _log_int(rng, 1, 1024)]))
        else:
            c["kind"] = "packed"
            c["T"] = _log_int(rng, 1, 8192)
            c["S"] = min(c["T"], _log_int(rng, 1, 16))
            c["fused"] = rng.random() < 0.5
        return c
    K = 8 * _log_int(rng, 8, 768)
    V = _log_int(rng, 100, 131072)
    M = max(1, min(_log_int(rng, 1, 4096), (1 << 41) // (K * V)))
    return dict(op=op, M=M, K=K, V=V, weights=rng.random() < 0.5, ignored=rng.choice([0.0, 0.1, 0.5]))


def _lengths(c):
    """(query lengths, key lengths) of the sequences; of a batch of several packed
    ones some may be empty."""
    rng = random.Random(c["mix"])
    S = c["S"]
    if c["kind"] == "cache":
        fill = [max(c["Lq"], rng.randint(c["cap"] // 8, c["cap"])) for _ in range(S)]
        return [c["Lq"]] * S, fill
    cuts = sorted(rng.randint(0, c["T"]) for _ in range(S - 1))
    n = [b - a for a, b in zip([0] + cuts, cuts + [c["T"]])]
    return n, n


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"].startswith("loss"):
        M, K, V = c["M"], c["K"], c["V"]
        grad = c["op"] == "loss_grad"
        b = V * K * 2 + M * K * 2 * (2 if grad else 1) + M * (8 + 4 + 4 + (4 if c["weights"] else 0)) + 4
        return {"bytes": b, "flops": 2 * M * K * V * (2 if grad else 1)}
    nq, nk = _lengths(c)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    pairs = sum(q * (k - q) + q * (q + 1) // 2 for q, k in zip(nq, nk))
    rows, keys = sum(nq) * Hq, sum(nk) * Hkv
    if c["op"] == "attn":
        return {"bytes": 2 * D * (2 * rows + 2 * keys) + (4 * rows if c["lse"] else 0), "flops": 4 * D * Hq * pairs}
    return {"bytes": 2 * D * (4 * rows + 4 * keys) + 4 * rows, "flops": 10 * D * Hq * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _offsets(n):
    at = [0]
    for x in n:
        at.append(at[-1] + x)
    return torch.tensor(at, dtype=torch.int64, device=DEV)


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=g, device=DEV) * std).to(BF)

    s = {"case": c}
    if c["op"].startswith("loss"):
        M, K, V = c["M"], c["K"], c["V"]
        s["W"] = normal(V, K, std=0.02)
        s["t"] = torch.randint(0, V, (M,), generator=g, device=DEV)
        # a normed hidden state, which leans towards its target's row more or less:
        # from words that are guessed to words that are known
        lean = torch.rand((M, 1), generator=g, device=DEV) * 12 / (0.02 * math.sqrt(K))
        x = torch.randn((M, K), generator=g, device=DEV)
        w = s["W"][s["t"]].float()
        s["X"] = (x + lean * w / w.norm(dim=1, keepdim=True)).to(BF)
        # prompt tokens and padding carry no loss
        s["t"][torch.rand(M, generator=g, device=DEV) < c["ignored"]] = IGNORE
        s["w"] = torch.rand(M, generator=g, device=DEV) / M if c["weights"] else None
        return s
    nq, nk = _lengths(c)
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    s["nq"], s["nk"] = nq, nk
    s["scale"] = 1 / math.sqrt(D)
    s["q_offsets"] = _offsets(nq)
    if c["kind"] == "cache":
        # what lies behind the filled part of a slab is left over from earlier use
        s["Q"] = normal(sum(nq), Hq, D, std=1.5)
        s["K"], s["V"] = normal(c["S"] * c["cap"], Hkv, D, std=1.5), normal(c["S"] * c["cap"], Hkv, D)
        s["k_offsets"] = _offsets([c["cap"]] * c["S"])
        s["k_lengths"] = torch.tensor(nk, dtype=torch.int64, device=DEV)
    else:
        T = c["T"]
        if c["fused"]:
            qkv = normal(T, Hq + 2 * Hkv, D, std=1.5)
            s["Q"], s["K"], s["V"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        else:
            s["Q"], s["K"], s["V"] = normal(T, Hq, D, std=1.5), normal(T, Hkv, D, std=1.5), normal(T, Hkv, D)
        s["k_offsets"] = s["k_lengths"] = None
    if c["op"] == "attn_bwd":
        s["dO"] = normal(T, Hq, D, std=0.02)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = case
    if c["op"].startswith("attn"):
        s["pad"] = _padding(s, c)
        if c["op"] == "attn_bwd":
            # what the forward has kept
            s["O"], s["lse"] = _attn_plain(s, c)
    if own:
        import lora_fine_tuning_amd as L
        s["L"] = L
        if c["op"].startswith("loss"):
            s["ws"] = L.head_loss_workspace(c["op"] == "loss_grad", c["M"], c["K"], c["V"], DEV)
        else:
            s["ws"] = L.attention_workspace(1 if c["op"] == "attn_bwd" else 0, s["Q"].shape[0], s["K"].shape[0], c["S"],
                                            c["Hq"], c["Hkv"], c["D"], DEV)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"].startswith("loss"):
        return _loss_plain(s, c)
    if c["op"] == "attn":
        o, lse = _attn_plain(s, c)
        return {"O": o, "lse": lse} if c["lse"] else {"O": o}
    return _attn_bwd_plain(s, c)


def _run_own(s, c):
    L = s["L"]
    if c["op"].startswith("loss"):
        o = L.head_loss(s["X"], s["W"], s["t"], weights=s["w"], ignore_index=IGNORE, want_grad=c["op"] == "loss_grad",
                        workspace=s["ws"])
    else:
        kw = dict(q_offsets=s["q_offsets"], k_offsets=s["k_offsets"], k_lengths=s["k_lengths"], workspace=s["ws"])
        if c["op"] == "attn":
            o = L.attention(s["Q"], s["K"], s["V"], s["scale"], want_lse=c["lse"], **kw)
        else:
            o = L.attention_backward(s["Q"], s["K"], s["V"], s["O"], s["lse"], s["dO"], s["scale"], **kw)
    return {k: v for k, v in o.items() if v is not None}


# ---- plain forms -----------------------------------------------------------

def _padding(s, c):
    """The padded form of a batch, as a program without packing keeps it: rows of
    the queries and keys of each sequence ([S, longest], the last row where a
    sequence has ended), which of them count, and the visible pairs."""
    nq, nk = (torch.tensor(n, device=DEV) for n in (s["nq"], s["nk"]))
    iq, ik = (torch.arange(max(1, max(n)), device=DEV) for n in (s["nq"], s["nk"]))
    k0 = (s["k_offsets"] if s["k_offsets"] is not None else s["q_offsets"])[:-1]
    rq = (s["q_offsets"][:-1, None] + iq).clamp_max(s["Q"].shape[0] - 1)
    rk = (k0[:, None] + ik).clamp_max(s["K"].shape[0] - 1)
    q_in, k_in = iq < nq[:, None], ik < nk[:, None]
    seen = (ik <= iq[:, None] + (nk - nq)[:, None, None]) & k_in[:, None]
    return {"rq": rq, "rk": rk, "q_in": q_in, "k_in": k_in, "seen": seen}


def _parts(s, c):
    """Key heads per piece: scores of at most 2^31 elements at a time."""
    pairs = s["pad"]["seen"].numel() * (c["Hq"] // c["Hkv"])
    n = max(1, (1 << 31) // pairs)
    return [slice(h, min(c["Hkv"], h + n)) for h in range(0, c["Hkv"], n)]


def _rows(x, rows):
    """[T, H, D] -> float32 [S, H, longest, D]."""
    return x[rows].float().transpose(1, 2)


def _scores(s, c, h):
    """The masked scores [S, heads, G, Lq, Lk] of the key heads h, and their operands."""
    p, G = s["pad"], c["Hq"] // c["Hkv"]
    q = _rows(s["Q"].unflatten(1, (c["Hkv"], G))[:, h].flatten(1, 2), p["rq"]).unflatten(1, (-1, G))
    k = _rows(s["K"][:, h], p["rk"])
    x = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (G, -1)) * s["scale"]
    return x.masked_fill(~p["seen"][:, None, None], -math.inf), q, k


def _attn_plain(s, c):
    p, G = s["pad"], c["Hq"] // c["Hkv"]
    O = torch.empty(s["Q"].shape, dtype=BF, device=DEV)
    lse = torch.empty(s["Q"].shape[:2], dtype=torch.float32, device=DEV)
    at = p["rq"][p["q_in"]]
    for h in _parts(s, c):
        x, _, _ = _scores(s, c, h)
        top = x.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        x = torch.exp(x - top)
        n = x.sum(-1, keepdim=True)
        v = _rows(s["V"][:, h], p["rk"])
        o = torch.matmul(x.flatten(2, 3), v).unflatten(2, (G, -1)) / n.clamp_min(1e-30)
        hq = slice(h.start * G, h.stop * G)
        O[at, hq] = o.flatten(1, 2).transpose(1, 2)[p["q_in"]].to(BF)
        lse[at, hq] = (top + torch.log(n)).squeeze(-1).flatten(1, 2).transpose(1, 2)[p["q_in"]]
    return O, lse


def _attn_bwd_plain(s, c):
    p, G = s["pad"], c["Hq"] // c["Hkv"]
    out = {"d" + n: torch.empty(s[n].shape, dtype=BF, device=DEV) for n in "QKV"}
    aq, ak = p["rq"][p["q_in"]], p["rk"][p["k_in"]]
    q_in = p["q_in"][:, None, None, :, None]
    for h in _parts(s, c):
        x, q, k = _scores(s, c, h)
        hq = slice(h.start * G, h.stop * G)
        v = _rows(s["V"][:, h], p["rk"])
        do = _rows(s["dO"][:, hq], p["rq"]).unflatten(1, (-1, G)) * q_in
        P = torch.softmax(x, -1).masked_fill(~p["seen"][:, None, None], 0.0)
        dP = torch.matmul(do.flatten(2, 3), v.transpose(-1, -2)).unflatten(2, (G, -1))
        dS = P * (dP - (P * dP).sum(-1, keepdim=True)) * s["scale"]
        dq = torch.matmul(dS.flatten(2, 3), k).unflatten(2, (G, -1))
        dk = torch.matmul(dS.flatten(2, 3).transpose(-1, -2), q.flatten(2, 3))
        dv = torch.matmul(P.flatten(2, 3).transpose(-1, -2), do.flatten(2, 3))
        out["dQ"][aq, hq] = dq.flatten(1, 2).transpose(1, 2)[p["q_in"]].to(BF)
        out["dK"][ak, h] = dk.transpose(1, 2)[p["k_in"]].to(BF)
        out["dV"][ak, h] = dv.transpose(1, 2)[p["k_in"]].to(BF)
    return out


def _loss_plain(s, c):
    t, w = s["t"], s["W"].float()
    counts = t != IGNORE
    at = t.clamp_min(0)[:, None]
    x = torch.matmul(s["X"].float(), w.t())
    lse = torch.logsumexp(x, 1)
    loss = torch.where(counts, lse - x.gather(1, at).squeeze(1), 0.0)
    weight = s["w"] if s["w"] is not None else 1.0 / counts.sum().clamp_min(1)
    weight = torch.where(counts, weight, 0.0)
    out = {"loss": loss, "total": (loss * weight).sum()[None]}
    if c["op"] == "loss_grad":
        x = torch.exp(x - lse[:, None])
        x.scatter_add_(1, at, torch.full_like(lse, -1.0)[:, None])
        out["dX"] = (weight[:, None] * torch.matmul(x, w)).to(BF)
    return out


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    return (_exact_loss if case["op"].startswith("loss") else _exact_attn)(s, case)


def _exact_loss(s, c):
    W = s["W"].double()
    rows = torch.arange(c["M"], device=DEV)
    valid = (s["t"] >= 0).double()
    target = torch.where(s["t"] >= 0, s["t"], 0)
    z = s["X"].double().matmul(W.T)
    z -= z[rows, target].unsqueeze(1)          # against the target's logit
    big = z.max(1, keepdim=True).values
    z = (z - big).exp_()
    total = z.sum(1, keepdim=True)
    loss = (big + total.log()).squeeze(1) * valid
    weight = valid / max(1.0, float(valid.sum())) if s["w"] is None else s["w"].double() * valid
    out = {"loss": loss, "total": torch.dot(loss, weight).reshape(1)}
    if c["op"] == "loss_grad":
        z /= total
        z[rows, target] = 0.0
        z[rows, target] = -z.sum(1)            # p - 1 without the cancellation
        z *= weight.unsqueeze(1)
        out["dX"] = z.matmul(W)
    return out


def _exact_attn(s, c):
    """Sequence by sequence and head by head."""
    f = dict(dtype=torch.float64, device=DEV)
    bwd, G = c["op"] == "attn_bwd", c["Hq"] // c["Hkv"]
    out = {n: torch.zeros(s[n[1:]].shape, **f) for n in ("dQ", "dK", "dV")} if bwd else {"O": torch.zeros(s["Q"].shape, **f)}
    if c["op"] == "attn" and c["lse"]:
        out["lse"] = torch.full(s["Q"].shape[:2], -math.inf, **f)
    q1 = k1 = 0
    for i, (m, n) in enumerate(zip(s["nq"], s["nk"])):
        q0, q1 = q1, q1 + m
        k0 = i * c["cap"] if c["kind"] == "cache" else k1
        k1 = k0 + n
        if m == 0 or n == 0:
            continue
        hidden = torch.ones((m, n), dtype=torch.bool, device=DEV).triu(n - m + 1)
        for hq in range(c["Hq"]):
            q, k, v = s["Q"][q0:q1, hq].double(), s["K"][k0:k1, hq // G].double(), s["V"][k0:k1, hq // G].double()
            x = (q * s["scale"]).matmul(k.T)
            x[hidden] = -math.inf
            lse = torch.logsumexp(x, 1)
            x = (x - lse.unsqueeze(1)).exp_()
            if not bwd:
                out["O"][q0:q1, hq] = x.matmul(v)
                if c["lse"]:
                    out["lse"][q0:q1, hq] = lse
                continue
            d = s["dO"][q0:q1, hq].double()
            out["dV"][k0:k1, hq // G] += x.T.matmul(d)
            y = d.matmul(v.T)
            y -= (y * x).sum(1, keepdim=True)
            y *= x * s["scale"]
            out["dQ"][q0:q1, hq] = y.matmul(k)
            out["dK"][k0:k1, hq // G] += y.T.matmul(q)
    return out
