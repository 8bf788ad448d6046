"""Measured cases of the feed-forward operators: the root-mean-square norm with
the residual's addition and an MXFP8 output, the gated projections of a 4-bit
base, and the linear layer with bias, activation and residual in its epilogue.

With ``own`` false, ``run`` computes an operator in its plain form (elementary
torch operations in float32, rounded once at the end); with ``own`` true it
makes the calls a user makes of the library. The frozen base is handed over
row-major, as checkpoints ship it: codes uint8 [G, N, K / 2] (element 2j in the
low nibble of byte j) and one scale per block of 64 (NF4), 32 (MXFP4) or 16
(NVFP4) elements of a row.

A case's ``op`` is one of norm, norm_bwd, gated, gated_bwd, linear, linear_bwd;
sizes: M tokens, K inputs, N outputs of one projection, r the adapter's rank,
E experts (1: a plain layer).
"""

import math
from statistics import NormalDist

import torch

own = False

BLOCK = {"nf4": 64, "nf4_dq": 64, "mxfp4": 32, "nvfp4": 16}
BF = torch.bfloat16
EPS = 1e-5
DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token enters the feed-forward half while decoding: latency
        dict(name="norm_decode", op="norm", M=1, D=4096, residual=True, mx=False),
        # prefill of an MX-native layer: bf16 for the adapter, MXFP8 for the base product
        dict(name="norm_mx", op="norm", M=8192, D=8192, residual=True, mx=True),
        # training with the norm's weight trained too; rows that are no multiple of a vector
        dict(name="norm_bwd_odd", op="norm_bwd", M=4097, D=5003, dh=True, dw=True),
        # one token through the gate and up projections of an 8B-shaped layer
        dict(name="gated_decode", op="gated", M=1, K=4096, N=14336, r=16, E=1, fmt="nf4", act="silu", save=False),
        # a serving batch, one token per sequence, on wide layers
        dict(name="gated_batch", op="gated", M=24, K=8192, N=28672, r=64, E=1, fmt="mxfp4", act="silu", save=False),
        # training forward of the 8B-shaped layer
        dict(name="gated_train", op="gated", M=4096, K=4096, N=14336, r=16, E=1, fmt="nf4", act="silu", save=True),
        # its backward, with double-quantized scales
        dict(name="gated_train_bwd", op="gated_bwd", M=4096, K=4096, N=14336, r=16, E=1, fmt="nf4_dq", act="silu"),
        # experts of a mixture, ragged row groups (one of them empty)
        dict(name="gated_experts", op="gated", M=2048, K=7168, N=2048, r=16, E=16, fmt="mxfp4", act="silu", save=False),
        # the down projection while decoding, with the residual added
        dict(name="linear_decode", op="linear", M=4, K=14336, N=4096, r=16, E=1, fmt="nvfp4", act="none", bias=True,
             residual=True, save=False),
        # the down projection of the training forward, with the residual added
        dict(name="linear_train", op="linear", M=4096, K=14336, N=4096, r=16, E=1, fmt="nf4", act="none", bias=False,
             residual=True, save=False),
        # a plain feed-forward's first projection on a ragged prompt
        dict(name="linear_gelu_odd", op="linear", M=333, K=2080, N=5003, r=24, E=1, fmt="mxfp4", act="gelu_tanh",
             bias=True, residual=False, save=True),
        # backward of that projection in training
        dict(name="linear_gelu_bwd", op="linear_bwd", M=2048, K=4096, N=4096, r=32, E=1, fmt="nf4", act="gelu",
             bias=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "gated", "gated", "gated_bwd", "linear", "linear", "linear_bwd"])
    if op in ("norm", "norm_bwd"):
        D = _log_int(rng, 32, 16384)
        M = _log_int(rng, 1, min(16384, (1 << 26) // D))
        if op == "norm_bwd":
            return dict(op=op, M=M, D=D, dh=rng.random() < 0.5, dw=rng.random() < 0.5)
        mx = rng.random() < 0.5
        return dict(op=op, M=M, D=max(32, D // 32 * 32) if mx else D, residual=rng.random() < 0.7, mx=mx)
    fmt = rng.choice(["nf4", "nf4_dq", "mxfp4", "nvfp4"])
    step = 64 if fmt in ("nf4", "nf4_dq") else 32
    E = rng.choice([1, 1, 1, rng.randint(2, 12)])
    K = max(2, _log_int(rng, 256, 8192) // step) * step
    N = _log_int(rng, 64, 14336 // E)
    if rng.random() < 0.5:
        N = max(64, N // 64 * 64)
    M = _log_int(rng, 1, 4096)
    M = max(1, min(M, int(4096 * 14336 * 4096 / (K * N))))
    r = rng.choice([1, 4, 8, 12, 16, 16, 32, 64, 128])
    c = dict(op=op, M=M, K=K, N=N, r=r, E=E, fmt=fmt)
    if op.startswith("gated"):
        c["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh"])
        if op == "gated":
            c["save"] = rng.random() < 0.5
        return c
    c["act"] = rng.choice(["none", "silu", "gelu", "gelu_tanh"])
    c["bias"] = rng.random() < 0.5
    if op == "linear":
        c["residual"] = rng.random() < 0.5
        c["save"] = c["act"] != "none" and rng.random() < 0.5
    return c


def work(c):
    """Bytes and operations that one pass cannot do without."""
    if c["op"] in ("norm", "norm_bwd"):
        M, D = c["M"], c["D"]
        if c["op"] == "norm":
            b = M * D * 2 * (1 + (2 if c["residual"] else 0) + 1) + D * 2
            b += M * D + M * D // 32 if c["mx"] else 0
            return {"bytes": b, "flops": 6 * M * D}
        return {"bytes": M * D * 2 * (3 + (1 if c["dh"] else 0)) + D * 2 * (2 if c["dw"] else 1), "flops": 10 * M * D}
    M, K, N, r, E = c["M"], c["K"], c["N"], c["r"], c["E"]
    P = 2 if c["op"].startswith("gated") else 1
    bits = {"nf4": 4.5, "nf4_dq": 4.127, "mxfp4": 4.25, "nvfp4": 4.5}[c["fmt"]]
    used = min(E, M)   # experts with no rows are not read
    w = used * P * N * K * bits / 8
    ab = used * P * r * (N + K) * 2
    if c["op"] in ("gated", "linear"):
        b = w + ab + M * K * 2 + M * N * 2 + (P * M * (N + r) * 2 if c["save"] else 0)
        b += (M * N * 2 if c.get("residual") else 0) + (E * N * 2 if c.get("bias") else 0)
        return {"bytes": b, "flops": 2 * P * M * (N * K + r * (N + K))}
    act_in = 2 * M * N * 2 if P == 2 else (M * N * 2 if c["act"] != "none" else 0)
    b = w + 2 * E * P * r * (N + K) * 2 + 2 * M * K * 2 + M * N * 2 + act_in + M * P * r * 2
    b += E * N * 2 if c.get("bias") else 0
    return {"bytes": b, "flops": 2 * P * M * (N * K + 2 * r * (N + K))}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _nf4_levels():
    """The 16 normal-float levels: quantiles of the normal distribution, eight
    above zero and seven below, with zero itself, over the largest."""
    inv = NormalDist().inv_cdf
    d = 0.5 * ((1 - 1 / 30) + (1 - 1 / 32))
    pos = [inv(d + (0.5 - d) * i / 8) for i in range(8)]
    neg = [-inv(d + (0.5 - d) * i / 7) for i in range(7)]
    v = sorted(pos + neg + [0.0])
    return [x / v[-1] for x in v]


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(BF)


def _quantize(W, fmt):
    """Row-major codes, scales and second-level scales of a base W [N, K]."""
    N, K = W.shape
    blk = BLOCK[fmt]
    w = W.float().reshape(N, K // blk, blk)
    amax = w.abs().amax(-1)
    second = None
    if fmt in ("nf4", "nf4_dq"):
        lv = torch.tensor(_nf4_levels(), device=DEV, dtype=torch.float32)
        x = w / amax.clamp_min(1e-30)[..., None]
        idx = torch.bucketize(x, (lv[1:] + lv[:-1]) / 2)
        scales = amax
        if fmt == "nf4_dq":
            flat = amax.reshape(-1)
            n = flat.numel()
            pad = torch.nn.functional.pad(flat, (0, -n % 256)).reshape(-1, 256)
            second = pad.amax(-1).clamp_min(1e-30)
            scales = (pad / second[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).reshape(-1)[:n].reshape(N, -1)
    else:
        if fmt == "mxfp4":
            e = torch.frexp(amax).exponent - 1 - 2
            scales = (e + 127).clamp(0, 254).to(torch.uint8)
            sv = torch.exp2(e.float())
        else:
            s8 = (amax / 6).clamp_max(448).to(torch.float8_e4m3fn)
            scales, sv = s8.view(torch.uint8), s8.float().clamp_min(2.0 ** -9)
        t = torch.tensor(E2M1, device=DEV)
        x = w / sv[..., None]
        idx = torch.bucketize(x.abs(), (t[1:] + t[:-1]) / 2) + 8 * (x < 0)
    idx = idx.reshape(N, K).to(torch.uint8)
    codes = idx[:, 0::2] | (idx[:, 1::2] << 4)
    return codes.contiguous(), scales.contiguous(), second


def _offsets(c, seed):
    """Row offsets of the experts: cut points drawn from the seed, one expert
    without rows."""
    E, M = c["E"], c["M"]
    g = torch.Generator().manual_seed(seed * 7 + 3)
    cuts = torch.randint(0, M + 1, (E - 1,), generator=g).sort().values.tolist()
    offs = [0] + cuts + [M]
    if E > 2:
        offs[1] = offs[2]
        offs[1:] = sorted(offs[1:])
    return offs


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] in ("norm", "norm_bwd"):
        M, D = c["M"], c["D"]
        # a residual stream grows over the layers, and a few channels carry large values
        chan = torch.where(torch.rand(D, generator=g, device=DEV) < 0.01, 20.0, 1.0)
        s["X"] = (torch.randn((M, D), generator=g, device=DEV) * chan).to(BF)
        s["w"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)).to(BF)
        if c["op"] == "norm":
            s["R"] = _normal(g, (M, D), 2.0) if c["residual"] else None
        else:
            s["dY"] = _normal(g, (M, D), 0.02)
            s["dH"] = _normal(g, (M, D), 0.02) if c["dh"] else None
        return s
    M, K, N, r, E = c["M"], c["K"], c["N"], c["r"], c["E"]
    P = 2 if c["op"].startswith("gated") else 1
    packs = [_quantize(_normal(g, (N, K), 0.02), c["fmt"]) for _ in range(E * P)]
    s["codes"] = torch.stack([p[0] for p in packs])
    s["scales"] = torch.stack([p[1] for p in packs])
    s["second"] = torch.stack([p[2] for p in packs]) if c["fmt"] == "nf4_dq" else None
    s["X"] = _normal(g, (M, K))
    s["A"] = ((torch.rand((E * P, r, K), generator=g, device=DEV) * 2 - 1) / math.sqrt(K)).to(BF)
    s["B"] = _normal(g, (E * P, N, r), 0.01)
    s["s"] = 2.0
    s["offs"] = _offsets(c, seed) if E > 1 else [0, M]
    s["offsets"] = torch.tensor(s["offs"], dtype=torch.int64, device=DEV) if E > 1 else None
    std = 0.02 * math.sqrt(K)   # of a projection's outputs
    if c.get("bias"):
        s["bias"] = _normal(g, (E, N), 0.1)
    if c["op"] == "linear" and c["residual"]:
        s["R"] = _normal(g, (M, N), 2.0)
    if c["op"] in ("gated_bwd", "linear_bwd"):
        s["dY"] = _normal(g, (M, N), 0.02)
        if P == 2 or c["act"] != "none":
            s["pre"] = _normal(g, (M, P * N), std)
        s["Z"] = _normal(g, (M, P * r), 1 / math.sqrt(3.0))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import lora_fine_tuning_amd as L
        s["L"] = L
        if case["op"] == "norm_bwd":
            s["ws"] = L.rmsnorm_workspace(case["M"], case["D"], s["X"].device)
        elif case["op"] != "norm":
            # the base as a program keeps it: in the library's tiled storage
            s["base"] = L.import_rowmajor(case["fmt"], s.pop("codes"), s.pop("scales"), s.pop("second"))
            which = 1 if case["op"].endswith("_bwd") else 0
            size = L.gated_workspace if case["op"].startswith("gated") else L.epilogue_workspace
            s["ws"] = size(which, s["base"], case["M"], case["r"])
            if case["E"] == 1 and case["op"].startswith("linear"):
                s["A"], s["B"] = s["A"][0], s["B"][0]
                s["bias"] = s["bias"][0] if "bias" in s else None
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    return {"norm": _norm, "norm_bwd": _norm_bwd, "gated": _gated, "gated_bwd": _gated_bwd, "linear": _linear,
            "linear_bwd": _linear_bwd}[c["op"]](s, c)


def _some(d):
    return {k: v for k, v in d.items() if v is not None}


def _run_own(s, c):
    L, op = s["L"], c["op"]
    if op == "norm":
        o = L.rmsnorm(s["X"], s["w"], EPS, residual=s["R"], mx=c["mx"])
        if c["mx"]:
            o["codes"] = o["codes"].view(torch.float8_e4m3fn)
            o["scales"] = o["scales"].view(torch.float8_e8m0fnu)
        return _some(o)
    if op == "norm_bwd":
        return _some(L.rmsnorm_backward(s["dY"], s["X"], s["w"], EPS, dH=s["dH"], want_dw=c["dw"], workspace=s["ws"]))
    kw = dict(activation=c["act"], group_offsets=s["offsets"], workspace=s["ws"])
    if op == "gated":
        return _some(L.gated_forward(s["base"], s["X"], s["A"], s["B"], s["s"], want_saved=c["save"], **kw))
    if op == "gated_bwd":
        return _some(L.gated_backward(s["base"], s["X"], s["dY"], s["pre"], s["A"], s["B"], s["s"], Z=s["Z"], **kw))
    if op == "linear":
        return _some(L.forward_epilogue(s["base"], s["X"], s["A"], s["B"], s["s"], bias=s.get("bias"),
                                        residual=s.get("R"), want_saved=c["save"], **kw))
    return _some(L.backward_epilogue(s["base"], s["X"], s["dY"], s["A"], s["B"], s["s"], P=s.get("pre"), Z=s["Z"],
                                     want_dbias=c["bias"], **kw))


# ---- plain forms -----------------------------------------------------------

def _norm(s, c):
    h = s["X"].float()
    out = {}
    if s["R"] is not None:
        h = h + s["R"].float()
        out["H"] = h.to(BF)
    y = (h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()).to(BF)
    out["Y"] = y
    if c["mx"]:
        # per 32 elements the power of two that brings the largest under 448,
        # the elements in E4M3; of the bf16 output, which the adapter reads too
        b = y.float().reshape(c["M"], -1, 32)
        amax = b.abs().amax(-1)
        e = torch.where(amax > 0, (torch.frexp(amax).exponent - 1 - 8).clamp(-127, 127), -127)
        q = torch.ldexp(b, -e[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        out["codes"] = q.reshape(c["M"], -1)
        out["scales"] = (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    return out


def _norm_bwd(s, c):
    h, dy, w = s["X"].float(), s["dY"].float(), s["w"].float()
    rstd = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
    n = h * rstd
    t = dy * w
    dx = rstd * (t - n * (t * n).mean(-1, keepdim=True))
    if s["dH"] is not None:
        dx = dx + s["dH"].float()
    out = {"dX": dx.to(BF)}
    if c["dw"]:
        out["dW"] = (dy * n).sum(0).to(BF)
    return out


def _deq(s, c, g):
    """deq(W) [N, K] of projection g, as float32 values of its bf16 elements."""
    codes, sc = s["codes"][g], s["scales"][g]
    blk = BLOCK[c["fmt"]]
    idx = torch.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1).int()
    if c["fmt"] in ("nf4", "nf4_dq"):
        lv = torch.tensor(_nf4_levels(), device=codes.device, dtype=torch.float32)
        if c["fmt"] == "nf4_dq":
            f = sc.view(torch.float8_e4m3fn).float()
            sc = f * s["second"][g].repeat_interleave(256)[:f.numel()].reshape(f.shape)
    else:
        t = torch.tensor(E2M1, device=codes.device)
        lv = torch.cat([t, -t])
        sc = torch.exp2(sc.float() - 127) if c["fmt"] == "mxfp4" else sc.view(torch.float8_e4m3fn).float()
    w = lv[idx].reshape(idx.shape[0], -1, blk) * sc[..., None]
    return w.to(BF).float().reshape(idx.shape)


def _act(x, name):
    if name == "none":
        return x
    if name == "silu":
        return x * torch.sigmoid(x)
    if name == "gelu":
        return 0.5 * x * (1 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _act_grad(x, name):
    if name == "none":
        return torch.ones_like(x)
    if name == "silu":
        p = torch.sigmoid(x)
        return p * (1 + x * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    t = torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * x * x)


def _project(s, c, x, g):
    """x deq(W)^T + s (x A^T) B^T of projection g, and x A^T."""
    z = x @ s["A"][g].float().t()
    return x @ _deq(s, c, g).t() + s["s"] * (z @ s["B"][g].float().t()), z


def _gated(s, c):
    parts = []
    for e in range(c["E"]):   # experts are separate layers
        x = s["X"][s["offs"][e]:s["offs"][e + 1]].float()
        if x.shape[0] == 0:
            continue
        gate, zg = _project(s, c, x, 2 * e)
        up, zu = _project(s, c, x, 2 * e + 1)
        h = (_act(gate, c["act"]) * up).to(BF)
        parts.append((h, torch.cat([gate, up], 1).to(BF), torch.cat([zg, zu], 1).to(BF)) if c["save"] else (h,))
    return dict(zip(("H", "GU", "Z"), (torch.cat(t) for t in zip(*parts))))


def _grads(s, c, g, x, d, z):
    """dX, dA and dB of projection g for the upstream gradient d of its outputs."""
    A, B = s["A"][g].float(), s["B"][g].float()
    dz = s["s"] * (d @ B)
    return d @ _deq(s, c, g) + dz @ A, dz.t() @ x, s["s"] * (d.t() @ z)


def _gated_bwd(s, c):
    N, r = c["N"], c["r"]
    dX, dA, dB = [], [], []
    for e in range(c["E"]):
        rows = slice(s["offs"][e], s["offs"][e + 1])
        x, dh, z = s["X"][rows].float(), s["dY"][rows].float(), s["Z"][rows].float()
        gate, up = s["pre"][rows, :N].float(), s["pre"][rows, N:].float()
        xg, ag, bg = _grads(s, c, 2 * e, x, dh * up * _act_grad(gate, c["act"]), z[:, :r])
        xu, au, bu = _grads(s, c, 2 * e + 1, x, dh * _act(gate, c["act"]), z[:, r:])
        dX.append(xg + xu)
        dA += [ag, au]
        dB += [bg, bu]
    return {"dX": torch.cat(dX).to(BF), "dA": torch.stack(dA).to(BF), "dB": torch.stack(dB).to(BF)}


def _linear(s, c):
    parts = []
    for e in range(c["E"]):
        rows = slice(s["offs"][e], s["offs"][e + 1])
        x = s["X"][rows].float()
        if x.shape[0] == 0:
            continue
        p, z = _project(s, c, x, e)
        if c["bias"]:
            p = p + s["bias"][e].float()
        y = _act(p, c["act"])
        if c["residual"]:
            y = y + s["R"][rows].float()
        parts.append((y.to(BF), p.to(BF), z.to(BF)) if c["save"] else (y.to(BF),))
    return dict(zip(("Y", "P", "Z"), (torch.cat(t) for t in zip(*parts))))


def _linear_bwd(s, c):
    dX, dA, dB, db = [], [], [], []
    for e in range(c["E"]):
        rows = slice(s["offs"][e], s["offs"][e + 1])
        d = s["dY"][rows].float()
        if c["act"] != "none":
            d = d * _act_grad(s["pre"][rows].float(), c["act"])
        x, a, b = _grads(s, c, e, s["X"][rows].float(), d, s["Z"][rows].float())
        dX.append(x)
        dA.append(a)
        dB.append(b)
        db.append(d.sum(0))
    one = (lambda t: t[0]) if c["E"] == 1 else torch.stack
    out = {"dX": torch.cat(dX).to(BF), "dA": one(dA).to(BF), "dB": one(dB).to(BF)}
    if c["bias"]:
        out["dbias"] = one(db).to(BF)
    return out


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def _w64(s, c, g):
    """The dequantized base, element for element as the formats define it: the
    fp32 product of level and scale rounded to bf16 (NF4), the exact product
    rounded to bf16 (MXFP4, NVFP4)."""
    packed = s["codes"][g]
    n, half = packed.shape
    nib = torch.empty((n, 2 * half), dtype=torch.uint8, device=packed.device)
    nib[:, ::2] = packed % 16
    nib[:, 1::2] = torch.div(packed, 16, rounding_mode="floor")
    blk = BLOCK[c["fmt"]]
    sc = s["scales"][g]
    if c["fmt"].startswith("nf4"):
        table = torch.tensor(_nf4_levels(), dtype=torch.float64, device=packed.device).to(torch.float32).double()
        if c["fmt"] == "nf4_dq":
            first = _e4m3_value(sc).reshape(-1)
            at = torch.arange(first.numel(), device=packed.device) // 256
            sc = (first * s["second"][g].double()[at]).to(torch.float32).reshape(n, -1)
        scale = sc.double()
    else:
        mag = torch.tensor(E2M1, dtype=torch.float64, device=packed.device)
        table = torch.cat((mag, mag.neg()))
        scale = 2.0 ** (sc.double() - 127) if c["fmt"] == "mxfp4" else _e4m3_value(sc)
    v = torch.take(table, nib.long()) * scale.repeat_interleave(blk, 1)
    return v.to(torch.float32).to(BF).double()


def _e4m3_value(code):
    c = code.long()
    m, e = (c & 7).double(), (c >> 3) & 15
    v = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e.double() - 7))
    return torch.where(c >= 128, -v, v)


def _value_and_slope(x, name):
    """The activation and its derivative at x."""
    if name == "none":
        return x, torch.ones_like(x)
    if name == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p + x * p * (1 - p)
    if name == "gelu":
        cdf = 0.5 * torch.special.erfc(-x / 2 ** 0.5)
        return x * cdf, cdf + x * torch.exp(-x ** 2 / 2) / (2 * math.pi) ** 0.5
    k = (2 / math.pi) ** 0.5
    p = 1 / (1 + torch.exp(-2 * k * (x + 0.044715 * x ** 3)))   # (1 + tanh u) / 2 = sigmoid(2 u)
    return x * p, p + x * 2 * p * (1 - p) * k * (1 + 0.134145 * x ** 2)


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"].startswith("norm"):
        return _exact_norm(s, c)
    P = 2 if c["op"].startswith("gated") else 1
    M, N, r, E = c["M"], c["N"], c["r"], c["E"]
    f = dict(dtype=torch.float64, device=DEV)
    X, A, B = s["X"].double(), s["A"].double(), s["B"].double()
    if c["op"] in ("gated", "linear"):
        pre, Z = torch.empty((M, P * N), **f), torch.empty((M, P * r), **f)
        for g in range(E * P):
            lo, hi, j = s["offs"][g // P], s["offs"][g // P + 1], g % P
            if lo == hi:
                continue
            Z[lo:hi, j * r:(j + 1) * r] = X[lo:hi].matmul(A[g].T)
            pre[lo:hi, j * N:(j + 1) * N] = X[lo:hi].matmul((_w64(s, c, g) + s["s"] * B[g].matmul(A[g])).T)
            if c.get("bias"):
                pre[lo:hi] += s["bias"][g].double()
        val = _value_and_slope(pre[:, :N], c["act"])[0]
        if P == 2:
            return {"H": val * pre[:, N:], **({"GU": pre, "Z": Z} if c["save"] else {})}
        if c["residual"]:
            val = val + s["R"].double()
        return {"Y": val, **({"P": pre, "Z": Z} if c["save"] else {})}
    d = s["dY"].double()
    if P == 2:
        val, slope = _value_and_slope(s["pre"][:, :N].double(), c["act"])
        D = torch.cat([d * s["pre"][:, N:].double() * slope, d * val], 1)
    else:
        D = d if c["act"] == "none" else d * _value_and_slope(s["pre"].double(), c["act"])[1]
    dX = torch.zeros((M, c["K"]), **f)
    dA, dB, db = torch.zeros_like(A), torch.zeros_like(B), torch.zeros((E, N), **f)
    Z = s["Z"].double()
    for g in range(E * P):
        lo, hi, j = s["offs"][g // P], s["offs"][g // P + 1], g % P
        Dg = D[lo:hi, j * N:(j + 1) * N]
        dX[lo:hi] += Dg.matmul(_w64(s, c, g) + s["s"] * B[g].matmul(A[g]))
        dA[g] = s["s"] * B[g].T.matmul(Dg.T.matmul(X[lo:hi]))
        dB[g] = s["s"] * Dg.T.matmul(Z[lo:hi, j * r:(j + 1) * r])
        if c.get("bias"):
            db[g] = Dg.sum(0)
    if P == 1 and E == 1:
        dA, dB, db = dA[0], dB[0], db[0]
    return {"dX": dX, "dA": dA, "dB": dB, **({"dbias": db} if c.get("bias") else {})}


def _exact_norm(s, c):
    h, w = s["X"].double(), s["w"].double()
    if c["op"] == "norm":
        out = {}
        if s["R"] is not None:
            h = h + s["R"].double()
            out["H"] = h
        y = h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS) * w
        out["Y"] = y
        if c["mx"]:
            b = y.to(BF).double().reshape(c["M"], -1, 32)
            top = b.abs().amax(2, keepdim=True)
            e = torch.where(top > 0, torch.floor(torch.log2(top)) - 8, -127.0).clamp(-127, 127)
            v = b / 2.0 ** e
            # the E4M3 grid: eight steps to each power of two, down to 2^-9
            step = 2.0 ** (torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            out["codes"] = (torch.round(v / step) * step).clamp(-448, 448).reshape(c["M"], -1)
            out["scales"] = (2.0 ** e).squeeze(2)
        return out
    dy = s["dY"].double()
    inv = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    dx = inv * dy * w - h * inv ** 3 * (dy * w * h).mean(1, keepdim=True)
    out = {"dX": dx + s["dH"].double() if s["dH"] is not None else dx}
    if c["dw"]:
        out["dW"] = (dy * h * inv).sum(0)
    return out
