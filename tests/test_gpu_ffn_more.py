"""GPU tests of the feed-forward operators where test_gpu_ffn.py does not reach:
every activation on the library's own backward over experts and on each forward
schedule, experts by the hundred, more rows than the norm's grid, offsets past 32
bits, the smallest sizes, two calls at once. The bounds are those of
test_gpu_ffn.py."""

import sys

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
import synth
import test_gpu_ffn
from gpu_util import compare_full, element_bound, f64, guarded, print_case, to_dev, to_host
from oracle import ffn
from test_gpu_ffn import (FMTS, POLICIES, Case, abs_mm, check_epilogue, check_gated, normal, run_epilogue, run_gated)

pytestmark = pytest.mark.gpu

EXPERTS = [[0, 0, 37, 100], [0, 150, 150, 460]]
# 90 experts, nine with rows; 200 with 0 to 9 rows each
MANY = [0] * 20 + list(range(0, 9)) + [8] * 62 + [11]
CROWD = np.concatenate([[0], np.cumsum(np.random.default_rng(1).integers(0, 10, 200))]).tolist()


def run_backward(c, act, with_z=True):
    """One backward of c (gated with two projections) on seeded saved tensors,
    every output and the workspace between guard bands, against the oracle."""
    rng = np.random.default_rng(9)
    pre, Zs = normal(rng, (c.M, c.P * c.N)), normal(rng, (c.M, c.P * c.r))
    X, A, B, dY = c.dev("X", "A", "B", "dY")
    out, checks = {}, []
    names = [("dX", (c.M, c.K)), ("dA", tuple(A.shape)), ("dB", tuple(B.shape))]
    if c.P == 1:
        names.append(("dbias", (c.N,) if c.E == 1 else (c.E, c.N)))
    for name, shp in names:
        out[name], chk = guarded(shp)
        checks.append((name, chk))
    size = L.lora4_gated_workspace_bytes if c.P == 2 else L.lora4_epilogue_workspace_bytes
    ws, chk = guarded((size(1, c.base.abi(), c.M, c.r),), torch.uint8)
    checks.append(("workspace", chk))
    kw = dict(activation=act, Z=to_dev(Zs) if with_z else None, group_offsets=c.offsets, workspace=ws, out=out)
    if c.P == 2:
        o = L.gated_backward(c.base, X, dY, to_dev(pre), A, B, c.s, **kw)
    else:
        o = L.backward_epilogue(c.base, X, dY, A, B, c.s, P=to_dev(pre), **kw)
    torch.cuda.synchronize()
    for name, chk in checks:
        chk(name)
    check_backward(c, act, o, pre, Zs if with_z else None)


def check_backward(c, act, o, pre, Zs):
    """o, the outputs of a backward of c at the saved bf16 bits pre and Zs (None:
    recomputed), against the oracle."""
    dX, IX = np.zeros((c.M, c.K)), np.zeros((c.M, c.K))
    dA, dB, IA, IB = [np.zeros(t.shape) for t in (c.A, c.B, c.A, c.B)]
    db, idb = np.zeros((c.E, c.N)), np.zeros((c.E, c.N))
    k = 0 if c.P == 1 and act == "none" else 1   # the gradient before the activation is rounded
    for e, sl in c.rows():
        x, g = f64(c.X[sl]), f64(pre[sl, :c.N])
        v, d = ffn.act(g, act)
        up = f64(c.dY[sl])
        grads = [up * f64(pre[sl, c.N:]) * d, up * v] if c.P == 2 else [up * d]
        for j, gr in enumerate(grads):
            i = e * c.P + j
            Ai, Bi = f64(c.A[i]), f64(c.B[i])
            z = x @ Ai.T if Zs is None else f64(Zs[sl, j * c.r:(j + 1) * c.r])
            dz = c.s * gr @ Bi
            dX[sl] += gr @ c.Wd[i] + dz @ Ai
            dA[i], dB[i] = dz.T @ x, c.s * gr.T @ z
            # the roundings on the way: of the gradient where it is an operand,
            # of dZ (made from the unrounded gradient), of a recomputed Z
            IX[sl] += k * abs_mm(gr, c.Wd[i]) + np.abs(dz) @ np.abs(Ai)
            IA[i] = np.abs(dz).T @ np.abs(x)
            IB[i] = c.s * abs_mm(gr.T, z) * (k + (1 if Zs is None else 0))
        if c.P == 1:
            db[e], idb[e] = grads[0].sum(0), 2.0 ** -13 * np.abs(grads[0]).sum(0)
    h = {n: f64(to_host(t)) for n, t in o.items() if t is not None}
    compare_full("dX", h["dX"], dX, IX)
    compare_full("dA", h["dA"].reshape(dA.shape), dA, IA)
    compare_full("dB", h["dB"].reshape(dB.shape), dB, IB)
    if c.P == 1:
        compare_full("dbias", h["dbias"].reshape(db.shape), db, idb)
    for e, sl in c.rows():                       # an expert with no rows: zeros
        if sl.start == sl.stop:
            for n in ("dA", "dB"):
                assert not h[n].reshape(dA.shape if n == "dA" else dB.shape)[e * c.P:(e + 1) * c.P].any()
            assert c.P == 2 or not h["dbias"].reshape(db.shape)[e].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("act", ffn.ACTIVATIONS)
@pytest.mark.parametrize("offsets", EXPERTS)
@pytest.mark.parametrize("P", [1, 2])
def test_experts_backward(fmt, act, offsets, P):
    print_case("experts bwd", fmt, act, offsets, P)
    run_backward(Case(offsets[-1], 256, 130, 8, fmt, P, offsets, seed=10), act, with_z=act != "silu")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offsets", [MANY, CROWD])
@pytest.mark.parametrize("P", [1, 2])
def test_many_experts_backward(fmt, offsets, P):
    print_case("many experts bwd", fmt, len(offsets) - 1, P)
    run_backward(Case(offsets[-1], 128, 70, 4, fmt, P, offsets, seed=11), "gelu")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("offsets", [MANY, CROWD])
@pytest.mark.parametrize("policy", ["", "8", "1064", "1256", "2032", "2128"])
def test_many_experts_forward(fmt, offsets, policy, monkeypatch):
    print_case("many experts", fmt, len(offsets) - 1, policy)
    monkeypatch.setenv("LORA4_FFN_ROWS", policy)
    c = Case(offsets[-1], 128, 70, 4, fmt, 2, offsets, seed=12)
    check_gated(c, "gelu_tanh", run_gated(c, "gelu_tanh"))
    c = Case(offsets[-1], 128, 70, 4, fmt, 1, offsets, seed=13)
    check_epilogue(c, "silu", True, True, run_epilogue(c, "silu", True, True))


@pytest.mark.parametrize("act", ffn.ACTIVATIONS)
@pytest.mark.parametrize("policy", POLICIES)
def test_every_activation_on_every_schedule(act, policy, monkeypatch):
    print_case("activation", act, policy)
    monkeypatch.setenv("LORA4_FFN_ROWS", policy)
    c = Case(70, 320, 200, 12, synth.NF4_DQ, 2, seed=14)
    check_gated(c, act, run_gated(c, act))
    c = Case(70, 320, 200, 12, synth.NVFP4, 1, seed=15)
    check_epilogue(c, act, True, True, run_epilogue(c, act, True, True))


def compare_elements(name, got, ref, inter=None):
    g = f64(got) if got.dtype == np.uint16 else got
    assert g.shape == ref.shape and np.all(np.isfinite(g)), name
    err, bound = np.abs(g - ref), element_bound(ref, inter)
    assert np.all(err <= bound), (name, float(np.max(err / np.maximum(bound, 1e-300))))


SMALL = [(1, 64, 1, 1), (2, 64, 2, 256), (1, 128, 65, 255), (9, 64, 63, 2), (33, 64, 7, 5), (17, 128, 1, 128)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("shape", SMALL + [(5, 32, 3, 2), (33, 96, 1, 7)])
@pytest.mark.parametrize("experts", [False, True])
def test_smallest_sizes(fmt, shape, experts, monkeypatch):
    # (outputs of a few elements: the bound of each, but no norm over them,
    # which one rounding can move by 2^-8)
    for module in (sys.modules[__name__], test_gpu_ffn):
        monkeypatch.setattr(module, "compare_full", compare_elements)
    M, K, N, r = shape
    if K % 64 and fmt in (synth.NF4, synth.NF4_DQ):
        K = 64
    print_case("smallest", fmt, M, K, N, r, experts)
    offsets = [0, 0, M - M // 2, M] if experts else None
    c = Case(M, K, N, r, fmt, 1, offsets, seed=16)
    check_epilogue(c, "gelu", True, True, run_epilogue(c, "gelu", True, True))
    run_backward(c, "gelu")
    run_backward(c, "none", with_z=False)
    c = Case(M, K, N, min(r, 128), fmt, 2, offsets, seed=17)
    check_gated(c, "silu", run_gated(c, "silu"))
    run_backward(c, "silu", with_z=False)


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

# more rows than the grid holds (65536 blocks of four rows, or of one row)
@pytest.mark.parametrize("M,D", [(262144 + 5, 8), (262144 + 5, 9), (65536 + 3, 1032), (65536 + 3, 1027)])
def test_norm_beyond_its_grid(M, D):
    print_case("norm grid", M, D)
    rng = np.random.default_rng(D)
    X, w, R, dY = normal(rng, (M, D)), normal(rng, (D,)), normal(rng, (M, D)), normal(rng, (M, D))
    x, wd, r, dy = (to_dev(t) for t in (X, w, R, dY))
    o = L.rmsnorm(x, wd, 1e-5, residual=r)
    frozen = L.rmsnorm_backward(dy, x, wd, 1e-5, dH=r, want_dw=False)["dX"]
    g = L.rmsnorm_backward(dy, x, wd, 1e-5, dH=r)
    torch.cuda.synchronize()
    assert torch.equal(frozen, g["dX"])
    dW, rows = np.zeros(D), 1 << 14
    for a in range(0, M, rows):
        sl = slice(a, min(M, a + rows))
        ref = ffn.rmsnorm(f64(X[sl]), f64(w), 1e-5, f64(R[sl]))
        compare_full("Y", to_host(o["Y"][sl]), ref["Y"])
        compare_full("H", to_host(o["H"][sl]), ref["H"])
        ref = ffn.rmsnorm_backward(f64(dY[sl]), f64(X[sl]), f64(w), 1e-5, f64(R[sl]))
        compare_full("dX", to_host(frozen[sl]), ref["dX"])
        dW += ref["dW"]
    compare_full("dW", to_host(g["dW"]), dW)


def test_norm_codes_of_special_rows():
    """Rows with infinities, NaNs, zeros and the type's ends give the codes that
    packing the bf16 output gives."""
    D = 256
    X = normal(np.random.default_rng(2), (8, D))
    for row, bits in ((0, 0x7F80), (1, 0xFF80), (2, 0x7FC0), (3, 0x0001), (4, 0x0080)):
        X[row, ::3] = bits
    X[5], X[6, 32:] = 0, 0
    w = normal(np.random.default_rng(3), (D,))
    w[:4] = [0x7F7F, 0xFF7F, 0x0001, 0x7F80]
    o = L.rmsnorm(to_dev(X), to_dev(w), 1e-6, mx=True)
    codes, scales = L.mxfp8(o["Y"])
    assert torch.equal(codes, o["codes"]) and torch.equal(scales, o["scales"])


# ---------------------------------------------------------------------------
# Offsets past 32 bits, two calls at once
# ---------------------------------------------------------------------------

def test_outputs_past_32_bit_offsets():
    """Outputs of more than 2^31 elements: the last rows are those of a call on
    the last rows alone."""
    M, K, N, r, tail = (1 << 18) + 70, 64, 8256, 8, 326
    c = Case(tail, K, N, r, synth.MXFP4, 1, seed=18)
    X, A, B, bias, R = c.dev("X", "A", "B", "bias", "R")
    Xl = torch.zeros((M, K), dtype=X.dtype, device=X.device)
    Xl[-tail:] = X
    Rl = torch.zeros((M, N), dtype=X.dtype, device=X.device)
    Rl[-tail:] = R
    assert Rl.numel() > 1 << 31
    o = L.forward_epilogue(c.base, Xl, A, B, c.s, bias=bias, activation="gelu", residual=Rl, out={"Y": Rl})
    last = {k: v[-tail:].contiguous() for k, v in o.items()}
    check_epilogue(c, "gelu", True, True, last)
    head = L.forward_epilogue(c.base, Xl[:tail], A, B, c.s, bias=bias, activation="gelu")
    assert torch.equal(o["Y"][:tail], head["Y"])        # (rows of zeros: act(bias))
    del head
    # backward: rows of zero gradient around the last ones add nothing to the sums
    dY = torch.zeros((M, N), dtype=X.dtype, device=X.device)
    dY[-tail:] = to_dev(c.dY)
    got = L.backward_epilogue(c.base, Xl, dY, A, B, c.s, P=o["P"], activation="gelu", Z=o["Z"], want_dbias=True)
    assert not got["dX"][:-tail].any()
    check_backward(c, "gelu", {**got, "dX": got["dX"][-tail:]}, to_host(last["P"]), to_host(last["Z"]))


def test_two_calls_at_once():
    """Calls on two streams, each with its own workspace, give the bits of one after the other."""
    c = [Case(300, 512, 640, 16, fmt, 2, seed=19 + i) for i, fmt in enumerate((synth.NF4, synth.MXFP4))]
    args = [x.dev("X", "A", "B", "dY") for x in c]

    def step(i):
        X, A, B, dY = args[i]
        f = L.gated_forward(c[i].base, X, A, B, c[i].s)
        b = L.gated_backward(c[i].base, X, dY, f["GU"], A, B, c[i].s, Z=f["Z"])
        return [f["H"], f["GU"], f["Z"], b["dX"], b["dA"], b["dB"]]

    want = [step(0), step(1)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(step(i))
    torch.cuda.synchronize()
    for i in (0, 1):
        for outs in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(outs, want[i]))


@pytest.mark.parametrize("double_quant", [False, True])
def test_joint_base_past_32_bit_offsets(double_quant):
    """Projections whose bases together pass 2 GiB of codes: dX of the gated backward is the
    sum of the plain layer's over each base."""
    M, K, N, r = 8, 8192, 262272, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s, std=1.0: (torch.randn(s, generator=g, device="cuda") * std).to(torch.bfloat16)
    base = L.pack_nf4(rand(2, N, K, std=0.05), double_quant=double_quant)
    assert base.codes.numel() > 1 << 31
    X, A, B, dH, GU = rand(M, K), rand(2, r, K, std=K ** -0.5), rand(2, N, r, std=0.01), rand(M, N), rand(M, 2 * N)
    Z = rand(M, 2 * r)
    o = L.gated_backward(base, X, dH, GU, A, B, 1.0, activation="none", Z=Z)
    grads = [(dH.float() * GU[:, (1 - j) * N:(2 - j) * N].float()).to(torch.bfloat16) for j in (0, 1)]
    dX, inter = np.zeros((M, K)), np.zeros((M, K))
    for j, d in enumerate(grads):
        one = L.PackedBase(base.fmt, N, K, 1, base.codes[j], base.scales[j],
                           base.scales2[j] if double_quant else None)
        b = L.backward(one, X, d, A[j], B[j], 1.0, Z=Z[:, j * r:(j + 1) * r].contiguous())
        h = f64(to_host(b["dX"]))
        dX += h
        # the plain results' own rounding, and dZ: there of the rounded gradient (off by
        # at most 2^-8 of each term), and rounded itself on both sides
        dz = d.double().abs() @ B[j].double().abs() + 2 * (d.double() @ B[j].double()).abs()
        inter += np.abs(h) + (dz @ A[j].double().abs()).cpu().numpy()
        compare_full("dB", f64(to_host(o["dB"][j])), f64(to_host(b["dB"])), np.abs(f64(to_host(b["dB"]))))
    compare_full("dX", f64(to_host(o["dX"])), dX, inter)
