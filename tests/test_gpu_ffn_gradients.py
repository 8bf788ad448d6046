"""GPU tests of the feed-forward gradients where their rounding matters: dZ (the
rank-r product of the gradient before the activation) is made from the unrounded
gradient, so it holds where bf16 loses the gradient. What is compared is dA =
dZ^T X, through which dZ leaves the library."""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import compare_full, f64, print_case, to_dev, to_host
from oracle import ffn
from test_gpu_ffn import Case, normal

pytestmark = pytest.mark.gpu

BF16_MAX = float(torch.finfo(torch.bfloat16).max)


def bf16(v):
    return synth.to_bf16(np.asarray(v, np.float32))


@pytest.mark.parametrize("M,E", [(3, 1), (70, 1), (9, 3)])
@pytest.mark.parametrize("P", [1, 2])
def test_gradient_past_bf16(M, E, P):
    """A gradient before the activation that fp32 holds and bf16 rounds to
    infinity: dZ is still the finite sum, and dA of it finite and right."""
    print_case("past bf16", M, E, P)
    c = Case(M, 256, 96, 8, synth.NF4, P, None if E == 1 else [0, 2, 2, M], seed=8)
    c.s = 0.25
    c.X = bf16(f64(c.X) * 0.25)
    X, A, B, dY = c.dev("X", "A", "B", "dY")
    rng = np.random.default_rng(3)
    pre, Z = f64(normal(rng, (M, P * c.N))), to_dev(normal(rng, (M, P * c.r)))
    up = f64(c.dY)
    if P == 2:     # dG = dH U (no activation): 181^2 2^-14 2^127, between bf16's largest and fp32's
        act = "none"
        up[1, 5], pre[1, c.N + 5] = 181 * 2.0 ** 56, 181 * 2.0 ** 57
        a = up[1, 5] * pre[1, c.N + 5]
    else:          # dP = dY silu'(8), silu'(8) = 1.00235
        act = "silu"
        up[1, 5], pre[1, 5] = -BF16_MAX, 8.0
        a = up[1, 5] * ffn.act(8.0, "silu")[1]
    assert BF16_MAX * (1 + 2.0 ** -9) < abs(a) < np.finfo(np.float32).max
    assert np.array_equal(f64(bf16(up)), up) and np.array_equal(f64(bf16(pre)), pre)
    up_d, pre_d = to_dev(bf16(up)), to_dev(bf16(pre))
    if P == 2:
        o = L.gated_backward(c.base, X, up_d, pre_d, A, B, c.s, activation=act, Z=Z, group_offsets=c.offsets)
    else:
        o = L.backward_epilogue(c.base, X, up_d, A, B, c.s, P=pre_d, activation=act, Z=Z, group_offsets=c.offsets)
    dA = f64(to_host(o["dA"])).reshape(c.A.shape)
    for e, sl in c.rows():
        x = f64(c.X[sl])
        v, d = ffn.act(pre[sl, :c.N], act)
        grads = [up[sl] * pre[sl, c.N:] * d, up[sl] * v] if P == 2 else [up[sl] * d]
        for j, g in enumerate(grads):
            dz = c.s * g @ f64(c.B[e * P + j])
            assert np.abs(dz).max(initial=0) < c.s * BF16_MAX     # (the sum before the scale is finite too)
            # dZ's own rounding is the one that dA carries in
            compare_full("dA", dA[e * P + j], dz.T @ x, np.abs(dz).T @ np.abs(x))


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_gradient(value):
    """An infinite gradient reaches dA as the infinities of its signs, a NaN as NaNs."""
    print_case("infinite", value)
    c = Case(5, 256, 96, 8, synth.NF4, 1, seed=9)
    X, A, B, dY = c.dev("X", "A", "B", "dY")
    pre, Z = torch.full((5, c.N), 2.0, device=X.device, dtype=torch.bfloat16), to_dev(c.R[:, :c.r])
    dY[1, 5] = value
    dA = L.backward_epilogue(c.base, X, dY, A, B, c.s, P=pre, activation="silu", Z=Z)["dA"].float()
    sign = B[5].float()[:, None] * X[1].float()[None, :]
    assert (sign != 0).all()
    assert torch.equal(dA.isnan(), (sign * value).isnan())
    if value == value:
        assert torch.equal(dA, torch.sign(sign) * value)


@pytest.mark.parametrize("pairs", [1, 20, 48])
def test_dz_keeps_what_bf16_drops(pairs):
    """Gradients that round to the same bf16 value and meet B's rows +1 and -1: the
    rounded parts cancel and dZ is what the rounding dropped. Gated, without an
    activation: dG = dH U is 129^2 2^-14 = 1 + 2^-6 + 2^-14 against 130 2^-7 =
    1 + 2^-6, both exact in fp32 and both 1 + 2^-6 in bf16."""
    print_case("dropped", pairs)
    N, K, r = 96, 128, 8
    c = Case(1, K, N, r, synth.NF4, 2, seed=10)
    dH, U, B = np.zeros((1, N)), np.zeros((1, N)), np.zeros((2, N, r))
    for i in range(pairs):
        dH[0, 2 * i:2 * i + 2] = 129 / 128, 130 / 128
        U[0, 2 * i:2 * i + 2] = 129 / 128, 1.0
        B[0, 2 * i], B[0, 2 * i + 1] = 1.0, -1.0
    X, A, _, _ = c.dev("X", "A", "B", "dY")
    GU, Z = np.concatenate([np.zeros((1, N)), U], 1), np.zeros((1, 2 * r))
    o = L.gated_backward(c.base, X, to_dev(bf16(dH)), to_dev(bf16(GU)), A, to_dev(bf16(B)), 1.0, activation="none",
                         Z=to_dev(bf16(Z)))
    # every product and sum is exact; dA = dZ^T X is rounded once
    want = pairs * 2.0 ** -14 * f64(c.X)[0]
    got = f64(to_host(o["dA"]))
    assert np.array_equal(got[0], np.broadcast_to(f64(bf16(want)), (r, K)))
    assert not got[1].any()


def test_dz_keeps_what_bf16_drops_behind_an_activation():
    """The same for one projection: two slopes of SiLU that differ and round alike."""
    N, K, r = 96, 128, 8
    c = Case(1, K, N, r, synth.NF4, 1, seed=11)
    p = f64(np.arange(0x4000, 0x4080, dtype=np.uint16))          # bf16 values of 2 to 4
    d = ffn.act(p, "silu")[1]
    q = f64(bf16(d))
    # (in [1, 1.1]; far from the middle between two bf16 values, which fp32 could round otherwise)
    safe = np.abs(d - q) < 2.0 ** -8 - 2.0 ** -16
    i, j = max(((i, j) for i in range(len(p)) for j in range(len(p)) if safe[i] and safe[j] and q[i] == q[j]),
               key=lambda t: d[t[0]] - d[t[1]])
    diff = d[i] - d[j]
    assert diff > 2.0 ** -10
    pre, B = np.empty((1, N)), np.empty((N, r))
    pre[0, ::2], pre[0, 1::2] = p[i], p[j]
    B[::2], B[1::2] = 1.0, -1.0
    X, A = c.dev("X", "A")
    o = L.backward_epilogue(c.base, X, torch.ones((1, N), dtype=torch.bfloat16, device=X.device), A, to_dev(bf16(B)),
                            1.0, P=to_dev(bf16(pre)), activation="silu", Z=torch.zeros((1, r), dtype=torch.bfloat16,
                                                                                      device=X.device))
    got, x = f64(to_host(o["dA"])), f64(c.X)[0]
    # per pair: the remainders (at most 2^-8) rounded to bf16, 2^-17 each, and the
    # fp32 slopes, within 2^-21 each; then dZ's and dA's own roundings, 2^-8 each
    ref = N // 2 * diff * x
    bound = N // 2 * 2 * (2.0 ** -17 + 2.0 ** -21) * np.abs(x) * (1 + 2.0 ** -6) + 2.01 * 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= bound)
    assert np.all(bound < 0.25 * np.abs(ref) + (x == 0))         # (dropping the remainders would miss it)
