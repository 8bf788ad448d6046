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
