"""CPU tests of attention's refusals: the C ABI's statuses and the binding's
errors, before anything reaches the GPU."""

import pytest
import torch

import lora_fine_tuning_amd as L

OK, ENULL, ESHAPE, EALIGN, EWS, EUNIMPL = 0, -1, -2, -3, -5, -7
P = 4096


def _a(**kw):
    a = dict(Tq=64, Tk=64, seqs=1, Hq=8, Hkv=2, D=128, scale=0.1, ldq=1024, ldk=256, ldv=256, q_offsets=None,
             k_offsets=None, k_lengths=None)
    a.update(kw)
    return L.lora4_attn(*a.values())


def fwd(attn=None, Q=P, K=P, V=P, O=P, lse=None, ws=P, n=1 << 40, **kw):
    return L.lora4_attention_forward(attn or _a(**kw), Q, K, V, O, lse, ws, n, None)


def bwd(attn=None, lse=P, dO=P, dQ=P, dK=P, dV=P, lds=(1024, 256, 256), ws=P, n=1 << 40, **kw):
    return L.lora4_attention_backward(attn or _a(**kw), P, P, P, P, lse, dO, dQ, dK, dV, *lds, ws, n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(Tq=-1), ESHAPE), (dict(Tk=-1), ESHAPE), (dict(seqs=0), ESHAPE), (dict(Hq=7), ESHAPE), (dict(Hkv=0), ESHAPE),
    (dict(Hq=130, Hkv=2, ldq=130 * 128), ESHAPE), (dict(D=4), ESHAPE), (dict(D=100), ESHAPE),
    (dict(D=136, ldq=8 * 136, ldk=272, ldv=272), EUNIMPL), (dict(scale=0.0), ESHAPE), (dict(scale=-1.0), ESHAPE),
    (dict(scale=float("nan")), ESHAPE), (dict(scale=float("inf")), ESHAPE), (dict(ldq=1016), ESHAPE),
    (dict(ldq=1028), ESHAPE), (dict(ldk=248), ESHAPE), (dict(ldv=260), ESHAPE), (dict(seqs=2), ENULL),
    (dict(q_offsets=P, Tk=65), ESHAPE), (dict(k_offsets=P), ESHAPE), (dict(Tq=1 << 31), ESHAPE),
    (dict(Tq=1 << 28), ESHAPE), (dict(ldq=1 << 23), ESHAPE)])
def test_problem(kw, want):
    assert fwd(**kw) == want
    assert bwd(**kw) == want


def test_pointers_and_workspace():
    assert L.lib().lora4_attention_forward(None, P, P, P, P, None, P, 1 << 40, None) == ENULL
    for n in ("Q", "K", "V", "O"):
        assert fwd(**{n: None}) == ENULL
        assert fwd(**{n: P + 8}) == EALIGN
    assert fwd(lse=P + 4) == EALIGN
    assert fwd(ws=None) == EWS
    need = L.lora4_attention_workspace_bytes(0, 1, 65536, 1, 8, 2, 128)
    assert need > 256                                     # key ranges
    assert fwd(Tq=1, Tk=65536, n=need - 1) == EWS
    for n in ("lse", "dO", "dQ", "dK", "dV"):
        assert bwd(**{n: None}) == ENULL
        assert bwd(**{n: P + 8}) == EALIGN
    assert bwd(lds=(1000, 256, 256)) == ESHAPE and bwd(lds=(1024, 128, 256)) == ESHAPE
    assert bwd(lds=(1024, 256, 257)) == ESHAPE
    assert bwd(n=L.lora4_attention_workspace_bytes(1, 64, 64, 1, 8, 2, 128) - 1) == EWS
    assert fwd(Tq=0, Q=None, O=None) == OK                # nothing to launch
    assert bwd(Tq=0, Tk=0) == OK


def test_workspace_sizes():
    f = L.lora4_attention_workspace_bytes
    assert f(0, 4096, 4096, 1, 32, 8, 128) > 0 and f(1, 4096, 4096, 1, 32, 8, 128) >= 4096 * 32 * 4
    for bad in [(2, 64, 64, 1, 8, 2, 128), (0, -1, 64, 1, 8, 2, 128), (0, 64, 64, 0, 8, 2, 128),
                (0, 64, 64, 1, 8, 3, 128), (1, 64, 64, 1, 8, 2, 132), (0, 64, 64, 1, 8, 2, 256)]:
        assert f(*bad) == 0, bad


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("args,kw", [
    ((_t(4, 16), _t(4, 2, 8), _t(4, 2, 8)), {}),                                   # Q 2-D
    ((_t(4, 2, 8, dtype=torch.float16), _t(4, 2, 8), _t(4, 2, 8)), {}),
    ((_t(4, 2, 8), _t(4, 2, 16), _t(4, 2, 16)), {}),                               # other D
    ((_t(4, 2, 8), _t(4, 2, 8), _t(5, 2, 8)), {}),                                 # V of another shape
    ((_t(4, 3, 8), _t(4, 2, 8), _t(4, 2, 8)), {}),                                 # 3 heads over 2
    ((_t(2, 4, 8).transpose(0, 1), _t(4, 2, 8), _t(4, 2, 8)), {}),                 # heads not contiguous
    ((_t(4, 2, 9)[:, :, :8], _t(4, 2, 8), _t(4, 2, 8)), {}),
    ((_t(4, 2, 8), _t(5, 2, 8), _t(5, 2, 8)), dict(q_offsets=_t(2, dtype=torch.int64))),   # keys are not the tokens
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(k_offsets=_t(2, dtype=torch.int64))),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(q_offsets=_t(2, dtype=torch.int32))),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(q_offsets=_t(1, dtype=torch.int64))),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(q_offsets=_t(3, dtype=torch.int64), k_offsets=_t(2, dtype=torch.int64))),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(k_lengths=_t(2, dtype=torch.int64))),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), dict(out={"O": _t(4, 2, 4)})),
    ((_t(4, 2, 8), _t(4, 2, 8), _t(4, 2, 8)), {}),                                 # not on a GPU
])
def test_binding(args, kw):
    with pytest.raises(ValueError):
        L.attention(*args, 0.1, **kw)


def test_binding_backward():
    t = [_t(4, 2, 8) for _ in range(5)]
    lse = _t(4, 2, dtype=torch.float32)
    for i in range(5):
        bad = list(t)
        bad[i] = _t(4, 2, 16)
        with pytest.raises(ValueError):
            L.attention_backward(bad[0], bad[1], bad[2], bad[3], lse, bad[4], 0.1)
    with pytest.raises(ValueError):
        L.attention_backward(*t[:4], _t(2, 4, dtype=torch.float32), t[4], 0.1)
    with pytest.raises(ValueError):
        L.attention_backward(*t[:4], lse, t[4], 0.1, out={"dK": _t(4, 1, 8)})
