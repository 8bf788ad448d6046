"""GPU tests of the loss over the vocabulary against the float64 oracle.

dX: every element passes |gpu - ref| <= 1.01 u (|ref| + I) + E and the whole output
||gpu - ref|| <= 5e-3 ||ref|| + ||E||, u = 2^-8 the bf16 unit roundoff. I = w sum of p
|W| over the other words is what rounding their exponentials carries into it (twice
where a row's reference moved: the cases that do so say so). E: a logit is a sum of
K exact products in fp32, off by at most e = K 2^-24 of the sum of their sizes, its
multiple of log2 e and the reference by 2^-24 each, exp2 by 2^-24 of its argument and
one unit: every p is off by at most r = 2^-24 (K + 8) size + 2^-20 of itself, as are
the sums that divide; the fp32 sums over V words add V 2^-24 at most (pairwise in
strips, far less). losses: their logits' error and the sums' (relative to the loss
itself where the target is nearly certain). Outputs and workspaces sit between
guard bands.
"""

import numpy as np
import pytest
import torch

import lora_fine_tuning_amd as L
import synth
from gpu_util import DEV, ELEM_U, TOL, f64, guarded, print_case, to_dev, to_host
from oracle import vocab_loss

pytestmark = pytest.mark.gpu


def normal(rng, shape, std=1.0):
    return synth.to_bf16((rng.standard_normal(shape) * std).astype(np.float32))


def fp32_guarded(n):
    raw, c = guarded((n * 2,))   # (bf16 guard bands around n floats)
    return raw.view(torch.float32), c


def check(o, ref, X, W, twice=False):
    V, K = W.shape
    r = 2.0 ** -24 * (K + 8) * ref["size"] + 2.0 ** -20 + V * 2.0 ** -24
    loss = o["loss"].cpu().numpy().astype(np.float64)
    # d loss = the error of the others' sum over the target's term, at most r of it
    # each, and the log of it; at most the error of lse - l_t as a number
    tol = 2 * r * np.minimum(1.0, np.abs(np.expm1(np.minimum(ref["loss"], 50)))) + 2.0 ** -22 * np.abs(ref["loss"]) + 2.0 ** -126
    assert np.all(np.abs(loss - ref["loss"]) <= tol), float((np.abs(loss - ref["loss"]) / tol).max())
    if o["lse"] is not None:
        lse = o["lse"].cpu().numpy().astype(np.float64)
        assert np.all(np.abs(lse - ref["lse"]) <= 2 * r + 2.0 ** -22 * np.abs(ref["lse"]))
    if o["dX"] is None:
        return
    g = f64(to_host(o["dX"]))
    assert np.all(np.isfinite(g))
    E = (2 * r + 2.0 ** -12)[:, None] * (ref["I_dX"] + ref["I_t"]) + 2.0 ** -120
    err = np.abs(g - ref["dX"])
    assert np.linalg.norm(err) <= TOL * np.linalg.norm(ref["dX"]) + np.linalg.norm(E)
    bound = 1.01 * ELEM_U * (np.abs(ref["dX"]) + ref["I_dX"] * (2 if twice else 1)) + E
    assert np.all(err <= bound), float((err / bound).max())


def run_case(M, K, V, seed, weights=False, ignored=0.2, std=0.3, boost=None, twice=False, grad=True):
    print_case("head_loss", M, K, V, weights, ignored)
    rng = np.random.default_rng(seed)
    X, W = normal(rng, (M, K)), normal(rng, (V, K), std)
    if boost is not None:
        X = boost(rng, X, W)
    t = rng.integers(0, V, M)
    t[rng.random(M) < ignored] = -100
    w = rng.random(M).astype(np.float32) if weights else None
    out, checks = {}, []
    for n, size in (("loss", M), ("lse", M), ("total", 1)):
        out[n], c = fp32_guarded(size)
        checks.append((n, c))
    if grad:
        out["dX"], c = guarded((M, K))
        checks.append(("dX", c))
    ws, c = guarded((L.lora4_head_loss_workspace_bytes(int(grad), M, K, V),), torch.uint8)
    checks.append(("workspace", c))
    td, wd = torch.from_numpy(t).to(DEV), None if w is None else torch.from_numpy(w).to(DEV)
    x, h = to_dev(X), to_dev(W)
    o = L.head_loss(x, h, td, weights=wd, want_grad=grad, workspace=ws, out=out)
    torch.cuda.synchronize()
    for n, c in checks:
        c(n)
    ref = vocab_loss.loss(f64(X), f64(W), t, None if w is None else w.astype(np.float64))
    check(o, ref, X, W, twice)
    total = float(o["total"])
    lw = np.abs(ref["loss"]) * (1.0 / max(1, (t != -100).sum()) if w is None else w)
    assert abs(total - ref["total"]) <= 1e-4 * lw.sum() + 1e-30
    again = L.head_loss(x, h, td, weights=wd, want_grad=grad, want_lse=True)
    for n in o:
        assert (o[n] is None and again[n] is None) or torch.equal(o[n], again[n]), n
    if grad:
        alone = L.head_loss(x, h, td, weights=wd, want_grad=False)
        assert torch.allclose(alone["loss"], o["loss"], rtol=1e-5, atol=1e-6) and alone["dX"] is None
    return o


@pytest.mark.parametrize("M,K,V", [(1, 8, 1), (1, 8, 2), (1, 64, 300), (3, 72, 129), (5, 200, 257), (64, 64, 64),
                                   (130, 520, 1000), (255, 128, 512), (257, 1000, 700), (300, 256, 5003),
                                   (600, 96, 33), (20, 2080, 4999)])
@pytest.mark.parametrize("weights", [False, True])
def test_sizes(M, K, V, weights):
    run_case(M, K, V, seed=M + K + V, weights=weights)


@pytest.mark.parametrize("M,K,V", [(1, 4096, 2000), (8, 256, 20000), (700, 64, 3001)])
def test_loss_alone(M, K, V):
    run_case(M, K, V, seed=M, grad=False)


@pytest.mark.parametrize("piece", ["1", "300", "1024"])
def test_pieces_of_the_vocabulary(monkeypatch, piece):
    """Several pieces: acc is added to in memory, the last one is ragged."""
    monkeypatch.setenv("LORA4_LOSS_PIECE", piece)
    run_case(300, 136, 2600, seed=3)
    run_case(70, 520, 777, seed=4, weights=True, grad=False)


@pytest.mark.parametrize("tiles", ["small", "big"])
@pytest.mark.parametrize("M,K,V", [(1, 8, 1), (5, 72, 130), (130, 520, 1000), (300, 256, 5003), (70, 2080, 129)])
def test_either_tiles(monkeypatch, tiles, M, K, V):
    monkeypatch.setenv("LORA4_LOSS_TILES", tiles)
    run_case(M, K, V, seed=M + V, weights=True)
    monkeypatch.setenv("LORA4_LOSS_PIECE", "256")
    run_case(M, K, V, seed=M + V + 1)
    run_case(M, K, V, seed=M + V + 2, grad=False)


def test_chunks_of_the_rows():
    run_case(4100, 40, 300, seed=5)
    run_case(9000, 16, 500, seed=6, weights=True, ignored=0.6)


def test_every_row_and_no_row_ignored():
    run_case(50, 64, 400, seed=7, ignored=0.0)
    o = run_case(50, 64, 400, seed=8, ignored=1.1)
    assert float(o["total"]) == 0 and not o["dX"].any() and not o["loss"].any() and not o["lse"].any()


@pytest.mark.parametrize("piece", ["100000", "512"])
@pytest.mark.parametrize("scale", [10.0, 40.0])
def test_targets_far_below_the_largest_logit(monkeypatch, piece, scale):
    """Logits further above the target's than the slack: rows move to another
    reference, in the first piece and in later ones."""
    monkeypatch.setenv("LORA4_LOSS_PIECE", piece)

    def boost(rng, X, W):
        f = np.where(rng.random((X.shape[0], 1)) < 0.5, scale, 1.0)
        return synth.to_bf16((f64(X) * f).astype(np.float32))
    run_case(200, 128, 3000, seed=9, boost=boost, twice=True)


def test_nearly_certain_targets():
    """p_t within 2^-20 and less of 1: loss and gradient keep their digits."""
    rng = np.random.default_rng(10)
    M, K, V = 64, 256, 900
    W = normal(rng, (V, K), 0.1)
    t = rng.integers(0, V, M)
    f = rng.uniform(2, 12, (M, 1))
    X = synth.to_bf16((f64(W)[t] * f * 2 + 0.1 * rng.standard_normal((M, K))).astype(np.float32))
    o = L.head_loss(to_dev(X), to_dev(W), torch.from_numpy(t).to(DEV), want_lse=True)
    ref = vocab_loss.loss(f64(X), f64(W), t)
    assert ref["loss"].min() < 1e-9
    check(o, ref, X, W)


def test_bad_targets_and_bad_rows():
    rng = np.random.default_rng(11)
    M, K, V = 40, 64, 300
    X, W, t = normal(rng, (M, K)), normal(rng, (V, K)), rng.integers(0, V, M)
    clean = L.head_loss(to_dev(X), to_dev(W), torch.from_numpy(t).to(DEV), weights=torch.ones(M, device=DEV))
    t[3], t[7], t[9], t[12] = V, -1, 1 << 40, -(1 << 40)
    X[20, 5], X[21, 6] = 0x7FC0, 0x7F80
    t[22] = -100
    X[22] = 0x7FC0                                     # an ignored row may hold anything
    bad = [3, 7, 9, 12, 20, 21]
    o = L.head_loss(to_dev(X), to_dev(W), torch.from_numpy(t).to(DEV), weights=torch.ones(M, device=DEV))
    loss, dX = o["loss"].cpu().numpy(), o["dX"].float().cpu().numpy()
    assert not np.isfinite(loss[bad]).any() and np.isnan(dX[bad]).all(axis=1).all()
    assert loss[22] == 0 and not dX[22].any() and torch.isnan(o["total"]).all()
    good = [i for i in range(M) if i not in bad + [22]]
    assert torch.equal(o["loss"][good], clean["loss"][good]) and torch.equal(o["dX"][good], clean["dX"][good])


def test_another_ignore_index_and_same_target_twice():
    rng = np.random.default_rng(12)
    X, W = to_dev(normal(rng, (6, 64))), to_dev(normal(rng, (50, 64)))
    t = torch.tensor([0, 7, 7, 0, 49, 7], device=DEV)
    a = L.head_loss(X, W, t, ignore_index=0)
    t2 = torch.tensor([-100, 7, 7, -100, 49, 7], device=DEV)
    b = L.head_loss(X, W, t2)
    for n in ("loss", "total", "dX"):
        assert torch.equal(a[n], b[n]), n


def test_empty_call():
    z = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    W = torch.ones(9, 64, dtype=torch.bfloat16, device=DEV)
    o = L.head_loss(z, W, torch.zeros(0, dtype=torch.int64, device=DEV))
    assert o["loss"].numel() == 0 and float(o["total"]) == 0


def test_another_stream_and_a_captured_graph():
    rng = np.random.default_rng(13)
    M, K, V = 300, 192, 2100
    X, W = to_dev(normal(rng, (M, K))), to_dev(normal(rng, (V, K), 0.2))
    t = torch.from_numpy(rng.integers(0, V, M)).to(DEV)
    ws = L.head_loss_workspace(True, M, K, V, DEV)
    out = {"loss": torch.empty(M, device=DEV), "total": torch.empty(1, device=DEV), "dX": torch.empty_like(X),
           "lse": torch.empty(M, device=DEV)}
    L.head_loss(X, W, t, workspace=ws, out=out)
    ref = {n: x.clone() for n, x in out.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.head_loss(X, W, t, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    for n in ref:
        assert torch.equal(out[n], ref[n]), n
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.head_loss(X, W, t, workspace=ws, out=out)
    for i in range(4):
        # other targets, and another number of rows that count, per replay
        t.copy_(torch.from_numpy(np.where(rng.random(M) < 0.3 * i, -100, rng.integers(0, V, M))))
        ws.fill_(0x7F if i % 2 else 0)
        g.replay()
        torch.cuda.synchronize()
        eager = L.head_loss(X, W, t, want_lse=True)
        for n in ref:
            assert torch.equal(out[n], eager[n]), (i, n)


def test_a_head_past_32_bit_offsets():
    """600000 words of 4096: 4.9 GB, the last words beyond 2^31 elements, in two
    pieces. The reference in float64 on the GPU, in ranges of the vocabulary."""
    M, K, V = 3, 4096, 600000
    g = torch.Generator(device=DEV).manual_seed(3)
    W = torch.empty(V, K, dtype=torch.bfloat16, device=DEV)
    for i in range(0, V, 100000):
        W[i:i + 100000] = torch.randn((100000, K), generator=g, device=DEV) * 0.02
    X = torch.randn((M, K), generator=g, device=DEV).to(torch.bfloat16)
    t = torch.tensor([V - 1, 7, 550000], device=DEV)
    o = L.head_loss(X, W, t, want_lse=True)
    alone = L.head_loss(X, W, t, want_grad=False)
    l = torch.cat([X.double() @ W[i:i + 50000].double().t() for i in range(0, V, 50000)], 1)
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    p[torch.arange(M), t] -= 1
    dX = sum(p[:, i:i + 50000] @ W[i:i + 50000].double() for i in range(0, V, 50000)) / M
    loss = lse - l[torch.arange(M), t]
    for r in (o, alone):
        assert torch.all((r["loss"].double() - loss).abs() <= 1e-5 * loss)
    err = (o["dX"].double() - dX).norm() / dX.norm()
    assert float(err) <= TOL


def test_two_calls_at_once():
    rng = np.random.default_rng(14)
    jobs = []
    for M, K, V in ((200, 256, 3000), (5, 512, 900)):
        a = (to_dev(normal(rng, (M, K))), to_dev(normal(rng, (V, K), 0.2)), torch.from_numpy(rng.integers(0, V, M)).to(DEV))
        jobs.append((a, L.head_loss(*a)))
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = [[] for _ in jobs]
    for _ in range(5):
        for i, (s, (a, _)) in enumerate(zip(streams, jobs)):
            with torch.cuda.stream(s):
                got[i].append(L.head_loss(*a))
    torch.cuda.synchronize()
    for g, (_, ref) in zip(got, jobs):
        assert all(torch.equal(x[n], ref[n]) for x in g for n in ("loss", "total", "dX"))


def test_gradient_against_differences():
    """d total along a direction, by the float64 loss around the bf16 inputs: off by
    at most 2 u of the sum of the gradient's terms."""
    rng = np.random.default_rng(15)
    X, W, t = normal(rng, (60, 96)), normal(rng, (700, 96), 0.2), rng.integers(0, 700, 60)
    t[::7] = -100
    g = f64(to_host(L.head_loss(to_dev(X), to_dev(W), torch.from_numpy(t).to(DEV))["dX"]))
    d = rng.standard_normal(g.shape)
    f = lambda x: vocab_loss.loss(x, f64(W), t)["total"]
    num = (f(f64(X) + 1e-5 * d) - f(f64(X) - 1e-5 * d)) / 2e-5
    assert abs(num - (g * d).sum()) <= 2 * 2.0 ** -8 * np.abs(g * d).sum()


def test_infinite_logits():
    """A target whose logit is -infinity costs infinity, one of +infinity NaN; the
    other rows are as without them."""
    rng = np.random.default_rng(16)
    X, W = normal(rng, (4, 64)), normal(rng, (50, 64))
    W[10] = 0
    t = np.array([3, 10, 10, 5])
    W2 = W.copy()
    W2[10, 0] = 0xFF80                    # -inf times X[., 0]
    X[1, 0], X[2, 0], X[0, 0], X[3, 0] = 0x3F80, 0xBF80, 0x3F80, 0x3F80   # 1, -1, 1, 1
    o = L.head_loss(to_dev(X), to_dev(W2), torch.from_numpy(t).to(DEV), weights=torch.ones(4, device=DEV), want_grad=False)
    l = o["loss"].cpu().numpy()
    assert np.isposinf(l[1]) and np.isnan(l[2])
    ref = vocab_loss.loss(f64(X)[[0, 3]], np.delete(f64(W), 10, 0), np.array([3, 5]))["loss"]
    assert np.allclose(l[[0, 3]], ref, rtol=1e-5)
