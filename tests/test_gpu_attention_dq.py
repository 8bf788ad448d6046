"""GPU tests of attention's dQ against the definition's, delta from P and dP in all
rows, with flat and with peaked scores over up to 700 keys.

Every element passes |gpu - ref| <= 1.01 u (|ref| + I) + E + 2^-12 I + D and the whole
output ||gpu - ref|| <= 5e-3 ||ref|| + ||E + 2^-12 I|| + ||N||: u, I, E and the sums'
2^-12 I as in test_gpu_attention; D and N are what the bf16 O, from which the rows of
many keys take delta, may cost, as the oracle derives them. Where a row's weight lies on
few keys its dS nearly cancels and N is the larger part, whatever number of keys the row
sees.
"""

import numpy as np
import pytest

import lora_fine_tuning_amd as L
from gpu_util import ELEM_U, TOL, f64, print_case, to_dev, to_host
from oracle import attention
from test_gpu_attention import normal, offsets, ranges

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("std", [0.5, 1.5, 3.0, 6.0])
@pytest.mark.parametrize("nq,Hq,Hkv,D", [([500], 4, 2, 64), ([330, 9, 90], 6, 1, 128), ([700], 2, 2, 40)])
def test_dq(nq, Hq, Hkv, D, std):
    print_case("dQ", nq, Hq, Hkv, D, std)
    rng = np.random.default_rng(D + int(10 * std))
    T, scale, r = sum(nq), D ** -0.5, ranges(nq)
    Q, K, V, dO = (normal(rng, (T, h, D), s) for h, s in ((Hq, std), (Hkv, std), (Hkv, 1.0), (Hq, 0.05)))
    q, k, v, do = map(to_dev, (Q, K, V, dO))
    o = L.attention(q, k, v, scale, q_offsets=offsets(nq))
    b = L.attention_backward(q, k, v, o["O"], o["lse"], do, scale, q_offsets=offsets(nq))
    ref = attention.dq(*map(f64, (Q, K, V, dO)), scale, r, r, ELEM_U)
    err = np.abs(f64(to_host(b["dQ"])) - ref["dQ"])
    E = ref["E_dQ"] + 2.0 ** -12 * ref["I_dQ"]
    share = np.linalg.norm(err) / np.linalg.norm(ref["dQ"])
    print("[error]", round(float(share), 5), "of it by O", round(float(np.linalg.norm(ref["N_dQ"]) / np.linalg.norm(ref["dQ"])), 5))
    assert np.linalg.norm(err) <= TOL * np.linalg.norm(ref["dQ"]) + np.linalg.norm(E) + np.linalg.norm(ref["N_dQ"])
    assert np.all(err <= 1.01 * ELEM_U * (np.abs(ref["dQ"]) + ref["I_dQ"]) + E + ref["D_dQ"])
