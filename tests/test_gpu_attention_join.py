"""GPU tests of attention over keys that are cut into many ranges, for every kind of
head size: single tokens, small batches and a few queries over long caches, against
the float64 oracle, O and lse.

Bounds as in test_gpu_attention. Its share for fp32 sums, 2^-12 of I, covers these
lengths: the keys of a range are summed one after the other and then the ranges, at
most 32768 / 64 + 64 keys and 64 ranges, so an element's sum is off by at most 640
2^-24 < 2^-14 of the sum of its terms' sizes.
"""

import pytest

import lora_fine_tuning_amd as L
from test_gpu_attention import run_case

pytestmark = pytest.mark.gpu


def ranges_of(Tq, Tk, seqs, Hq, Hkv, D, keys):
    """Ranges that hold keys, of a sequence of `keys` keys in a forward call: the number
    of ranges from the workspace (per range, row and head a maximum and a sum, then D
    partial results, all fp32), each of whole steps of 64 keys."""
    size = L.lora4_attention_workspace_bytes(0, Tq, Tk, seqs, Hq, Hkv, D)
    up = lambda n: (n + 255) // 256 * 256
    for n in range(2, 65):
        if up(n * Tq * Hq * 8) + up(n * Tq * Hq * D * 4) == size:
            steps = -(-keys // 64)
            return -(-steps // -(-steps // n))
    return 1


@pytest.mark.parametrize("D,cap", [(8, 2048), (8, 9000), (16, 4096), (24, 9001), (64, 8448), (64, 20480), (72, 32768),
                                   (80, 10496), (96, 16384), (112, 32768), (120, 16384), (128, 32768)])
def test_one_token(D, cap):
    n = ranges_of(1, cap, 1, 32, 8, D, cap - 3)
    assert n > D // 2 or n == 64
    run_case([1], [cap - 3], 32, 8, D, seed=D + cap, cap=cap, bwd=False)


@pytest.mark.parametrize("D", [16, 64, 104])
def test_a_batch_of_single_tokens(D):
    """Caches filled to the end, in part, with one key and not at all."""
    cap, fill = 32768, [32768, 20001, 1, 0]
    assert ranges_of(4, cap * 4, 4, 8, 8, D, cap) > D // 2
    run_case([1] * 4, fill, 8, 8, D, seed=D, cap=cap, tail=2, bwd=False)


@pytest.mark.parametrize("Lq,Hq,D", [(20, 1, 64), (20, 4, 64), (3, 5, 40), (130, 1, 112)])
def test_few_queries_of_one_key_head(Lq, Hq, D):
    assert ranges_of(Lq, 32768, 1, Hq, 1, D, 32768) > D // 2
    run_case([Lq], [32768], Hq, 1, D, seed=Lq + D, cap=32768, bwd=False)
