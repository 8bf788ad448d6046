"""CPU tests of the ends of attention's ranges: a scale whose multiple of log2 e is past
fp32 would make scores of NaN, also from zeros, and is refused."""

import numpy as np
import pytest

import lora_fine_tuning_amd as L

ESHAPE, EWS = -2, -5
P = 4096


def calls(scale):
    a = L.lora4_attn(64, 64, 1, 8, 2, 128, scale, 1024, 256, 256, None, None, None)
    # (a workspace of no bytes: nothing is launched where the scale is taken)
    return (L.lora4_attention_forward(a, P, P, P, P, None, P, 0, None),
            L.lora4_attention_backward(a, P, P, P, P, P, P, P, P, P, 1024, 256, 256, P, 0, None))


LARGEST = float(np.float32(3.4028234e38 / 1.4426950408889634))


@pytest.mark.parametrize("scale,want", [(1e-45, EWS), (1.0, EWS), (2.3e38, EWS), (LARGEST * 1.000001, ESHAPE),
                                        (3e38, ESHAPE), (float("inf"), ESHAPE)])
def test_scales(scale, want):
    assert calls(scale) == (want, want)
