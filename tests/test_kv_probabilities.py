"""GPU test of kv_attention over bf16 rows: what is left of the error is the
output's rounding, not the probabilities'."""
import math

import numpy as np
import pytest

from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention
from tests._parity import bf16_values, host_bits
from tests.test_kv_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("R", [1, 4, 12])
def test_probabilities_keep_16_bits(D, R):
    # values that nearly cancel: the output is far smaller than its terms
    lens, H = [2, 3, 5, 16, 40, 333, 2500], 2
    hc = HostCache(lens, H, D, 16, 0, 16, seed=D + R)
    q = synth.normal_bf16((len(lens), H * R, D), 81)
    scale = 1 / math.sqrt(D)
    ref, bound, probs = attention(hc, q, H * R, scale)
    # the bound with each probability the sum of two bf16 numbers, off by half a
    # step of the second (2^-16), in place of one (2^-8)
    for b, n in enumerate(lens):
        _, va = hc.dense("v", b, n)
        for h in range(H * R):
            bound[b, h] -= (2.0 ** -8 - 2.0 ** -16) * (probs[b][0][h] @ va[h // R])
    y = bf16_values(host_bits(run(hc, q, H * R, scale)))
    bad = np.abs(y - ref) > bound
    assert not bad.any(), (int(bad.sum()), bad.size, float((np.abs(y - ref) / bound).max()))
