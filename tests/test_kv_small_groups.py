"""GPU test of kv_attention where one group's value scales are far below
another's: what the contract says is lost of them, and no more."""
import numpy as np
import pytest
import torch

from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention
from tests._parity import bf16_values, host_bits
from tests.test_kv_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("power", [-12, -20, -24, -27, -30, -33])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_a_small_group_beside_a_large_one(bits, power, n):
    # groups of 64: the first of ordinary scales, the second 2^power of it, and
    # the other way round in the second head
    H, R, D = 2, 2, 128
    hc = HostCache([n], H, D, bits, 64, 16, seed=n - power)
    _, s, b = hc.q["v"]
    top = 1.25
    for h in range(H):
        s[:, h, :, h] = synth.bf16_bits(torch.full((1,), top))[0]
        s[:, h, :, 1 - h] = synth.bf16_bits(torch.full((1,), 1.5 * 2.0 ** power))[0]
    b[...] = 0
    q = synth.normal_bf16((1, H * R, D), 61)
    out = bf16_values(host_bits(run(hc, q, H * R, 0.02)))
    ref, _, probs = attention(hc, q, H * R, 0.02)
    _, va = hc.dense("v", 0, n)
    for h in range(H * R):
        p, e = probs[0][0][h], probs[0][1][h]
        # half of fp16's steps: relative 2^-11, or 2^-34 of the largest scale (its
        # power of two is 2^9, the last step 2^-24) a slot and code; the sum of
        # probabilities that it is divided by is 1 or more
        low = 2.0 ** -34 * top * (2 ** bits - 1) * n
        tol = (2.0 ** -8 * np.abs(ref[0, h]) + (2.0 ** -11 + 2.0 ** -20) * (p @ va[h // R])
               + e.max() * (p @ va[h // R]) + low)
        err = np.abs(out[0, h] - ref[0, h])
        assert (err <= tol).all(), (h, (err / tol).max())
