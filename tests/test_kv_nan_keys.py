"""GPU tests of kv_attention with NaN keys: a NaN among a sequence's keys shows in
its outputs and weights and nowhere else."""
import numpy as np
import pytest
import torch

from affine_group_quantized_b200 import synth
from tests._kv import BF16_NAN, HostCache
from tests._parity import bf16_values, host_bits
from tests.test_kv_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits, D, gs", [(4, 128, 64), (8, 64, 32), (16, 128, 0)])
@pytest.mark.parametrize("n", [9, 33, 900])
def test_nan_keys_show_in_outputs_and_weights(bits, D, gs, n):
    # sequence 0 holds nothing but NaN keys, sequence 2 one, 1 and 3 none
    H, R = 2, 3
    hc = HostCache([n, 40, n, 5], H, D, bits, gs, 16, seed=n)
    q = synth.normal_bf16((4, H * R, D), 54)
    width = hc.width * 16
    clean = torch.zeros((4, H, width), device="cuda")
    good = run(hc, q, H * R, 0.1, weights=clean, state_width=width)
    target = hc.q["k"][0 if bits == 16 else 2]
    for j in range(n):
        target[hc.table[0, j // 16], :, j % 16] = BF16_NAN
    target[hc.table[2, (n // 2) // 16], :, (n // 2) % 16] = BF16_NAN
    w = torch.zeros((4, H, width), device="cuda")
    out = run(hc, q, H * R, 0.1, weights=w, state_width=width)
    for b in (0, 2):
        assert torch.isnan(out[b]).all() and torch.isnan(w[b, :, :n]).all(), b
        assert (w[b, :, n:] == 0).all()
    for b in (1, 3):
        assert torch.isfinite(out[b]).all() and torch.isfinite(w[b]).all()
        y, z = bf16_values(host_bits(out[b])), bf16_values(host_bits(good[b]))
        assert np.abs(y - z).max() <= 2.0 ** -7 * np.abs(z).max()
