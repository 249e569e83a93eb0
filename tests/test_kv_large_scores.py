"""GPU tests of kv_attention where scores are far larger than the steps of
binary32: the probabilities are those of the scores' differences, never of a
score's own rounding."""
import numpy as np
import pytest
import torch

from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention, values
from tests._parity import bf16_values, host_bits
from tests.test_kv_attention import run

pytestmark = pytest.mark.gpu

SHAPES = [(4, 64, 32), (4, 128, 64), (4, 256, 128), (8, 128, 128), (8, 96, 32), (16, 64, 0),
          (16, 128, 0), (16, 256, 0)]


def _grow(hc, b, slot, by):
    """Slot `slot` of sequence b's key, `by` (a power of two) times as large."""
    at = hc.table[b, slot // hc.S], slice(None), slot % hc.S
    c, s, bias = hc.q["k"]
    for a in ((c,) if hc.bits == 16 else (s, bias)):
        a[at] = synth.bf16_bits(torch.from_numpy((values(a[at]) * by).astype(np.float32)))


def _queries(hc, winners, Hq):
    """For every head, the key of its sequence's winning slot: that slot's score is
    far above the others'."""
    R = Hq // hc.H
    q = np.zeros((len(hc.lens), Hq, hc.D))
    for b, n in enumerate(hc.lens):
        k, _ = hc.dense("k", b, n)
        q[b] = np.repeat(k[:, winners[b]], R, 0)
    return synth.bf16_bits(torch.from_numpy(q.astype(np.float32)))


@pytest.mark.parametrize("bits, D, gs", SHAPES)
@pytest.mark.parametrize("power", [0, 18, 24, 40, 90])
def test_one_slot_far_above_the_others(bits, D, gs, power):
    lens, winners, H, R = [40, 700, 1, 33], [39, 350, 0, 7], 2, 4
    hc = HostCache(lens, H, D, bits, gs, 16, seed=bits + D + power)
    for b, w in enumerate(winners):
        _grow(hc, b, w, 4.0)
    q = _queries(hc, winners, H * R)
    scale = 2.0 ** power
    w = torch.zeros((4, H, hc.width * 16), device="cuda")
    out = bf16_values(host_bits(run(hc, q, H * R, scale, weights=w, state_width=hc.width * 16)))
    ref, _, probs = attention(hc, q, H * R, scale)
    for b, n in enumerate(lens):
        v, va = hc.dense("v", b, n)
        for h in range(H * R):
            p = probs[b][0][h]
            assert p[winners[b]] > 1 - 2.0 ** -40       # the others count nothing
            # the probability's rounding (times the scale), the output's, and the fp32 steps
            tol = ((2.0 ** -8 if bits == 16 else 2.0 ** -11) * va[h // R, winners[b]]
                   + 2.0 ** -8 * np.abs(ref[b, h])
                   + 2.0 ** -20 * (va[h // R, winners[b]] + np.abs(v[h // R, winners[b]])) + 1e-30)
            assert (np.abs(out[b, h] - ref[b, h]) <= tol).all(), (b, h, out[b, h][:4], ref[b, h][:4])
        want = np.zeros((H, hc.width * 16))
        want[:, winners[b]] = R
        got = w[b].cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -20 * R).all(), (b, got[:, winners[b]])


@pytest.mark.parametrize("bits, D, gs", [(4, 128, 64), (8, 64, 32), (16, 128, 0)])
@pytest.mark.parametrize("power", [0, 22, 30, 60])
def test_slots_that_are_all_alike(bits, D, gs, power):
    # one key and one value in every slot: equal probabilities, the value itself,
    # and equal weights, however large the scores (rows over many CTAs too)
    lens, H, R = [5, 3000, 64], 1, 2
    hc = HostCache(lens, H, D, bits, gs, 16, seed=power + D)
    for name in "kv":
        for a in hc.q[name]:
            if a is not None:
                a[...] = a[:1, :, :1]
    q = _queries(hc, [0, 0, 0], R)
    w = torch.zeros((3, H, hc.width * 16), device="cuda")
    out = bf16_values(host_bits(run(hc, q, R, 2.0 ** power, weights=w, state_width=hc.width * 16)))
    for b, n in enumerate(lens):
        v, va = hc.dense("v", b, n)
        # as above, with the sums of n equal terms in binary32
        sums = 2.0 ** -23 * (n / 16 + 64)
        tol = ((2.0 ** -8 if bits == 16 else 2.0 ** -11) + sums) * va[0, 0] \
            + (2.0 ** -8 + sums) * np.abs(v[0, 0]) + 1e-30
        assert (np.abs(out[b] - v[0, 0]) <= tol).all(), b
        got = w[b, 0].cpu().numpy()
        assert (np.abs(got[:n] * n - R) <= R * (sums + 2.0 ** -20)).all() and (got[n:] == 0).all()


@pytest.mark.parametrize("bits", [4, 16])
def test_scores_one_step_apart(bits):
    # scores that rise by a step or two of binary32 from slot to slot: the last
    # tenth's differences are far above 1, so the largest takes all
    n, D, H = 320, 64, 1
    hc = HostCache([n], H, D, bits, 64, 16, seed=3)
    k = np.zeros((n, D))
    k[:, 0] = 1 + np.arange(n) // 40 * 2.0 ** -7        # bf16 numbers, 40 slots each
    if bits == 16:
        rows = synth.bf16_bits(torch.from_numpy(k.astype(np.float32)))
        for j in range(n):
            hc.q["k"][0][hc.table[0, j // 16], 0, j % 16] = rows[j]
    else:                                               # code 1 at the first element, scaled
        c, s, b = hc.q["k"]
        c[...], b[...] = 0, 0
        for j in range(n):
            at = hc.table[0, j // 16], 0, j % 16
            c[at][0] = 1
            s[at] = synth.bf16_bits(torch.from_numpy(k[j:j + 1, :1].astype(np.float32)))[0]
    q = np.zeros((1, 2, D), np.float32)
    q[..., 0] = 1.5
    q16 = synth.bf16_bits(torch.from_numpy(q))
    for power in (20, 29, 45):
        w = torch.zeros((1, 1, hc.width * 16), device="cuda")
        out = bf16_values(host_bits(run(hc, q16, 2, 2.0 ** power, weights=w, state_width=hc.width * 16)))
        v, va = hc.dense("v", 0, n)
        want = v[0, 280:320].mean(0)
        tol = ((2.0 ** -8 if bits == 16 else 2.0 ** -11) + 2.0 ** -16) * va[0, 280:320].mean(0) \
            + 2.0 ** -8 * np.abs(want) + 1e-30
        assert (np.abs(out[0] - want) <= tol).all(), power
        got = w[0, 0].cpu().numpy()
        assert (got[:280] == 0).all() and (np.abs(got[280:320] - 2 / 40) <= 2.0 ** -20).all(), power
