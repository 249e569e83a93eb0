"""GPU tests of kv_* kernels and loops that the other files do not reach: every
attention kernel for more than 8 query heads to a kv head, more than 64 of them
with weights, weights of a row over many CTAs, the largest room of an eviction,
values beside keys in an append."""
import math

import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention
from tests._parity import dev_bf16
from tests.test_kv_attention import SHAPES, check, check_weights, run
from tests.test_kv_evict import case, state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits, D, gs", SHAPES)
@pytest.mark.parametrize("R, page", [(12, 16), (16, 48)])
def test_many_heads_of_a_group(bits, D, gs, R, page):
    lens = [0, 1, 15, 16, 17, 33, -2, 64, 257, 700]
    hc = HostCache(lens, 2, D, bits, gs, page, seed=bits + D + gs + R)
    hc.poison_unused()
    q = synth.normal_bf16((len(lens), 2 * R, D), 91)
    ref, bound, _ = attention(hc, q, 2 * R, 1 / math.sqrt(D))
    check(run(hc, q, 2 * R, 1 / math.sqrt(D)), ref, bound)


@pytest.mark.parametrize("bits, D, gs, R", [(4, 128, 32, 65), (8, 96, 32, 70), (16, 64, 0, 130),
                                            (4, 256, 64, 67)])
def test_weights_of_more_than_64_heads(bits, D, gs, R):
    lens, H = [40, 0, 600, 1], 2
    hc = HostCache(lens, H, D, bits, gs, 32, seed=R)
    q = synth.normal_bf16((4, H * R, D), 92)
    width = hc.width * 32
    before = np.random.default_rng(2).random((4, H, width)).astype(np.float32)
    w = torch.from_numpy(before.copy()).cuda()
    out = run(hc, q, H * R, 0.05, weights=w, state_width=width)
    ref, bound, probs = attention(hc, q, H * R, 0.05)
    check(out, ref, bound)
    check_weights(w, before.astype(np.float64), hc, probs, R)


@pytest.mark.parametrize("bits, D, gs", [(4, 128, 64), (8, 64, 64), (16, 128, 0), (8, 256, 128)])
@pytest.mark.parametrize("H, R", [(1, 2), (3, 9)])
def test_weights_of_a_row_over_many_ctas(bits, D, gs, H, R):
    lens = [20011, 3] if H == 1 else [9001, 0, 5003]
    hc = HostCache(lens, H, D, bits, gs, 64, seed=bits + H)
    q = synth.normal_bf16((len(lens), H * R, D), 93)
    width = hc.width * 64 + 1
    before = np.zeros((len(lens), H, width), np.float32)
    w = torch.zeros(before.shape, device="cuda")
    out = run(hc, q, H * R, 1 / math.sqrt(D), weights=w, state_width=width)
    ref, bound, probs = attention(hc, q, H * R, 1 / math.sqrt(D))
    check(out, ref, bound)
    check_weights(w, before.astype(np.float64), hc, probs, R)


@pytest.mark.parametrize("n, budget", [(196608, 100001), (196607, 196606), (131073, 4096)])
@pytest.mark.parametrize("in_place", [False, True])
def test_the_largest_room(n, budget, in_place):
    hc = HostCache([n], 1, 64, 4, 64, 4096, seed=budget, room=196608, spare=0)
    assert hc.width * hc.S == 196608
    for kind in ("skewed", "ties"):
        w, pos, width = state(hc, n, kind=kind)
        case(hc, w, pos, [n], budget, budget // 4, 4, width, in_place=in_place)


@pytest.mark.parametrize("bits, gs", [(4, 64), (8, 32), (16, 0)])
def test_keys_and_values_of_one_append_are_their_own(bits, gs):
    # the same rows as keys and as values give the same bits, others others
    H, D, T, page = 8, 128, 1500, 64
    hc = HostCache([T], H, D, bits, gs, page, seed=94)
    one, two = (dev_bf16(synth.normal_bf16((T, H, D), s)) for s in (95, 96))
    zero, starts = (torch.tensor(i, dtype=torch.int32, device="cuda") for i in ([0], [0, T]))
    stored = []
    for k, v in ((one, one), (one, two), (two, one)):
        cache, table, _ = hc.device()
        agq.kv_append(cache, k, v, table, zero, starts, 1, T, hc.width)
        j = torch.arange(T, device="cuda")
        pages, at = table[0].long()[j // page], j % page
        rows = [None if t is None else t.view(hc.num_pages, H, page, -1)[pages, :, at]
                for t in cache.buffers]
        stored.append([[rows[i] for i in side if rows[i] is not None] for side in ((0, 2, 3), (1, 4, 5))])

    def same(a, b):
        return all(torch.equal(x, y) for x, y in zip(a, b))

    (k0, v0), (k1, v1), (k2, v2) = stored
    assert same(k0, v0) and same(k0, k1) and same(k0, v2) and same(v1, k2)
    assert not same(k1, v1) and not same(k2, v2)


@pytest.mark.parametrize("bits", [4, 16])
def test_many_sequences_with_state(bits):
    # more sequences than token_starts in shared memory, each with its state
    B, H, D, page = 1100, 2, 64, 16
    rng = np.random.default_rng(5)
    new = rng.integers(0, 3, B)
    before = rng.integers(-1, 14, B)
    hc = HostCache([16] * B, H, D, bits, 32, page, seed=97)
    starts = np.concatenate(([0], np.cumsum(new)))
    T = int(starts[-1])
    x = dev_bf16(synth.normal_bf16((T, H, D), 98))
    cache, table, _ = hc.device()
    dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()  # noqa: E731
    pos = torch.full((B, H, 16), -7, dtype=torch.int32, device="cuda")
    w = torch.full((B, H, 16), 3.0, device="cuda")
    agq.kv_append(cache, x, x, table, dev(before), dev(starts), B, T, hc.width, seen=dev(before + 50),
                  positions=pos, weights=w, state_width=16)
    want_p, want_w = np.full((B, H, 16), -7), np.full((B, H, 16), 3.0)
    for b in range(B):
        for i in range(new[b] if before[b] >= 0 else 0):
            want_p[b, :, before[b] + i], want_w[b, :, before[b] + i] = before[b] + 50 + i, 0.0
    assert np.array_equal(pos.cpu().numpy(), want_p) and np.array_equal(w.cpu().numpy(), want_w)
