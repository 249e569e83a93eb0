"""GPU tests of kv_append and kv_read: the rows that append writes are the
oracle quantizer's bits (bf16 rows: the input's), everything else in the cache
is left alone, and read gives back the oracle's dequantized values."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
import oracle
from affine_group_quantized_b200 import synth
from tests._kv import HostCache
from tests._parity import dev_bf16, host_bits

pytestmark = pytest.mark.gpu

SHAPES = [(4, 64, 32), (4, 96, 32), (4, 128, 64), (4, 256, 128), (8, 64, 64), (8, 96, 32),
          (8, 128, 128), (8, 256, 32), (16, 96, 32), (16, 128, 64), (16, 256, 0)]


def _i32(*x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _rows(T, H, D, seed, strange=True):
    x = synth.normal_bf16((T, H, D), seed).copy()
    if strange and T > 2:
        x[1] = 0                                   # all-zero groups
        x[2, :, : D // 2] = synth.bf16_bits(torch.full((1,), 0.375))[0]   # constant groups
    return x


def _expect(hc, x, seqs, slots, name):
    """The host cache's buffers after rows x[t] go to (sequence, slot)."""
    T, H, D = x.shape
    c, s, b = (None if a is None else a.copy() for a in hc.q[name])
    if hc.bits == 16:
        new = (x, None, None)
    else:
        w, ss, bb = oracle.affine_quantize(x.reshape(-1, D), T * H, D, hc.bits, hc.gs)
        new = (w.reshape(T, H, -1), ss.reshape(T, H, -1), bb.reshape(T, H, -1))
    for t in range(T):
        if seqs[t] < 0:
            continue
        page, at = hc.table[seqs[t], slots[t] // hc.S], slots[t] % hc.S
        for a, n in zip((c, s, b), new):
            if a is not None:
                a[page, :, at] = n[t]
    return c, s, b


@pytest.mark.parametrize("bits, D, gs", SHAPES)
@pytest.mark.parametrize("page", [16, 48])
def test_append_then_read(bits, D, gs, page):
    H, B = 3, 5
    before, new = [0, 15, 40, 7, 33], [1, 17, 0, 9, 30]   # rows cross pages; one adds nothing
    hc = HostCache([a + n for a, n in zip(before, new)], H, D, bits, gs, page, seed=bits + D + page)
    starts = np.concatenate(([0], np.cumsum(new)))
    T = int(starts[-1]) + 3                                # three padding tokens at the end
    seqs = np.full(T, -1)
    slots = np.zeros(T, int)
    for b in range(B):
        seqs[starts[b]:starts[b + 1]] = b
        slots[starts[b]:starts[b + 1]] = before[b] + np.arange(new[b])
    # keys and values as slices of one wider projection output
    wide = synth.normal_bf16((T, 2 * H + 1, D), 5)
    wide[:, :H], wide[:, H + 1:] = _rows(T, H, D, 6), _rows(T, H, D, 7)
    X = dev_bf16(wide)
    cache, table, _ = hc.device()
    agq.kv_append(cache, X[:, :H], X[:, H + 1:], table, _i32(*before), _i32(*starts), B, T,
                  hc.width)
    torch.cuda.synchronize()
    got = hc.host(cache)
    for name, x in (("k", wide[:, :H]), ("v", wide[:, H + 1:])):
        for g, w in zip(got[name], _expect(hc, np.ascontiguousarray(x), seqs, slots, name)):
            assert (g is None and w is None) or np.array_equal(g.reshape(w.shape), w), name

    # read everything back, into wider rows whose other columns stay
    total = [a + n for a, n in zip(before, new)]
    starts = np.concatenate(([0], np.cumsum(total)))
    T = int(starts[-1]) + 2
    K = torch.full((T, H + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    V = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    agq.kv_read(cache, K[:, 1:H + 1], V, table, _i32(*[0] * B), _i32(*starts), B, T, hc.width)
    torch.cuda.synchronize()
    assert (K[:, 0] == 7).all() and (K[:, -1] == 7).all()
    assert (K[-2:] == 7).all() and (V[-2:] == 7).all()     # rows of no sequence
    hc.q = {n: tuple(None if a is None else a.reshape(b.shape) for a, b in zip(got[n], hc.q[n]))
            for n in "kv"}
    for name, t in (("k", K[:, 1:H + 1]), ("v", V)):
        out = host_bits(t.contiguous())
        for b in range(B):
            j = np.arange(total[b])
            pages, at = hc.table[b, j // page], j % page
            c, s, bi = (None if a is None else np.ascontiguousarray(a[pages, :, at])
                        for a in hc.q[name])
            if bits == 16:
                want = c
            else:
                n = total[b] * H
                want = oracle.dequantize_bf16(c.reshape(n, -1), s.reshape(n, -1),
                                              bi.reshape(n, -1), n, D, bits, gs)
            assert np.array_equal(out[starts[b]:starts[b + 1]].reshape(-1), want.reshape(-1))


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_one_token_each_with_state(bits):
    H, D, gs, page = 40, 64, 32, 16                        # more heads than a warp has lanes
    before = [0, 16, 31, -1, 5]                            # the fourth row is not in use
    hc = HostCache([max(0, n) + 1 for n in before], H, D, bits, gs, page, seed=3, room=64)
    x, y = _rows(5, H, D, 8), _rows(5, H, D, 9)
    cache, table, _ = hc.device()
    width = hc.width * page + 5                            # wider state than room
    pos = torch.full((5, H, width), -7, dtype=torch.int32, device="cuda")
    w = torch.full((5, H, width), 3.0, device="cuda")
    agq.kv_append(cache, dev_bf16(x), dev_bf16(y), table, _i32(*before), None, 5, 5, hc.width,
                  seen=_i32(100, 200, 300, 400, 500), positions=pos, weights=w, state_width=width)
    torch.cuda.synchronize()
    want_p, want_w = np.full((5, H, width), -7), np.full((5, H, width), 3.0)
    for b, n in enumerate(before):
        if n >= 0:
            want_p[b, :, n], want_w[b, :, n] = 100 * (b + 1), 0.0
    assert np.array_equal(pos.cpu().numpy(), want_p) and np.array_equal(w.cpu().numpy(), want_w)
    seqs = [b if n >= 0 else -1 for b, n in enumerate(before)]
    got = hc.host(cache)
    for name, v in (("k", x), ("v", y)):
        for g, e in zip(got[name], _expect(hc, v, seqs, before, name)):
            assert (g is None and e is None) or np.array_equal(g.reshape(e.shape), e)


def test_state_of_several_tokens():
    hc = HostCache([20, 3], 2, 64, 8, 64, 16, seed=4)
    cache, table, _ = hc.device()
    pos = torch.full((2, 2, 32), -7, dtype=torch.int32, device="cuda")
    w = torch.full((2, 2, 32), 3.0, device="cuda")
    x = dev_bf16(_rows(6, 2, 64, 8))
    agq.kv_append(cache, x, x, table, _i32(15, 2), _i32(0, 5, 6), 2, 6, hc.width,
                  seen=_i32(1000, 0), positions=pos, weights=w, state_width=32)
    assert (pos[0, :, 15:20] == torch.arange(1000, 1005, device="cuda")).all()
    assert (w[0, :, 15:20] == 0).all() and (pos[1, :, 2] == 0).all()
    assert (pos == -7).sum() == 2 * 64 - 2 * 6 and (w == 3).sum() == 2 * 64 - 2 * 6


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_bad_indices_are_flagged_and_left_alone(bits):
    H, D, page = 2, 128, 16
    hc = HostCache([32, 32, 32], H, D, bits, 64, page, seed=11)
    bad = hc.table.copy()
    bad[0, 1], bad[1, 0] = hc.num_pages, -3                # past the cache, and negative
    good = hc.table
    cache, _, _ = hc.device()
    x = dev_bf16(_rows(6, H, D, 12))
    status = _i32(0)
    # sequence 0: its second page is bad; 1: its first; 2: runs out of room
    hc.table = bad
    agq.kv_append(cache, x, x, torch.from_numpy(bad).cuda(), _i32(15, 3, 31), _i32(0, 2, 4, 6), 3,
                  6, hc.width, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 1
    hc.table = good
    seqs, slots = [0, -1, -1, -1, 2, -1], [15, 0, 0, 0, 31, 0]
    got = hc.host(cache)
    for name in "kv":
        for g, e in zip(got[name], _expect(hc, host_bits(x), seqs, slots, name)):
            assert (g is None and e is None) or np.array_equal(g.reshape(e.shape), e)
    K = torch.full((6, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    status.zero_()
    agq.kv_read(cache, K, V, torch.from_numpy(bad).cuda(), _i32(15, 3, 31), _i32(0, 2, 4, 6), 3, 6,
                hc.width, d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 1
    for t in (1, 2, 3, 5):
        assert (K[t] == 7).all() and (V[t] == 7).all()
    assert not (K[0] == 7).all() and not (K[4] == 7).all()
    status.zero_()                                         # good indices: nothing is flagged
    agq.kv_read(cache, K, V, torch.from_numpy(good).cuda(), _i32(15, 3, 30), _i32(0, 2, 4, 6), 3,
                6, hc.width, d_status=status)
    assert status.item() == 0


def test_long_prompt_against_affine_quantize():
    # the same rows through the library's own quantizer, one launch each
    H, D, bits, gs, page, T = 8, 128, 4, 64, 64, 1500
    hc = HostCache([T], H, D, bits, gs, page, seed=21)
    cache, table, _ = hc.device()
    x = dev_bf16(_rows(T, H, D, 22))
    agq.kv_append(cache, x, x, table, _i32(0), _i32(0, T), 1, T, hc.width)
    w = torch.empty((T * H, D * bits // 32), dtype=torch.int32, device="cuda")
    s = torch.empty((T * H, D // gs), dtype=torch.bfloat16, device="cuda")
    b = torch.empty_like(s)
    agq.affine_quantize(x, w, s, b, T * H, D, bits, gs)
    j = torch.arange(T, device="cuda")
    pages, at = table[0].long()[j // page], j % page
    shape = (hc.num_pages, H, page, -1)
    for buf, want in zip((0, 2, 3), (w, s, b)):
        assert torch.equal(cache.buffers[buf].view(shape)[pages, :, at].reshape(want.shape), want)
    assert torch.equal(cache.buffers[1], cache.buffers[1])
    for a, c in ((0, 1), (2, 4), (3, 5)):
        ka, va = (cache.buffers[i].view(shape)[pages, :, at] for i in (a, c))
        assert torch.equal(ka, va)                         # the same rows as values
