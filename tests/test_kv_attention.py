"""GPU tests of kv_attention against the definition in 64 bits, within a bound
that counts the operator's roundings (tests/_kv.py)."""
import math

import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention
from tests._parity import bf16_values, dev_bf16, host_bits

pytestmark = pytest.mark.gpu

SHAPES = [(4, 64, 32), (4, 64, 64), (4, 96, 32), (4, 128, 32), (4, 128, 64), (4, 128, 128),
          (4, 256, 32), (4, 256, 64), (4, 256, 128), (8, 64, 32), (8, 64, 64), (8, 96, 32),
          (8, 128, 32), (8, 128, 64), (8, 128, 128), (8, 256, 32), (8, 256, 64), (8, 256, 128),
          (16, 64, 0), (16, 96, 0), (16, 128, 0), (16, 256, 0)]


def run(hc, q16, Hq, scale, weights=None, state_width=0, dev=None, status=None, stream=None):
    B = len(hc.lens)
    cache, table, lens = dev or hc.device()
    Q = dev_bf16(q16)
    out = torch.full((B, Hq, hc.D), 7.0, dtype=torch.bfloat16, device="cuda")
    n = agq.kv_attention_workspace(cache, B, Hq, hc.width, weights is not None)
    ws = torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN where read as floats
    agq.kv_attention(cache, Q, table, lens, out, B, Hq, hc.width, scale, ws, weights=weights,
                     state_width=state_width, d_status=status, stream=stream)
    torch.cuda.synchronize()
    return out


def check(out, ref, bound, what=""):
    y = bf16_values(host_bits(out))
    assert np.isfinite(y).all(), what
    bad = np.abs(y - ref) > bound
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3],
                           float((np.abs(y - ref) / bound).max()))


def check_weights(w, before, hc, probs, R):
    got = w.cpu().numpy().astype(np.float64)
    for b, n in enumerate(hc.lens):
        n = max(0, n)
        p, e = probs[b]
        want = before[b].copy()
        tol = np.full(want.shape, 0.0)
        for g in range(hc.H):
            pg, eg = p[g * R:(g + 1) * R], e[g * R:(g + 1) * R]
            want[g, :n] += pg.sum(0)
            tol[g, :n] = (pg * eg).sum(0) + 2.0 ** -22 * (pg.sum(0) + np.abs(before[b][g, :n])) + 1e-30
        assert (np.abs(got[b] - want) <= tol).all(), (b, np.abs(got[b] - want).max())


@pytest.mark.parametrize("bits, D, gs", SHAPES)
def test_shapes(bits, D, gs):
    # lengths around every 16- and 32-slot edge, an empty row, a row not in use
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 48, -5, 100, 257]
    for H, R, page in ((2, 4, 16), (1, 1, 48)):
        hc = HostCache(lens, H, D, bits, gs, page, seed=bits * 7 + D + gs + R)
        hc.poison_unused()
        q = synth.normal_bf16((len(lens), H * R, D), 31)
        out = run(hc, q, H * R, 1 / math.sqrt(D))
        ref, bound, _ = attention(hc, q, H * R, 1 / math.sqrt(D))
        check(out, ref, bound, f"H={H} R={R} page={page}")
        assert (out[0] == 0).all() and (out[9] == 0).all()


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("R", [1, 2, 3, 5, 7, 8, 9, 12, 16, 17, 33])
def test_heads_of_a_group(bits, R):
    lens = [70, 3, 0, 200]
    for D in (64, 128, 256):
        hc = HostCache(lens, 2, D, bits, 64, 32, seed=R + D)
        q = synth.normal_bf16((4, 2 * R, D), 32)
        ref, bound, _ = attention(hc, q, 2 * R, 0.11)
        check(run(hc, q, 2 * R, 0.11), ref, bound, f"D={D}")


@pytest.mark.parametrize("bits, D, gs, page", [(4, 128, 64, 16), (8, 128, 64, 64), (16, 128, 0, 48),
                                               (4, 256, 128, 256), (8, 64, 32, 16), (4, 96, 32, 80)])
def test_long_rows_split_and_joined(bits, D, gs, page):
    # one long row beside short ones: it is split, they are not
    for lens, H, R in (([5000], 1, 2), ([7, 6001, 900, 1, 64], 2, 4), ([4096, 4095, 4097], 3, 16)):
        hc = HostCache(lens, H, D, bits, gs, page, seed=sum(lens))
        hc.poison_unused()
        q = synth.normal_bf16((len(lens), H * R, D), 33)
        ref, bound, _ = attention(hc, q, H * R, 1 / math.sqrt(D))
        check(run(hc, q, H * R, 1 / math.sqrt(D)), ref, bound, str(lens))


@pytest.mark.parametrize("bits, D, gs", [(4, 128, 64), (4, 64, 32), (8, 128, 128), (16, 256, 0)])
@pytest.mark.parametrize("R", [1, 4, 16])
def test_weights(bits, D, gs, R):
    lens = [0, 1, 33, 500, -1, 2100, 47]
    H = 2
    hc = HostCache(lens, H, D, bits, gs, 16, seed=bits + D + R)
    hc.poison_unused()
    q = synth.normal_bf16((len(lens), H * R, D), 34)
    width = hc.width * 16 + 3
    before = np.random.default_rng(1).random((len(lens), H, width)).astype(np.float32)
    w = torch.from_numpy(before.copy()).cuda()
    out = run(hc, q, H * R, 1 / math.sqrt(D), weights=w, state_width=width)
    ref, bound, probs = attention(hc, q, H * R, 1 / math.sqrt(D))
    check(out, ref, bound)
    check_weights(w, before.astype(np.float64), hc, probs, R)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_peaked_and_flat_scores(bits):
    # one slot takes all (scores far apart, rising along the row, so the
    # running maximum moves at every step), and all slots alike
    lens = [700, 700]
    hc = HostCache(lens, 1, 128, bits, 64, 16, seed=77, k_scale=4.0)
    q = synth.normal_bf16((2, 4, 128), 35).copy()
    q[1] = 0
    for scale in (1.0, -1.0, 3.0, 0.0):
        ref, bound, _ = attention(hc, q, 4, scale)
        check(run(hc, q, 4, scale), ref, bound, str(scale))


@pytest.mark.parametrize("bits", [4, 8])
def test_scales_over_many_binades(bits):
    # value scales from 2^-30 to 2^30 of each other, both signs, rising and
    # falling along the row; zero scales; a zero query
    lens = [300, 300, 64]
    hc = HostCache(lens, 2, 128, bits, 64, 16, seed=5)
    c, s, b = hc.q["v"]
    rng = np.random.default_rng(6)
    j = np.zeros(s.shape)
    for bb, n in enumerate(lens):
        for t in range(n):
            e = (t / n * 60 - 30) if bb == 0 else (30 - t / n * 60) if bb == 1 else 0
            j[hc.table[bb, t // 16], :, t % 16] = e
    sv = (2.0 ** np.round(j)) * rng.choice([-1.0, 1.0], s.shape) * (rng.random(s.shape) < 0.9)
    s[...] = synth.bf16_bits(torch.from_numpy(sv.astype(np.float32)))
    b[...] = synth.bf16_bits(torch.from_numpy((sv * -3.0).astype(np.float32)))
    q = synth.normal_bf16((3, 8, 128), 36).copy()
    q[2] = 0
    ref, bound, _ = attention(hc, q, 8, 0.05)
    check(run(hc, q, 8, 0.05), ref, bound)


@pytest.mark.parametrize("bits", [4, 16])
def test_queries_over_many_binades(bits):
    # every head's query is a power of two of its own, and inside a head some
    # elements are far smaller than the rest
    hc = HostCache([130, 40], 1, 128, bits, 64, 16, seed=8)
    q = synth.bits_to_float(synth.normal_bf16((2, 8, 128), 37)).astype(np.float64)
    for h in range(8):
        q[:, h] *= 2.0 ** (10 * h - 40)
    q[:, :, ::3] *= 2.0 ** -9
    q16 = synth.bf16_bits(torch.from_numpy(q.astype(np.float32)))
    for scale in (2.0 ** 10, 2.0 ** -30):
        qs = q16.copy()
        if scale > 1:
            qs[:, 4:] = 0                                  # keep the scores finite and modest
        ref, bound, _ = attention(hc, qs, 8, scale)
        check(run(hc, qs, 8, scale), ref, bound, str(scale))


def test_lengths_past_the_room_are_cut_and_flagged():
    hc = HostCache([64, 10], 2, 128, 4, 64, 16, seed=9)
    q = synth.normal_bf16((2, 8, 128), 38)
    ref, bound, _ = attention(hc, q, 8, 0.1)
    cache, table, _ = hc.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    over = torch.tensor([1000000, 10], dtype=torch.int32, device="cuda")
    check(run(hc, q, 8, 0.1, dev=(cache, table, over), status=status), ref, bound)
    assert status.item() == 1
    status.zero_()
    check(run(hc, q, 8, 0.1, status=status), ref, bound)
    assert status.item() == 0


@pytest.mark.parametrize("bits", [4, 16])
def test_slots_of_bad_pages_take_no_part(bits):
    hc = HostCache([100, 40, 16], 2, 64, bits, 64, 16, seed=10)
    q = synth.normal_bf16((3, 4, 64), 39)
    cache, table, lens = hc.device()
    bad = table.clone()
    bad[0, 2], bad[1, 0], bad[2, 0] = hc.num_pages, -1, 1 << 30   # the third has no good page
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.zeros((3, 2, hc.width * 16), device="cuda")
    out = run(hc, q, 4, 0.125, dev=(cache, bad, lens), status=status, weights=w,
              state_width=hc.width * 16)
    assert status.item() == 1
    # the same rows with the bad pages' slots left out
    keep = HostCache([100 - 16, 40 - 16, 0], 2, 64, bits, 64, 16, seed=10, room=112)
    keep.q, keep.num_pages = hc.q, hc.num_pages
    t = np.full((3, keep.width), -1, np.int32)
    t[0, :6] = np.delete(hc.table[0, :7], 2)
    t[1, :2] = hc.table[1, 1:3]
    keep.table = t
    ref, bound, probs = attention(keep, q, 4, 0.125)
    check(out, ref, bound)
    assert (w[0, :, 32:48] == 0).all() and (w[1, :, :16] == 0).all() and (w[2] == 0).all()
    back = torch.cat((w[0, :, :32], w[0, :, 48:100]), -1).cpu().numpy()
    p, e = probs[0]
    assert (np.abs(back[0] - p[:2].sum(0)) <= (p[:2] * e[:2]).sum(0) + 2.0 ** -22).all()


def test_query_slices_and_streams_and_repeats():
    # q as columns of a wider projection, on a side stream; the same bits twice
    hc = HostCache([900, 333, 20], 2, 128, 8, 64, 16, seed=12)
    wide = synth.normal_bf16((3, 12, 128), 40)
    cache, table, lens = hc.device()
    Q = dev_bf16(wide)
    ref, bound, _ = attention(hc, np.ascontiguousarray(wide[:, 2:10]), 8, 0.09)
    ws = torch.empty(agq.kv_attention_workspace(cache, 3, 8, hc.width), dtype=torch.uint8,
                     device="cuda")
    outs = []
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
        agq.kv_attention(cache, Q[:, 2:10], table, lens, out, 3, 8, hc.width, 0.09, ws, stream=st)
        st.synchronize()
        outs.append(out)
        check(out, ref, bound)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_two_calls_at_once_and_a_graph_that_sees_new_lengths():
    hc = HostCache([2000, 2000], 2, 128, 4, 64, 16, seed=13)
    q = synth.normal_bf16((2, 8, 128), 41)
    cache, table, lens = hc.device()
    Q = dev_bf16(q)
    n = agq.kv_attention_workspace(cache, 2, 8, hc.width, True)
    state = hc.width * 16

    def buffers():
        return (torch.empty(n, dtype=torch.uint8, device="cuda"),
                torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda"),
                torch.zeros((2, 2, state), device="cuda"))

    sets = [buffers(), buffers()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for (ws, out, w), s in zip(sets, streams):
            agq.kv_attention(cache, Q, table, lens, out, 2, 8, hc.width, 0.1, ws, weights=w,
                             state_width=state, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(sets[0][1], sets[1][1]) and torch.equal(sets[0][2], sets[1][2])
    ref, bound, _ = attention(hc, q, 8, 0.1)
    check(sets[0][1], ref, bound)

    ws, out, w = sets[0]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        agq.kv_attention(cache, Q, table, lens, out, 2, 8, hc.width, 0.1, ws)
    for new in ([5, 1999], [0, 17], [2000, 1]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        hc.lens = new
        ref, bound, _ = attention(hc, q, 8, 0.1)
        check(out, ref, bound, str(new))


def test_large_batch_of_short_rows():
    rng = np.random.default_rng(14)
    lens = rng.integers(0, 70, 600).tolist()
    hc = HostCache(lens, 2, 64, 8, 32, 16, seed=15)
    q = synth.normal_bf16((600, 4, 64), 42)
    ref, bound, _ = attention(hc, q, 4, 0.125)
    check(run(hc, q, 4, 0.125), ref, bound)


def test_cache_rows_past_32_bit_offsets():
    # rows that start more than 2^32 bytes into a buffer, and a table that
    # points there
    H, D, page = 4, 128, 256
    pages = (1 << 32) // (H * page * D * 2) + 3
    small = HostCache([300], H, D, 16, 0, page, seed=16, spare=0)
    k = torch.zeros((pages, H, page, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    c, t, lens = small.device()
    last = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    for buf, big in zip(c.buffers[:2], (k, v)):
        big[last[0].long()] = buf.view(small.num_pages, H, page, D)[t[0].long()]
    cache = agq.KVCache(k, v, None, None, None, None, pages, H, page, D, 16, 0)
    q = synth.normal_bf16((1, 8, D), 43)
    ref, bound, _ = attention(small, q, 8, 0.1)
    check(run(small, q, 8, 0.1, dev=(cache, last, lens)), ref, bound)
