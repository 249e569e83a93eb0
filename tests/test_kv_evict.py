"""GPU tests of kv_evict: the choice, the moves and the state are compared
exactly with a plain implementation (tests/_kv.py)."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from tests._kv import HostCache, evict

pytestmark = pytest.mark.gpu


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def case(hc, w, pos, seen, budget, recent, sinks, state, in_place=False, lens=None, status=None,
         stream=None):
    """Runs one call and compares everything it may write."""
    B, H = len(hc.lens), hc.H
    cache, table, dev_lens = hc.device()
    if lens is not None:
        dev_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    W, P = _dev(w), _dev(pos)
    new_lens = torch.full((B,), -9, dtype=torch.int32, device="cuda")
    NW, NP = (W, P) if in_place else (torch.full_like(W, 5.5), torch.full_like(P, -5))
    agq.kv_evict(cache, table, dev_lens, _dev(np.asarray(seen, np.int32)), W, P, new_lens, NW, NP,
                 B, hc.width, state, budget, recent, sinks, d_status=status, stream=stream)
    torch.cuda.synchronize()
    want_w = w.copy() if in_place else np.full_like(w, 5.5)
    want_p = pos.copy() if in_place else np.full_like(pos, -5)
    want_q = {n: [None if a is None else a.copy() for a in hc.q[n]] for n in "kv"}
    for b, n in enumerate(hc.lens):
        n = max(0, n)
        left = min(n, budget)
        for h in range(H):
            _, src = evict(w[b, h], pos[b, h], n, seen[b], budget, recent, sinks)
            want_w[b, h, :n], want_p[b, h, :n] = 0, -1
            want_w[b, h, :left], want_p[b, h, :left] = w[b, h, src], pos[b, h, src]
            for name in "kv":
                for a, o in zip(want_q[name], hc.q[name]):
                    for j in np.flatnonzero(src != np.arange(left)):
                        if a is not None:
                            a[hc.table[b, j // hc.S], h, j % hc.S] = \
                                o[hc.table[b, src[j] // hc.S], h, src[j] % hc.S]
    assert new_lens.tolist() == [min(max(0, n), budget) for n in hc.lens]
    assert np.array_equal(NW.cpu().numpy().view(np.uint32), want_w.view(np.uint32))
    assert np.array_equal(NP.cpu().numpy(), want_p)
    got = hc.host(cache)
    for name in "kv":
        for g, e in zip(got[name], want_q[name]):
            assert (g is None and e is None) or np.array_equal(g.reshape(e.shape), e), name


def state(hc, seed, extra=0, kind="random"):
    rng = np.random.default_rng(seed)
    B, width = len(hc.lens), hc.width * hc.S + extra
    shape = (B, hc.H, width)
    w = rng.random(shape).astype(np.float32)
    if kind == "skewed":
        w = np.exp(rng.standard_normal(shape) * 6).astype(np.float32)
    elif kind == "ties":
        w = rng.integers(0, 3, shape).astype(np.float32)
    elif kind == "alike":
        w = np.full(shape, 0.25, np.float32)
    elif kind == "strange":
        w = rng.choice(np.array([np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-45, -1.0, 1.0,
                                 3.4e38], np.float32), shape)
    pos = np.broadcast_to(np.arange(width, dtype=np.int32), shape).copy()
    return w, pos, width


@pytest.mark.parametrize("bits, D, gs", [(4, 64, 32), (4, 128, 64), (4, 96, 32), (8, 128, 128),
                                         (8, 256, 32), (16, 96, 0), (16, 256, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths_and_types(bits, D, gs, in_place):
    lens = [0, 1, 39, 40, 41, 64, 100, 217, -3]
    hc = HostCache(lens, 2, D, bits, gs, 16, seed=bits + D)
    w, pos, width = state(hc, 1, extra=3)
    case(hc, w, pos, [max(0, n) for n in lens], 40, 8, 4, width, in_place=in_place)


@pytest.mark.parametrize("kind", ["skewed", "ties", "alike", "strange"])
@pytest.mark.parametrize("in_place", [False, True])
def test_weights_of_every_kind(kind, in_place):
    lens = [300, 77, 500]
    hc = HostCache(lens, 3, 64, 8, 64, 32, seed=2)
    w, pos, width = state(hc, 3, kind=kind)
    for budget, recent, sinks in ((64, 0, 0), (64, 32, 0), (64, 60, 4), (1, 0, 0), (1, 1, 0),
                                  (76, 10, 3)):
        case(hc, w, pos, lens, budget, recent, sinks, width, in_place=in_place)


@pytest.mark.parametrize("n, budget", [(1025, 1024), (4097, 1000), (9000, 8999), (20000, 640),
                                       (33000, 16500)])
def test_long_rows(n, budget):
    # rows shared out over clusters of 1, 4 and 8 CTAs, beside a short one
    hc = HostCache([n, n // 3, 5], 1, 64, 4, 64, 64, seed=n, spare=1)
    for kind in ("random", "ties"):
        w, pos, width = state(hc, n, kind=kind)
        case(hc, w, pos, hc.lens, budget, budget // 4, 4, width)


def test_positions_out_of_order():
    # after earlier evictions slots are not in order of position; some
    # positions are protected wherever they lie, more than once even
    lens = [200, 200]
    hc = HostCache(lens, 2, 128, 4, 64, 16, seed=4)
    w, pos, width = state(hc, 5)
    rng = np.random.default_rng(6)
    pos = rng.integers(0, 1000, pos.shape).astype(np.int32)
    case(hc, w, pos, [1000, 500], 50, 30, 20, width)
    case(hc, w, np.full_like(pos, 999), [1000, 1000], 50, 30, 20, width)  # all protected: lower slots


def test_length_past_the_room_is_cut_and_flagged():
    hc = HostCache([64, 30], 2, 64, 16, 0, 16, seed=7)
    w, pos, width = state(hc, 8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    case(hc, w, pos, [64, 30], 20, 4, 0, width, lens=[70000, 30], status=status)
    assert status.item() == 1
    status.zero_()
    case(hc, w, pos, [64, 30], 20, 4, 0, width, status=status)
    assert status.item() == 0


def test_bad_pages_move_only_state():
    hc = HostCache([64], 1, 64, 8, 64, 16, seed=9)
    w, pos, width = state(hc, 10)
    w[0, 0, :16], w[0, 0, 48:] = 0.0, 2.0        # the first page's slots go, the last page's come
    cache, table, lens = hc.device()
    bad = table.clone()
    bad[0, 3] = hc.num_pages + 1
    before = [t.clone() for t in cache.buffers]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    W, P = _dev(w), _dev(pos)
    NW, NP = torch.empty_like(W), torch.empty_like(P)
    agq.kv_evict(cache, bad, lens, lens, W, P, new_lens, NW, NP, 1, hc.width, width, 48,
                 d_status=status)
    torch.cuda.synchronize()
    assert status.item() == 1 and new_lens.item() == 48
    assert NP[0, 0, :16].tolist() == list(range(48, 64)) and (NW[0, 0, :16] == 2).all()
    assert all(torch.equal(a, b) for a, b in zip(before, cache.buffers))


def test_side_stream_and_graph():
    hc = HostCache([300, 20], 2, 128, 4, 64, 16, seed=11)
    w, pos, width = state(hc, 12)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    case(hc, w, pos, [300, 20], 100, 10, 4, width, stream=st)
    cache, table, lens = hc.device()
    W, P = _dev(w), _dev(pos)
    new_lens, NW, NP = torch.zeros_like(lens), torch.zeros_like(W), torch.zeros_like(P)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        agq.kv_evict(cache, table, lens, lens, W, P, new_lens, NW, NP, 2, hc.width, width, 100,
                     10, 4)
    for new in ([300, 20], [101, 0], [100, 99]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert new_lens.tolist() == [min(100, n) for n in new]
        for b in range(2):
            _, src = evict(w[b, 0], pos[b, 0], new[b], new[b], 100, 10, 4)
            assert np.array_equal(NP[b, 0, :len(src)].cpu().numpy(), pos[b, 0][src])
