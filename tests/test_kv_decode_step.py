"""The key-value cache operators as they are used: a decode step of quantized
products around append, attention and eviction, prompts first, eagerly and as a
captured graph, on several widths of the cache."""
import math

import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
import oracle
from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention, evict
from tests._parity import bf16_values, check, dev_bf16, dev_u32, host_bits

pytestmark = pytest.mark.gpu

HIDDEN, HQ, H, D, GS = 512, 8, 2, 64, 64
COLS = (HQ + 2 * H) * D


class Model:
    """One attention layer: a quantized qkv product, the cache, a quantized
    output product.  `host` mirrors the cache on the CPU."""

    def __init__(self, bits, lens, room, page=16):
        self.B = len(lens)
        self.hc = HostCache([room] * self.B, H, D, bits, GS, page, seed=50)
        self.cache, self.table, _ = self.hc.device()
        self.room = self.hc.width * page
        self.w = [synth.qmv_inputs(1, n, k, 4, GS, seed=s)[1:] for n, k, s in
                  ((COLS, HIDDEN, 60), (HIDDEN, HQ * D, 61))]
        self.dw = [(dev_u32(w), dev_bf16(s), dev_bf16(b)) for w, s, b in self.w]
        self.qkv = torch.zeros((self.B, HQ + 2 * H, D), dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros((self.B, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.y = torch.zeros((self.B, HIDDEN), dtype=torch.bfloat16, device="cuda")
        n = agq.kv_attention_workspace(self.cache, self.B, HQ, self.hc.width, True)
        self.ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
        self.weights = torch.zeros((self.B, H, self.room), device="cuda")
        self.positions = torch.full((self.B, H, self.room), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.seen = self.lens.clone()
        self.new_lens = torch.zeros_like(self.lens)
        self.x = torch.zeros((self.B, HIDDEN), dtype=torch.bfloat16, device="cuda")

    def step(self, budget=0, recent=0, sinks=0):
        W, st = self.hc.width, dict(state_width=self.room)
        agq.qmv(self.x, *self.dw[0], self.qkv, self.B, COLS, HIDDEN, 4, GS)
        agq.kv_append(self.cache, self.qkv[:, HQ:HQ + H], self.qkv[:, HQ + H:], self.table,
                      self.lens, None, self.B, self.B, W, seen=self.seen,
                      positions=self.positions, weights=self.weights, **st)
        self.lens += 1
        self.seen += 1
        agq.kv_attention(self.cache, self.qkv[:, :HQ], self.table, self.lens, self.out, self.B,
                         HQ, W, 1 / math.sqrt(D), self.ws, weights=self.weights, **st)
        if budget:
            agq.kv_evict(self.cache, self.table, self.lens, self.seen, self.weights,
                         self.positions, self.new_lens, self.weights, self.positions, self.B, W,
                         self.room, budget, recent, sinks)
            self.lens.copy_(self.new_lens)
        agq.qmv(self.out, *self.dw[1], self.y, self.B, HIDDEN, HQ * D, 4, GS)


def _mirror(m, lens):
    """The host cache with the device's rows and these lengths."""
    got = m.hc.host(m.cache)
    m.hc.q = {n: tuple(None if a is None else a.reshape(b.shape) for a, b in zip(got[n], m.hc.q[n]))
              for n in "kv"}
    m.hc.lens = list(lens)
    return m.hc


def _check_step(m, lens):
    """The step's products against the oracle, its attention against the
    definition over the rows that the cache now holds."""
    y_ref, a_ref = oracle.qmv(host_bits(m.x), *m.w[0], m.B, COLS, HIDDEN, 4, GS)
    check(host_bits(m.qkv).reshape(m.B, COLS), y_ref, a_ref, "qkv")
    hc = _mirror(m, lens)
    q = host_bits(m.qkv)[:, :HQ]
    ref, bound, probs = attention(hc, np.ascontiguousarray(q), HQ, 1 / math.sqrt(D))
    out = host_bits(m.out)
    assert (np.abs(bf16_values(out) - ref) <= bound).all()
    y_ref, a_ref = oracle.qmv(out.reshape(m.B, -1), *m.w[1], m.B, HIDDEN, HQ * D, 4, GS)
    check(host_bits(m.y), y_ref, a_ref, "o")
    return probs


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_prompt_then_steps(bits):
    # prompts of different lengths in one call, then steps that cross pages
    lens = [14, 0, 31]
    m = Model(bits, [0, 0, 0], room=48)
    T = sum(lens)
    p = synth.normal_bf16((T, 2 * H, D), 70)
    P = dev_bf16(p)
    starts = torch.tensor([0, 14, 14, 45], dtype=torch.int32, device="cuda")
    agq.kv_append(m.cache, P[:, :H], P[:, H:], m.table, m.lens, starts, 3, T, m.hc.width,
                  seen=m.seen, positions=m.positions, weights=m.weights, state_width=m.room)
    # the prompt's rows, dense again, are what the cache stands for
    K = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    agq.kv_read(m.cache, K, V, m.table, m.lens, starts, 3, T, m.hc.width)
    hc = _mirror(m, lens)
    for t, name in ((K, "k"), (V, "v")):
        dense = np.concatenate([hc.dense(name, b, n)[0].transpose(1, 0, 2) for b, n in enumerate(lens)])
        assert np.array_equal(bf16_values(host_bits(t)), bf16_values(synth.bf16_bits(
            torch.from_numpy(dense)))) or bits != 16
        assert (np.abs(bf16_values(host_bits(t)) - dense) <= 2.0 ** -8 * np.abs(dense)).all()
    m.lens.copy_(torch.tensor(lens))
    m.seen.copy_(m.lens)
    total = np.zeros((3, H, m.room))
    for s in range(4):
        m.x.copy_(dev_bf16(synth.normal_bf16((3, HIDDEN), 80 + s)))
        m.step()
        lens = [n + 1 for n in lens]
        probs = _check_step(m, lens)
        for b, n in enumerate(lens):
            for g in range(H):
                total[b, g, :n] += probs[b][0][g * HQ // H:(g + 1) * HQ // H].sum(0)
    w = m.weights.cpu().numpy()
    assert (np.abs(w - total) <= 2.0 ** -10 * total + 1e-30).all()
    pos = m.positions.cpu().numpy()
    for b, n in enumerate(lens):
        assert (pos[b, :, :n] == np.arange(n)).all() and (pos[b, :, n:] == -1).all()


@pytest.mark.parametrize("bits", [4, 16])
def test_steps_at_a_full_budget(bits):
    # every step appends one slot and evicts one; attention sees slots out of
    # order of position; the choice is checked from the step's own weights
    budget, recent, sinks = 40, 10, 2
    m = Model(bits, [38, 5], room=48)
    m.positions.copy_(torch.arange(m.room, dtype=torch.int32).expand(2, H, -1))
    m.positions[0, :, 38:] = -1
    m.positions[1, :, 5:] = -1
    m.weights[0, :, :38] = torch.rand((H, 38), device="cuda")
    lens = [38, 5]
    for s in range(6):
        m.x.copy_(dev_bf16(synth.normal_bf16((2, HIDDEN), 90 + s)))
        m.step()
        lens = [n + 1 for n in lens]
        _check_step(m, lens)
        w, pos = m.weights.cpu().numpy(), m.positions.cpu().numpy()
        rows = {n: [None if a is None else a.copy() for a in m.hc.q[n]] for n in "kv"}
        seen = m.seen.tolist()
        agq.kv_evict(m.cache, m.table, m.lens, m.seen, m.weights, m.positions, m.new_lens,
                     m.weights, m.positions, 2, m.hc.width, m.room, budget, recent, sinks)
        m.lens.copy_(m.new_lens)
        got = _mirror(m, lens).q
        nw, npos = m.weights.cpu().numpy(), m.positions.cpu().numpy()
        for b in range(2):
            left = min(lens[b], budget)
            for h in range(H):
                _, src = evict(w[b, h], pos[b, h], lens[b], seen[b], budget, recent, sinks)
                assert np.array_equal(npos[b, h, :left], pos[b, h, src])
                assert np.array_equal(nw[b, h, :left], w[b, h, src])
                assert (nw[b, h, left:] == 0).all() and (npos[b, h, left:] == -1).all()
                for name in "kv":
                    for g, a in zip(got[name], rows[name]):
                        if a is not None:
                            j = np.arange(left)
                            at = (m.hc.table[b, j // 16], h, j % 16)
                            of = (m.hc.table[b, src // 16], h, src % 16)
                            assert np.array_equal(g[at], a[of])
        lens = m.lens.tolist()
    assert lens == [40, 11]


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_a_captured_step_equals_the_eager_one(bits):
    # one graph, replayed as the lengths grow past pages and into eviction; a
    # second one on another stream with a workspace of its own, alive meanwhile
    models = [Model(bits, [20, 3, 37], room=64) for _ in range(3)]
    args = (40, 8, 4)
    eager, graphs = models[0], []
    for m in models:
        m.positions.copy_(torch.arange(m.room, dtype=torch.int32).expand(3, H, -1))
    state = [(m.lens.clone(), m.seen.clone(), m.weights.clone(), m.positions.clone(),
              [t if t is None else t.clone() for t in m.cache.buffers]) for m in models]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for m, st, old in zip(models[1:], streams, state[1:]):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            m.step(*args)                       # warm up, then put everything back
            for t, o in zip((m.lens, m.seen, m.weights, m.positions), old):
                t.copy_(o)
            for t, o in zip(m.cache.buffers, old[4]):
                if t is not None:
                    t.copy_(o)
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            m.step(*args)
        graphs.append(g)
    for s in range(8):
        x = dev_bf16(synth.normal_bf16((3, HIDDEN), 100 + s))
        for m in models:
            m.x.copy_(x)
        torch.cuda.synchronize()
        eager.step(*args)
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for m in models[1:]:
            assert m.lens.tolist() == eager.lens.tolist()
            for a, b in ((m.y, eager.y), (m.out, eager.out), (m.weights, eager.weights),
                         (m.positions, eager.positions), (m.cache.buffers[0], eager.cache.buffers[0]),
                         (m.cache.buffers[1], eager.cache.buffers[1])):
                assert torch.equal(a, b)
    assert eager.lens.tolist() == [28, 11, 40]
    del graphs
