"""Helpers for the key-value cache tests: a cache built on the CPU with the
oracle's quantizer, the operators' definitions in 64 bits, and the bounds their
results are held to."""
from __future__ import annotations

import numpy as np
import torch

import oracle
from affine_group_quantized_b200 import synth

BF16_NAN = 0x7FC1


def values(bits16: np.ndarray) -> np.ndarray:
    return synth.bits_to_float(bits16).astype(np.float64)


class HostCache:
    """num_pages pages of random rows: bf16 bit patterns, or the oracle's
    codes, scales and biases of such rows; `table` names each sequence's pages
    (scattered; entries past its slots are -1)."""

    def __init__(self, lens, H, D, bits, gs, page, seed, room=None, spare=2, k_scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.H, self.D, self.bits, self.gs, self.S = list(lens), H, D, bits, gs, page
        longest = max([1] + [n for n in lens]) if room is None else room
        self.width = -(-longest // page)
        need = [-(-max(0, n) // page) for n in lens]
        self.num_pages = sum(need) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(lens), self.width), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        shape = (self.num_pages, H, page, D)
        self.rows, self.q = {}, {}
        for i, name in enumerate("kv"):
            x = rng.standard_normal(shape).astype(np.float32)
            if name == "k":
                x[..., : max(1, D // 16)] *= 4.0 * k_scale
            bits16 = synth.bf16_bits(torch.from_numpy(x))
            if bits == 16:
                self.q[name] = (bits16, None, None)
            else:
                n = self.num_pages * H * page
                w, s, b = oracle.affine_quantize(bits16.reshape(n, D), n, D, bits, gs)
                self.q[name] = (w.reshape(*shape[:3], -1), s.reshape(*shape[:3], -1),
                                b.reshape(*shape[:3], -1))

    def poison_unused(self):
        """NaN wherever no sequence has a slot: rows, or scales and biases with
        every code bit set."""
        used = np.zeros((self.num_pages, self.S), bool)
        for b, n in enumerate(self.lens):
            for j in range(max(0, n)):
                used[self.table[b, j // self.S], j % self.S] = True
        off = ~used
        for name in "kv":
            c, s, b = self.q[name]
            for a, bad in ((c, BF16_NAN if self.bits == 16 else 0xFFFFFFFF), (s, BF16_NAN),
                           (b, BF16_NAN)):
                if a is not None:
                    t = a.transpose(0, 2, 1, 3)
                    t[off] = bad

    def dense(self, name, b, n):
        """[H, n, D] values in 64 bits, and [H, n, D] of |scale| * code (|value|
        for bf16 rows), the size of what a product term rounds."""
        j = np.arange(n)
        pages, at = self.table[b, j // self.S], j % self.S
        c, s, bias = self.q[name]
        rows = c[pages, :, at].transpose(1, 0, 2)
        if self.bits == 16:
            v = values(rows)
            return v, np.abs(v)
        by = rows.copy().view(np.uint8).reshape(self.H, n, self.D * self.bits // 8)
        codes = by if self.bits == 8 else np.stack((by & 15, by >> 4), -1).reshape(self.H, n, self.D)
        sv = np.repeat(values(s[pages, :, at].transpose(1, 0, 2)), self.gs, -1)
        bv = np.repeat(values(bias[pages, :, at].transpose(1, 0, 2)), self.gs, -1)
        return sv * codes + bv, np.abs(sv) * codes + (np.abs(bv) if name == "k" else 0.0)

    def device(self):
        """(KVCache, device table, device lens) with fresh copies of the buffers."""
        import affine_group_quantized_b200 as agq

        def dev(a):
            if a is None:
                return None
            a = np.ascontiguousarray(a)
            if a.dtype == np.uint16:
                return torch.from_numpy(a.view(np.int16).copy()).view(torch.bfloat16).cuda()
            return torch.from_numpy(a.view(np.int32).copy()).cuda()

        bufs = [dev(a) for a in (self.q["k"][0], self.q["v"][0], self.q["k"][1], self.q["k"][2],
                                 self.q["v"][1], self.q["v"][2])]
        cache = agq.KVCache(*bufs, self.num_pages, self.H, self.S, self.D, self.bits, self.gs)
        return (cache, torch.from_numpy(self.table.copy()).cuda(),
                torch.tensor(self.lens, dtype=torch.int32).cuda())

    def host(self, cache):
        """The device cache's buffers as numpy arrays, keyed like self.q."""
        k, v, ks, kb, vs, vb = (None if t is None else
                                t.cpu().view(torch.int16).numpy().view(np.uint16)
                                if t.element_size() == 2 else
                                t.cpu().numpy().view(np.uint32) for t in cache.buffers)
        return {"k": (k, ks, kb), "v": (v, vs, vb)}


def attention(hc: HostCache, q16, Hq, scale):
    """The definition in 64 bits.  Returns out [B, Hq, D], the bound on |out -
    kernel| and, per sequence, p [Hq, n] with the bound on p's relative error.

    The bound counts: the fp32 sums of a score (2^-23 a term over its D terms
    and a few joins: it moves a probability by twice that), the probability
    times the group's scale rounded to half precision before the value product
    (2^-11 of |scale| * code), or the probability rounded to bf16 for bf16 rows
    (2^-8 of |value|), fp32 sums over the slots, and the output's rounding to
    bf16 (2^-8)."""
    B, R, D = len(hc.lens), Hq // hc.H, hc.D
    qv = values(q16).reshape(B, Hq, D)
    out, bound, probs = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), []
    for b, n in enumerate(hc.lens):
        if n <= 0:
            probs.append((np.zeros((Hq, 0)), np.zeros((Hq, 0))))
            continue
        k, ka = hc.dense("k", b, n)
        v, va = hc.dense("v", b, n)
        ps, es = [], []
        for h in range(Hq):
            g = h // R
            s = scale * (k[g] @ qv[b, h])
            size = abs(scale) * (ka[g] @ np.abs(qv[b, h]))
            e = np.exp(s - s.max())
            p = e / e.sum()
            # two scores' errors (the slot's and the sum's), and exp's own
            rel = 2 * (D / 2 + 8) * 2.0 ** -23 * size.max() + 2.0 ** -18 * (1 + np.abs(s).max() / 16)
            out[b, h] = p @ v[g]
            term = 2.0 ** -8 if hc.bits == 16 else 2.0 ** -11
            sums = (n / 16 + 64) * 2.0 ** -23
            bound[b, h] = (2.0 ** -8 * np.abs(out[b, h]) + (term + rel + sums) * (p @ va[g])
                           + (rel + sums) * (p @ np.abs(v[g])) + 1e-30)
            if hc.bits != 16:  # the biases' own sum
                bound[b, h] += (rel + sums) * (p @ (va[g] + np.abs(v[g])))
            ps.append(p)
            es.append(np.full(n, rel))
        probs.append((np.array(ps), np.array(es)))
    return out, bound, probs


def evict(w, pos, n, seen, budget, recent, sinks):
    """One (sequence, head): (kept mask over n, source slot of each slot below
    the new length)."""
    left = min(n, budget)
    if n <= budget:
        return np.ones(n, bool), np.arange(left)
    w, pos = w[:n].astype(np.float64), pos[:n].astype(np.int64)
    held = (pos < sinks) | (pos >= seen - recent)
    rank = np.where(held, 2, np.where(np.isnan(w), 0, 1))
    w = np.where(rank == 1, w, 0.0)     # protected slots, and NaNs, by slot alone
    order = np.lexsort((np.arange(n), -w, -rank))
    keep = np.zeros(n, bool)
    keep[order[:left]] = True
    src = np.arange(left)
    src[np.flatnonzero(~keep[:left])] = left + np.flatnonzero(keep[left:])
    return keep, src
