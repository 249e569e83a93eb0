"""CPU models of the key-value cache kernels' index arithmetic: how tiles are
shared out over CTAs and warps, the swizzle and slot order of a tile in shared
memory (bijective, every read of a warp over all 32 banks, or how near it
comes), which element an accumulator holds, codes as fp16 subnormals, the packed
codes of the quantizer, and the order of eviction keys."""
import numpy as np
import pytest

HEADS = {4: {64: (32, 64), 96: (32,), 128: (32, 64, 128), 256: (32, 64, 128)},
         8: {64: (32, 64), 96: (32,), 128: (32, 64, 128), 256: (32, 64, 128)},
         16: {64: (64,), 96: (96,), 128: (128,), 256: (256,)}}
CASES = [(b, d, g) for b, v in HEADS.items() for d, gs in v.items() for g in gs]


def share(total, most, few=8):
    ctas = min(-(-total // few), most)
    base = total // ctas if ctas else 0
    return ctas, base, total - base * ctas


@pytest.mark.parametrize("most", [148, 296])
def test_every_tile_has_one_cta_and_one_warp(most):
    rng = np.random.default_rng(0)
    for total in [1, 7, 8, 9, most * 8 - 1, most * 8, most * 8 + 1, 12345, 10 ** 7 + 3] + \
            rng.integers(1, 10 ** 6, 50).tolist():
        ctas, base, extra = share(total, most)
        first = [c * base + min(c, extra) for c in range(ctas + 1)]
        assert first[0] == 0 and first[-1] == total
        sizes = np.diff(first)
        assert sizes.min() >= 1 and sizes.max() - sizes.min() <= 1

        def cta_of(tile):
            bound = extra * (base + 1)
            return tile // (base + 1) if tile < bound else extra + (tile - bound) // base

        for c in range(ctas):
            assert cta_of(first[c]) == c and cta_of(first[c + 1] - 1) == c
        for warps in (4, 8, 12):
            for c in (0, ctas // 2, ctas - 1):
                n = int(sizes[c])
                each, more = divmod(n, warps)
                u = [w * each + min(w, more) for w in range(warps)] + [n]
                counts = [each + (w < more) for w in range(warps)]
                assert [b - a for a, b in zip(u, u[1:])] == counts
                # warps without tiles come last: a segment's pieces are neighbours
                assert sorted(counts, reverse=True) == counts


def bits_of(ch):
    return {3: 0, 2: 1, 6: 1, 4: 3, 12: 3}.get(ch, 7)


def swizzle(ch, r):
    if ch in (2, 6):
        return (r >> 2) & 1
    if ch in (4, 12):
        return (r >> 1) & 3
    return 0 if ch == 3 else r & 7


def slot_of(ch, r):
    if ch == 2:
        return ((r & 1) << 2) | (r >> 1)
    if ch == 4:
        return (r & 4) | ((r & 1) << 1) | ((r >> 1) & 1)
    return r


def chunk_at(ch, row0, chunk):
    k = bits_of(ch)
    return (row0 ^ ((chunk & k) << 4)) + ((chunk & ~k) << 4)


def stored(ch, r, chunk):
    """Where the copies put chunk `chunk` of row r (16 rows to a block)."""
    return r * 16 * ch + ((chunk ^ swizzle(ch, r & 7)) << 4)


@pytest.mark.parametrize("bits, D, gs", CASES)
def test_tiles_in_shared_memory(bits, D, gs):
    ch = D * bits // 128
    rb = 16 * ch
    at = {(r, c): stored(ch, r, c) for r in range(16) for c in range(ch)}
    assert sorted(at.values()) == list(range(0, 16 * rb, 16))
    assert sorted(slot_of(ch, r) for r in range(8)) == list(range(8))
    # lane i of copy c writes chunk 32 c + i of the block, as the kernel computes it
    for c in range((ch + 1) // 2):
        for lane in range(32):
            ix = 32 * c + lane
            if ix >= 16 * ch:
                continue
            if 32 % ch == 0:
                rows = 32 // ch
                to = (lane // ch) * rb + ((lane % ch ^ swizzle(ch, (lane // ch) & 7)) << 4)
                dst = (to ^ (swizzle(ch, (c * rows) & 7) << 4)) + c * rows * rb
            else:
                r = ix // ch
                dst = r * rb + ((ix % ch ^ swizzle(ch, r & 7)) << 4)
            assert dst == at[ix // ch, ix % ch]
    if bits == 16:
        for i in range(D // 16):
            # ldmatrix: 8 rows of 16 bytes at a time, for keys and for values
            for lane in range(32):
                k0 = (lane & 15) * rb + (((lane >> 4) ^ swizzle(ch, lane & 7)) << 4)
                assert chunk_at(ch, k0, 2 * i) == at[lane & 15, 2 * i + (lane >> 4)]
                r = (lane & 7) + ((lane >> 4) << 3)
                v0 = r * rb + ((((lane >> 3) & 1) ^ swizzle(ch, lane & 7)) << 4)
                assert chunk_at(ch, v0, 2 * i) == at[r, 2 * i + ((lane >> 3) & 1)]
            assert len({at[r, 2 * i] // 16 % 8 for r in range(8)}) == 8   # all banks
        return
    # scores: lane (g, t) reads word t + 4 i of slot slot_of(g), and of the slot 8 on
    for i in range(ch):
        banks = []
        for lane in range(32):
            g, t = lane >> 2, lane & 3
            row = slot_of(ch, g)
            a = chunk_at(ch, row * rb + (swizzle(ch, row) << 4) + 4 * t, i)
            assert a == at[row, i] + 4 * t and a + 8 * rb == at[row + 8, i] + 4 * t
            banks.append(a // 4 % 32)
        assert len(set(banks)) == 32
    # values: words of four slots, for the elements that the accumulators say
    vch = 64 if bits == 4 and gs >= 64 else 32
    worst = 0
    for c in range(D // vch):
        for half in range(2):
            words = {}
            for lane in range(32):
                g, t = lane >> 2, lane & 3
                w0 = g & 3 if vch == 32 and bits == 4 else g
                word = 8 * c + g if bits == 8 or vch == 64 else 4 * c + (g & 3)
                r = slot_of(ch, 2 * t + half)
                base = r * rb + (((w0 >> 2) ^ swizzle(ch, r)) << 4) + ((w0 & 3) << 2)
                a = chunk_at(ch, base, c * (1 if vch == 32 and bits == 4 else 2))
                assert a == at[r, word // 4] + 4 * (word % 4)
                words.setdefault(a // 4 % 32, set()).add(a)
            worst = max(worst, max(len(v) for v in words.values()))
    assert worst == (2 if ch == 6 else 1)     # heads of 96 in 8 bits: two rows meet


@pytest.mark.parametrize("bits, D, gs", CASES)
def test_accumulators_hold_every_element_once(bits, D, gs):
    vch = 64 if bits == 4 and gs >= 64 else 32
    seen = []
    for mt in range(D // 16):
        for half in range(2):
            for g in range(8):
                if bits == 16:
                    d = 16 * mt + g + 8 * half
                elif bits == 8:
                    d = 32 * (mt // 2) + 4 * g + 2 * half + mt % 2
                elif vch == 64:
                    d = 64 * (mt // 4) + 8 * g + 4 * half + mt % 4
                else:
                    d = 32 * (mt // 2) + 8 * (g & 3) + 4 * (g >> 2) + 2 * half + mt % 2
                seen.append(d)
                if bits != 16:                # one group, one factor, for a whole tile
                    assert d // gs == mt * 16 // gs
                if bits == 4:                 # odd tiles hold the bytes' sums
                    assert d % 2 == mt % 2
    assert sorted(seen) == list(range(D))


def half_value(b):
    return np.array([b], np.uint16).view(np.float16).astype(np.float64)[0]


def test_codes_are_fp16_subnormals():
    for q in range(256):
        assert half_value(q) == q * 2.0 ** -24
    for q in range(16):
        assert half_value(q << 4) == q * 2.0 ** -20
    # the sums of bytes and of low nibbles give those of the high ones
    rng = np.random.default_rng(1)
    b, p = rng.integers(0, 256, 1000), rng.random(1000)
    assert abs(((p * b).sum() - (p * (b & 15)).sum()) / 16 - (p * (b >> 4)).sum()) < 1e-9


def test_sixteen_bits_of_codes_are_an_exact_binary32_number():
    f = np.float32
    for c in ((15, 15, 15, 15), (0, 0, 0, 0), (1, 2, 4, 8), (15, 0, 15, 0)):
        y = f(c[0]) + f(16) * f(c[1]) + f(256) * f(c[2]) + f(4096) * f(c[3])
        assert (f(y + f(8388608)).view(np.uint32) & 0xffff) == sum(v << (4 * i) for i, v in enumerate(c))
    for c in ((255, 255), (0, 255), (7, 200)):
        y = f(c[0]) + f(256) * f(c[1])
        assert (f(y + f(8388608)).view(np.uint32) & 0xffff) == c[0] | c[1] << 8


def test_quantizer_margin_covers_the_reciprocal():
    # t = d * fl(1 / s) against fl(d / s): within 3 * 2^-24 of it, relative, so
    # within 2^-22 * (n_bins + 1) / 1.33 for |t| <= n_bins + 1
    rng = np.random.default_rng(2)
    f = np.float32
    for n_bins in (15, 255):
        s = (rng.random(200000).astype(f) + f(0.01))
        d = (s * (rng.random(200000) * (n_bins + 1))).astype(f)
        t = d * (f(1) / s)
        q = (d / s).astype(f)
        err = np.abs(t.astype(np.float64) - q.astype(np.float64))
        assert (err <= 3 * 2.0 ** -24 * np.abs(q)).all()
        assert err.max() < (n_bins + 1) * 2.0 ** -22


def test_eviction_keys_are_in_order():
    def key(w, pos=5, sinks=0, frm=100):
        if pos < sinks or pos >= frm:
            return 0xffffffff
        w = np.float32(w)
        if np.isnan(w):
            return 0
        u = int((w + np.float32(0)).view(np.uint32))
        return (~u & 0xffffffff) if u >> 31 else u | 0x80000000

    order = [float("nan"), float("-inf"), -3.4e38, -1.0, -1e-45, 0.0, 1e-45, 1e-38, 0.5, 1.0, 3.4e38,
             float("inf")]
    keys = [key(w) for w in order]
    assert keys == sorted(keys) and len(set(keys)) == len(keys)
    assert key(-0.0) == key(0.0)
    assert key(float("inf")) < key(0.0, pos=100) == key(float("nan"), pos=0, sinks=1)


@pytest.mark.parametrize("units", [4, 8, 12, 16, 24, 32, 64])
def test_a_warp_copies_every_unit_of_its_moves_once(units):
    u = min(units, 32)
    per = 32 // u
    for count in (1, 3, 14, 31, 32):
        seen = []
        for m0 in range(0, count, 4 * per):
            for a in range(4):
                for lane in range(32):
                    sub = min(lane // u, per)
                    m = m0 + a * per + sub
                    if m < count and sub < per:
                        seen.append((m, lane - (lane // u) * u))
        assert sorted(seen) == [(m, i) for m in range(count) for i in range(u)]
