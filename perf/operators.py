"""What is measured of the key-value cache operators: kv_append, kv_read,
kv_attention and kv_evict over a paged cache whose rows are bf16 (bits = 16)
or hold the packed affine format (bits = 4 or 8: codes, and one bf16 scale and
bias per group).

Every operator has a plain form of elementary torch operations in 32 bits
(used where ``own`` is false) and the framework's call (where it is true).
``exact`` evaluates the definitions in 64 bits, apart from the plain form.
"""
import math
import random

import numpy as np
import torch

own = False

GROUPS = {64: (32, 64), 96: (32,), 128: (32, 64, 128), 256: (32, 64, 128)}


def _case(name, kind, **kw):
    c = dict(name=name, kind=kind, batch=1, heads=8, group_heads=4, dim=128, bits=4, group=64,
             page=64, longest=1024, ragged=False, weights=False, new=0, budget=0)
    c.update(kw)
    return c


def listed():
    return [
        # one user's chat, a few hundred tokens in: the call's latency counts
        _case("attend_short", "attend", page=16, longest=611),
        # a serving batch of different ages over an 8-bit cache
        _case("attend_ragged", "attend", batch=32, bits=8, longest=4096, ragged=True),
        # four long documents, eight query heads to each key-value head
        _case("attend_long", "attend", batch=4, group_heads=8, page=128, longest=131072),
        # unquantized pages that end inside a tile, wide heads
        _case("attend_bf16", "attend", batch=16, heads=4, group_heads=4, dim=256, bits=16,
              page=48, longest=2047, ragged=True),
        # a head of its own for every query head, weights kept for eviction
        _case("attend_weights", "attend", batch=8, heads=16, group_heads=1, dim=64, group=32,
              page=32, longest=8190, ragged=True, weights=True),
        # one new token for each sequence of a serving batch, and its rows as stored
        _case("append_step", "append", batch=64, longest=4096, ragged=True, new=1, weights=True),
        # prompts of different lengths in one call
        _case("append_prompts", "append", batch=4, bits=8, longest=8192, ragged=True, new=4096,
              weights=True),
        # a chunk behind a prefix, bf16 pages, heads of 96
        _case("append_chunk", "append", batch=3, dim=96, bits=16, group=32, page=16, longest=5000,
              new=1000),
        # one cached system prompt, dense again for the next chunk's attention
        _case("read_prefix", "read", longest=1500),
        # long prefixes of a batch
        _case("read_long", "read", batch=4, page=128, longest=32768, ragged=True),
        # every step of a full cache: one slot has to go
        _case("evict_step", "evict", batch=16, longest=1025, budget=1024),
        # prompts cut to an eighth
        _case("evict_prompt", "evict", batch=4, bits=16, longest=16384, budget=2048, ragged=True),
    ]


def draw(rng: random.Random):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.choice(["attend", "attend", "append", "read", "evict"])
    dim = rng.choice([64, 96, 128, 128, 256])
    c = dict(kind=kind, dim=dim, bits=rng.choice([4, 4, 8, 16]), group=rng.choice(GROUPS[dim]),
             heads=rng.choice([1, 2, 4, 5, 8, 16]), group_heads=rng.choice([1, 2, 3, 4, 7, 8, 16]),
             page=rng.choice([16, 32, 48, 64, 128, 256]), batch=spread(1, 64),
             ragged=rng.random() < 0.6, weights=rng.random() < 0.4, new=0, budget=0)
    row = c["heads"] * 2 * dim * c["bits"] // 8
    room = 16 << 20 if kind == "evict" else 12 << 20 if kind in ("append", "read") else 300 << 20
    most = max(8, min(131072 if kind == "attend" else 16384, room * (1 if kind == "attend" else 8)
                      // (c["batch"] * row)))
    c["longest"] = spread(min(8, most), most)
    if kind == "append":
        c["new"] = 1 if rng.random() < 0.3 else spread(1, c["longest"])
        c["weights"] = rng.random() < 0.5
    if kind == "evict":
        c["budget"] = max(4, spread(max(4, c["longest"] // 16), c["longest"]))
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _lengths(case):
    """Slots in use for each sequence (after an append: the new tokens too), and
    how many of them the call appends or reads; ragged ones spread evenly."""
    n, b = case["longest"], case["batch"]
    low = max(1, n // 8) if case["ragged"] else n
    lens = [n - (n - low) * i // max(1, b - 1) for i in range(b)]
    if case["kind"] == "append":
        new = [min(case["new"], x) for x in lens]
        if case["ragged"]:
            new = [max(1, x * (i + 1) // b) for i, x in enumerate(new)]
        return lens, new
    return lens, lens


def _pages_of(case):
    return -(-case["longest"] // case["page"])


def _round_away(x):
    """Halves away from zero, in 64 bits: a sum with 0.5 is exact there."""
    x = x.double()
    return torch.trunc(x + torch.copysign(torch.full_like(x, 0.5), x)).float()


def _quantize(w, bits, group):
    """The affine quantizer's binary32 steps: bytes of codes, bf16 scales and biases."""
    v = w.float().unflatten(-1, (-1, group))
    n_bins = float(2 ** bits - 1)
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True).clamp(min=0)
    # (a plain number as the divisor would be multiplied by its reciprocal)
    step = ((hi - lo) / torch.full_like(hi, n_bins)).clamp(min=1e-7)
    low = lo.abs() > hi.abs()
    edge, step = torch.where(low, lo, hi), torch.where(low, step, -step)
    q0 = _round_away(edge / step)
    scale = torch.where(q0 != 0, edge / torch.where(q0 != 0, q0, torch.ones_like(q0)), step)
    bias = torch.where(q0 != 0, edge, torch.zeros_like(edge))
    codes = _round_away((v - bias) / scale).clamp(max=n_bins).flatten(-2).to(torch.uint8)
    if bits == 4:
        codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return (codes.contiguous().view(torch.int32), scale.squeeze(-1).bfloat16(),
            bias.squeeze(-1).bfloat16())


def _values(codes, scales, biases, bits, group):
    """scale * q + bias in 32 bits; bf16 rows as they are."""
    if bits == 16:
        return codes.float()
    b = codes.contiguous().view(torch.uint8)
    q = b.float() if bits == 8 else torch.stack((b & 15, b >> 4), -1).flatten(-2).float()
    return (q.unflatten(-1, (-1, group)) * scales.float().unsqueeze(-1)
            + biases.float().unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    B, H, D, S = case["batch"], case["heads"], case["dim"], case["page"]
    bits, group, W = case["bits"], case["group"], _pages_of(case)
    P = B * W + 3
    both = list(zip(*_lengths(case)))
    r.shuffle(both)
    lens, count = map(list, zip(*both))
    st = dict(case=case)

    def dev(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    # some channels of the keys are larger than the others, as in trained models
    channel = 1 + 2 * (torch.rand((H, 1, D), generator=g, device="cuda") < 0.06)
    for name in "kv":
        empty = case["kind"] == "append"
        rows = torch.zeros((P, H, S, D), device="cuda") if empty else normal(P, H, S, D)
        rows = (rows * channel if name == "k" else rows).bfloat16()
        if bits == 16:
            st[name], st[name + "_scales"], st[name + "_biases"] = rows, None, None
        else:
            st[name], st[name + "_scales"], st[name + "_biases"] = _quantize(rows, bits, group)
        del rows
    # every sequence's pages, scattered over the pool
    st["table"] = (torch.randperm(P, generator=g, device="cuda")[:B * W].to(torch.int32)
                   .view(B, W).contiguous())
    st["width"], st["pages"] = W, P
    n_state = W * S
    if case["kind"] == "attend":
        q = normal(B, H * case["group_heads"], D)
        st["q"] = q.bfloat16()
        st["lens"] = dev(lens)
        st["longest"] = max(lens)
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
        st["weights"] = torch.zeros((B, H, n_state), device="cuda") if case["weights"] else None
    elif case["kind"] in ("append", "read"):
        starts = [sum(count[:i]) for i in range(B + 1)]
        T = starts[-1]
        st["lens"] = dev([n - c for n, c in zip(lens, count)])
        st["starts"], st["tokens"] = dev(starts), T
        # keys and values as columns of one projection's output
        st["qkv"] = torch.cat((normal(T, H, D) * channel.view(1, H, D), normal(T, H, D)),
                              1).bfloat16() if case["kind"] == "append" else None
        st["k_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda")
        st["v_out"] = torch.empty_like(st["k_out"])
        if case["weights"]:
            st["seen"] = dev([n - c + 7 for n, c in zip(lens, count)])
            st["weights"] = torch.ones((B, H, n_state), device="cuda")
            st["positions"] = torch.full((B, H, n_state), -1, dtype=torch.int32, device="cuda")
    else:
        st["lens"], st["seen"] = dev(lens), dev(lens)
        u = torch.rand((B, H, n_state), generator=g, device="cuda")
        st["weights"] = 1.0 / (u * 40 + 0.01)  # few slots hold most of the weight
        st["positions"] = torch.arange(n_state, dtype=torch.int32, device="cuda").expand(
            B, H, -1).contiguous()
        st["recent"], st["sinks"] = case["budget"] // 4, min(4, case["budget"] // 4)
        st["new_lens"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        st["new_weights"] = torch.zeros_like(st["weights"])
        st["new_positions"] = torch.full_like(st["positions"], -1)
    if own:
        import affine_group_quantized_b200 as agq
        st["cache"] = agq.KVCache(st["k"], st["v"], st["k_scales"], st["k_biases"],
                                  st["v_scales"], st["v_biases"], P, H, S, D, bits, group)
        if case["kind"] == "attend":
            n = agq.kv_attention_workspace(st["cache"], B, H * case["group_heads"], W,
                                           case["weights"])
            st["workspace"] = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def run(st):
    kind = st["case"]["kind"]
    if kind == "attend":
        return _attend_own(st) if own else _attend(st)
    if kind == "append":
        return _append_own(st) if own else _append(st)
    if kind == "read":
        return _read_own(st) if own else _read(st)
    return _evict_own(st) if own else _evict(st)


def _attend_own(st):
    import affine_group_quantized_b200 as agq
    c = st["case"]
    agq.kv_attention(st["cache"], st["q"], st["table"], st["lens"], st["out"], c["batch"],
                     c["heads"] * c["group_heads"], st["width"], st["scale"], st["workspace"],
                     weights=st["weights"], state_width=st["width"] * c["page"])
    return {"out": st["out"], "weights": st["weights"]}


def _append_own(st):
    import affine_group_quantized_b200 as agq
    c = st["case"]
    H = c["heads"]
    state = dict(seen=st["seen"], positions=st["positions"], weights=st["weights"],
                 state_width=st["width"] * c["page"]) if c["weights"] else {}
    agq.kv_append(st["cache"], st["qkv"][:, :H], st["qkv"][:, H:], st["table"], st["lens"],
                  st["starts"], c["batch"], st["tokens"], st["width"], **state)
    return _read_own(st)


def _read_own(st):
    import affine_group_quantized_b200 as agq
    c = st["case"]
    agq.kv_read(st["cache"], st["k_out"], st["v_out"], st["table"], st["lens"], st["starts"],
                c["batch"], st["tokens"], st["width"])
    return _stored(st)


def _stored(st):
    """The rows as the cache holds them (an 8- or 4-bit row as its values), and the state."""
    got = {"k": st["k_out"], "v": st["v_out"]}
    if st["case"]["kind"] == "append" and st["case"]["weights"]:
        got["positions"], got["weights"] = st["positions"], st["weights"]
    return got


def _evict_own(st):
    import affine_group_quantized_b200 as agq
    c = st["case"]
    agq.kv_evict(st["cache"], st["table"], st["lens"], st["seen"], st["weights"],
                 st["positions"], st["new_lens"], st["new_weights"], st["new_positions"],
                 c["batch"], st["width"], st["width"] * c["page"], c["budget"], st["recent"],
                 st["sinks"])
    return _kept(st)


def _kept(st):
    # rows are moved, never computed: words of codes are returned as they lie
    # and have to be equal
    return {n: st[n] for n in ("k", "v", "k_scales", "k_biases", "v_scales", "v_biases",
                               "new_lens", "new_weights", "new_positions")}


def _dense(st, name, pages):
    """[B, H, slots, D] of the sequences' pages, in 32 bits."""
    c = st["case"]
    part = [None if st[name + x] is None else st[name + x][pages] for x in
            ("", "_scales", "_biases")]
    return _values(*part, c["bits"], c["group"]).transpose(1, 2).flatten(2, 3)


def _attend(st):
    c = st["case"]
    B, H, R, D = c["batch"], c["heads"], c["group_heads"], c["dim"]
    pages = st["table"][:, :-(-st["longest"] // c["page"])].long()
    k = _dense(st, "k", pages)
    s = torch.matmul(st["q"].float().view(B, H, R, D), k.transpose(2, 3)) * st["scale"]
    del k
    live = torch.arange(s.shape[-1], device="cuda") < st["lens"].view(B, 1, 1, 1)
    s = s.masked_fill(~live, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    out = torch.matmul(p, _dense(st, "v", pages)).view(B, H * R, D).to(torch.bfloat16)
    if st["weights"] is not None:
        st["weights"][:, :, :p.shape[-1]] += p.sum(2)
    return {"out": out, "weights": st["weights"]}


def _slots(st):
    """Sequence, page and offset of every token of the call."""
    t = torch.arange(st["tokens"], device="cuda")
    seq = torch.searchsorted(st["starts"][1:].long(), t, right=True)
    slot = st["lens"].long()[seq] + t - st["starts"].long()[seq]
    S = st["case"]["page"]
    return seq, slot, st["table"].long()[seq, slot // S], slot % S


def _append(st):
    c = st["case"]
    H = c["heads"]
    seq, slot, page, at = _slots(st)
    k, v = st["qkv"][:, :H], st["qkv"][:, H:]
    if c["bits"] == 16:
        st["k"][page, :, at], st["v"][page, :, at] = k, v
    else:
        parts = ("", "_scales", "_biases")
        kq, vq = _quantize(k, c["bits"], c["group"]), _quantize(v, c["bits"], c["group"])
        (st["k" + parts[0]][page, :, at], st["k" + parts[1]][page, :, at],
         st["k" + parts[2]][page, :, at]) = kq
        (st["v" + parts[0]][page, :, at], st["v" + parts[1]][page, :, at],
         st["v" + parts[2]][page, :, at]) = vq
    if c["weights"]:
        pos = st["seen"].long()[seq] + slot - st["lens"].long()[seq]
        st["positions"][seq, :, slot] = pos.to(torch.int32).unsqueeze(1).expand(-1, H)
        st["weights"][seq, :, slot] = 0.0
    return _read(st)


def _read(st):
    c = st["case"]
    _, _, page, at = _slots(st)

    def rows(name):
        part = [None if st[name + x] is None else st[name + x][page, :, at] for x in
                ("", "_scales", "_biases")]
        return _values(*part, c["bits"], c["group"]).to(torch.bfloat16)

    st["k_out"], st["v_out"] = rows("k"), rows("v")
    return _stored(st)


def _evict(st):
    c = st["case"]
    B, H, S, budget = c["batch"], c["heads"], c["page"], c["budget"]
    w, pos = st["weights"], st["positions"]
    L = w.shape[-1]
    j = torch.arange(L, device="cuda")
    n = st["lens"].long().view(B, 1, 1)
    held = (pos < st["sinks"]) | (pos >= st["seen"].view(B, 1, 1) - st["recent"])
    key = torch.where(held, math.inf, w).masked_fill(j >= n, -math.inf)
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    left = n.clamp(max=budget)
    keep = (rank < left) & (j < n)
    hole = ~keep & (j < left)
    mover = keep & (j >= left)
    # the i-th mover's slot, in order, for the i-th hole
    nth = torch.where(mover, mover.cumsum(-1) - 1, L)
    src = torch.zeros((B, H, L + 1), dtype=torch.long, device="cuda").scatter_(
        -1, nth, j.expand_as(nth).contiguous())
    src = torch.where(hole, src.gather(-1, (hole.cumsum(-1) - 1).clamp(min=0)), j)
    state = ((st["new_weights"], w, 0.0), (st["new_positions"], pos, -1))
    new = [torch.where(j < left, x.gather(-1, src), torch.where(j < n, torch.full_like(x, z), y))
           for y, x, z in state]
    st["new_weights"], st["new_positions"] = new
    st["new_lens"] = left.view(B).to(torch.int32)
    # the first `budget` slots of every sequence, from where they come
    m = min(budget, L)
    seq = torch.arange(B, device="cuda").view(B, 1, 1)
    head = torch.arange(H, device="cuda").view(1, H, 1)
    table, src, to = st["table"].long(), src[..., :m], j[:m].view(1, 1, m)
    from_at = (table[seq, src // S], head, src % S)
    to_at = (table[seq, to // S], head, (to % S).expand(B, H, m))
    moved = [x[from_at] for x in _rows(st)]
    _ = [x.index_put_(to_at, y) for x, y in zip(_rows(st), moved)]
    return _kept(st)


def _rows(st):
    return [st[n] for n in ("k", "v", "k_scales", "k_biases", "v_scales", "v_biases")
            if st[n] is not None]


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------


def _row_bytes(case):
    """Bytes of one slot's key and value rows."""
    if case["bits"] == 16:
        return 4 * case["dim"]
    return 2 * (case["dim"] * case["bits"] // 8 + 4 * (case["dim"] // case["group"]))


def work(case):
    H, D = case["heads"], case["dim"]
    lens, new = _lengths(case)
    if case["kind"] == "attend":
        slots = H * sum(lens)
        by = slots * _row_bytes(case) + 4 * case["batch"] * H * case["group_heads"] * D
        by += 8 * slots if case["weights"] else 0
        return {"bytes": by, "flops": 4 * slots * case["group_heads"] * D}
    if case["kind"] in ("append", "read"):
        rows = H * sum(new)
        by = rows * (_row_bytes(case) + 4 * D)
        if case["kind"] == "append":  # the rows come in, and their stored values go out
            by += rows * (4 * D + (8 if case["weights"] else 0))
        return {"bytes": by, "flops": rows * D * (2 if case["kind"] == "read" else 20)}
    state = sum(8 * n + 8 * n for n in lens)
    # a kept slot lies at or above the budget with the share of slots that do
    moved = sum(case["budget"] * (1 - case["budget"] / n) for n in lens if n > case["budget"])
    return {"bytes": H * (state + 2 * moved * _row_bytes(case)), "flops": 4 * H * sum(lens)}


def exact(case, seed):
    def values(codes, scales, biases, bits):
        if bits == 16:
            return codes.double()
        D = codes.shape[-1] * 32 // bits
        wide = codes.repeat_interleave(32 // bits, -1).long() & 0xffffffff
        shift = (torch.arange(D, device=codes.device) % (32 // bits)) * bits
        q = (wide >> shift) & ((1 << bits) - 1)
        rep = D // scales.shape[-1]
        return (q.double() * scales.double().repeat_interleave(rep, -1)
                + biases.double().repeat_interleave(rep, -1))

    def attend(st):
        c = st["case"]
        H, R, S = c["heads"], c["group_heads"], c["page"]
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        wts = None if st["weights"] is None else st["weights"].double()
        lens, table = st["lens"].tolist(), st["table"].long()
        for b, n in enumerate(lens):
            if n <= 0:
                continue
            pages = table[b, :-(-n // S)]
            for h in range(H):
                kv = [values(st[x][pages, h], *(
                    None if st[x + y] is None else st[x + y][pages, h] for y in
                    ("_scales", "_biases")), c["bits"]).flatten(0, 1)[:n] for x in "kv"]
                q = st["q"][b, h * R:(h + 1) * R].double()
                p = torch.softmax((q @ kv[0].T) / math.sqrt(c["dim"]), -1)
                out[b, h * R:(h + 1) * R] = p @ kv[1]
                if wts is not None:
                    wts[b, h, :n] += p.sum(0)
        return {"out": out, "weights": wts}

    def quantized(x, bits, group):
        """The values an affine row stands for: codes by the quantizer's binary32
        steps on the CPU, scale * q + bias in 64 bits."""
        v = x.float().cpu().numpy().reshape(*x.shape[:-1], -1, group)
        f = np.float32
        lo, hi = v.min(-1), np.maximum(v.max(-1), f(0))
        nb = f(2 ** bits - 1)
        d = np.maximum((hi - lo) / nb, f(1e-7))
        edge = np.where(np.abs(lo) > np.abs(hi), lo, hi)
        s = np.where(np.abs(lo) > np.abs(hi), d, -d)

        def away(t):
            t = t.astype(np.float64)
            return np.sign(t) * np.floor(np.abs(t) + 0.5)

        q0 = away(edge / s).astype(f)
        with np.errstate(divide="ignore", invalid="ignore"):
            s = np.where(q0 != 0, edge / q0, s).astype(f)
        b = np.where(q0 != 0, edge, f(0)).astype(f)
        q = np.minimum(away((v - b[..., None]) / s[..., None]), nb)
        s, b = (torch.from_numpy(t).bfloat16().double() for t in (s, b))
        return (torch.from_numpy(q).double() * s[..., None] + b[..., None]).flatten(-2)

    def stored(st):
        c = st["case"]
        H, S = c["heads"], c["page"]
        starts, lens = st["starts"].tolist(), st["lens"].tolist()
        got = {}
        if c["kind"] == "append":
            for name, x in (("k", st["qkv"][:, :H]), ("v", st["qkv"][:, H:])):
                got[name] = x.double() if c["bits"] == 16 else quantized(x, c["bits"], c["group"])
            if c["weights"]:
                w = st["weights"].double()
                for b, n in enumerate(lens):
                    w[b, :, n:n + starts[b + 1] - starts[b]] = 0
                got["positions"], got["weights"] = None, w
            return got
        for name in "kv":
            rows = []
            for b, n in enumerate(lens):
                m = starts[b + 1] - starts[b]
                pages = st["table"][b, :-(-(n + m) // S)].long()
                x = values(st[name][pages], *(None if st[name + y] is None else st[name + y][pages]
                                              for y in ("_scales", "_biases")), c["bits"])
                rows.append(x.transpose(1, 2).flatten(0, 1)[n:n + m])
            got[name] = torch.cat(rows)
        return got

    def evict(st):
        """Nothing is computed but the choice: the weights where they end up."""
        c = st["case"]
        new = st["new_weights"].double().cpu().numpy()
        w, pos = st["weights"].cpu().numpy(), st["positions"].cpu().numpy()
        seen, lens = st["seen"].tolist(), st["lens"].tolist()
        for b, n in enumerate(lens):
            left = min(n, c["budget"])
            for h in range(c["heads"]):
                p, x = pos[b, h, :n], w[b, h, :n].astype(np.float64)
                held = (p < st["sinks"]) | (p >= seen[b] - st["recent"])
                kept = np.zeros(n, bool)
                kept[np.lexsort((np.arange(n), -np.where(held, np.inf, x)))[:left]] = True
                new[b, h, :n] = 0
                new[b, h, :left] = x[:left]
                new[b, h, np.flatnonzero(~kept[:left])] = x[left + np.flatnonzero(kept[left:])]
        got = dict.fromkeys(_kept(st))
        got["new_weights"] = torch.from_numpy(new)
        return got

    st = prepare(case, seed)
    if case["kind"] == "attend":
        return attend(st)
    return stored(st) if case["kind"] in ("append", "read") else evict(st)
