"""GPU tests of calls at the edges of what the key-value cache operators allow:
rows that are only 16-byte aligned, one head, large batches, no slots at all,
refusals that need a device."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
import oracle
from affine_group_quantized_b200 import synth
from tests._kv import HostCache, attention, evict
from tests._parity import bf16_values, dev_bf16, host_bits
from tests.test_kv_attention import check, run

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bits, D, gs", [(4, 64, 32), (8, 96, 32), (16, 64, 0), (16, 256, 0)])
@pytest.mark.parametrize("H", [1, 2])
def test_rows_aligned_to_16_bytes_only(bits, D, gs, H):
    # strides that are odd multiples of 16 bytes, and a buffer that begins at one
    T = 37
    hc = HostCache([T], H, D, bits, gs, 16, seed=1)
    x = synth.normal_bf16((T, H, D), 2)
    stride = H * D + 8

    def strided(fill):
        flat = torch.full((T * stride + 8,), fill, dtype=torch.bfloat16, device="cuda")
        return flat, flat[8:].as_strided((T, H, D), (stride, D, 1))

    flat, X = strided(0.0)
    X.copy_(dev_bf16(x))
    results = []
    for src in (X, dev_bf16(x)):
        cache, table, _ = hc.device()
        agq.kv_append(cache, src, src, table, _i32([0]), _i32([0, T]), 1, T, hc.width)
        results.append([t for t in cache.buffers if t is not None])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    dense = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    flat, K = strided(7.0)
    other, V = strided(7.0)
    agq.kv_read(cache, K, V, table, _i32([0]), _i32([0, T]), 1, T, hc.width)
    agq.kv_read(cache, dense, dense.clone(), table, _i32([0]), _i32([0, T]), 1, T, hc.width)
    assert torch.equal(K, dense) and torch.equal(V, dense)
    gaps = flat[8:8 + T * stride].view(T, stride)[:, H * D:]
    assert (gaps == 7).all() and (flat[:8] == 7).all()


def test_many_sequences():
    # more sequences than the tables in shared memory take, some without slots
    B, H, D = 1500, 1, 64
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 20, B)
    hc = HostCache(lens.tolist(), H, D, 4, 32, 16, seed=4, room=32)
    new = np.minimum(lens, rng.integers(0, 3, B))
    starts = np.concatenate(([0], np.cumsum(new)))
    T = int(starts[-1])
    x = synth.normal_bf16((T, H, D), 5)
    cache, table, dlens = hc.device()
    agq.kv_append(cache, dev_bf16(x), dev_bf16(x), table, _i32(lens - new), _i32(starts), B, T,
                  hc.width)
    K = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    agq.kv_read(cache, K, V, table, _i32(lens - new), _i32(starts), B, T, hc.width)
    assert torch.equal(K, V)
    wq, s, b = oracle.affine_quantize(x.reshape(-1, D), T * H, D, 4, 32)
    want = oracle.dequantize_bf16(wq, s, b, T * H, D, 4, 32)
    assert np.array_equal(host_bits(K).reshape(-1), want.reshape(-1))
    hc.q = {n: tuple(None if a is None else a.reshape(b.shape) for a, b in
                     zip(hc.host(cache)[n], hc.q[n])) for n in "kv"}
    q = synth.normal_bf16((B, 2, D), 6)
    ref, bound, _ = attention(hc, q, 2, 0.125)
    check(run(hc, q, 2, 0.125, dev=(cache, table, dlens)), ref, bound)


def test_the_largest_batch():
    B, H, D = 4096, 1, 64
    hc = HostCache([1] * B, H, D, 16, 0, 16, seed=7, room=16)
    q = synth.normal_bf16((B, 1, D), 8)
    out = run(hc, q, 1, 0.125)
    for b in (0, 1, 2047, 4095):              # one slot: its value, as it is
        v, _ = hc.dense("v", b, 1)
        assert np.array_equal(bf16_values(host_bits(out[b, 0])), v[0, 0])


@pytest.mark.parametrize("bits", [4, 16])
def test_no_slots_at_all(bits):
    hc = HostCache([0, 0, -1], 2, 128, bits, 64, 16, seed=9, room=64)
    q = synth.normal_bf16((3, 8, 128), 10)
    w = torch.full((3, 2, 64), 2.0, device="cuda")
    out = run(hc, q, 8, 0.1, weights=w, state_width=64)
    assert (out == 0).all() and (w == 2).all()
    cache, table, lens = hc.device()
    K = torch.full((4, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    agq.kv_read(cache, K, K, table, lens, _i32([0, 0, 0, 0]), 3, 4, hc.width)   # four padding rows
    assert (K == 7).all()
    p = torch.full((3, 2, 64), 5, dtype=torch.int32, device="cuda")
    new = _i32([9, 9, 9])
    agq.kv_evict(cache, table, lens, lens, w, p, new, w, p, 3, hc.width, 64, 8)
    assert new.tolist() == [0, 0, 0] and (w == 2).all() and (p == 5).all()


def test_refusals_on_a_device():
    hc = HostCache([10], 2, 64, 8, 64, 16, seed=11)
    cache, table, lens = hc.device()
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    n = agq.kv_attention_workspace(cache, 1, 4, hc.width)
    small = torch.empty(n - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(agq.QmvError, match="workspace") as ei:
        agq.kv_attention(cache, q, table, lens, out, 1, 4, hc.width, 0.1, small)
    assert ei.value.status == agq.QMV_ERR_SHAPE
    assert agq.kv_attention_workspace(cache, 1, 4, hc.width, True) > n
    with pytest.raises(ValueError, match="lens"):
        agq.kv_attention(cache, q, table, lens.cpu(), out, 1, 4, hc.width, 0.1, small)
    with pytest.raises(ValueError, match="block_table: must hold 4-byte"):
        agq.kv_attention(cache, q, table.long(), lens, out, 1, 4, hc.width, 0.1, small)
    with pytest.raises(ValueError, match="out"):
        agq.kv_attention(cache, q, table, lens, out[:, :3], 1, 4, hc.width, 0.1, small)


def test_evicting_everything_but_one_of_a_long_row():
    # the room's largest cluster, a budget of one, every key in one bin but one
    n = 60000
    hc = HostCache([n], 1, 64, 4, 64, 256, seed=12, spare=0)
    width = hc.width * 256
    w = np.full((1, 1, width), 0.5, np.float32)
    w[0, 0, 43210] = 0.75
    pos = np.arange(width, dtype=np.int32).reshape(1, 1, -1)
    cache, table, lens = hc.device()
    W, P = torch.from_numpy(w).cuda(), torch.from_numpy(pos).cuda()
    new = _i32([0])
    agq.kv_evict(cache, table, lens, lens, W, P, new, W, P, 1, hc.width, width, 1)
    assert new.item() == 1 and P[0, 0, 0].item() == 43210 and W[0, 0, 0].item() == 0.75
    assert (W[0, 0, 1:n] == 0).all() and (P[0, 0, 1:n] == -1).all()
    keep, src = evict(w[0, 0], pos[0, 0], n, n, 1, 0, 0)
    assert src.tolist() == [43210]
    k = hc.host(cache)["k"][0].reshape(hc.q["k"][0].shape)
    assert np.array_equal(k[hc.table[0, 0], 0, 0], hc.q["k"][0][hc.table[0, 43210 // 256], 0, 43210 % 256])
